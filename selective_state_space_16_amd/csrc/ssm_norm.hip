// The norms of a Mamba block for gfx950, forward and backward: the residual
// sum with the root-mean-square norm ahead of the block's projection, and the
// gate with the (grouped) root-mean-square norm behind its scan.
//
//   add norm    r = residual + scale o x;   y = r rstd w,  rstd = (mean r^2 + eps)^-1/2
//   gate norm   u = x silu(z);              y = u rstd w   per group of D / groups channels
//
// Backward, with g = dy w and hat = r rstd (or u rstd), the norm's chain rule is
//   dr = rstd (g - hat mean(g hat)),   dw = sum over rows of dy hat,
// so one reduction per row gives both sums that a row needs (sum r^2 and
// sum g r). Every kernel reads each input once and writes each output once:
// HBM bounds them all. A row is held in registers by the lanes that read it
// (a wave, or a workgroup for long rows), so a row costs one pass. Measured, with
// bfloat16 activations and a float32 residual, against 5.4 TB/s of a large copy:
//   gate norm 32768 x 5120    forward  174 us, 1.01 GB, 5.8 TB/s
//   add norm  32768 x 2560    backward 291 us, 1.51 GB, 5.2 TB/s (its reduction 4 us of it)
//   add norm  16384 x 2560    forward   95 us, 0.50 GB, 5.3 TB/s
//   gate norm 8193 x 1536/2   backward  30 us, 0.13 GB (reduction 4 us)
//   add norm  4097 x 1001     forward   14 us, float32, 66 MB
// Streaming loads or stores in the backward passes were not worth it (at 40
// values per lane 305 us: stores 302, loads 322), nor were all of a row's loads
// ahead of its reduction (340: more registers than two waves per SIMD leave).
//
// dw (and dscale) sum over all rows: a workgroup keeps its rows' sums in
// registers, adds its waves' in a fixed order through LDS and writes one
// partial row; a second kernel adds the partial rows in order. Equal inputs
// give equal bits.
#include "ssm_internal.h"
#include "ssm_norm_rows.h"

namespace ssm {

namespace {

// Rows beyond the last-level cache (256 MB) that a kernel passes over once are
// loaded and stored as data without reuse (STREAM).
constexpr int64_t kStreamBytes = 256ll << 20;

template <int TPR, bool ODD, int ITER, typename T, typename R>
__global__ __launch_bounds__(block_threads(TPR)) void add_norm_fwd_kernel(AddNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ double sh[2][16][1];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const int64_t base = row * D;
        float r[ITER][kVec], ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float x[kVec];
                ld_vec<ODD>((const T *)a.x + base + c, left, x);
                if (a.residual) ld_vec<ODD>((const R *)a.residual + base + c, left, r[k]);
                float s[kVec];
                if (a.scale) ld_vec<ODD>(a.scale + c, left, s);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float add = a.scale ? s[i] * x[i] : x[i];
                    r[k][i] = a.residual ? r[k][i] + add : add;
                    ss[0] = __builtin_fmaf(r[k][i], r[k][i], ss[0]);
                }
            }
        }
        double sum[1];
        row_sum<TPR, 1>(ss, sum, sh, turn);
        const float rstd = inv_rms(sum[0], inv, a.eps);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec], y[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
                st_vec<ODD>((R *)a.residual_out + base + c, left, r[k]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) y[i] = r[k][i] * rstd * w[i];
                st_vec<ODD>((T *)a.y + base + c, left, y);
            }
        }
    }
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
__global__ __launch_bounds__(block_threads(TPR)) void add_norm_bwd_kernel(AddNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ double sh[2][16][2];
    __shared__ float cols[RPB > 1 ? TPR * kVec * ITER : 1];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    float dw[ITER][kVec], ds[ITER][kVec];
#pragma unroll
    for (int k = 0; k < ITER; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[k][i] = ds[k][i] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const int64_t base = row * D;
        float r[ITER][kVec], dy[ITER][kVec], ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec];
                ld_vec<ODD>((const R *)a.residual + base + c, left, r[k]);
                ld_vec<ODD>((const T *)a.dy + base + c, left, dy[k]);
                ld_vec<ODD>(a.weight + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    ss[0] = __builtin_fmaf(r[k][i], r[k][i], ss[0]);
                    ss[1] = __builtin_fmaf(dy[k][i] * w[i], r[k][i], ss[1]);
                }
            }
        }
        double sum[2];
        row_sum<TPR, 2>(ss, sum, sh, turn);
        const float rstd = inv_rms(sum[0], inv, a.eps);
        const float m = (float)(sum[1] * inv) * rstd;  // mean(g hat)
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec], dr[kVec], up[kVec], x[kVec], s[kVec], dx[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
                if (a.dres) ld_vec<ODD>((const R *)a.dres + base + c, left, up);
                if (a.scale) {
                    ld_vec<ODD>((const T *)a.x + base + c, left, x);
                    ld_vec<ODD>(a.scale + c, left, s);
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float hat = r[k][i] * rstd;
                    dw[k][i] = __builtin_fmaf(dy[k][i], hat, dw[k][i]);
                    float v = rstd * __builtin_fmaf(-m, hat, dy[k][i] * w[i]);
                    if (a.dres) v += up[i];
                    dr[i] = v;
                    if (a.scale) {
                        dx[i] = v * s[i];
                        ds[k][i] = __builtin_fmaf(v, x[i], ds[k][i]);
                    } else {
                        dx[i] = v;
                    }
                }
                st_vec<ODD>((R *)a.residual_out + base + c, left, dr);
                st_vec<ODD>((T *)a.dx + base + c, left, dx);
            }
        }
    }
    write_partial<TPR, ODD, ITER>(dw, cols, a.part + (int64_t)blockIdx.x * D, D);
    if (a.scale) write_partial<TPR, ODD, ITER>(ds, cols, a.part + ((int64_t)gridDim.x + blockIdx.x) * D, D);
}

// u = x silu(z) and the factors of its gradient.
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-z * kLog2e)); }

template <int TPR, bool ODD, int ITER, typename T, bool STREAM>
__global__ __launch_bounds__(block_threads(TPR)) void gate_norm_fwd_kernel(GateNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ double sh[2][16][1];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t Dg = a.D / a.groups, g0 = (int64_t)blockIdx.y * Dg;
    const double inv = 1.0 / (double)Dg;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const T *xp = (const T *)a.x + row * a.x_stride + g0, *zp = (const T *)a.z + row * a.z_stride + g0;
        T *yp = (T *)a.y + row * a.D + g0;
        float u[ITER][kVec], ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)Dg - c;
            if (left > 0) {
                float x[kVec], z[kVec];
                ld_vec<ODD, STREAM>(xp + c, left, x);
                ld_vec<ODD, STREAM>(zp + c, left, z);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    u[k][i] = x[i] * silu(z[i]);
                    ss[0] = __builtin_fmaf(u[k][i], u[k][i], ss[0]);
                }
            }
        }
        double sum[1];
        row_sum<TPR, 1>(ss, sum, sh, turn);
        const float rstd = inv_rms(sum[0], inv, a.eps);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)Dg - c;
            if (left > 0) {
                float w[kVec], y[kVec];
                ld_vec<ODD>(a.weight + g0 + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) y[i] = u[k][i] * rstd * w[i];
                st_vec<ODD, STREAM>(yp + c, left, y);
            }
        }
    }
}

template <int TPR, bool ODD, int ITER, typename T>
__global__ __launch_bounds__(block_threads(TPR)) void gate_norm_bwd_kernel(GateNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ double sh[2][16][2];
    __shared__ float cols[RPB > 1 ? TPR * kVec * ITER : 1];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D, Dg = D / a.groups, g0 = (int64_t)blockIdx.y * Dg;
    const double inv = 1.0 / (double)Dg;
    float dw[ITER][kVec];
#pragma unroll
    for (int k = 0; k < ITER; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[k][i] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const T *xp = (const T *)a.x + row * a.x_stride + g0, *zp = (const T *)a.z + row * a.z_stride + g0;
        const T *dyp = (const T *)a.dy + row * D + g0;
        float x[ITER][kVec], z[ITER][kVec], dy[ITER][kVec], ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)Dg - c;
            if (left > 0) {
                float w[kVec];
                ld_vec<ODD>(xp + c, left, x[k]);
                ld_vec<ODD>(zp + c, left, z[k]);
                ld_vec<ODD>(dyp + c, left, dy[k]);
                ld_vec<ODD>(a.weight + g0 + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float u = x[k][i] * silu(z[k][i]);
                    ss[0] = __builtin_fmaf(u, u, ss[0]);
                    ss[1] = __builtin_fmaf(dy[k][i] * w[i], u, ss[1]);
                }
            }
        }
        double sum[2];
        row_sum<TPR, 2>(ss, sum, sh, turn);
        const float rstd = inv_rms(sum[0], inv, a.eps);
        const float m = (float)(sum[1] * inv) * rstd;  // mean(g hat)
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)Dg - c;
            if (left > 0) {
                float w[kVec], dx[kVec], dz[kVec];
                ld_vec<ODD>(a.weight + g0 + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float s = sigmoid(z[k][i]), gate = z[k][i] * s, u = x[k][i] * gate;
                    const float hat = u * rstd;
                    dw[k][i] = __builtin_fmaf(dy[k][i], hat, dw[k][i]);
                    const float du = rstd * __builtin_fmaf(-m, hat, dy[k][i] * w[i]);
                    dx[i] = du * gate;
                    // silu'(z) = s + z s (1 - s)
                    dz[i] = du * x[k][i] * __builtin_fmaf(gate, 1.0f - s, s);
                }
                st_vec<ODD>((T *)a.dx + row * D + g0 + c, left, dx);
                st_vec<ODD>((T *)a.dz + row * a.dz_stride + g0 + c, left, dz);
            }
        }
    }
    write_partial<TPR, ODD, ITER>(dw, cols, a.part + (int64_t)blockIdx.x * D + g0, Dg);
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
hipError_t add_fwd_n(const AddNormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((add_norm_fwd_kernel<TPR, ODD, ITER, T, R>), dim3(norm_grid(a.rows, TPR, 8192)),
                       dim3(block_threads(TPR)), 0, s, a);
    return hipGetLastError();
}
template <typename T, typename R>
hipError_t add_fwd(const AddNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) add_fwd_n<TPR, ODD, ITER, T, R>(a, s)
    SSM_NORM_DISPATCH(a.D, a.D % 8 == 0, false, SSM_CALL);
#undef SSM_CALL
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
hipError_t add_bwd_n(const AddNormArgs &a, hipStream_t s) {
    const unsigned g = norm_grid(a.rows, TPR, kNormBwdBlocks);
    hipLaunchKernelGGL((add_norm_bwd_kernel<TPR, ODD, ITER, T, R>), dim3(g), dim3(block_threads(TPR)), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_reduce(a.part, g, a.D, {{a.dweight, a.scale ? a.dscale : nullptr}}, s);
}
template <typename T, typename R>
hipError_t add_bwd(const AddNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) add_bwd_n<TPR, ODD, ITER, T, R>(a, s)
    SSM_NORM_DISPATCH(a.D, a.D % 8 == 0, false, SSM_CALL);
#undef SSM_CALL
}

template <int TPR, bool ODD, int ITER, typename T>
hipError_t gate_fwd_n(const GateNormArgs &a, hipStream_t s) {
    const dim3 grid(norm_grid(a.rows, TPR, 8192), (unsigned)a.groups);
    if (!ODD && a.rows * a.D * (int64_t)sizeof(T) > kStreamBytes)
        hipLaunchKernelGGL((gate_norm_fwd_kernel<TPR, ODD, ITER, T, !ODD>), grid, dim3(block_threads(TPR)), 0, s, a);
    else
        hipLaunchKernelGGL((gate_norm_fwd_kernel<TPR, ODD, ITER, T, false>), grid, dim3(block_threads(TPR)), 0, s, a);
    return hipGetLastError();
}
template <int TPR, bool ODD, int ITER, typename T>
hipError_t gate_bwd_n(const GateNormArgs &a, hipStream_t s) {
    const unsigned g = norm_grid(a.rows, TPR, kNormBwdBlocks);
    hipLaunchKernelGGL((gate_norm_bwd_kernel<TPR, ODD, ITER, T>), dim3(g, (unsigned)a.groups), dim3(block_threads(TPR)),
                       0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_reduce(a.part, g, a.D, {{a.dweight}}, s);
}
// whole 16-byte pieces: the group's width, and the row strides of what is read and written
bool gate_vec(const GateNormArgs &a) {
    return (a.D / a.groups) % 8 == 0 && a.x_stride % 8 == 0 && a.z_stride % 8 == 0 && a.dz_stride % 8 == 0;
}
template <typename T>
hipError_t gate_fwd(const GateNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) gate_fwd_n<TPR, ODD, ITER, T>(a, s)
    SSM_NORM_DISPATCH(a.D / a.groups, gate_vec(a), true, SSM_CALL);
#undef SSM_CALL
}
template <typename T>
hipError_t gate_bwd(const GateNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) gate_bwd_n<TPR, ODD, ITER, T>(a, s)
    SSM_NORM_DISPATCH(a.D / a.groups, gate_vec(a), false, SSM_CALL);
#undef SSM_CALL
}

}  // namespace

// Workgroups of a backward pass, each of which writes one partial row.
int64_t norm_bwd_blocks(int64_t rows) { return rows < kNormBwdBlocks ? rows : kNormBwdBlocks; }

hipError_t launch_add_norm(const AddNormArgs &a, bool backward, int dtype, int res_dtype, hipStream_t s) {
    if (dtype == 0) return backward ? add_bwd<float, float>(a, s) : add_fwd<float, float>(a, s);
    if (res_dtype == 0) return backward ? add_bwd<uint16_t, float>(a, s) : add_fwd<uint16_t, float>(a, s);
    return backward ? add_bwd<uint16_t, uint16_t>(a, s) : add_fwd<uint16_t, uint16_t>(a, s);
}

hipError_t launch_gate_norm(const GateNormArgs &a, bool backward, int dtype, hipStream_t s) {
    if (dtype == 0) return backward ? gate_bwd<float>(a, s) : gate_fwd<float>(a, s);
    return backward ? gate_bwd<uint16_t>(a, s) : gate_fwd<uint16_t>(a, s);
}

}  // namespace ssm
