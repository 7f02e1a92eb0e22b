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
#include <type_traits>

#include "ssm_common.h"
#include "ssm_internal.h"

namespace ssm {

namespace {

typedef float f32x4n __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4n __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8n __attribute__((ext_vector_type(8)));
typedef f32x4n f32x4u __attribute__((aligned(4)));  // at an element's alignment
typedef u32x4n u32x4u __attribute__((aligned(2)));
typedef bf16x8n bf16x8u __attribute__((aligned(2)));

// Rows beyond the last-level cache (256 MB) that a kernel passes over once are
// loaded and stored as data without reuse (STREAM).
constexpr int64_t kStreamBytes = 256ll << 20;

constexpr int kVec = 8;

// kVec consecutive elements as floats. ODD: the row's length or stride is not
// whole 16-byte pieces; the accesses are as wide, at the elements' own alignment
// (the hardware takes any address), and a row's last elements, `left` of them,
// are taken one by one, zeros behind them. Against one element per lane and
// access (us, rows of 84 MB of bfloat16 in all): add norm of 1001 channels
// forward 131 -> 106, backward 371 -> 164, gate norm of 4095 122 -> 69 and
// 366 -> 165; as many rows of 1000 take 95 and 126, 41 and 92.
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void ld_vec(const float *p, int left, float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
        return;
    }
    using Piece = std::conditional_t<ODD, f32x4u, f32x4n>;
    const Piece *q = (const Piece *)p;
    const f32x4n a = STREAM ? __builtin_nontemporal_load(q) : q[0];
    const f32x4n b = STREAM ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void ld_vec(const uint16_t *p, int left, float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? ld_act(p, i) : 0.0f;
        return;
    }
    using Piece = std::conditional_t<ODD, u32x4u, u32x4n>;
    const u32x4n a = STREAM ? __builtin_nontemporal_load((const Piece *)p) : *(const Piece *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void st_vec(float *p, int left, const float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
        return;
    }
    using Piece = std::conditional_t<ODD, f32x4u, f32x4n>;
    const f32x4n a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    Piece *q = (Piece *)p;
    if constexpr (STREAM) {
        __builtin_nontemporal_store(a, q);
        __builtin_nontemporal_store(b, q + 1);
    } else {
        q[0] = a;
        q[1] = b;
    }
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void st_vec(uint16_t *p, int left, const float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) st_act(p, i, v[i]);
        return;
    }
    using Piece = std::conditional_t<ODD, bf16x8u, bf16x8n>;
    bf16x8n o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
    if constexpr (STREAM) __builtin_nontemporal_store(o, (Piece *)p);
    else *(Piece *)p = o;
}

// Sums of NV values over the TPR lanes that share a row, in every one of them.
// A wave adds by lane exchanges; more waves meet through LDS (two buffers in
// turn, so that one barrier per row is enough). In double precision: what rounds
// in the last steps of a tree is a whole row's error, and no other row averages it
// (two rows of 3088 channels, 40 seeds: at most 6.0e-8 of y, 8.0e-8 with float32
// sums and the hardware's root as it is; 1 % of the time of large batches).
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(const float (&part)[NV], double (&v)[NV], double (*sh)[16][NV], int &turn) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = (double)part[i];
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m *= 2)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], m);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) sh[turn][w][i] = v[i];
        __syncthreads();
        if constexpr (TPR <= 512) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = 0.0;
#pragma unroll
                for (int k = 0; k < TPR / 64; ++k) v[i] += sh[turn][k][i];
            }
        } else {  // a lane per wave, four times over: 16 pairs at once cost registers that a workgroup of 16 waves has not
            const int k = threadIdx.x & 15;
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = k < TPR / 64 ? sh[turn][k][i] : 0.0;
#pragma unroll
            for (int m = 1; m < 16; m *= 2)
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], m);
        }
        turn ^= 1;
    }
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// (sum / n + eps)^-1/2 rounded once: its error is a whole row's. The hardware's
// reciprocal root and one step of Newton's in double precision, four
// instructions per row.
__device__ __forceinline__ float inv_rms(double sum, double inv, float eps) {
    const double v = __builtin_fma(sum, inv, (double)eps);
    const double r = (double)rsqrtf((float)v);
    const float rstd = (float)__builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
    return finite(rstd) ? rstd : (float)r;  // of zero, infinity and NaN
}

constexpr int block_threads(int TPR) { return TPR < 256 ? 256 : TPR; }

// Adds a workgroup's column sums (one set per row-sharing group of lanes) in
// the order of the groups and writes them as one partial row of D columns.
template <int TPR, bool ODD, int ITER>
__device__ __forceinline__ void write_partial(const float (&acc)[ITER][kVec], float *sh, float *part, int64_t D) {
    constexpr int RPB = block_threads(TPR) / TPR;
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    for (int w = 0; w < RPB; ++w) {
        if (RPB > 1) __syncthreads();
        if (mine != w) continue;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left <= 0) continue;
            if (RPB == 1) {
                st_vec<ODD>(part + c, left, acc[k]);
            } else {
                float t[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    t[i] = w == 0 ? acc[k][i] : sh[c + i] + acc[k][i];
                    sh[c + i] = t[i];
                }
                if (w == RPB - 1) st_vec<ODD>(part + c, left, t);
            }
        }
    }
    if (RPB > 1) __syncthreads();
}

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

// out[c] = sum over the partial rows, in order: 64 columns per workgroup, 16
// slices of the rows, whose sums are added in the order of the slices.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *part, int64_t nblk, int64_t D, float *out0,
                                                           float *out1) {
    __shared__ float sh[16][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int s = threadIdx.x >> 6;
    const float *p = part + (int64_t)blockIdx.y * nblk * D;
    const int64_t per = (nblk + 15) / 16, lo = s * per, hi = lo + per < nblk ? lo + per : nblk;
    float v = 0.0f;
    if (c < D)
#pragma unroll 8
        for (int64_t i = lo; i < hi; ++i) v += p[i * D + c];
    sh[s][threadIdx.x & 63] = v;
    __syncthreads();
    if (s == 0 && c < D) {
#pragma unroll
        for (int k = 1; k < 16; ++k) v += sh[k][threadIdx.x & 63];
        (blockIdx.y ? out1 : out0)[c] = v;
    }
}

// Lanes per row and elements per lane by the row's length: a wave per row as
// long as it holds at most 24 elements per lane (1536 channels), then a
// workgroup of as many waves as give each lane 8. Short rows share a wave (rows of
// 24 channels, a wave each: add norm 423 us forward and 1146 backward, three
// lanes each: 102 and 195).
//
// Both sides at rows of 84 MB of bfloat16 (float32 residual), us: add norm
// forward / backward, gate norm forward / backward,
//   1536   a wave, 24 per lane       99 133  42  96     3 waves, 8 per lane    97 144  40 135
//   2048   a wave, 32 per lane      103 134  49  98     4 waves                94 132  42 102
//   2560   a wave, 40 per lane      103 137  44 102     5 waves                94 134  40  98
//   4096   4 waves, 16 per lane      94 136  43 107     8 waves                90 133  42  92
//   5120   4 waves, 24 per lane      98 141  44 120     10 waves               93 141  48  93
//   8192   4 waves, 32 per lane     100 138  42 105     16 waves               95 137  41  97
// Only the gate norm's forward pass keeps 4 waves for rows above 4096 (FEW):
// 32768 rows of 5120 channels take 173 us so and 182 with 10 waves.
#define SSM_NORM_ROWS(n, ODD, FEW, CALL)             \
    do {                                             \
        if (n <= 64) return CALL(8, ODD, 1);         \
        if (n <= 128) return CALL(16, ODD, 1);       \
        if (n <= 256) return CALL(32, ODD, 1);       \
        if (n <= 512) return CALL(64, ODD, 1);       \
        if (n <= 1024) return CALL(64, ODD, 2);      \
        if (n <= 1536) return CALL(64, ODD, 3);      \
        if (n <= 2048) return CALL(256, ODD, 1);     \
        if (n <= 2560) return CALL(320, ODD, 1);     \
        if (n <= 4096) return CALL(512, ODD, 1);     \
        if (n > 8192) return CALL(1024, ODD, 2);     \
        if constexpr (FEW) {                         \
            if (n <= 6144) return CALL(256, ODD, 3); \
            return CALL(256, ODD, 4);                \
        } else {                                     \
            if (n <= 5120) return CALL(640, ODD, 1); \
            if (n <= 6144) return CALL(768, ODD, 1); \
            return CALL(1024, ODD, 1);               \
        }                                            \
    } while (0)
#define SSM_NORM_DISPATCH(LEN, EVEN, FEW, CALL)         \
    do {                                                \
        const int64_t n_ = (LEN);                       \
        if (EVEN) SSM_NORM_ROWS(n_, false, FEW, CALL);  \
        else SSM_NORM_ROWS(n_, true, FEW, CALL);        \
    } while (0)

unsigned norm_grid(int64_t rows, int tpr, int64_t cap) {
    const int64_t rpb = tpr < 256 ? 256 / tpr : 1, b = (rows + rpb - 1) / rpb;
    return (unsigned)(b < cap ? b : cap);
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

hipError_t launch_reduce(const float *part, int64_t nblk, int64_t D, float *o0, float *o1, hipStream_t s) {
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((D + 63) / 64), o1 ? 2 : 1), dim3(1024), 0, s, part, nblk, D,
                       o0, o1);
    return hipGetLastError();
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
hipError_t add_bwd_n(const AddNormArgs &a, hipStream_t s) {
    const unsigned g = norm_grid(a.rows, TPR, kNormBwdBlocks);
    hipLaunchKernelGGL((add_norm_bwd_kernel<TPR, ODD, ITER, T, R>), dim3(g), dim3(block_threads(TPR)), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_reduce(a.part, g, a.D, a.dweight, a.scale ? a.dscale : nullptr, s);
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
    return e != hipSuccess ? e : launch_reduce(a.part, g, a.D, a.dweight, nullptr, s);
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
