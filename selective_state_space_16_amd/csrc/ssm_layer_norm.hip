// The residual sum and the layer norm ahead of a block for gfx950, forward and
// backward.
//
//   r = residual + scale o x;   m = mean r,  rstd = (mean (r - m)^2 + eps)^-1/2
//   y = (r - m) rstd w + b
//
// Backward, with g = dy w and hat = (r - m) rstd:
//   dr = rstd (g - mean g - hat mean(g hat)) + dres,   dx = scale o dr,
//   dw = sum over rows of dy hat,   db = sum over rows of dy,   dscale = sum of dr x.
//
// A row is held in registers by the lanes that read it, as in the root-mean-square
// norms. The variance as a difference of two sums over the whole row would lose a row
// whose mean is large against its spread, and two sums one after the other cost a
// barrier more where several waves share a row; so each wave takes its own elements'
// mean off first, and what the waves found is joined at one barrier (row_stats). Each input is read once and each output written once.
// Measured, against 5.4 TB/s of a large copy:
//   layer norm 32768 x 2560   backward 392 us, bfloat16 with float32 sums and a scale,
//                             1.51 GB, 3.9 TB/s (the root-mean-square norm's 291)
//   layer norm 32768 x 2560   forward 221 us, bfloat16 with a float32 residual, 1.01 GB,
//                             4.6 TB/s (the root-mean-square norm's 195); float32 265,
//                             5.1 TB/s; bfloat16 without a residual 133, 2.5 TB/s
//   layer norm 4097 x 1001    forward 9.0 us, float32, 33 MB: every row is on the chip at
//                             once, so the time is one row's chain of loads and sums
// The backward pass is bound by its 158 registers per lane, which leave two workgroups of
// five waves a CU to hide a row's loads and sums: held to 128 it spills (590 us), with the
// next row's loads ahead it takes 182 (455 us).
//
// dw, db and dscale sum over all rows: a workgroup keeps its rows' sums in
// registers and writes one partial row of each, a second kernel adds them in
// order. Equal inputs give equal bits.
#include "ssm_internal.h"
#include "ssm_norm_rows.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

// The lanes that share a row each take its elements' part (cnt of them in a wave, or in
// the row's lanes where they are fewer) less a centre of their own wave, near its mean:
// part = sums of d = r - centre, of d^2, and of g and g d in the backward pass. From
// these the row's statistics, exactly as from one centre:
//   mean   = (sum over waves of (sum d + cnt centre)) / D
//   spread = sum over waves of (sum d^2 - 2 e sum d + cnt e^2),  e = mean - centre
//   sum g (r - mean) = sum over waves of (sum g d - e sum g)
// for one barrier per row. The squares are added in double precision (what rounds in
// the last steps of a tree is a whole row's error), and so are the means; sums that are
// small beside what they are taken from (of d, and of g and g d for the means that the
// gradient takes off) in float32: 32768 x 2560 backward 415 us with all four in double.
struct RowStats {
    float rest, rstd, mg, mh;  // mean - centre, 1 / sd, mean(g), mean(g hat)
};
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_addf(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <int TPR>
__device__ __forceinline__ double lanes_sum(double v) {
    if constexpr (TPR >= 64) {
        const uint64_t u = __builtin_bit_cast(uint64_t, wave_prefix_sum(v));
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, 63), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), 63);
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    } else {
#pragma unroll
        for (int m = 1; m < TPR; m *= 2) v += __shfl_xor(v, m);
        return v;
    }
}
template <int TPR>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (TPR >= 64) {  // wave_prefix_sum's steps
        v = dpp_addf<0x111, 0xF>(v);
        v = dpp_addf<0x112, 0xF>(v);
        v = dpp_addf<0x114, 0xF>(v);
        v = dpp_addf<0x118, 0xF>(v);
        v = dpp_addf<0x142, 0xA>(v);
        v = dpp_addf<0x143, 0xC>(v);
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
    } else {
#pragma unroll
        for (int m = 1; m < TPR; m *= 2) v += __shfl_xor(v, m);
        return v;
    }
}
// What a wave knows of a row: sums of d^2, d, g and g d, its centre and number of elements.
struct Share {
    double dd;
    float d, centre, cnt, g, gd, pad;
};
template <int TPR, int NV>
__device__ __forceinline__ RowStats row_stats(const float (&part)[NV], float centre, float cnt, Share (*sh)[16], int &turn,
                                              double inv, float eps) {
    Share own{};
    own.dd = lanes_sum<TPR>((double)part[1]);
    own.d = lanes_sum<TPR>(part[0]);
    own.centre = centre;
    own.cnt = cnt;
    if constexpr (NV == 4) own.g = lanes_sum<TPR>(part[2]), own.gd = lanes_sum<TPR>(part[3]);
    double mean, spread = 0.0;
    float g = 0.0f, gd = 0.0f;
    auto sum = [&](const Share &p) { return (double)p.d + (double)p.cnt * p.centre; };
    auto add = [&](const Share &p) {
        const double e = mean - p.centre;
        spread += p.dd - e * (2.0 * p.d - p.cnt * e);
        if constexpr (NV == 4) g += p.g, gd += __builtin_fmaf(-(float)e, p.g, p.gd);
    };
    if constexpr (TPR <= 64) {
        mean = sum(own) * inv;
        add(own);
    } else {
        constexpr int WAVES = TPR / 64;
        if ((threadIdx.x & 63) == 0) sh[turn][threadIdx.x >> 6] = own;
        __syncthreads();
        double all = 0.0;
        if constexpr (WAVES <= 8) {
#pragma unroll
            for (int k = 0; k < WAVES; ++k) all += sum(sh[turn][k]);
            mean = all * inv;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) add(sh[turn][k]);
        } else {  // a lane per wave, four times over, as row_sum does
            const int k = threadIdx.x & 15;
            Share p{};
            if (k < WAVES) p = sh[turn][k];
            all = sum(p);
#pragma unroll
            for (int m = 1; m < 16; m *= 2) all += __shfl_xor(all, m);
            mean = all * inv;
            add(p);
#pragma unroll
            for (int m = 1; m < 16; m *= 2) {
                spread += __shfl_xor(spread, m);
                if constexpr (NV == 4) g += __shfl_xor(g, m), gd += __shfl_xor(gd, m);
            }
        }
        turn ^= 1;
    }
    RowStats s;
    s.rest = (float)(mean - (double)centre);
    s.rstd = inv_rms(spread > 0.0 || spread != spread ? spread : 0.0, inv, eps);
    s.mg = g * (float)inv;
    s.mh = gd * (float)inv * s.rstd;
    return s;
}

// A wave's (or a row's fewer lanes') centre and number of elements.
template <int TPR, int ITER>
__device__ __forceinline__ void row_centre(float sum, int64_t D, float &centre, float &cnt) {
    constexpr int LANES = TPR < 64 ? TPR : 64;
    sum = lanes_sum<TPR>(sum);
    const int base = TPR > 64 ? (int)(threadIdx.x % TPR) / 64 * 64 : 0;
    int n = 0;
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
        const int left = (int)D - (k * TPR + base) * kVec;
        n += left < 0 ? 0 : left < LANES * kVec ? left : LANES * kVec;
    }
    cnt = (float)n;
    centre = n > 0 ? sum / cnt : 0.0f;
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
__global__ __launch_bounds__(block_threads(TPR)) void layer_norm_fwd_kernel(LayerNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ Share sh[2][16];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const int64_t base = row * D;
        float r[ITER][kVec], sum = 0.0f, part[2] = {0.0f, 0.0f}, centre, cnt;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float x[kVec], s[kVec];
                ld_vec<ODD>((const T *)a.x + base + c, left, x);
                if (a.residual) ld_vec<ODD>((const R *)a.residual + base + c, left, r[k]);
                if (a.scale) ld_vec<ODD>(a.scale + c, left, s);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float add = a.scale ? s[i] * x[i] : x[i];
                    r[k][i] = a.residual ? r[k][i] + add : add;
                    sum += r[k][i];
                }
            }
        }
        row_centre<TPR, ITER>(sum, D, centre, cnt);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                if (a.residual_out) st_vec<ODD>((R *)a.residual_out + base + c, left, r[k]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    r[k][i] = ODD && i >= left ? 0.0f : r[k][i] - centre;
                    part[0] += r[k][i];
                    part[1] = __builtin_fmaf(r[k][i], r[k][i], part[1]);
                }
            }
        }
        const RowStats st = row_stats<TPR, 2>(part, centre, cnt, sh, turn, inv, a.eps);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec], b[kVec], y[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
                if (a.bias) ld_vec<ODD>(a.bias + c, left, b);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float hat = (r[k][i] - st.rest) * st.rstd;
                    y[i] = a.bias ? __builtin_fmaf(hat, w[i], b[i]) : hat * w[i];
                }
                st_vec<ODD>((T *)a.y + base + c, left, y);
            }
        }
    }
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
__global__ __launch_bounds__(block_threads(TPR)) void layer_norm_bwd_kernel(LayerNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ Share sh[2][16];
    __shared__ float cols[RPB > 1 ? TPR * kVec * ITER : 1];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    float dw[ITER][kVec], db[ITER][kVec], ds[ITER][kVec];
#pragma unroll
    for (int k = 0; k < ITER; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dw[k][i] = db[k][i] = ds[k][i] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const int64_t base = row * D;
        float r[ITER][kVec], dy[ITER][kVec], sum = 0.0f, part[4] = {0.0f, 0.0f, 0.0f, 0.0f}, centre, cnt;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                ld_vec<ODD>((const R *)a.residual + base + c, left, r[k]);
                ld_vec<ODD>((const T *)a.dy + base + c, left, dy[k]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) sum += r[k][i];
            }
        }
        row_centre<TPR, ITER>(sum, D, centre, cnt);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float g = dy[k][i] * w[i];
                    r[k][i] = ODD && i >= left ? 0.0f : r[k][i] - centre;
                    part[0] += r[k][i];
                    part[1] = __builtin_fmaf(r[k][i], r[k][i], part[1]);
                    part[2] += g;
                    part[3] = __builtin_fmaf(g, r[k][i], part[3]);
                }
            }
        }
        const RowStats st = row_stats<TPR, 4>(part, centre, cnt, sh, turn, inv, a.eps);
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
                    const float hat = (r[k][i] - st.rest) * st.rstd;
                    dw[k][i] = __builtin_fmaf(dy[k][i], hat, dw[k][i]);
                    db[k][i] += dy[k][i];
                    float v = st.rstd * __builtin_fmaf(-st.mh, hat, __builtin_fmaf(dy[k][i], w[i], -st.mg));
                    if (a.dres) v += up[i];
                    dr[i] = v;
                    if (a.scale) {
                        dx[i] = v * s[i];
                        ds[k][i] = __builtin_fmaf(v, x[i], ds[k][i]);
                    } else {
                        dx[i] = v;
                    }
                }
                if (a.residual_out) st_vec<ODD>((R *)a.residual_out + base + c, left, dr);
                st_vec<ODD>((T *)a.dx + base + c, left, dx);
            }
        }
    }
    const int64_t set = (int64_t)gridDim.x * D;
    float *part = a.part + (int64_t)blockIdx.x * D;
    write_partial<TPR, ODD, ITER>(dw, cols, part, D);
    write_partial<TPR, ODD, ITER>(db, cols, part + set, D);
    if (a.scale) write_partial<TPR, ODD, ITER>(ds, cols, part + 2 * set, D);
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
hipError_t layer_fwd_n(const LayerNormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((layer_norm_fwd_kernel<TPR, ODD, ITER, T, R>), dim3(norm_grid(a.rows, TPR, 8192)),
                       dim3(block_threads(TPR)), 0, s, a);
    return hipGetLastError();
}
template <typename T, typename R>
hipError_t layer_fwd(const LayerNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) layer_fwd_n<TPR, ODD, ITER, T, R>(a, s)
    SSM_NORM_DISPATCH(a.D, a.D % 8 == 0, false, SSM_CALL);
#undef SSM_CALL
}

template <int TPR, bool ODD, int ITER, typename T, typename R>
hipError_t layer_bwd_n(const LayerNormArgs &a, hipStream_t s) {
    const unsigned g = norm_grid(a.rows, TPR, kNormBwdBlocks);
    hipLaunchKernelGGL((layer_norm_bwd_kernel<TPR, ODD, ITER, T, R>), dim3(g), dim3(block_threads(TPR)), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_reduce(a.part, g, a.D, {{a.dweight, a.dbias, a.scale ? a.dscale : nullptr}}, s);
}
template <typename T, typename R>
hipError_t layer_bwd(const LayerNormArgs &a, hipStream_t s) {
#define SSM_CALL(TPR, ODD, ITER) layer_bwd_n<TPR, ODD, ITER, T, R>(a, s)
    SSM_NORM_DISPATCH(a.D, a.D % 8 == 0, false, SSM_CALL);
#undef SSM_CALL
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs &a, bool backward, int dtype, int res_dtype, hipStream_t s) {
    if (dtype == 0) return backward ? layer_bwd<float, float>(a, s) : layer_fwd<float, float>(a, s);
    if (res_dtype == 0) return backward ? layer_bwd<uint16_t, float>(a, s) : layer_fwd<uint16_t, float>(a, s);
    return backward ? layer_bwd<uint16_t, uint16_t>(a, s) : layer_fwd<uint16_t, uint16_t>(a, s);
}

}  // namespace ssm
