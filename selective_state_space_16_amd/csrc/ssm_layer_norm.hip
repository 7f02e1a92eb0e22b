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
// norms, and summed twice: first for its mean (and that of g), then the squares of
// what is left (and g times it). The variance as a difference of two sums would
// take one pass over registers instead of two, and lose a row whose mean is large
// against its spread; for the same reason the second pass also sums what the
// first mean's rounding left, and takes it off (where mean / spread is 2^12, the
// mean's last bit alone is 2^-12 of y). HBM bounds both passes: each input is read once, each output
// written once.
//
// dw, db and dscale sum over all rows: a workgroup keeps its rows' sums in
// registers and writes one partial row of each, a second kernel adds them in
// order. Equal inputs give equal bits.
#include "ssm_internal.h"
#include "ssm_norm_rows.h"

namespace ssm {

namespace {

template <int TPR, bool ODD, int ITER, typename T, typename R>
__global__ __launch_bounds__(block_threads(TPR)) void layer_norm_fwd_kernel(LayerNormArgs a) {
    constexpr int RPB = block_threads(TPR) / TPR;
    __shared__ double sh[2][16][1], sh2[2][16][2];
    int turn = 0;
    const int lane = threadIdx.x % TPR;
    const int64_t D = a.D;
    const double inv = 1.0 / (double)D;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        const int64_t base = row * D;
        float r[ITER][kVec], part[1] = {0.0f}, part2[2] = {0.0f, 0.0f};
        double sum[1], sum2[2];
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
                    part[0] += r[k][i];
                }
            }
        }
        row_sum<TPR, 1>(part, sum, sh, turn);
        const float mean = (float)(sum[0] * inv);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                if (a.residual_out) st_vec<ODD>((R *)a.residual_out + base + c, left, r[k]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    r[k][i] = ODD && i >= left ? 0.0f : r[k][i] - mean;
                    part2[0] = __builtin_fmaf(r[k][i], r[k][i], part2[0]);
                    part2[1] += r[k][i];
                }
            }
        }
        row_sum<TPR, 2>(part2, sum2, sh2, turn);
        const double low = sum2[1] * inv;  // what the rounding of the mean left
        const float rstd = inv_rms(sum2[0] - low * sum2[1], inv, a.eps), rest = (float)low;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec], b[kVec], y[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
                if (a.bias) ld_vec<ODD>(a.bias + c, left, b);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float hat = (r[k][i] - rest) * rstd;
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
    __shared__ double sh[2][16][2], sh3[2][16][3];
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
        float r[ITER][kVec], dy[ITER][kVec], part[2] = {0.0f, 0.0f}, part3[3] = {0.0f, 0.0f, 0.0f};
        double sum[2], sum3[3];
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
                    part[0] += r[k][i];
                    part[1] = __builtin_fmaf(dy[k][i], w[i], part[1]);
                }
            }
        }
        row_sum<TPR, 2>(part, sum, sh, turn);
        const float mean = (float)(sum[0] * inv), mg = (float)(sum[1] * inv);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left > 0) {
                float w[kVec];
                ld_vec<ODD>(a.weight + c, left, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    r[k][i] = ODD && i >= left ? 0.0f : r[k][i] - mean;
                    part3[0] = __builtin_fmaf(r[k][i], r[k][i], part3[0]);
                    part3[1] = __builtin_fmaf(dy[k][i] * w[i], r[k][i], part3[1]);
                    part3[2] += r[k][i];
                }
            }
        }
        row_sum<TPR, 3>(part3, sum3, sh3, turn);
        const double low = sum3[2] * inv;  // what the rounding of the mean left
        const float rstd = inv_rms(sum3[0] - low * sum3[2], inv, a.eps), rest = (float)low;
        const float mh = (float)((sum3[1] - low * sum[1]) * inv) * rstd;  // mean(g hat)
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
                    const float hat = (r[k][i] - rest) * rstd;
                    dw[k][i] = __builtin_fmaf(dy[k][i], hat, dw[k][i]);
                    db[k][i] += dy[k][i];
                    float v = rstd * __builtin_fmaf(-mh, hat, __builtin_fmaf(dy[k][i], w[i], -mg));
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
