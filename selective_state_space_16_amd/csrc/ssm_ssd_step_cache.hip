// The SSD decode step on a cache of states for gfx950: one token per request,
// from the layer's projected row (x | B | C before the convolution, and the
// step size before its softplus) to y, with the request's convolution window
// and state updated in place in the cache slot that the request names.
//
//   u[c]    = conv_b[c] + sum_j conv_w[c][j] raw[t-3+j][c],  x | B | C = silu(u)
//   dt      = softplus(dt_raw + dt_bias),   a = exp(dt A)
//   S[p][n] = a S[p][n] + dt x[p] B[n],     y[p] = sum_n C[n] S[p][n] + D x[p]
//
// Two launches. B and C of a request are read by all of its heads, so the
// window can be shifted only when every head has its values: the first kernel
// convolves a request's channels once, writes them (and dt, a) to the
// workspace in float32 and shifts the window; the second reads and writes the
// state, 8 bytes per element of it, which is what bounds the step (HBM).
//
// A slot outside [0, num_slots), or one that an earlier request of the batch
// names, marks a padding row: its y is zeros and no cache entry is touched.
#include "ssm_common.h"
#include "ssm_internal.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kConvPer = 2;  // channels per thread of the convolution

template <int DT>
__global__ __launch_bounds__(kThreads) void step_cache_conv_kernel(SsdCacheArgs a) {
    using T = typename Act<DT>::T;
    const int64_t b = blockIdx.y, C = a.C;
    const int32_t slot = a.slots[b];
    bool dead = slot < 0 || slot >= a.num_slots;
    if (!dead) {
        bool same = false;
        for (int64_t i = threadIdx.x; i < b; i += kThreads) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.ws_slot[b] = dead ? -1 : slot;
    if (dead) return;
    float *row = a.ws_act + b * a.ws_row;
#pragma unroll
    for (int k = 0; k < kConvPer; ++k) {
        const int64_t c = ((int64_t)blockIdx.x * kConvPer + k) * kThreads + threadIdx.x;
        if (c < C) {
            T *win = (T *)a.conv_cache + ((int64_t)slot * C + c) * 3;
            const float xm3 = ld_act(win, 0), xm2 = ld_act(win, 1), xm1 = ld_act(win, 2);
            const float x0 = ld_act((const T *)a.xBC, b * a.xBC_stride + c);
            const float4 w = *(const float4 *)(a.conv_w + 4 * c);
            row[c] = conv_silu(w.x, w.y, w.z, w.w, a.conv_b ? a.conv_b[c] : 0.0f, xm3, xm2, xm1, x0);
            st_act(win, 0, xm2);
            st_act(win, 1, xm1);
            st_act(win, 2, x0);
        } else if (c < C + a.H) {
            const int64_t h = c - C;
            const float dt = softplus(ld_act((const T *)a.dt_raw, b * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
            row[c] = dt;
            row[c + a.H] = fast_exp2(dt * a.A[h] * kLog2e);
        }
    }
}

// One workgroup per (request, head, 64 rows of the state): a state row is N / 4
// lanes of 16 bytes, so every access of a wave covers whole rows; all loads of
// the state are issued before the first use.
template <int N, int DT>
__global__ __launch_bounds__(kThreads) void step_cache_state_kernel(SsdCacheArgs a) {
    using T = typename Act<DT>::T;
    using F4 = float __attribute__((ext_vector_type(4)));
    constexpr int TPR = N / 4, RPP = kThreads / TPR, PASSES = 64 / RPP;
    const int64_t H = a.H, pb = a.P / 64;
    const int64_t id = blockIdx.x, b = id / (H * pb), hp = id % (H * pb), h = hp / pb, g = h / (H / a.G);
    const int tid = threadIdx.x, r0 = tid / TPR, n0 = (tid % TPR) * 4;
    const int32_t slot = a.ws_slot[b];
    const int64_t p0 = (hp % pb) * 64 + r0;  // pass q: row p0 + q RPP
    T *y = (T *)a.y + (b * H + h) * a.P + p0;
    if (slot < 0) {
        if (tid % TPR == 0)
#pragma unroll
            for (int q = 0; q < PASSES; ++q) st_act(y, q * RPP, 0.0f);
        return;
    }
    F4 *S = (F4 *)(a.state_cache + (((int64_t)slot * H + h) * a.P + p0) * N + n0);
    F4 s[PASSES];
#pragma unroll
    for (int q = 0; q < PASSES; ++q) s[q] = S[q * RPP * N / 4];
    const float *row = a.ws_act + b * a.ws_row;
    const float dt = row[a.C + h], av = row[a.C + H + h];
    const F4 B = *(const F4 *)(row + H * a.P + g * N + n0), Cv = *(const F4 *)(row + H * a.P + (a.G + g) * N + n0);
    float xv[PASSES];
#pragma unroll
    for (int q = 0; q < PASSES; ++q) xv[q] = row[h * a.P + p0 + q * RPP];
    const float dsk = a.Dskip ? a.Dskip[h] : 0.0f;
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
        const float dx = dt * xv[q];
        float acc = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = __builtin_fmaf(av, s[q][e], dx * B[e]);
            s[q][e] = v;
            acc = __builtin_fmaf(Cv[e], v, acc);
        }
        S[q * RPP * N / 4] = s[q];
#pragma unroll
        for (int m = 1; m < TPR; m *= 2) acc += __shfl_xor(acc, m);
        if (tid % TPR == 0) st_act(y, q * RPP, a.Dskip ? __builtin_fmaf(dsk, xv[q], acc) : acc);
    }
}

template <int DT>
hipError_t step_cache(const SsdCacheArgs &a, int N, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.C + a.H + kThreads * kConvPer - 1) / (kThreads * kConvPer));
    hipLaunchKernelGGL((step_cache_conv_kernel<DT>), dim3(blocks, (unsigned)a.seqs), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.seqs * a.H * (a.P / 64)));
    if (N == 64) hipLaunchKernelGGL((step_cache_state_kernel<64, DT>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((step_cache_state_kernel<128, DT>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssd_step_cache(const SsdCacheArgs &a, int N, int dtype, hipStream_t s) {
    return dtype == 0 ? step_cache<0>(a, N, s) : step_cache<1>(a, N, s);
}

}  // namespace ssm
