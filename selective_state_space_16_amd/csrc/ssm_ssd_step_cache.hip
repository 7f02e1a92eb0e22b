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
constexpr int64_t kStreamBytes = 400ll << 20;  // of states: see step_cache_state_kernel
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Four values of the activation type: 8 or 16 bytes.
__device__ __forceinline__ f32x4 ld4(const float *p) { return *(const f32x4 *)p; }
__device__ __forceinline__ f32x4 ld4(const uint16_t *p) {
    const uint2 v = *(const uint2 *)p;
    return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                 __uint_as_float(v.y & 0xffff0000u)};
}
__device__ __forceinline__ void st4(float *p, f32x4 v) { *(f32x4 *)p = v; }
__device__ __forceinline__ void st4(uint16_t *p, f32x4 v) {  // values that are bfloat16 already
    uint2 o;
    o.x = __float_as_uint(v[0]) >> 16 | (__float_as_uint(v[1]) & 0xffff0000u);
    o.y = __float_as_uint(v[2]) >> 16 | (__float_as_uint(v[3]) & 0xffff0000u);
    *(uint2 *)p = o;
}

// A thread takes four neighbouring channels: their windows are twelve
// consecutive values, read and written as three pieces (256 requests of 5376
// channels: 8.6 us; a channel per thread took 12.1).
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
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x, c = id * 4;
    if (c < C) {
        T *win = (T *)a.conv_cache + ((int64_t)slot * C + c) * 3;
        const f32x4 p = ld4(win), q = ld4(win + 4), r = ld4(win + 8), x = ld4((const T *)a.xBC + b * a.xBC_stride + c);
        const float past[12] = {p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3], r[0], r[1], r[2], r[3]};
        const f32x4 bias = a.conv_b ? *(const f32x4 *)(a.conv_b + c) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f32x4 w = *(const f32x4 *)(a.conv_w + 4 * (c + k));
            v[k] = conv_silu(w[0], w[1], w[2], w[3], bias[k], past[3 * k], past[3 * k + 1], past[3 * k + 2], x[k]);
        }
        *(f32x4 *)(row + c) = v;
        st4(win, f32x4{past[1], past[2], x[0], past[4]});
        st4(win + 4, f32x4{past[5], x[1], past[7], past[8]});
        st4(win + 8, f32x4{x[2], past[10], past[11], x[3]});
    } else if (id - C / 4 < a.H) {
        const int64_t h = id - C / 4;
        const float dt = softplus(ld_act((const T *)a.dt_raw, b * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
        row[C + h] = dt;
        row[C + a.H + h] = fast_exp2(dt * a.A[h] * kLog2e);
    }
}

// One workgroup per (request, head, 64 rows of the state): a state row is N / 4
// lanes of 16 bytes, so every access of a wave covers whole rows; all loads of
// the state are issued before the first use.
//
// STREAM: the states do not fit the last-level cache (256 MB), where lines that
// are kept only push each other out; they are loaded and stored as data without
// reuse. Whole steps at 80 heads with 64 x 128 states, called over and over:
// 256 requests (671 MB of states) 275 -> 251 us (5.5 TB/s), 192 requests
// 207 -> 188; but 128 requests (336 MB) 122 -> 126 and 64 (168 MB) 56 -> 65,
// where the last step's states are still there in part or whole.
template <int N, int DT, bool STREAM>
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
    for (int q = 0; q < PASSES; ++q) s[q] = STREAM ? __builtin_nontemporal_load(&S[q * RPP * N / 4]) : S[q * RPP * N / 4];
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
        if (STREAM) __builtin_nontemporal_store(s[q], &S[q * RPP * N / 4]);
        else S[q * RPP * N / 4] = s[q];
#pragma unroll
        for (int m = 1; m < TPR; m *= 2) acc += __shfl_xor(acc, m);
        if (tid % TPR == 0) st_act(y, q * RPP, a.Dskip ? __builtin_fmaf(dsk, xv[q], acc) : acc);
    }
}

template <int N, int DT>
hipError_t step_cache_state(const SsdCacheArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)(a.seqs * a.H * (a.P / 64)));
    if (a.seqs * a.H * a.P * N * 4 > kStreamBytes)
        hipLaunchKernelGGL((step_cache_state_kernel<N, DT, true>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((step_cache_state_kernel<N, DT, false>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t step_cache(const SsdCacheArgs &a, int N, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.C / 4 + a.H + kThreads - 1) / kThreads);
    hipLaunchKernelGGL((step_cache_conv_kernel<DT>), dim3(blocks, (unsigned)a.seqs), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return N == 64 ? step_cache_state<64, DT>(a, s) : step_cache_state<128, DT>(a, s);
}

}  // namespace

hipError_t launch_ssd_step_cache(const SsdCacheArgs &a, int N, int dtype, hipStream_t s) {
    return dtype == 0 ? step_cache<0>(a, N, s) : step_cache<1>(a, N, s);
}

}  // namespace ssm
