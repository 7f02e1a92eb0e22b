// The short causal convolution and SiLU ahead of a layer, on a cache of windows
// (gfx950): over packed prompts, and over one token per request.
//
//   u[t][c] = conv_b[c] + sum_j conv_w[c][j] raw[t-3+j][c],  y = u / (1 + exp(-u))
//
// The rows before a sequence's first are its slot's window, or zeros; behind its
// last token the slot holds its last three raw rows. Each row of x is read once
// and each of y written once, which is what bounds the prompts (HBM). A lane
// takes the channels of 16 bytes along a run of tokens with the taps and the last
// three rows in registers.
//
// The window is read by the lanes of a sequence's first tokens and written by
// those of its first token, which stand in the same workgroup: a barrier lies
// between. A sequence whose slot is out of range or named by an earlier one is
// left out: zeros in its rows of y, no access to the cache.
#include "ssm_common.h"
#include "ssm_internal.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;  // tokens of a workgroup

// VEC elements as floats; 16 bytes, 8 or one element.
template <int VEC>
__device__ __forceinline__ void ld(const float *p, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const f32x4 a = *(const f32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i];
    } else {
        v[0] = p[0];
    }
}
template <int VEC>
__device__ __forceinline__ void ld(const uint16_t *p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const u32x4 a = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    } else {
        v[0] = ld_act(p, 0);
    }
}
template <int VEC>
__device__ __forceinline__ void st(float *p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
    else p[0] = v[0];
}
template <int VEC>
__device__ __forceinline__ void st(uint16_t *p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        bf16x8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
        *(bf16x8 *)p = o;
    } else {
        st_act(p, 0, v[0]);
    }
}

// Whether sequence (or request) s has no slot of its own. Called by a whole workgroup.
__device__ __forceinline__ bool without_slot(const ConvCacheArgs &a, int64_t s) {
    const int32_t slot = a.slots[s];
    if (slot < 0 || slot >= a.num_slots) return true;
    bool same = false;
    for (int64_t i = threadIdx.x; i < s; i += kThreads) same |= a.slots[i] == slot;
    return __syncthreads_or(same);
}

template <int VEC>
struct Taps {
    float w[4][VEC], b[VEC];
    __device__ __forceinline__ Taps(const ConvCacheArgs &a, int64_t c) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const f32x4 t = *(const f32x4 *)(a.conv_w + 4 * (c + i));
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j][i] = t[j];
            b[i] = a.conv_b ? a.conv_b[c + i] : 0.0f;
        }
    }
    // `past`: the three rows before, oldest first
    __device__ __forceinline__ void at(const float (&past)[3][VEC], const float (&x)[VEC], float (&y)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            y[i] = conv_silu(w[0][i], w[1][i], w[2][i], w[3][i], b[i], past[0][i], past[1][i], past[2][i], x[i]);
    }
};

// A workgroup: one piece of 64 tokens of one sequence, and up to 256 lanes' worth of
// channels; where there are fewer, `per` lanes, the others take other tokens of it.
template <int DT, int VEC>
__global__ __launch_bounds__(kThreads) void conv_cache_kernel(ConvCacheArgs a, int per) {
    using T = typename Act<DT>::T;
    const uint32_t id = blockIdx.x;
    const int s = find_seq(a, id, kTokens);
    if (s < 0) return;
    const uint32_t begin = seq_begin(a, s), len = seq_length(a, s, begin);
    const uint32_t piece = id - (begin / kTokens + s);
    if (piece > 0 && piece * kTokens >= len) return;
    const bool dead = without_slot(a, s);
    const int64_t slot = dead ? 0 : a.slots[s];
    const int subs = kThreads / per, sub = threadIdx.x / per, run = (kTokens + subs - 1) / subs;
    const int64_t c = ((int64_t)blockIdx.y * per + threadIdx.x % per) * VEC;
    const bool mine = sub < subs && c < a.C;
    const int64_t lo = (int64_t)piece * kTokens + sub * run, end = lo + run, most = (int64_t)(piece + 1) * kTokens;
    const int64_t stop = end < most ? end : most, hi = stop < (int64_t)len ? stop : (int64_t)len;
    T *y = (T *)a.y + (int64_t)begin * a.C + c;
    const T *x = (const T *)a.x + (int64_t)begin * a.x_stride + c;
    T *win = (T *)a.conv_cache + (slot * a.C + c) * 3;
    const bool resume = !dead && a.resume && a.resume[s] != 0;
    float past[3][VEC], keep[3][VEC];
    if (dead) {
        const float zero[VEC] = {};
        if (mine)
            for (int64_t t = lo; t < hi; ++t) st<VEC>(y + t * a.C, zero);
        return;
    }
    // the row of token t, or the window's
    auto row = [&](int64_t t, float (&v)[VEC]) {
        if (t >= 0) {
            ld<VEC>(x + t * a.x_stride, v);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = resume ? ld_act(win, i * 3 + 3 + t) : 0.0f;
        }
    };
    const bool keeper = mine && piece == 0 && sub == 0;
    if (mine && lo < hi) {
#pragma unroll
        for (int k = 0; k < 3; ++k) row(lo - 3 + k, past[k]);
    }
    if (keeper) {
#pragma unroll
        for (int k = 0; k < 3; ++k) row((int64_t)len - 3 + k, keep[k]);
    }
    if (piece == 0) __syncthreads();  // everyone has read the window
    if (keeper) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int k = 0; k < 3; ++k) st_act(win, i * 3 + k, keep[k][i]);
    }
    if (!mine || lo >= hi) return;
    const Taps<VEC> taps(a, c);
    constexpr int kAhead = 8;  // rows loaded at once
    int64_t t = lo;
    for (; t + kAhead <= hi; t += kAhead) {
        float raw[kAhead][VEC], out[VEC];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ld<VEC>(x + (t + k) * a.x_stride, raw[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            taps.at(past, raw[k], out);
            st<VEC>(y + (t + k) * a.C, out);
#pragma unroll
            for (int i = 0; i < VEC; ++i) past[0][i] = past[1][i], past[1][i] = past[2][i], past[2][i] = raw[k][i];
        }
    }
    for (; t < hi; ++t) {
        float raw[VEC], out[VEC];
        ld<VEC>(x + t * a.x_stride, raw);
        taps.at(past, raw, out);
        st<VEC>(y + t * a.C, out);
#pragma unroll
        for (int i = 0; i < VEC; ++i) past[0][i] = past[1][i], past[1][i] = past[2][i], past[2][i] = raw[i];
    }
}

// One token per request: a lane takes a channel, its window three values.
template <int DT>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvCacheArgs a) {
    using T = typename Act<DT>::T;
    const int64_t b = blockIdx.y, c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool dead = without_slot(a, b);
    if (c >= a.C) return;
    T *y = (T *)a.y + b * a.C;
    if (dead) {
        st_act(y, c, 0.0f);
        return;
    }
    T *win = (T *)a.conv_cache + ((int64_t)a.slots[b] * a.C + c) * 3;
    const T raw = ((const T *)a.x)[b * a.x_stride + c], w1 = win[1], w2 = win[2];
    const Taps<1> taps(a, c);
    const float past[3][1] = {{ld_act(win, 0)}, {ld_act(&w1, 0)}, {ld_act(&w2, 0)}}, x[1] = {ld_act(&raw, 0)};
    float out[1];
    taps.at(past, x, out);
    st_act(y, c, out[0]);
    win[0] = w1;
    win[1] = w2;
    win[2] = raw;
}

template <int DT, int VEC>
hipError_t conv_prompt(const ConvCacheArgs &a, hipStream_t s) {
    const int64_t lanes = (a.C + VEC - 1) / VEC;
    const int per = (int)(lanes < kThreads ? lanes : kThreads);
    const dim3 grid((unsigned)(a.rows / kTokens + a.seqs), (unsigned)((lanes + per - 1) / per));
    hipLaunchKernelGGL((conv_cache_kernel<DT, VEC>), grid, dim3(kThreads), 0, s, a, per);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_cache(const ConvCacheArgs &a, bool prompt, int dtype, hipStream_t s) {
    if (!prompt) {
        const dim3 grid((unsigned)((a.C + kThreads - 1) / kThreads), (unsigned)a.seqs);
        if (dtype == 0) hipLaunchKernelGGL((conv_step_kernel<0>), grid, dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((conv_step_kernel<1>), grid, dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    // 16 bytes per access where every row is whole pieces of them, else one element. 32768
    // tokens, us: bfloat16, 8192 channels 225 (rows 8256 apart 246), by one element 261 (rows
    // 8193 apart) and 302 (8191 channels); float32, 4096 channels 221, 4097 by one element 293.
    if (dtype == 0) return a.C % 4 == 0 && a.x_stride % 4 == 0 ? conv_prompt<0, 4>(a, s) : conv_prompt<0, 1>(a, s);
    return a.C % 8 == 0 && a.x_stride % 8 == 0 ? conv_prompt<1, 8>(a, s) : conv_prompt<1, 1>(a, s);
}

}  // namespace ssm
