// The gated delta rule for one token per request on a cache of states (gfx950),
// each state updated in place in the slot that its request names.
//
//   q' = q scale / sqrt(|q|^2 + eps),  k' = k / sqrt(|k|^2 + eps)
//   a  = exp(softplus(dt_raw + dt_bias) A),  beta = 1 / (1 + exp(-beta_raw))
//   u[p]    = beta (v[p] - a sum_n S[p][n] k'[n])
//   S[p][n] = a S[p][n] + u[p] k'[n],   y[p] = sum_n S[p][n] q'[n]
//
// With S the old state, y = a S q' + u (k'.q'), so S k' and S q' come from one pass
// over the registers that hold a state row. Reading and writing the states, 8 bytes
// per element, bounds the step (HBM). A workgroup takes 64 rows of one head's state:
// eight lanes per row, pieces of 16 bytes of the row in turn, so that a row's sums
// need three exchanges.
//
// A slot outside [0, num_slots), or one that an earlier request of the batch names,
// marks a padding row: its y is zeros and no cache entry is touched.
#include "ssm_delta_device.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

constexpr int kThreads = 256, kLanes = 8, kRows = 64, kPasses = kRows / (kThreads / kLanes);
constexpr int64_t kStreamBytes = 400ll << 20;  // of states: see delta_step_kernel

__device__ __forceinline__ f32x4 ld4(const float *p) { return *(const f32x4 *)p; }
__device__ __forceinline__ f32x4 ld4(const uint16_t *p) {
    const uint2 v = *(const uint2 *)p;
    return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                 __uint_as_float(v.y & 0xffff0000u)};
}

// STREAM: the states do not fit the last-level cache (256 MB) and are loaded and
// stored as data without reuse.
template <int N, int DT, bool STREAM>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(DeltaArgs a) {
    using T = typename Act<DT>::T;
    constexpr int PIECES = N / (4 * kLanes);
    const int64_t H = a.H, pb = a.P / kRows;
    const int64_t id = blockIdx.x, b = id / (H * pb), hp = id % (H * pb), h = hp / pb, g = h / (H / a.G);
    const int tid = threadIdx.x, lane = tid % kLanes, n0 = lane * 4;
    const int64_t p0 = (hp % pb) * kRows + tid / kLanes;  // pass r: row p0 + r kThreads / kLanes
    const int32_t slot = a.slots[b];
    bool dead = slot < 0 || slot >= a.num_slots;
    T *y = (T *)a.y + (b * H + h) * a.P + p0;
    f32x4 *S = (f32x4 *)(a.state_cache + (((int64_t)(dead ? 0 : slot) * H + h) * a.P + p0) * N + n0);
    constexpr int kNext = kThreads / kLanes * N / 4;  // 16-byte pieces from pass to pass
    f32x4 s[kPasses][PIECES];
    if (!dead) {
#pragma unroll
        for (int r = 0; r < kPasses; ++r)
#pragma unroll
            for (int j = 0; j < PIECES; ++j)
                s[r][j] = STREAM ? __builtin_nontemporal_load(&S[r * kNext + j * kLanes]) : S[r * kNext + j * kLanes];
        bool same = false;
        for (int64_t i = tid; i < b; i += kThreads) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (dead) {
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < kPasses; ++r) st_act(y, r * (kThreads / kLanes), 0.0f);
        return;
    }
    const T *qp = (const T *)a.q + b * a.q_stride + g * N + n0, *kp = (const T *)a.k + b * a.k_stride + g * N + n0;
    f32x4 q[PIECES], k[PIECES];
#pragma unroll
    for (int j = 0; j < PIECES; ++j) q[j] = ld4(qp + 4 * kLanes * j), k[j] = ld4(kp + 4 * kLanes * j);
    float v[kPasses];
#pragma unroll
    for (int r = 0; r < kPasses; ++r) v[r] = ld_act((const T *)a.v + b * a.v_stride + h * a.P, p0 + r * (kThreads / kLanes));
    const float dt = softplus(ld_act((const T *)a.dt_raw, b * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
    const float beta = delta_gate(ld_act((const T *)a.beta_raw, b * a.beta_stride + h));
    const float decay = fast_exp2(dt * a.A[h] * kLog2e);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            kk = __builtin_fmaf(k[j][e], k[j][e], kk);
            qq = __builtin_fmaf(q[j][e], q[j][e], qq);
        }
    const float rk = unit_scale(sum8(kk), a.norm_eps), rq = unit_scale(sum8(qq), a.norm_eps) * a.scale;
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[j][e] *= rk;
            q[j][e] *= rq;
            kq = __builtin_fmaf(k[j][e], q[j][e], kq);
        }
    kq = sum8(kq);
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
        float sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[r][j][e] *= decay;
                sk = __builtin_fmaf(s[r][j][e], k[j][e], sk);
                sq = __builtin_fmaf(s[r][j][e], q[j][e], sq);
            }
        const float u = beta * (v[r] - sum8(sk));
        sq = __builtin_fmaf(u, kq, sum8(sq));
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[r][j][e] = __builtin_fmaf(u, k[j][e], s[r][j][e]);
            if (STREAM) __builtin_nontemporal_store(s[r][j], &S[r * kNext + j * kLanes]);
            else S[r * kNext + j * kLanes] = s[r][j];
        }
        if (lane == 0) st_act(y, r * (kThreads / kLanes), sq);
    }
}

template <int N, int DT>
hipError_t delta_step(const DeltaArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)(a.seqs * a.H * (a.P / kRows)));
    if (a.seqs * a.H * a.P * N * 4 > kStreamBytes)
        hipLaunchKernelGGL((delta_step_kernel<N, DT, true>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((delta_step_kernel<N, DT, false>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs &a, int N, int dtype, hipStream_t s) {
    if (dtype == 0) return N == 64 ? delta_step<64, 0>(a, s) : delta_step<128, 0>(a, s);
    return N == 64 ? delta_step<64, 1>(a, s) : delta_step<128, 1>(a, s);
}

}  // namespace ssm
