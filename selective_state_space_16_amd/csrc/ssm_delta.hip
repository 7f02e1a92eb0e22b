// The gated delta rule over packed prompts, on a cache of states (gfx950):
// sequences of different lengths lie one behind the other in one array of rows,
// each starts from zero or from the state in its cache slot, and leaves it there.
//
//   q' = q scale / sqrt(|q|^2 + eps),  k' = k / sqrt(|k|^2 + eps)
//   a  = exp(softplus(dt_raw + dt_bias) A),  beta = 1 / (1 + exp(-beta_raw))
//   u[p]    = beta (v[p] - a sum_n S[p][n] k'[n])
//   S[p][n] = a S[p][n] + u[p] k'[n],   y[p] = sum_n S[p][n] q'[n]
//
// The rows p of a state never meet: a wave walks a sequence with 16 of them, a lane
// with N / 4 elements of one row.
#include "ssm_delta_device.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

constexpr int kCols = 16;  // state rows p of a wave

// Which slot each sequence owns, -1 for none.
__global__ __launch_bounds__(256) void delta_slots_kernel(DeltaArgs a) {
    const int64_t s = blockIdx.x;
    const int32_t slot = a.slots[s];
    bool dead = slot < 0 || slot >= a.num_slots;
    if (!dead) {
        bool same = false;
        for (int64_t i = threadIdx.x; i < s; i += 256) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (threadIdx.x == 0) a.ws_slot[s] = dead ? -1 : slot;
}

// Eight bfloat16 as floats.
__device__ __forceinline__ void ld8(const uint16_t *p, float *v) {
    const u32x4 u = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// v summed over the four lanes that share a state row.
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <int N>
__global__ __launch_bounds__(64) void delta_walk_kernel(DeltaArgs a) {
    constexpr int KB = N / 32;
    const int64_t h = blockIdx.y, s = blockIdx.z, g = h / (a.H / a.G);
    const int lane = threadIdx.x, grp = lane >> 4;
    const int64_t p = (int64_t)blockIdx.x * kCols + (lane & 15);
    const uint32_t begin = seq_begin(a, s), len = seq_length(a, s, begin);
    const int32_t slot = a.ws_slot[s];
    uint16_t *y = (uint16_t *)a.y + ((int64_t)begin * a.H + h) * a.P + p;
    if (slot < 0) {
        if (grp == 0)
            for (uint32_t t = 0; t < len; ++t) y[(int64_t)t * a.H * a.P] = 0;
        return;
    }
    float *cache = a.state_cache + (((int64_t)slot * a.H + h) * a.P + p) * N + 8 * grp;
    const bool resume = a.resume && a.resume[s] != 0;
    float S[KB][8];  // n = 32 b + 8 grp + e
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) S[b][e] = resume ? cache[32 * b + e] : 0.0f;
    const uint16_t *qp = (const uint16_t *)a.q + begin * a.q_stride + g * N + 8 * grp;
    const uint16_t *kp = (const uint16_t *)a.k + begin * a.k_stride + g * N + 8 * grp;
    const uint16_t *vp = (const uint16_t *)a.v + begin * a.v_stride + h * a.P + p;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f, A = a.A[h] * kLog2e;
    for (uint32_t t = 0; t < len; ++t) {
        float k[KB][8], q[KB][8], kk = 0.0f, qq = 0.0f, sk = 0.0f, sq = 0.0f;
        const float v = ld_act(vp, t * a.v_stride);
        const float dt = softplus(ld_act((const uint16_t *)a.dt_raw, (begin + t) * a.dt_stride + h) + bias);
        const float beta = delta_gate(ld_act((const uint16_t *)a.beta_raw, (begin + t) * a.beta_stride + h));
        const float decay = fast_exp2(dt * A);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            ld8(kp + t * a.k_stride + 32 * b, k[b]);
            ld8(qp + t * a.q_stride + 32 * b, q[b]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kk = __builtin_fmaf(k[b][e], k[b][e], kk);
                qq = __builtin_fmaf(q[b][e], q[b][e], qq);
                S[b][e] *= decay;
                sk = __builtin_fmaf(S[b][e], k[b][e], sk);
            }
        }
        const float rk = unit_scale(sum_groups(kk), a.norm_eps), rq = unit_scale(sum_groups(qq), a.norm_eps) * a.scale;
        const float u = beta * __builtin_fmaf(-rk, sum_groups(sk), v) * rk;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                S[b][e] = __builtin_fmaf(u, k[b][e], S[b][e]);
                sq = __builtin_fmaf(S[b][e], q[b][e], sq);
            }
        sq = sum_groups(sq);
        if (grp == 0) st_act(y, t * a.H * a.P, sq * rq);
    }
    if (len > 0 || !resume)
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) cache[32 * b + e] = S[b][e];
}

}  // namespace

size_t delta_workspace(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N) {
    return ((size_t)seqs * 4 + 255) / 256 * 256;
}

hipError_t launch_delta(DeltaArgs a, int N, void *workspace, hipStream_t s) {
    a.ws_slot = (int32_t *)workspace;
    hipLaunchKernelGGL(delta_slots_kernel, dim3((unsigned)a.seqs), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.P / kCols), (unsigned)a.H, (unsigned)a.seqs);
    if (N == 64) hipLaunchKernelGGL((delta_walk_kernel<64>), grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((delta_walk_kernel<128>), grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace ssm
