// The SSD layer behind its short causal convolution, over packed prompts, on a
// cache of states (gfx950): sequences of different lengths lie one behind the
// other in one array of rows, each starts from zero or from the window and
// state in its cache slot, and leaves both there.
//
//   u[t][c] = conv_b[c] + sum_j conv_w[c][j] raw[t-3+j][c],  x | B | C = silu(u)
//   dt      = softplus(dt_raw + dt_bias),   a = exp(dt A)
//   S[p][n] = a S[p][n] + dt x[p] B[n],     y[p] = sum_n C[n] S[p][n] + D x[p]
//
// The simple form: one workgroup per (sequence, head, 64 rows of the state)
// walks the tokens in order; four lanes share a state row.
#include "ssm_common.h"
#include "ssm_internal.h"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 8;  // tokens convolved at a time

// The sequence's rows, kept inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ void seq_rows(const SsdCacheArgs &a, int64_t s, int64_t &t0, int64_t &len) {
    const int64_t lo = a.cu_seqlens[s], hi = a.cu_seqlens[s + 1];
    t0 = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
    const int64_t t1 = hi < t0 ? t0 : hi > a.rows ? a.rows : hi;
    len = t1 - t0;
}

// Which slot each sequence owns (-1: none), and the windows the sequences
// start from, copied so that the caches can be written while they are read.
__global__ __launch_bounds__(kThreads) void seq_start_kernel(SsdCacheArgs a) {
    const int64_t s = blockIdx.y;
    const int32_t slot = a.slots[s];
    bool dead = slot < 0 || slot >= a.num_slots;
    if (!dead) {
        bool same = false;
        for (int64_t i = threadIdx.x; i < s; i += kThreads) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.ws_slot[s] = dead ? -1 : slot;
    const bool resume = !dead && a.resume && a.resume[s] != 0;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c < a.C)
        for (int k = 0; k < 3; ++k)
            a.ws_win[(s * 3 + k) * a.C + c] = resume ? ((const uint16_t *)a.conv_cache)[((int64_t)slot * a.C + c) * 3 + k] : 0;
}

template <int N>
__global__ __launch_bounds__(kThreads) void seq_walk_kernel(SsdCacheArgs a) {
    __shared__ float X[kTile][64], Bs[kTile][N], Cs[kTile][N], Dt[kTile];
    constexpr int E = N / 4;  // state elements per lane
    const int64_t H = a.H, pb = a.P / 64, C = a.C;
    const int64_t s = blockIdx.y, hp = blockIdx.x, h = hp / pb, p0 = (hp % pb) * 64, g = h / (H / a.G);
    const int tid = threadIdx.x, p = tid / 4, n0 = (tid % 4) * E;
    int64_t t0, len;
    seq_rows(a, s, t0, len);
    const int32_t slot = a.ws_slot[s];
    uint16_t *y = (uint16_t *)a.y + (t0 * H + h) * a.P + p0;
    if (slot < 0) {
        for (int64_t i = tid; i < len * 64; i += kThreads) y[(i / 64) * H * a.P + i % 64] = 0;
        return;
    }
    float *st = a.state_cache + (((int64_t)slot * H + h) * a.P + p0 + p) * N + n0;
    const bool resume = a.resume && a.resume[s] != 0;
    float S[E];
    for (int e = 0; e < E; ++e) S[e] = resume ? st[e] : 0.0f;
    const float A2 = a.A[h] * kLog2e, dsk = a.Dskip ? a.Dskip[h] : 0.0f, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const uint16_t *raw = (const uint16_t *)a.xBC;
    // raw row k of the sequence (k >= -3; before 0 the window) of channel c
    auto at = [&](int64_t k, int64_t c) {
        return ld_act(k < 0 ? a.ws_win : raw, k < 0 ? (s * 3 + k + 3) * C + c : (t0 + k) * a.xBC_stride + c);
    };
    for (int64_t k0 = 0; k0 < len; k0 += kTile) {
        const int m = len - k0 < kTile ? (int)(len - k0) : kTile;
        __syncthreads();
        for (int i = tid; i < m * (64 + 2 * N); i += kThreads) {
            const int j = i / (64 + 2 * N), q = i % (64 + 2 * N);
            const int64_t k = k0 + j;
            const int64_t c = q < 64 ? h * a.P + p0 + q : q < 64 + N ? H * a.P + g * N + q - 64 : H * a.P + (a.G + g) * N + q - 64 - N;
            const float4 w = *(const float4 *)(a.conv_w + 4 * c);
            const float v = conv_silu(w.x, w.y, w.z, w.w, a.conv_b ? a.conv_b[c] : 0.0f, at(k - 3, c), at(k - 2, c), at(k - 1, c), at(k, c));
            if (q < 64) X[j][q] = v;
            else if (q < 64 + N) Bs[j][q - 64] = v;
            else Cs[j][q - 64 - N] = v;
        }
        if (tid < m) Dt[tid] = softplus(ld_act((const uint16_t *)a.dt_raw, (t0 + k0 + tid) * a.dt_stride + h) + bias);
        __syncthreads();
        for (int j = 0; j < m; ++j) {
            const float av = fast_exp2(Dt[j] * A2), dx = Dt[j] * X[j][p];
            float acc = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                S[e] = __builtin_fmaf(av, S[e], dx * Bs[j][n0 + e]);
                acc = __builtin_fmaf(Cs[j][n0 + e], S[e], acc);
            }
            acc += __shfl_xor(acc, 1);
            acc += __shfl_xor(acc, 2);
            if (tid % 4 == 0) st_act(y, (k0 + j) * H * a.P + p, __builtin_fmaf(dsk, X[j][p], acc));
        }
    }
    for (int e = 0; e < E; ++e) st[e] = S[e];
    // the window the sequence leaves; the first head of a group writes its B and C
    const bool first = h % (H / a.G) == 0 && p0 == 0;
    for (int q = tid; q < 64 + (first ? 2 * N : 0); q += kThreads) {
        const int64_t c = q < 64 ? h * a.P + p0 + q : q < 64 + N ? H * a.P + g * N + q - 64 : H * a.P + (a.G + g) * N + q - 64 - N;
        for (int k = 0; k < 3; ++k) st_act((uint16_t *)a.conv_cache, ((int64_t)slot * C + c) * 3 + k, at(len - 3 + k, c));
    }
}

}  // namespace

size_t ssd_cache_workspace(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N) {
    return ((size_t)seqs * 4 + 255) / 256 * 256 + (size_t)seqs * 3 * (H * P + 2 * G * N) * 2;
}

hipError_t launch_ssd_cache(SsdCacheArgs a, int N, void *workspace, hipStream_t s) {
    a.ws_slot = (int32_t *)workspace;
    a.ws_win = (uint16_t *)((char *)workspace + ((size_t)a.seqs * 4 + 255) / 256 * 256);
    hipLaunchKernelGGL(seq_start_kernel, dim3((unsigned)((a.C + kThreads - 1) / kThreads), (unsigned)a.seqs), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.H * (a.P / 64)), (unsigned)a.seqs);
    if (N == 64) hipLaunchKernelGGL((seq_walk_kernel<64>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((seq_walk_kernel<128>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ssm
