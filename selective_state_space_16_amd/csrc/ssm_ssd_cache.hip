// The SSD layer behind its short causal convolution, over packed prompts, on a
// cache of states (gfx950): sequences of different lengths lie one behind the
// other in one array of rows, each starts from zero or from the window and
// state in its cache slot, and leaves both there.
//
//   u[t][c] = conv_b[c] + sum_j conv_w[c][j] raw[t-3+j][c],  x | B | C = silu(u)
//   dt      = softplus(dt_raw + dt_bias),   a = exp(dt A)
//   S[p][n] = a S[p][n] + dt x[p] B[n],     y[p] = sum_n C[n] S[p][n] + D x[p]
//
// Every sequence is cut into chunks of 64 tokens. With cum_t the log2 decay
// from the chunk's start through token t, sfx_t from behind t to its end and
// w_t = dt_t exp2(sfx_t), a chunk is three matrix products on the matrix cores:
//
//   y   = diag(exp2(cum)) C S^T + (G o exp2(cum_t - cum_s) dt_s, s <= t) x + D x,   G = C B^T
//   S^T = exp2(cum_last) S^T + B^T (w o x)
//
// Launches, in order:
//   prepare   per (chunk, group): the convolution of B and C, G, and the layouts
//             that the products load; per (chunk, head): the decays. B, C and G
//             are shared by all heads of a group, so they are formed once.
//   walk A    every segment of every sequence: the convolution of x, kept as the
//             operand of the later products, and the segment's end state, from
//             zero where the sequence is longer than one segment;
//   join      those end states in order: the state that enters each segment, and
//             the sequence's last state into the cache;
//   walk C    every segment from its entering state: y.
// A long sequence so keeps the whole chip busy. The offsets are read on the
// device. Chunk i of sequence s has the id cu[s] / 64 + s + i: disjoint ranges
// without a prefix sum, as ceil(len / 64) <= cu[s+1] / 64 - cu[s] / 64 + 1. The
// segments of several sequences are chosen and numbered on the device, by one wave
// of the first launch; otherwise their length is the host's and their ids as above.
//
// Precision. The state must come out as a float32 state would, so the products
// of walk A take both operands as sums of three bfloat16 (24 bits; six products,
// those left out are below 2^-24 of the whole). bfloat16 has float32's range, so
// no scale is needed that channels, columns or tokens of unlike size would share.
// The products for y, which is
// rounded to bfloat16 in the end, take single float16 operands (11 bits, against
// 8 of the result). float16 has little range, so they carry power-of-two
// scales: C one per token, B one per chunk, x one per chunk and wave, w one per
// chunk; walk C's state accumulates in units 2^K that follow a running bound of its
// size. Scales are exact, and they cancel in one factor per token at the end.
#include "ssm_common.h"
#include "ssm_device.h"
#include "ssm_internal.h"

namespace ssm {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kQ = 64;            // tokens per chunk
// Threads of a workgroup ahead of the walks: a lane convolves four channels of
// four tokens (256 threads and 16 tokens: 11.8 us for one chunk against 7).
constexpr int prep_threads(int N) { return 8 * N; }
constexpr int kBlocksA = 2;       // column blocks of 64 per workgroup of walk A, two waves each
constexpr int kBlocksC = 4;       // of walk C

// Workspace of one (chunk, group), in 16-bit elements: B in three parts as operand
// registers (lane-major; half, part, n tile), B and C in float16, G as operand
// registers, 2^eC per token (float32), filled up to whole 1 KiB pieces.
constexpr int frag_elems(int N) { return 5 * kQ * N + kQ * kQ + 512; }
// Floats per (chunk, head) for walk C: cum, cum - log2 dt, exp2(cum), and w as
// scaled float16, filled up to 1 KiB.
constexpr int kHead = 4 * kQ;
// Heads of a wave that forms decays (80 heads then take one workgroup per chunk at
// N = 128: 16384 tokens 22.2 -> 18.5 us against two heads, a short prompt the same).
constexpr int kDtHeads = 5;
constexpr int dt_heads(int N) { return prep_threads(N) / 64 * kDtHeads; }

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// a and b rounded to bfloat16, and what that leaves of them, exactly.
__device__ __forceinline__ uint32_t bf16_pair(float &a, float &b) {
    const uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xffff0000u);
    return u;
}
// Eight values as sums of PARTS bfloat16 each, 8 bits a part.
template <int PARTS>
__device__ __forceinline__ void split(float (&v)[8], bf16x8 (&out)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        u32x4 u;
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
        out[p] = __builtin_bit_cast(bf16x8, u);
    }
}
// The product of two operands of three parts each, as six, the small ones first.
constexpr int kTerm[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};
// Buffer accesses: bytes from a wave-uniform base, a range that the hardware
// checks (loads outside it give 0, stores outside it are dropped).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
// Smallest e with |v| < 2^e, for a normal v; -126 for zero.
__device__ __forceinline__ int exponent(float v) { return (int)((__float_as_uint(v) >> 23) & 255) - 126; }
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
__device__ __forceinline__ float finite_abs(float v) { return finite(v) ? __builtin_fabsf(v) : 0.0f; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// v plus the value of lane (lane - S) of its row of 16 (0 below it).
template <int S>
__device__ __forceinline__ float shr_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x110 + S, 0xF, 0xF,
                                                                      false));
}
// Inclusive prefix sum over the 64 lanes.
__device__ __forceinline__ float wave_prefix_sum(float v) {
    v = shr_add<1>(v);
    v = shr_add<2>(v);
    v = shr_add<4>(v);
    v = shr_add<8>(v);
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xA, 0xF, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xC, 0xF, false));
    return v;
}

// The largest of the values in a lane's row of 16, none negative.
__device__ __forceinline__ float row_top(float v) {
    auto step = [&](int o) { v = __builtin_fmaxf(v, __int_as_float(o)); };
    step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));  // row_ror:8, 4, 2, 1
    step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xF, 0xF, false));
    return v;
}
// The largest of the wave's values, none negative (or NaN, which stays): the
// order of their bits.
__device__ __forceinline__ float wave_top(float v) {
    uint32_t u = __float_as_uint(v);
    auto step = [&](uint32_t o) { u = o > u ? o : u; };
    step(__builtin_amdgcn_update_dpp(0, u, 0x128, 0xF, 0xF, false));  // row_ror:8, 4, 2, 1
    step(__builtin_amdgcn_update_dpp(0, u, 0x124, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, u, 0x122, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, u, 0x121, 0xF, 0xF, false));
    const uint32_t a = __builtin_amdgcn_readlane(u, 0), b = __builtin_amdgcn_readlane(u, 16);
    const uint32_t c = __builtin_amdgcn_readlane(u, 32), d = __builtin_amdgcn_readlane(u, 48);
    const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
    return __uint_as_float(ab > cd ? ab : cd);
}

// The rows of sequence s, kept inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ uint32_t seq_begin(const SsdCacheArgs &a, uint32_t s) {
    const int32_t lo = a.cu_seqlens[s], rows = (int32_t)a.rows;
    return lo < 0 ? 0 : lo > rows ? rows : lo;
}
__device__ __forceinline__ uint32_t seq_length(const SsdCacheArgs &a, uint32_t s, uint32_t begin) {
    const int32_t hi = a.cu_seqlens[s + 1], rows = (int32_t)a.rows, end = hi > rows ? rows : hi;
    return end < (int32_t)begin ? 0 : end - begin;
}

// The last s < n with key(s) <= id, or -1, for a key that does not decrease: 64
// candidates at a time, one per lane.
template <typename Key>
__device__ __forceinline__ int find(uint32_t id, uint32_t n, Key key) {
    uint32_t lo = 0;
    const uint32_t lane = threadIdx.x & 63;
    do {
        const uint32_t step = (n + 63) / 64, at = lane * step;
        const bool below = at < n && key(lo + at) <= id;
        const int cnt = __popcll(__ballot(below));
        if (cnt == 0) return -1;
        const uint32_t skip = (cnt - 1) * step;
        n = n - skip < step ? n - skip : step;
        lo += skip;
    } while (n > 1);
    return uniform((int)lo);
}

// The sequence whose pieces of `unit` tokens include piece `id`: the last s with
// cu[s] / unit + s <= id.
__device__ __forceinline__ int find_seq(const SsdCacheArgs &a, uint32_t id, uint32_t unit) {
    if (a.seqs == 1) return 0;
    return find(id, (uint32_t)a.seqs, [&](uint32_t s) { return seq_begin(a, s) / unit + s; });
}

// Tokens per segment.
__device__ __forceinline__ uint32_t segment(const SsdCacheArgs &a) {
    return a.ws_plan ? (uint32_t)uniform(a.ws_plan[0]) : (uint32_t)a.seg;
}

// Segments of a sequence (one without tokens has one too), the id of its first
// and the number of ids. From the device's plan the ids have no gaps; offsets that
// overlap may ask for more of them than the workspace holds, which are left out.
__device__ __forceinline__ uint32_t segments(uint32_t len, uint32_t seg) { return len > 0 ? (len + seg - 1) / seg : 1; }
__device__ __forceinline__ uint32_t first_segment(const SsdCacheArgs &a, uint32_t s, uint32_t begin, uint32_t seg) {
    return a.ws_plan ? (uint32_t)a.ws_plan[1 + s] : begin / seg + s;
}
__device__ __forceinline__ uint32_t segment_ids(const SsdCacheArgs &a) {
    if (!a.ws_plan) return (uint32_t)a.nseg;
    const uint32_t n = (uint32_t)uniform(a.ws_plan[1 + a.seqs]);
    return n < (uint32_t)a.nseg ? n : (uint32_t)a.nseg;
}

// -------------------------------------------------------------------- prepare

// The segment length, a lane per candidate, and the ids of the segments. The chip
// holds 512 workgroups of walk A and 256 of walk C at once. A workgroup costs its
// chunks and about two more (the first loads, the states); all of them either
// rounds of the longest (walk A's last round two thirds where it leaves every
// second place empty) or their sum over the places and one longest, whichever is
// less; a segment's state passes through the join besides. Against a length that
// suits the worst case of as many tokens, whole calls (us): eight prompts of 3600
// to 4900 tokens, 80 heads 548 -> 528, 13 of 4099, 32 heads 56 -> 53, 9 of 4148 tokens, 68 heads 118 -> 99, 3 of
// 19798 tokens, 34 heads 159 -> 139; 45 of 5143 tokens, 4 heads 56 -> 62.
__device__ __forceinline__ void plan_segments(const SsdCacheArgs &a) {
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x, least = (int)(a.seg / kQ);
    const float m = (float)(least + lane), inv = 1.0f / m, seqs = (float)a.seqs;
    float n = 0.0f, all = 0.0f, longest = 0.0f;
    for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
        float c = 0.0f;
        if (s0 + lane < a.seqs) c = (float)((seq_length(a, s0 + lane, seq_begin(a, s0 + lane)) + kQ - 1) / kQ);
        const int many = a.seqs - s0 < 64 ? (int)(a.seqs - s0) : 64;
        for (int k = 0; k < many; ++k) {
            const float ck = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(c), k));
            n += __builtin_fmaxf(__builtin_ceilf(__builtin_fmaf(ck, inv, -1e-3f)), 1.0f);
            all += ck;
            longest = __builtin_fmaxf(longest, ck);
        }
    }
    const int64_t ncb = a.H / a.G * (a.P / 64);
    const float ua = (float)(a.G * ((ncb + kBlocksA - 1) / kBlocksA)) * (1.0f / 512.0f);
    const float uc = (float)(a.G * ((ncb + kBlocksC - 1) / kBlocksC)) * (1.0f / 256.0f);
    const float one = __builtin_fminf(m, longest) + 2.0f, work = all + 2.0f * n;
    const float whole = __builtin_floorf(n * ua), rest = n * ua - whole;
    const float ra = whole + (rest > 0.5f ? 1.0f : rest > 0.0f ? 0.67f : 0.0f);
    const float cost = __builtin_fminf(ra * one, work * ua + one) + __builtin_fminf(__builtin_ceilf(n * uc) * one, work * uc + one) +
                       (n > seqs ? 2.2f * n * ua : 0.0f);
    float best = cost;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) best = __builtin_fminf(best, __shfl_xor(best, d));
    const int first = __ffsll((unsigned long long)__ballot(cost == best)) - 1;
    const uint32_t seg = uniform((least + (first < 0 ? 0 : first)) * kQ);
    uint32_t base = 0;
    for (int64_t s0 = 0; s0 < a.seqs; s0 += 64) {
        uint32_t k = 0;
        if (s0 + lane < a.seqs) k = segments(seq_length(a, s0 + lane, seq_begin(a, s0 + lane)), seg);
        uint32_t sum = k;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t below = __shfl_up(sum, d);
            sum += lane >= d ? below : 0;
        }
        if (s0 + lane < a.seqs) a.ws_plan[1 + s0 + lane] = base + sum - k;
        base += __shfl(sum, 63);
    }
    if (lane == 0) {
        a.ws_plan[0] = seg;
        a.ws_plan[1 + a.seqs] = base;
    }
}

template <int N>
struct PrepShared {
    static constexpr int R = N + 4;
    alignas(16) float B[kQ][R], C[kQ][R];
    float maxb[16];
    int ec[kQ];
};

// Which slot a sequence owns (-1: none), and the raw rows before its start.
template <int THREADS>
__device__ __forceinline__ void start_seq(const SsdCacheArgs &a, int64_t s, int64_t part) {
    const int32_t slot = a.slots[s];
    bool dead = slot < 0 || slot >= a.num_slots;
    if (!dead) {
        bool same = false;
        for (int64_t i = threadIdx.x; i < s; i += THREADS) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (part == 0 && threadIdx.x == 0) a.ws_slot[s] = dead ? -1 : slot;
    const bool resume = !dead && a.resume && a.resume[s] != 0;
    const int64_t c = part * THREADS + threadIdx.x;
    if (c < a.C)
        for (int k = 0; k < 3; ++k)
            a.ws_win[(s * 3 + k) * a.C + c] = resume ? ((const uint16_t *)a.conv_cache)[((int64_t)slot * a.C + c) * 3 + k] : 0;
}

// The decays of the chunk for a wave's heads h0 .., a lane per token.
__device__ __forceinline__ void chunk_decays(const SsdCacheArgs &a, uint32_t id, uint32_t row, int rem, uint32_t h0) {
    const int lane = threadIdx.x & 63;
    const uint32_t H = (uint32_t)a.H;
    const uint16_t *src = (const uint16_t *)a.dt_raw + (int64_t)(row + (lane < rem ? lane : rem - 1)) * a.dt_stride;
    float raw[kDtHeads], bias[kDtHeads], A2[kDtHeads];
#pragma unroll
    for (int k = 0; k < kDtHeads; ++k) {
        const uint32_t h = h0 + k < H ? h0 + k : H - 1;
        raw[k] = ld_act(src, h);
        bias[k] = a.dt_bias ? a.dt_bias[h] : 0.0f;
        A2[k] = a.A[h] * kLog2e;
    }
#pragma unroll
    for (int k = 0; k < kDtHeads; ++k) {
        if (h0 + k >= H) break;
        const int64_t at = (int64_t)id * H + h0 + k;
        const float dt = lane < rem ? softplus(raw[k] + bias[k]) : 0.0f;
        // A decay of 2^-256 leaves nothing of a float32 state: no more than that,
        // so that the sums keep bits for the tokens behind (2^14 at most). A step
        // that is not finite is a NaN from here on, not a decay to nothing.
        float step = dt * A2[k];
        step = step < -256.0f ? -256.0f : step;
        if (!finite(dt)) step = __builtin_nanf("");
        const float cum = wave_prefix_sum(step);
        // from the end, without subtracting: exact where little decays
        const float back = wave_prefix_sum(__shfl(step, 63 - lane));
        const float sfx = lane < 63 ? __shfl(back, 62 - lane) : 0.0f;
        const float wt = dt * fast_exp2(sfx);
        const int ed = exponent(wave_top(finite_abs(dt))), ew = exponent(wave_top(finite_abs(wt)));
        float *o = a.ws_head + at * kHead;
        o[lane] = cum;
        o[kQ + lane] = cum - __builtin_amdgcn_logf(dt) + (float)ed;
        o[2 * kQ + lane] = fast_exp2(cum);
        ((_Float16 *)(o + 3 * kQ))[lane] = (_Float16)__builtin_ldexpf(wt, -ew);  // below 1, as for walk A below
        a.ws_w[at * kQ + lane] = wt;
        if (lane == 63) *(f32x4 *)(a.ws_meta + at * 4) = f32x4{fast_exp2(cum), __int_as_float(ew), __int_as_float(ed), 0.0f};
    }
}

// Bound by latency and by its stores of 1.3 KB per (chunk, head) and 58 KB per
// (chunk, group) together: 9.1 us for one chunk (3 of them an empty launch, 1.6
// the loads and the convolution, the rest LDS and its barriers: with the low
// parts of B and C in one array in turn 10.0), 19 us for 16384 tokens of 80 heads
// (52 MB). The heads' decays have workgroups of their own, so that a short
// prompt waits for neither: done by the workgroups that convolve B and C, one
// chunk took 2 us more and 16384 tokens 23 in all.
// PLAN: one workgroup more, the first, chooses the segments (in every launch, its
// code alone took 3 of those 19 us).
template <int N, bool PLAN>
__global__ __launch_bounds__(prep_threads(N)) void prepare_kernel(SsdCacheArgs a) {
    __shared__ PrepShared<N> sh;
    constexpr int THREADS = prep_threads(N), WAVES = THREADS / 64, HEADS = dt_heads(N);
    uint32_t blk = blockIdx.x;
    if constexpr (PLAN) {
        if (blk-- == 0) {
            plan_segments(a);
            return;
        }
    }
    const uint32_t nbc = (uint32_t)(a.nchunk * a.G), per = ((uint32_t)a.H + HEADS - 1) / HEADS;
    const uint32_t ndt = (uint32_t)a.nchunk * per;
    if (blk >= nbc + ndt) {
        const uint32_t parts = (uint32_t)((a.C + THREADS - 1) / THREADS);
        blk -= nbc + ndt;
        start_seq<THREADS>(a, blk / parts, blk % parts);
        return;
    }
    const bool decays = blk >= nbc;
    if (decays) blk -= nbc;
    const uint32_t id = blk / (decays ? per : (uint32_t)a.G), g = blk % (decays ? per : (uint32_t)a.G);
    const int s = find_seq(a, id, kQ);
    if (s < 0) return;
    // all of the sequence's words at once, ahead of the branches
    const int32_t slot = a.slots[s], flag = a.resume ? a.resume[s] : 0;
    const uint32_t begin = seq_begin(a, s), len = seq_length(a, s, begin);
    const uint32_t first = (id - (begin / kQ + s)) * kQ;  // token of the sequence
    if (first >= len) return;
    const int rem = len - first < kQ ? (int)(len - first) : kQ;
    const bool resume = flag != 0 && slot >= 0 && slot < a.num_slots;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    if (decays) {
        chunk_decays(a, id, begin + first, rem, g * HEADS + wave * kDtHeads);
        return;
    }

    // The convolution: a lane takes four channels of TPB tokens; N / 4 lanes
    // hold a token's B, the next N / 4 its C.
    constexpr int LPR = 2 * N / 4, NB = THREADS / LPR, TPB = kQ / NB;
    const int cl = tid % LPR, tb = tid / LPR, isC = cl / (N / 4), n0 = (cl % (N / 4)) * 4;
    const int64_t c0 = a.H * a.P + (isC * a.G + g) * N + n0;
    float w[4][4], bias[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const f32x4 t = *(const f32x4 *)(a.conv_w + 4 * (c0 + k));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k][j] = t[j];
        bias[k] = a.conv_b ? a.conv_b[c0 + k] : 0.0f;
    }
    uint2 raw[TPB + 3];
    const int t0 = tb * TPB;
    const uint16_t *rows = (const uint16_t *)a.xBC + c0;
#pragma unroll
    for (int i = 0; i < TPB + 3; ++i) {
        const int t = (int)first + t0 + i - 3, last = (int)len - 1;  // token of the sequence
        if (t >= 0) {
            raw[i] = *(const uint2 *)(rows + (int64_t)(begin + (t < last ? t : last)) * a.xBC_stride);
        } else {
            uint32_t v[4];
            for (int k = 0; k < 4; ++k)
                v[k] = resume ? ((const uint16_t *)a.conv_cache)[((int64_t)slot * a.C + c0 + k) * 3 + t + 3] : 0;
            raw[i] = uint2{v[0] | v[1] << 16, v[2] | v[3] << 16};
        }
    }
    float v[TPB][4], big = 0.0f;
#pragma unroll
    for (int i = 0; i < TPB; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            auto at = [&](int j) {
                const uint32_t u = k < 2 ? raw[i + j].x : raw[i + j].y;
                return __uint_as_float(k % 2 ? u & 0xffff0000u : u << 16);
            };
            v[i][k] = t0 + i < rem ? conv_silu(w[k][0], w[k][1], w[k][2], w[k][3], bias[k], at(0), at(1), at(2), at(3)) : 0.0f;
            top = __builtin_fmaxf(top, finite_abs(v[i][k]));
        }
        // the largest value of the token's C, and of the chunk's B
        top = row_top(top);
        if constexpr (N == 128) top = __builtin_fmaxf(top, __shfl_xor(top, 16));
        if (isC) {
            if (cl == N / 4) sh.ec[t0 + i] = clampi(exponent(top), -100, 120);
        } else {
            big = __builtin_fmaxf(big, top);
        }
    }
    big = wave_top(big);
    if (lane == 0) sh.maxb[wave] = big;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WAVES; ++k) big = __builtin_fmaxf(big, sh.maxb[k]);
    const int eB = clampi(exponent(big), -100, 128);
#pragma unroll
    for (int i = 0; i < TPB; ++i) *(f32x4 *)(isC ? &sh.C[t0 + i][n0] : &sh.B[t0 + i][n0]) = f32x4{v[i][0], v[i][1], v[i][2], v[i][3]};
    __syncthreads();

    _Float16 *out = (_Float16 *)a.ws_frag + ((int64_t)id * a.G + g) * frag_elems(N);
    const int r = lane & 15, q = lane >> 4;
    // Each wave forms one of B^T's operands, (h, nt): row n = 16 nt + r, k = token
    // 16 q + 8 h + j;
    static_assert(2 * (N / 16) == WAVES && 4 * (N / 32) == WAVES);
    _Float16 *const out16 = out + 3 * kQ * N;
    {
        constexpr int NT = N / 16;
        const int h = wave / NT, nt = wave % NT;
        float t[8];
        f16x8 hi;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            t[j] = sh.B[16 * q + 8 * h + j][16 * nt + r];
            hi[j] = (_Float16)__builtin_ldexpf(t[j], 7 - eB);
        }
        *(f16x8 *)(out16 + (wave * 64 + lane) * 8) = hi;
        bf16x8 part[3];
        split(t, part);
#pragma unroll
        for (int p = 0; p < 3; ++p) *((bf16x8 *)out + ((h * 3 + p) * NT + nt) * 64 + lane) = part[p];
    }
    // one of C's, (tt, m): row r is token 16 (r / 4) + 4 tt + r % 4, and k runs
    // over n in the order in which two accumulator tiles hold the state;
    const int row = 16 * (r / 4) + r % 4;
    {
        const int tt = wave / (N / 32), m = wave % (N / 32), e = 7 - sh.ec[row + 4 * tt];
        const float *src = &sh.C[row + 4 * tt][32 * m + 4 * q];
        const f32x4 lo = *(const f32x4 *)src, hi = *(const f32x4 *)(src + 16);
        f16x8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (_Float16)__builtin_ldexpf(lo[j], e), o[4 + j] = (_Float16)__builtin_ldexpf(hi[j], e);
        *(f16x8 *)(out16 + kQ * N + (wave * 64 + lane) * 8) = o;
    }
    // and of G's, (tt, h) with row r as in C and k = token s = 16 q + 8 h + j, one
    // or two of the sixteen products (tt, h, b), whose row 4 q + e is token
    // 16 q + 8 h + 4 b + e.
    constexpr int PER = 16 / WAVES;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int f = wave * PER + k, tt = f / 4, sr = row + 4 * (f % 4), s0 = 16 * q + 4 * (f % 4);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < N / 32; ++m) {
            float cv[8], bv[8];
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *(f32x4 *)(cv + j) = *(const f32x4 *)&sh.C[row + 4 * tt][32 * m + 8 * q + j];
                *(f32x4 *)(bv + j) = *(const f32x4 *)&sh.B[sr][32 * m + 8 * q + j];
            }
            bf16x8 cp[3], bp[3];
            split(cv, cp);
            split(bv, bp);
#pragma unroll
            for (int p = 0; p < 6; ++p) acc = mfma(bp[kTerm[p][0]], cp[kTerm[p][1]], acc);
        }
        f16x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = s0 + e <= row + 4 * tt ? (_Float16)__builtin_ldexpf(acc[e], 7 - sh.ec[row + 4 * tt] - eB) : (_Float16)0.0f;
        *(f16x4 *)(out16 + 2 * kQ * N + ((f / 2) * 64 + lane) * 8 + 4 * (f % 2)) = o;
    }
    if (tid < kQ) ((float *)(out16 + 2 * kQ * N + kQ * kQ))[tid] = __builtin_ldexpf(1.0f, sh.ec[tid]);
    if (tid == 0) a.ws_eb[id * a.G + g] = eB;
}

// ---------------------------------------------------------------------- walks

// What a workgroup of a walk works on: one segment of one sequence, and BLOCKS
// column blocks (64 rows of a head's state each) of one group; two waves share a
// block, 32 columns each. Lane (r, q) = (l % 16, l / 16) holds the channels p =
// 2 r + c of the wave's 32 for the tokens 16 q + i of a chunk: what the 16 x 16
// x 32 product takes as its B operand (column r, k = 8 consecutive tokens), and,
// with the output's rows numbered to match, the place where y comes out.
struct Unit {
    uint32_t begin, len, k, nseg, from, to, g, hb, h, hfirst, ch0, sid, chunk0;
    int s;
    int32_t slot;
    bool resume;
    bool on;    // the wave has columns
    bool some;  // there is anything to do
};

template <int BLOCKS>
__device__ __forceinline__ Unit find_unit(const SsdCacheArgs &a) {
    Unit u;
    u.some = false;
    const uint32_t wave = uniform(threadIdx.x >> 6);
    // Workgroups are dealt to the 8 XCDs in turn: neighbours in the order of
    // the work (the column blocks of one segment, which load the same B, C and
    // G) go to one XCD and its L2.
    const uint32_t P = (uint32_t)a.P, pb = P / 64, G = (uint32_t)a.G, hpg = (uint32_t)a.H / G, seg = segment(a);
    const uint32_t ncb = hpg * pb, nhb = (ncb + BLOCKS - 1) / BLOCKS;
    const uint32_t total = segment_ids(a) * G * nhb, per = (total + 7) / 8;
    const uint32_t unit = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || unit >= total) return u;
    u.sid = unit / (G * nhb);
    u.g = unit / nhb % G;
    u.hb = unit % nhb;
    u.s = a.ws_plan ? find(u.sid, (uint32_t)a.seqs, [&](uint32_t s) { return (uint32_t)a.ws_plan[1 + s]; }) : find_seq(a, u.sid, seg);
    if (u.s < 0) return u;
    // all of the sequence's words at once, ahead of the branches
    u.slot = a.ws_slot[u.s];
    u.resume = a.resume && a.resume[u.s] != 0;
    u.begin = seq_begin(a, u.s);
    u.len = seq_length(a, u.s, u.begin);
    u.k = u.sid - first_segment(a, u.s, u.begin, seg);
    u.nseg = segments(u.len, seg);
    if (u.k >= u.nseg) return u;
    u.from = u.k * seg;
    u.to = u.len - u.from < seg ? u.len : u.from + seg;
    const uint32_t cb = u.hb * BLOCKS + wave / 2;
    u.on = cb < ncb;
    u.hfirst = u.g * hpg + u.hb * BLOCKS / pb;
    u.h = u.g * hpg + (u.on ? cb / pb : 0);
    u.ch0 = u.h * P + (u.on ? cb % pb : 0) * 64 + 32 * (wave % 2);  // the wave's first channel
    u.chunk0 = u.begin / kQ + u.s;
    u.some = true;
    return u;
}

// Pieces of 1 KiB from `src` straight into LDS, dealt to the waves in turn.
template <int PIECES, int WAVES>
__device__ __forceinline__ void pieces(const void *src, const void *to_lds, int wave, int lane) {
    const uint32_t dst = lds_addr(to_lds);
#pragma unroll
    for (int i = 0; i < (PIECES + WAVES - 1) / WAVES; ++i) {
        const int p = i * WAVES + wave;
        if (p < PIECES) dma16_s((const char *)src + p * 1024, lane * 16, dst + p * 1024);
    }
}

constexpr int pieces_b(int N) { return 3 * kQ * N / 512; }
constexpr int pieces_cg(int N) { return (kQ * N + kQ * kQ) / 512; }

// Walk A: x, and the segment's end state. B lies in LDS by halves of a chunk (48 KB
// of three parts each chunk at N = 128), three of them in turn, so that two
// workgroups share a CU, two waves a SIMD; a barrier before each half's products
// says that it has come and that the one before it may be overwritten.
//
// Bound by instruction issue: per chunk and wave the convolution and SiLU of 32
// values a lane, their split into three bfloat16 and 192 products (N = 128), from
// two waves per SIMD, which is what the state's 64 registers and the operands
// leave room for (249 of 256). 16384 tokens of 80 heads: 148 us for 168 MB of x
// read and as much written. Operands of two float16 (22 bits, three products, 114
// us) need scales that channels, columns and tokens share, and lose what is small
// beside a neighbour. Workgroups of 6 waves (which do not pair up on a CU) and of 12
// took 1.7 and 1.35 times as long.
template <int N>
__global__ __launch_bounds__(128 * kBlocksA, 2) void walk_state_kernel(SsdCacheArgs a) {
    constexpr int NT = N / 16;
    struct Shared {
        alignas(16) __bf16 B[3][3 * kQ / 2 * N];  // halves of a chunk, in turn
        alignas(16) float w[2][4][kQ];
    };
    __shared__ Shared sh;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const Unit u = find_unit<kBlocksA>(a);
    if (!u.some) return;
    const int32_t slot = u.slot;
    if (slot < 0) return;
    const uint32_t from = u.from, to = u.to, H = (uint32_t)a.H, G = (uint32_t)a.G;

    // The convolution times -log2(e): its exp2 is SiLU's exponential, and the
    // factor comes out again with the scales.
    float w[2][4], bias[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const f32x4 t = *(const f32x4 *)(a.conv_w + 4 * (int64_t)(u.ch0 + 2 * r + c));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[c][j] = t[j] * -kLog2e;
        bias[c] = a.conv_b ? a.conv_b[u.ch0 + 2 * r + c] * -kLog2e : 0.0f;
    }

    // The raw rows of a chunk: tokens 16 q - 3 .. 16 q + 15, two channels each.
    // Behind the sequence's end zeros; before its start the window.
    uint32_t raw[19];
    const uint32_t rowb = (uint32_t)a.xBC_stride * 2, chb = (u.ch0 + 2 * r) * 2;
    const uint32_t xlane = 16 * q * rowb + chb;
    auto load = [&](uint32_t t) {  // the chunk that starts at token t of the sequence
        const char *base = (const char *)a.xBC + (int64_t)(u.begin + t) * rowb;
        const uint32_t rem = to - t < kQ ? to - t : kQ;
        const auto rows = buffer(base, rem * rowb);
        uint32_t o = xlane;
        asm volatile("" : "+v"(o));  // one running offset, not sixteen kept between chunks
        if (t > 0) {
            const auto before = buffer(base - 3 * (int64_t)rowb, (rem + 3) * rowb);
#pragma unroll
            for (int i = 0; i < 3; ++i) raw[i] = __builtin_amdgcn_raw_buffer_load_b32(before, o + i * rowb, 0, 0);
        } else {
            const uint16_t *win = a.ws_win + (int64_t)u.s * 3 * a.C;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t first = *(const uint32_t *)((const char *)(win + i * a.C) + chb);
                const uint32_t later = __builtin_amdgcn_raw_buffer_load_b32(rows, o + i * rowb - 3 * rowb, 0, 0);
                raw[i] = q == 0 ? first : later;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            raw[3 + i] = __builtin_amdgcn_raw_buffer_load_b32(rows, o, 0, 0);
            o += rowb;
        }
    };
    auto stage = [&](uint32_t t, int half, int slot) {
        const uint32_t id = u.chunk0 + t / kQ;
        pieces<pieces_b(N) / 2, 2 * kBlocksA>((const char *)a.ws_frag + ((int64_t)id * G + u.g) * (frag_elems(N) * 2) + half * (pieces_b(N) / 2 * 1024),
                                              sh.B[slot], wave, lane);
        // w of four heads, the first two or all of them needed
        if (half == 0 && wave == 0) dma16_s(a.ws_w + ((int64_t)id * H + u.hfirst) * kQ, lane * 16, lds_addr(sh.w[(t - from) / kQ & 1]));
    };
    int at0 = 0;  // where the chunk's first half lies

    float segdec = 1.0f;
    if (from < to) {
        stage(from, 0, 0);
        stage(from, 1, 1);
        if (u.on) load(from);
    }

    // the state: acc[nt][c][e] = S[p = 2 r + c][n = 16 nt + 4 q + e], from the
    // cache where the sequence is one segment and resumes
    f32x4 acc[NT][2];
    const int64_t off = (int64_t)(u.ch0 + 2 * r) * N + 4 * q, hpn = a.H * a.P * N;
    const bool resume = u.resume, one = u.nseg == 1;
    float *const cache = a.state_cache + (int64_t)slot * hpn + off;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[nt][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (one && resume && u.on) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[nt][c] = *(const f32x4 *)(cache + c * N + 16 * nt);
    }
    for (uint32_t t = from; t < to; t += kQ) {
        const uint32_t id = u.chunk0 + t / kQ;
        const int rem = to - t < kQ ? (int)(to - t) : kQ;
        const bool more = t + kQ < to;
        const int at1 = at0 == 2 ? 0 : at0 + 1, at2 = at1 == 2 ? 0 : at1 + 1;

        float x[2][16], top = 0.0f;
        if (u.on) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    auto at = [&](int j) { return __uint_as_float(c ? raw[i + j] & 0xffff0000u : raw[i + j] << 16); };
                    float v = __builtin_fmaf(w[c][0], at(0), bias[c]);
                    v = __builtin_fmaf(w[c][1], at(1), v);
                    v = __builtin_fmaf(w[c][2], at(2), v);
                    v = __builtin_fmaf(w[c][3], at(3), v);
                    x[c][i] = v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(v)) * -kLn2;
                }
            if (rem < kQ) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[c][i] = 16 * q + i < rem ? x[c][i] : 0.0f;
            }
        }
        vm_wait();
        lds_barrier();  // the chunk is in LDS, and every wave is done with the one before
        if (more) stage(t + kQ, 0, at2);
        float dec = 0.0f;
        const float *wt = sh.w[(t - from) / kQ & 1][u.h - u.hfirst] + 16 * q;
        bf16x8 bo[2][3][2], v[2][3];
        auto read_b = [&](int slot, int g) {  // two operands, in three parts each
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int j = 0; j < 2; ++j) bo[g & 1][p][j] = *(const bf16x8 *)(sh.B[slot] + ((p * NT + 2 * g + j) * 64 + lane) * 8);
        };
        // w o x of eight tokens a lane, and their products with B
        auto products = [&](int hh, int slot) {
            read_b(slot, 0);
            f32x4 wq[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) wq[j] = *(const f32x4 *)(wt + 8 * hh + 4 * j);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float wx[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) wx[j] = x[c][8 * hh + j] * wq[j / 4][j % 4];
                split(wx, v[c]);
            }
            if (hh == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[nt][c] *= dec;
            }
#pragma unroll
            for (int g = 0; g < NT / 2; ++g) {
                if (g + 1 < NT / 2) read_b(slot, g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < 6; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            acc[2 * g + j][c] = mfma(bo[g & 1][kTerm[k][0]][j], v[c][kTerm[k][1]], acc[2 * g + j][c]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (u.on) {
            if (more) load(t + kQ);
            dec = ((cf32_ptr)(a.ws_meta + ((int64_t)id * H + u.h) * 4))[0];
            segdec *= dec;
            // x as walk C's operand: float16 times 2^(14 - ex). A value that is not
            // finite would reach earlier tokens there as 0 times itself: it is marked.
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(__builtin_fabsf(x[c][i]), top);  // keeps a NaN
            top = wave_top(top);
            const bool anybad = !finite(top);
            if (anybad) {
                top = 0.0f;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, finite_abs(x[c][i]));
                top = wave_top(top);
            }
            const int ex = clampi(uniform(exponent(top)), -100, 127);
            const float sx = __builtin_ldexpf(1.0f, 14 - ex);
            const int64_t at = (int64_t)id * (a.H * a.P / 32) + u.ch0 / 32;
            if (lane == 0) a.ws_ex[at] = ex + (anybad ? 1 << 16 : 0);
            f16x8 xo[2][2], *dst = (f16x8 *)a.ws_x + at * 256 + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) xo[c][i / 8][i % 8] = (_Float16)(x[c][i] * sx);
            if (anybad) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!finite(x[c][i])) xo[c][i / 8][i % 8] = (_Float16)__builtin_nanf("");
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) dst[(c * 2 + hh) * 64] = xo[c][hh];
            // The convolution stands before the products of the SIMD's other wave: the
            // matrix cores are then fed while it runs (16384 tokens 124 -> 117 us; the
            // products first: 123).
            __builtin_amdgcn_s_setprio(0);
            products(0, at0);
        }
        lds_barrier();  // every wave is done with the chunk's first half
        if (more) stage(t + kQ, 1, at0);
        if (u.on) {
            products(1, at1);
            __builtin_amdgcn_s_setprio(1);
        }
        at0 = at2;
    }
    if (!u.on) return;
    // A sequence of one segment that does not resume is done; one that does is
    // stored aside, as walk C still reads its first state (without tokens it
    // keeps its bits); others are joined.
    float *dst = one && !resume ? cache : a.ws_state + (int64_t)u.sid * hpn + off;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) *(f32x4 *)(dst + c * N + 16 * nt) = acc[nt][c];
    if (lane == 0) a.ws_segdec[(int64_t)u.sid * H + u.h] = segdec;
}

// Bound by HBM where there are many heads: 63 MB of segment states in 13 us (16384
// tokens, 80 heads, 12 segments), 131 MB in 25 us (eight prompts of 4096). With
// few heads there are many segments, and the loads of one after the other are:
// four ahead take a prompt batch of 21507 tokens, 8 heads, from 70 to 64 us.
// enter[k] in place of end[k]: enter[0] the sequence's first state, enter[k+1] =
// dec[k] enter[k] + end[k]; the last one goes into the cache.
__global__ __launch_bounds__(256) void join_kernel(SsdCacheArgs a, int N) {
    constexpr uint32_t kAhead = 4;  // segments loaded ahead of the chain
    const uint32_t s = blockIdx.y, seg = segment(a);
    const int32_t slot = a.ws_slot[s], flag = a.resume ? a.resume[s] : 0;
    const uint32_t begin = seq_begin(a, s), len = seq_length(a, s, begin), nseg = segments(len, seg);
    if (nseg < 2 || slot < 0) return;
    const int64_t hpn = a.H * a.P * N, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= hpn) return;
    const int64_t h = i / (a.P * N), first = first_segment(a, s, begin, seg);
    if (first + nseg > a.nseg) return;
    float *const cache = a.state_cache + slot * hpn + i;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (flag != 0) v = *(const f32x4 *)cache;
    for (uint32_t k0 = 0; k0 < nseg; k0 += kAhead) {
        f32x4 end[kAhead];
        float dec[kAhead];
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) {
            const int64_t k = first + (k0 + j < nseg ? k0 + j : nseg - 1);
            end[j] = *(const f32x4 *)(a.ws_state + k * hpn + i);
            dec[j] = a.ws_segdec[k * a.H + h];
        }
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) {
            if (k0 + j >= nseg) break;
            *(f32x4 *)(a.ws_state + (first + k0 + j) * hpn + i) = v;
            v = end[j] + v * dec[j];
        }
    }
    *(f32x4 *)cache = v;
}

// Walk C: y of a segment. The two waves of a block each form half of the block's
// masked matrix and put it into LDS as operand registers. An iteration finishes
// one chunk (the masked product, y, the state) and begins the next one (C S^T and
// the masked matrix), so that one barrier per chunk is enough and products and
// vector instructions of both stand side by side; B, C, G and the decays are
// held twice and loaded a whole iteration ahead. One workgroup fills a CU (160 KB
// of LDS at N = 128).
//
// Bound by instruction issue, as walk A: 48 products for y and 32 for the state
// per chunk and wave, the masked matrix's exponentials (16 per lane), the
// operands' LDS reads. 16384 tokens of 80 heads: 112 us; with two barriers per
// chunk and operands read at their use 126. 6 waves per workgroup 188, 12 waves 140.
template <int N>
__global__ __launch_bounds__(128 * kBlocksC, 2) void walk_out_kernel(SsdCacheArgs a) {
    constexpr int NT = N / 16, KB = N / 32, WAVES = 2 * kBlocksC;
    struct Shared {
        alignas(16) _Float16 B[2][kQ * N];  // the high parts
        alignas(16) _Float16 CG[2][kQ * N + kQ * kQ];
        alignas(16) float scale[3][256];  // 2^eC per token
        alignas(16) float head[3][kBlocksC][kHead];
        alignas(16) _Float16 M[2][kBlocksC][8][64][8];
    };
    __shared__ Shared sh;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const Unit u = find_unit<kBlocksC>(a);
    if (!u.some) return;
    const uint32_t from = u.from, to = u.to, H = (uint32_t)a.H, G = (uint32_t)a.G;
    const int32_t slot = u.slot;
    const uint32_t yrow = (uint32_t)(a.H * a.P) * 2;
    if (slot < 0) {
        if (u.on)
            for (uint32_t t = from + q; t < to; t += 4)
                *(uint32_t *)((char *)a.y + (int64_t)(u.begin + t) * yrow + (u.ch0 + 2 * r) * 2) = 0u;
        return;
    }

    auto operands = [&](uint32_t t) {  // in float16
        return (const char *)a.ws_frag + ((int64_t)(u.chunk0 + t / kQ) * G + u.g) * (frag_elems(N) * 2) + pieces_b(N) * 1024;
    };
    auto stage_b = [&](uint32_t t) {
        pieces<pieces_b(N) / 3, WAVES>(operands(t), sh.B[(t - from) / kQ & 1], wave, lane);
    };
    auto stage_cg = [&](uint32_t t) {
        const uint32_t i = (t - from) / kQ, i3 = i % 3;
        const char *f = operands(t) + pieces_b(N) / 3 * 1024;
        pieces<pieces_cg(N), WAVES>(f, sh.CG[i & 1], wave, lane);
        if (wave == WAVES - 1) dma16_s(f + pieces_cg(N) * 1024, lane * 16, lds_addr(sh.scale[i3]));
        if (wave % 2 == 0 && u.on)
            dma16_s(a.ws_head + ((int64_t)(u.chunk0 + t / kQ) * H + u.h) * kHead, lane * 16, lds_addr(sh.head[i3][wave / 2]));
    };
    if (from < to) {
        stage_b(from);
        stage_cg(from);
        if (from + kQ < to) stage_cg(from + kQ);
    }
    if (!u.on) {  // no columns: the wave only carries its share of the loads
        if (from < to) {
            vm_wait();
            lds_barrier();
        }
        for (uint32_t t = from; t < to; t += kQ) {
            vm_wait();
            lds_barrier();
            if (t + kQ < to) stage_b(t + kQ);
            if (t + 2 * kQ < to) stage_cg(t + 2 * kQ);
        }
    }

    // the state: acc[nt][c][e] = S[p = 2 r + c][n = 16 nt + 4 q + e] 2^-K, kept
    // below 2^15 by its bound, so that its float16 copy needs no scale of its own
    const int64_t off = (int64_t)(u.ch0 + 2 * r) * N + 4 * q, hpn = a.H * a.P * N;
    const bool resume = u.resume, one = u.nseg == 1;
    float *const cache = a.state_cache + (int64_t)slot * hpn + off;
    const float *const own = a.ws_state + (int64_t)u.sid * hpn + off;
    if (u.on && from < to) {
        f32x4 acc[NT][2];
        int K = 0;
        float bound = 0.0f;  // of |acc|
        f16x8 xn[2][2];
        auto load = [&](uint32_t t) {
            const f16x8 *src = (const f16x8 *)a.ws_x + ((int64_t)(u.chunk0 + t / kQ) * (a.H * a.P / 32) + u.ch0 / 32) * 256 + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) xn[c][hh] = src[(c * 2 + hh) * 64];
        };
        load(from);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[nt][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (resume || u.k > 0) {
            const float *src = one ? cache : own;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    acc[nt][c] = *(const f32x4 *)(src + c * N + 16 * nt);
#pragma unroll
                    for (int e = 0; e < 4; ++e) bound = __builtin_fmaxf(bound, finite_abs(acc[nt][c][e]));
                }
            bound = wave_top(bound);
            if (bound > 0.0f) {
                K = uniform(exponent(bound)) - 14;
                bound = 0x1p14f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][c][e] = __builtin_ldexpf(acc[nt][c][e], -K);
            }
        }
        const float dsk = a.Dskip ? a.Dskip[u.h] : 0.0f;

        // What a chunk is begun with: its exponents and its decay over all.
        float dec, decn;
        int ew, ewn, ed, edn, eB, eBn, exb, exbn;
        auto scalars = [&](uint32_t t) {
            const uint32_t id = u.chunk0 + t / kQ;
            const cf32_ptr meta = (cf32_ptr)(a.ws_meta + ((int64_t)id * H + u.h) * 4);
            decn = meta[0];
            ewn = __float_as_int(meta[1]), edn = __float_as_int(meta[2]);
            eBn = ((const __attribute__((address_space(4))) int *)a.ws_eb)[(int64_t)id * G + u.g];
            exbn = ((const __attribute__((address_space(4))) int *)a.ws_ex)[(int64_t)id * (a.H * a.P / 32) + u.ch0 / 32];
        };
        f32x4 Y[4][2];
        int E2 = 0, E2n = 0;
        // C S^T of the chunk with the scalars above and the wave's half of its
        // masked matrix, M[t][s] = G[t][s] exp2(cum_t - cum_s) dt_s.
        auto begin_chunk = [&](uint32_t i, int ex, int edx, int eBx) {
            const float *hd = sh.head[i % 3][wave / 2];
            const _Float16 *CG = sh.CG[i & 1];
            // C S^T in units 2^(eC + E1), the masked product in units 2^(eC + E2)
            const int E1 = K - 7;
            E2n = ex + edx + eBx - 21;
            const bool small = E1 - E2n > 60;  // nothing beside the state: the factor below stays in range
            if (small) E2n = E1 - 60;
            const float cap = small ? -200.0f : 15.0f;
            // operands are read from LDS one group of products ahead
            f32x4 cs[4], ec[4];
            float ct[2];
            f16x8 gv[2][2], co[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[j] = *(const f32x4 *)(hd + kQ + 16 * q + 4 * j);
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                ct[k2] = hd[16 * (r / 4) + r % 4 + 4 * (2 * (wave % 2) + k2)];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    gv[k2][hh] = *(const f16x8 *)(CG + kQ * N + (((2 * (wave % 2) + k2) * 2 + hh) * 64 + lane) * 8);
            }
            auto read_c = [&](int m) {
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) co[m & 1][tt] = *(const f16x8 *)(CG + ((tt * KB + m) * 64 + lane) * 8);
            };
            read_c(0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int c = 0; c < 2; ++c) Y[tt][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < KB; ++m) {
                if (m + 1 < KB) {
                    read_c(m + 1);
                } else {
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt) ec[tt] = *(const f32x4 *)(hd + 2 * kQ + 16 * q + 4 * tt);
                }
                __builtin_amdgcn_sched_barrier(0);
                // C S^T, and in between the masked matrix
                f16x8 so[2];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) so[c][e] = (_Float16)acc[2 * m + e / 4][c][e % 4];
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) Y[tt][c] = mfma(co[m & 1][tt], so[c], Y[tt][c]);
#pragma unroll
                for (int k = m * 4 / KB; k < (m + 1) * 4 / KB; ++k) {
                    const int k2 = k / 2, hh = k % 2;
                    f16x8 me;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        // G is zero above the diagonal, where the exponent may be large
                        me[j] = (_Float16)fast_exp2(__builtin_fminf(ct[k2] - cs[2 * hh + j / 4][j % 4], cap));
                    *(f16x8 *)&sh.M[i & 1][wave / 2][(2 * (wave % 2) + k2) * 2 + hh][lane][0] = me * gv[k2][hh];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            const float al = __builtin_ldexpf(1.0f, E1 - E2n);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                ec[tt] *= al;
#pragma unroll
                for (int c = 0; c < 2; ++c) Y[tt][c] *= ec[tt];
            }
        };
        auto of_ex = [](int e) { return e >= 1 << 15 ? e - (1 << 16) : e; };  // without the mark of values that are not finite

        scalars(from);
        vm_wait();
        lds_barrier();
        begin_chunk(0, of_ex(exbn), edn, eBn);
        for (uint32_t t = from; t < to; t += kQ) {
            const uint32_t i = (t - from) / kQ;
            dec = decn, ew = ewn, ed = edn, eB = eBn, exb = exbn, E2 = E2n;
            const bool anybad = exb >= 1 << 15;
            const int ex = of_ex(exb), rem = to - t < kQ ? (int)(to - t) : kQ;
            const bool more = t + kQ < to;
            if (more) scalars(t + kQ);
            f16x8 x16[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) x16[c][hh] = xn[c][hh];
            // Issued since the barrier before: the loads of two chunks ahead, x,
            // and the last chunk's 16 stores of y, which may stay in flight
            // (accesses complete in order).
            if (t > from) asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
            else vm_wait();
            lds_barrier();  // M is whole, and the next chunk's C, G and decays and this one's B are in LDS
            if (more) {
                stage_b(t + kQ);
                if (t + 2 * kQ < to) stage_cg(t + 2 * kQ);
                load(t + kQ);
            }
            uint32_t badm[2] = {0u, 0u};
            if (anybad) {
                // values that are not finite: zero for the products, and what
                // they reach (their channel, from their token on) becomes NaN
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const _Float16 v = x16[c][j / 8][j % 8];
                        if (v != v) {
                            badm[c] |= 1u << j;
                            x16[c][j / 8][j % 8] = (_Float16)0.0f;
                        }
                    }
                    bool low = false;  // the channel is marked in an earlier lane's tokens
#pragma unroll
                    for (int d = 16; d < 64; d += 16) {
                        const uint32_t o = __shfl(badm[c], (lane - d) & 63);
                        low |= lane >= d && o != 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (low || (badm[c] & ((2u << j) - 1))) Y[j / 4][c][j % 4] = __builtin_nanf("");
                }
            }
            const float *hd = sh.head[i % 3][wave / 2];
            // LDS reads stand a group of products ahead of their use
            f16x8 mo[4][2], wv[2], bq[2][4];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) mo[tt][hh] = *(const f16x8 *)&sh.M[i & 1][wave / 2][tt * 2 + hh][lane][0];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) wv[hh] = *(const f16x8 *)((const _Float16 *)(hd + 3 * kQ) + 16 * q + 8 * hh);
            __builtin_amdgcn_sched_barrier(0);
            // the state: x 2^-sc times w (w < 1 as stored) in units that keep
            // dec |acc| + 64 |x w B| below 2^15
            const int c0 = ex + ew + eB - 21;
            int e1 = K - c0 + uniform(exponent(bound * dec));
            e1 = e1 > 27 ? e1 : 27;
            const int sc = e1 - 14, Kn = c0 + sc;
            const float f = __builtin_ldexpf(dec, K - Kn < 120 ? K - Kn : 120);
            bound = __builtin_fmaf(bound, f, __builtin_ldexpf(1.0f, 27 - sc));
            if (!finite(bound)) bound = 0x1p14f;
            K = Kn;
            const _Float16 sf = (_Float16)__builtin_ldexpf(1.0f, sc < 24 ? -sc : -24);
            const _Float16 sw = (_Float16)__builtin_ldexpf(1.0f, sc < 24 ? 0 : 24 - sc);
            auto read_b = [&](int g) {  // four operands in the order (hh, nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) bq[g & 1][k] = *(const f16x8 *)(sh.B[i & 1] + ((4 * g + k) * 64 + lane) * 8);
            };
            read_b(0);
            f32x4 rv[4];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) rv[tt] = *(const f32x4 *)(sh.scale[i % 3] + 16 * q + 4 * tt);
            __builtin_amdgcn_sched_barrier(0);
            // the masked product
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) Y[tt][c] = mfma(mo[tt][hh], x16[c][hh], Y[tt][c]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) acc[nt][c] *= f;
            f16x8 v[2][2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int c = 0; c < 2; ++c) v[c][hh] = (x16[c][hh] * sf) * (wv[hh] * sw);
            __builtin_amdgcn_sched_barrier(0);
            // the state's products, and in between y: ahead of what the SIMD's other
            // wave begins (eight prompts of 4096 tokens 255 -> 249 us)
            __builtin_amdgcn_s_setprio(1);
            const float dx = __builtin_ldexpf(dsk, ex - 14);
            const auto yb = buffer((const char *)a.y + (int64_t)(u.begin + t) * yrow + u.ch0 * 2, (rem - 1) * yrow + 64);
            uint32_t yo = 16 * q * yrow + 4 * r;
            asm volatile("" : "+v"(yo));
            constexpr int GB = NT / 2;  // groups of four operands
#pragma unroll
            for (int g = 0; g < GB; ++g) {
                if (g + 1 < GB) read_b(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int hh = (4 * g + k) / NT, nt = (4 * g + k) % NT;
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[nt][c] = mfma(bq[g & 1][k], v[c][hh], acc[nt][c]);
                }
#pragma unroll
                for (int tt = g * 4 / GB; tt < (g + 1) * 4 / GB; ++tt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * tt + e;
                        const float be = __builtin_ldexpf(rv[tt][e], E2);
                        float o[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) o[c] = __builtin_fmaf((float)x16[c][j / 8][j % 8], dx, Y[tt][c][e] * be);
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, bf16x2{(__bf16)o[0], (__bf16)o[1]}), yb, yo, 0, 0);
                        yo += yrow;
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (anybad) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o = badm[c];
                    o |= __shfl_xor(o, 16);
                    o |= __shfl_xor(o, 32);
                    if (o)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[nt][c][e] = __builtin_nanf("");
                }
            }
            __builtin_amdgcn_s_setprio(0);
            if (more) begin_chunk(i + 1, of_ex(exbn), edn, eBn);
        }
    }

    if (u.k != u.nseg - 1) return;
    if (u.on && one && resume && from < to) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) *(f32x4 *)(cache + c * N + 16 * nt) = *(const f32x4 *)(own + c * N + 16 * nt);
    }
    // the window: the last three raw rows, of the wave's channels and, once per
    // group, of its B and C
    auto row = [&](int t, int64_t c) {
        return t < 0 ? a.ws_win[((int64_t)u.s * 3 + t + 3) * a.C + c]
                     : ((const uint16_t *)a.xBC)[(int64_t)(u.begin + t) * a.xBC_stride + c];
    };
    uint16_t *win = (uint16_t *)a.conv_cache + (int64_t)slot * a.C * 3;
    if (u.on && q < 3)
#pragma unroll
        for (int c = 0; c < 2; ++c) win[(int64_t)(u.ch0 + 2 * r + c) * 3 + q] = row((int)u.len - 3 + q, u.ch0 + 2 * r + c);
    if (u.hb == 0)
        for (int i = threadIdx.x; i < 2 * N * 3; i += 64 * WAVES) {
            const int n = i / 3;
            const int64_t c = a.H * a.P + ((n / N) * a.G + u.g) * N + n % N;
            win[c * 3 + i % 3] = row((int)u.len - 3 + i % 3, c);
        }
}

template <int N>
hipError_t launch_n(const SsdCacheArgs &a, hipStream_t s) {
    constexpr int64_t threads = prep_threads(N);
    const int64_t parts = (a.C + threads - 1) / threads, dts = (a.H + dt_heads(N) - 1) / dt_heads(N);
    const unsigned prep = (unsigned)(a.nchunk * (a.G + dts) + a.seqs * parts);
    if (a.ws_plan) hipLaunchKernelGGL((prepare_kernel<N, true>), dim3(prep + 1), dim3(threads), 0, s, a);
    else hipLaunchKernelGGL((prepare_kernel<N, false>), dim3(prep), dim3(threads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t ncb = a.H / a.G * (a.P / 64);
    auto grid = [&](int blocks) { return dim3((unsigned)((a.nseg * a.G * ((ncb + blocks - 1) / blocks) + 7) / 8 * 8)); };
    hipLaunchKernelGGL((walk_state_kernel<N>), grid(kBlocksA), dim3(128 * kBlocksA), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.rows > a.seg) {  // some sequence may be longer than a segment: at least this long
        hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.H * a.P * N + 1023) / 1024), (unsigned)a.seqs), dim3(256), 0, s, a, N);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((walk_out_kernel<N>), grid(kBlocksC), dim3(128 * kBlocksC), 0, s, a);
    return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether the segment length is chosen on the device, which knows the lengths: a
// wave looks at every sequence in turn, up to 5 us for this many.
bool planned(int64_t seqs) { return seqs > 1 && seqs <= 256; }

// Tokens per segment, the least of them where the device chooses: at most 4
// rounds of 512 workgroups of walk A whatever the lengths are, (rows + seqs (seg -
// 1)) / seg segments in the worst case, for the workspace and the launches. One
// sequence: the length that costs least over 1 to 8 rounds, a round costing a
// segment's chunks and about two more (16384 tokens of 80 heads in one round 270
// us, in two 287).
int64_t segment_tokens(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G) {
    const int64_t units = G * ((H / G * (P / 64) + kBlocksA - 1) / kBlocksA);
    if (seqs > 1) {
        const int64_t most = 512 * 4 / units;  // segments
        if (most <= seqs) return 2048;
        const int64_t seg = (rows - seqs + most - seqs) / (most - seqs);
        return seg > 2048 ? 2048 : seg < kQ ? kQ : (seg + kQ - 1) / kQ * kQ;
    }
    int64_t best = (rows + kQ - 1) / kQ * kQ, cost = INT64_MAX;
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
        const int64_t most = 512 * rounds / units;
        if (most < 1) continue;
        int64_t seg = (rows + most - 1) / most;
        seg = (seg < kQ ? kQ : seg + kQ - 1) / kQ * kQ;
        const int64_t c = rounds * (seg / kQ + 2);
        if (c < cost) cost = c, best = seg;
    }
    return best < kQ ? kQ : best;
}

// Cuts the workspace up; returns its size.
size_t plan(SsdCacheArgs &a, int N, char *base) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = base + at;
        at += up256(bytes);
        return p;
    };
    a.seg = segment_tokens(a.seqs, a.rows, a.H, a.P, a.G);
    a.nchunk = a.rows / kQ + a.seqs;
    a.nseg = a.rows / a.seg + a.seqs;
    const size_t chunks = (size_t)a.nchunk;
    a.ws_slot = (int32_t *)take((size_t)a.seqs * 4);
    a.ws_plan = planned(a.seqs) ? (int32_t *)take((size_t)(a.seqs + 2) * 4) : nullptr;
    a.ws_win = (uint16_t *)take((size_t)a.seqs * 3 * a.C * 2);
    a.ws_frag = take(chunks * a.G * frag_elems(N) * 2);
    a.ws_head = (float *)take(chunks * a.H * kHead * 4);
    a.ws_w = (float *)take(chunks * a.H * kQ * 4 + 1024);  // read four heads at a time
    a.ws_meta = (float *)take(chunks * a.H * 16);
    a.ws_eb = (int32_t *)take(chunks * a.G * 4);
    a.ws_ex = (int32_t *)take(chunks * (a.H * a.P / 32) * 4);
    a.ws_x = take(chunks * (a.H * a.P / 32) * 4096);
    a.ws_state = (float *)take((size_t)a.nseg * a.H * a.P * N * 4);
    a.ws_segdec = (float *)take((size_t)a.nseg * a.H * 4);
    return at;
}

}  // namespace

size_t ssd_cache_workspace(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N) {
    SsdCacheArgs a{};
    a.seqs = seqs;
    a.rows = rows;
    a.H = H;
    a.P = P;
    a.G = G;
    a.C = H * P + 2 * G * N;
    return plan(a, (int)N, nullptr);
}

hipError_t launch_ssd_cache(SsdCacheArgs a, int N, void *workspace, hipStream_t s) {
    plan(a, N, (char *)workspace);
    return N == 64 ? launch_n<64>(a, s) : launch_n<128>(a, s);
}

}  // namespace ssm
