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
// Precision. Operands are sums of bfloat16, 8 bits a part: bfloat16 has float32's
// range, so nothing carries a scale that channels, columns or tokens of unlike size
// would share. The state must come out as a float32 state would, so the products
// of walk A take both operands in three parts (24 bits; six products, those left
// out are below 2^-24 of the whole). The products for y, which is rounded to
// bfloat16 (8 bits) in the end, take them in two (16 bits; three products): the
// state as walk C reads it, C, the masked matrix (with D on its diagonal), x and,
// for walk C's own copy of the state, B and w o x. G, the decays, every sum and
// the state itself are float32, the summed exponents of the decays float64. x goes through as x times -log2(e), which SiLU's
// exponential needs; the other factor, -ln(2), stands in w, in dt and in D.
#include "ssm_common.h"
#include "ssm_device.h"
#include "ssm_internal.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

constexpr int kQ = 64;            // tokens per chunk
// Threads of a workgroup ahead of the walks: a lane convolves four channels of
// four tokens (256 threads and 16 tokens took 1.6 times as long for one chunk).
constexpr int prep_threads(int N) { return 8 * N; }
constexpr int kBlocksA = 2;       // column blocks of 64 per workgroup of walk A, two waves each
constexpr int kBlocksC = 4;       // of walk C

// Workspace of one (chunk, group), in pieces of 1 KiB, a register of 16 bytes of
// each lane: B (half, part of 3, n tile), C (part of 2, token tile, 32 of n), G in
// float32 (token tile, half, four tokens).
constexpr int pieces_b(int N) { return 6 * N / 16; }
constexpr int pieces_c(int N) { return 8 * N / 32; }
constexpr int pieces_g() { return 16; }
constexpr int64_t frag_bytes(int N) { return (pieces_b(N) + pieces_c(N) + pieces_g()) * 1024; }
// Floats per (chunk, head) for walk C: cum rounded to float32, -ln(2) dt 2^-rest,
// exp2(cum), 2^rest, where rest is what that rounding leaves of cum.
constexpr int kHead = 4 * kQ;
// Heads of a wave that forms decays (80 heads then take one workgroup per chunk at
// N = 128: 16384 tokens 21.9 -> 18.9 us against two heads, a short prompt the same).
constexpr int kDtHeads = 5;
constexpr int dt_heads(int N) { return prep_threads(N) / 64 * kDtHeads; }

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
// to 4900 tokens, 80 heads 830 -> 786, 13 of 4099, 32 heads 81 -> 64, 9 of 4148
// tokens, 68 heads 162 -> 128, 3 of 19798 tokens, 34 heads 300 -> 228; 45 of 5143
// tokens, 4 heads 50 both ways.
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
    float raw[kDtHeads], bias[kDtHeads];
    double A2[kDtHeads];
#pragma unroll
    for (int k = 0; k < kDtHeads; ++k) {
        const uint32_t h = h0 + k < H ? h0 + k : H - 1;
        raw[k] = ld_act(src, h);
        bias[k] = a.dt_bias ? a.dt_bias[h] : 0.0f;
        A2[k] = (double)a.A[h] * 1.4426950408889634;
    }
#pragma unroll
    for (int k = 0; k < kDtHeads; ++k) {
        if (h0 + k >= H) break;
        const int64_t at = (int64_t)id * H + h0 + k;
        const float dt = lane < rem ? softplus(raw[k] + bias[k]) : 0.0f;
        // A decay of 2^-256 leaves nothing of a float32 state: no more than that. The
        // sums reach 2^14 and are differenced, so they are held in double precision
        // and handed on in two parts. A step that is not finite is a NaN from here on,
        // not a decay to nothing.
        double step = (double)dt * A2[k];
        step = step < -256.0 ? -256.0 : step;
        if (!finite(dt)) step = __builtin_nan("");
        const double cum = wave_prefix_sum(step), total = __shfl(cum, 63);
        const float top = (float)cum, rest = (float)(cum - (double)top);
        const float own = dt * -kLn2 * fast_exp2(-rest), decay = fast_exp2(top) * fast_exp2(rest);
        float *o = a.ws_head + at * kHead;
        o[lane] = top;
        o[kQ + lane] = finite(own) ? own : 0.0f;  // stands beside zeros of G for the tokens before
        o[2 * kQ + lane] = decay;
        o[3 * kQ + lane] = fast_exp2(rest);
        a.ws_w[at * kQ + lane] = dt * -kLn2 * fast_exp2((float)(total - cum));
        if (lane == 63) a.ws_dec[at] = decay;
    }
}

// Bound by latency and by its stores of 1.3 KB per (chunk, head) and 96 KB per
// (chunk, group) together: 8.2 us for one chunk (3 of them an empty launch), 18.9 us
// for 16384 tokens of 80 heads (52 MB). B and C are held as float32 in LDS and split
// where they are read. The heads' decays have workgroups of their own, so that a
// short prompt waits for neither: done by the workgroups that convolve B and C, one
// chunk took 2 us more and 16384 tokens 4.
// PLAN: one workgroup more, the first, chooses the segments (in every launch, its
// code alone takes 3 us more).
template <int N, bool PLAN>
__global__ __launch_bounds__(prep_threads(N), 8) void prepare_kernel(SsdCacheArgs a) {
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
#pragma unroll
    for (int i = 0; i < TPB; ++i) {
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            auto at = [&](int j) {
                const uint32_t u = k < 2 ? raw[i + j].x : raw[i + j].y;
                return __uint_as_float(k % 2 ? u & 0xffff0000u : u << 16);
            };
            v[k] = t0 + i < rem ? conv_silu(w[k][0], w[k][1], w[k][2], w[k][3], bias[k], at(0), at(1), at(2), at(3)) : 0.0f;
        }
        *(f32x4 *)(isC ? &sh.C[t0 + i][n0] : &sh.B[t0 + i][n0]) = v;
    }
    __syncthreads();

    constexpr int NT = N / 16, KB = N / 32;
    char *const out = (char *)a.ws_frag + ((int64_t)id * a.G + g) * frag_bytes(N);
    const int r = lane & 15, q = lane >> 4;
    // Each wave forms one of B^T's operands, (h, nt): row n = 16 nt + r, k = token
    // 16 q + 8 h + j;
    static_assert(2 * NT == WAVES && 4 * KB == WAVES);
    {
        const int h = wave / NT, nt = wave % NT;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = sh.B[16 * q + 8 * h + j][16 * nt + r];
        bf16x8 part[3];
        split(t, part);
#pragma unroll
        for (int p = 0; p < 3; ++p) ((bf16x8 *)out)[((h * 3 + p) * NT + nt) * 64 + lane] = part[p];
    }
    // one of C's, (tt, m): row r is token 16 (r / 4) + 4 tt + r % 4, and k runs
    // over n in the order in which two accumulator tiles hold the state;
    const int row = 16 * (r / 4) + r % 4;
    {
        const int tt = wave / KB, m = wave % KB;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) *(f32x4 *)(t + j) = *(const f32x4 *)&sh.C[row + 4 * tt][32 * m + 4 * q + 4 * j];
        bf16x8 part[2];
        split(t, part);
#pragma unroll
        for (int p = 0; p < 2; ++p) ((bf16x8 *)(out + pieces_b(N) * 1024))[(p * 4 * KB + wave) * 64 + lane] = part[p];
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
        for (int m = 0; m < KB; ++m) {
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
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = s0 + e <= row + 4 * tt ? acc[e] : 0.0f;
        ((f32x4 *)(out + (pieces_b(N) + pieces_c(N)) * 1024))[f * 64 + lane] = acc;
    }
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
        if (PIECES % WAVES == 0 || p < PIECES) dma16_s((const char *)src + p * 1024, lane * 16, dst + p * 1024);
    }
}

// Walk A: x, and the segment's end state. B lies in LDS by halves of a chunk (48 KB
// of three parts each chunk at N = 128), three of them in turn, so that two
// workgroups share a CU, two waves a SIMD; a barrier before each half's products
// says that it has come and that the one before it may be overwritten.
//
// Bound by instruction issue: per chunk and wave the convolution and SiLU of 32
// values a lane, their split into three bfloat16 and 192 products (N = 128), from
// two waves per SIMD, which is what the state's 64 registers and the operands
// leave room for (235 of 256). 16384 tokens of 80 heads: 153 us for 168 MB of x
// read and twice as much written. Operands of two float16 (22 bits, three products, 114
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

    // The convolution times -log2(e): its exp2 is SiLU's exponential.
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
        pieces<pieces_b(N) / 2, 2 * kBlocksA>((const char *)a.ws_frag + ((int64_t)id * G + u.g) * frag_bytes(N) + half * (pieces_b(N) / 2 * 1024),
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
                    x[c][i] = v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(v));
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
            dec = ((cf32_ptr)a.ws_dec)[(int64_t)id * H + u.h];
            segdec *= dec;
            // x as walk C's operand, in two parts. One whose first is not finite would
            // reach earlier tokens there as 0 times itself: that is marked.
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(__builtin_fabsf(x[c][i]), top);  // keeps a NaN
            const int64_t at = (int64_t)id * (a.H * a.P / 32) + u.ch0 / 32;
            const bool anybad = __ballot(!(top < 0x1.ffp127f)) != 0;
            if (lane == 0) a.ws_bad[at] = anybad;
            bf16x8 *dst = (bf16x8 *)a.ws_x + at * 512 + lane;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float t[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) t[j] = x[c][8 * hh + j];
                    bf16x8 part[2];
                    split(t, part);
#pragma unroll
                    for (int p = 0; p < 2; ++p) dst[((p * 2 + c) * 2 + hh) * 64] = part[p];
                }
            // The convolution stands before the products of the SIMD's other wave: the
            // matrix cores are then fed while it runs (16384 tokens 171 -> 153 us).
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
// four ahead take a prompt of 21507 tokens, 8 heads, from 117 to 100 us.
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
// masked matrix and put it into LDS as operand registers. A chunk is begun (C S^T
// and the masked matrix, from C, G and the decays in LDS) and finished (the masked
// product, y, the state, from B), with a barrier behind each; what one phase has
// read is loaded again for the next chunk during the other. One workgroup fills a
// CU (154 KB of LDS at N = 128).
//
// Two waves per SIMD run 240 products each per chunk (N = 128) in 0.38 of its cycles
// and issue vector instructions (the splits of the state, of the masked matrix and
// of w o x, its exponentials) in 0.44; the rest waits for LDS and at the barriers.
// 16384 tokens of 80 heads: 207 us. With single float16 operands (80 products, no
// splits, one barrier per chunk) 113, but those hold 11 bits and need scales that
// channels and tokens share. Steps interleaved by hand, priorities and x loaded a
// phase earlier changed nothing.
template <int N>
__global__ __launch_bounds__(128 * kBlocksC, 2) void walk_out_kernel(SsdCacheArgs a) {
    constexpr int NT = N / 16, KB = N / 32, WAVES = 2 * kBlocksC;
    struct Shared {
        bf16x8 B[2][2][NT][64];  // half, part, n tile
        bf16x8 C[2][4][KB][64];  // part, token tile, 32 of n
        f32x4 G[4][2][2][64];    // token tile, half, four tokens
        f32x4 head[2][kBlocksC][kHead / 4];
        f32x4 w[2][4][kQ / 4];
        bf16x8 M[kBlocksC][2][4][2][64];  // part, token tile, half
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

    auto operands = [&](uint32_t t) {
        return (const char *)a.ws_frag + ((int64_t)(u.chunk0 + t / kQ) * G + u.g) * frag_bytes(N);
    };
    auto stage_b = [&](uint32_t t) {  // two parts of the three
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) pieces<2 * NT, WAVES>(operands(t) + hh * 3 * NT * 1024, sh.B[hh], wave, lane);
    };
    auto stage_cg = [&](uint32_t t) {
        const int b = (int)((t - from) / kQ & 1);
        const uint32_t first = (u.chunk0 + t / kQ) * H;  // chunks times heads: below 2^24
        static_assert(offsetof(Shared, G) == offsetof(Shared, C) + pieces_c(N) * 1024);
        pieces<pieces_c(N) + pieces_g(), WAVES>(operands(t) + pieces_b(N) * 1024, sh.C, wave, lane);
        if (wave % 2 == 0 && u.on) dma16_s(a.ws_head + (int64_t)uniform(first + u.h) * kHead, lane * 16, lds_addr(sh.head[b][wave / 2]));
        // w of four heads, the first one or all of them needed
        if (wave == WAVES - 1) dma16_s(a.ws_w + (int64_t)uniform(first + u.hfirst) * kQ, lane * 16, lds_addr(sh.w[b]));
    };
    if (from < to) {
        stage_cg(from);
        stage_b(from);
        if (!u.on) {  // no columns: the wave only carries its share of the loads
            vm_wait();
            lds_barrier();
            for (uint32_t t = from; t < to; t += kQ) {
                vm_wait();
                lds_barrier();
                if (t + kQ >= to) break;
                stage_cg(t + kQ);
                vm_wait();
                lds_barrier();
                stage_b(t + kQ);
            }
        }
    }

    // the state: acc[nt][c][e] = S[p = 2 r + c][n = 16 nt + 4 q + e]
    const int64_t off = (int64_t)(u.ch0 + 2 * r) * N + 4 * q, hpn = a.H * a.P * N;
    const bool resume = u.resume, one = u.nseg == 1;
    float *const cache = a.state_cache + (int64_t)slot * hpn + off;
    const float *const own = a.ws_state + (int64_t)u.sid * hpn + off;
    if (u.on && from < to) {
        f32x4 acc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[nt][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (resume || u.k > 0) {
            const float *src = one ? cache : own;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) acc[nt][c] = *(const f32x4 *)(src + c * N + 16 * nt);
        }
        // D on the diagonal of the masked matrix, for the wave's half: of the token
        // tiles tt = 2 (wave % 2) + k2 the elements (h = wave % 2, j = 4 k2 + r % 4)
        // of the lanes with q = r / 4
        const float dsk = a.Dskip && q == r / 4 ? a.Dskip[u.h] * -kLn2 : 0.0f;
        float diag[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) diag[j] = j == r % 4 ? dsk : 0.0f;
        const int mine = wave % 2;

        vm_wait();
        lds_barrier();  // the first chunk is in LDS
        for (uint32_t t = from; t < to; t += kQ) {
            const int b = (int)((t - from) / kQ & 1), rem = to - t < kQ ? (int)(to - t) : kQ;
            const bool more = t + kQ < to;
            const int64_t id = u.chunk0 + t / kQ, at = id * (a.H * a.P / 32) + u.ch0 / 32;
            const f32x4 *hd = sh.head[b][wave / 2];
            const float *hf = (const float *)hd;

            bf16x8 x[2][2][2];  // part, c, half
            {
                const bf16x8 *src = (const bf16x8 *)a.ws_x + at * 512 + lane;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) x[p][c][hh] = src[((p * 2 + c) * 2 + hh) * 64];
            }
            const bool anybad = ((const __attribute__((address_space(4))) int *)a.ws_bad)[at] != 0;
            const float dec = hf[2 * kQ + kQ - 1];

            // C S^T of the chunk, and in between the wave's half of the masked matrix,
            // M[t][s] = G[t][s] exp2(cum_t - cum_s) dt_s: steps of two token tiles and 32
            // of n, their operands read from LDS one step ahead
            f32x4 Y[4][2];
            bf16x8 co[2][2][2];  // step, part, tile
            auto read_c = [&](int i) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k) co[i & 1][p][k] = sh.C[p][2 * (i & 1) + k][i / 2][lane];
            };
            read_c(0);
            const float *hrow = hf + 16 * (r / 4) + r % 4 + 8 * mine;
            const float ct[2] = {hrow[0], hrow[4]}, rest[2] = {hrow[3 * kQ], hrow[3 * kQ + 4]};
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int c = 0; c < 2; ++c) Y[tt][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 so[2][2];  // part, c
#pragma unroll
            for (int i = 0; i < 2 * KB; ++i) {
                const int m = i / 2;
                if (i + 1 < 2 * KB) read_c(i + 1);
                __builtin_amdgcn_sched_barrier(0);
                if (i % 2 == 0)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = acc[2 * m + e / 4][c][e % 4];
                        bf16x8 part[2];
                        split(v, part);
                        so[0][c] = part[0], so[1][c] = part[1];
                    }
#pragma unroll
                for (int p = kTwo; p < 6; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            Y[2 * (i & 1) + k][c] = mfma(co[i & 1][kTerm[p][0]][k], so[kTerm[p][1]][c], Y[2 * (i & 1) + k][c]);
#pragma unroll
                for (int o = i * 4 / (2 * KB); o < (i + 1) * 4 / (2 * KB); ++o) {
                    const int k2 = o / 2, hh = o % 2, tt = 2 * mine + k2;
                    float v[8];
#pragma unroll
                    for (int h4 = 0; h4 < 2; ++h4) {
                        const f32x4 gv = sh.G[tt][hh][h4][lane], cs = hd[4 * q + 2 * hh + h4], dt = hd[kQ / 4 + 4 * q + 2 * hh + h4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            // G is zero above the diagonal, where the exponent may be large
                            v[4 * h4 + j] = gv[j] * dt[j] * fast_exp2(__builtin_fminf(ct[k2] - cs[j], 126.0f)) * rest[k2];
                    }
                    const float dg = hh == mine ? 1.0f : 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * k2 + j] = __builtin_fmaf(diag[j], dg, v[4 * k2 + j]);
                    bf16x8 part[2];
                    split(v, part);
#pragma unroll
                    for (int p = 0; p < 2; ++p) sh.M[wave / 2][p][tt][hh][lane] = part[p];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                const f32x4 ec = hd[2 * kQ / 4 + 4 * q + tt];
#pragma unroll
                for (int c = 0; c < 2; ++c) Y[tt][c] *= ec;
            }

            vm_wait();
            lds_barrier();  // M is whole, B is in LDS, and every wave is done with C, G and the decays
            if (more) stage_cg(t + kQ);
            uint32_t badm[2] = {0u, 0u};
            if (anybad) {
                // values that are not finite: zero for the products, and what
                // they reach (their channel, from their token on) becomes NaN
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        u32x4 v[2] = {__builtin_bit_cast(u32x4, x[0][c][hh]), __builtin_bit_cast(u32x4, x[1][c][hh])};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t bits = 0x7f80u << 16 * (j % 2);
                            if ((v[0][j / 2] & bits) == bits) {
                                badm[c] |= 1u << (8 * hh + j);
                                v[0][j / 2] &= ~(0xffffu << 16 * (j % 2));
                                v[1][j / 2] &= ~(0xffffu << 16 * (j % 2));
                            }
                        }
                        x[0][c][hh] = __builtin_bit_cast(bf16x8, v[0]);
                        x[1][c][hh] = __builtin_bit_cast(bf16x8, v[1]);
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
            // the masked product; steps of two token tiles and a half, as above. In
            // between w o x and the state's decay.
            bf16x8 mo[2][2][2], v[2][2][2];  // step, part, tile; part, c, half
            auto read_m = [&](int i) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k) mo[i & 1][p][k] = sh.M[wave / 2][p][2 * (i & 1) + k][i / 2][lane];
            };
            read_m(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hh = i / 2;
                if (i + 1 < 4) read_m(i + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int p = kTwo; p < 6; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            Y[2 * (i & 1) + k][c] = mfma(mo[i & 1][kTerm[p][0]][k], x[kTerm[p][1]][c][hh], Y[2 * (i & 1) + k][c]);
                {
                    const int c = i & 1;
                    const f32x4 *wt = sh.w[b][u.h - u.hfirst] + 4 * q + 2 * hh;
                    const f32x4 w0 = wt[0], w1 = wt[1];
                    const u32x4 hi = __builtin_bit_cast(u32x4, x[0][c][hh]), lo = __builtin_bit_cast(u32x4, x[1][c][hh]);
                    float wx[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        wx[j] = (__uint_as_float(hi[j / 2] << 16) + __uint_as_float(lo[j / 2] << 16)) * (j < 4 ? w0[j % 4] : w1[j % 4]);
                        wx[j + 1] = (__uint_as_float(hi[j / 2] & 0xffff0000u) + __uint_as_float(lo[j / 2] & 0xffff0000u)) *
                                    (j < 4 ? w0[j % 4 + 1] : w1[j % 4 + 1]);
                    }
                    bf16x8 part[2];
                    split(wx, part);
                    v[0][c][hh] = part[0], v[1][c][hh] = part[1];
                }
#pragma unroll
                for (int nt = i * NT / 4; nt < (i + 1) * NT / 4; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[nt][c] *= dec;
                __builtin_amdgcn_sched_barrier(0);
            }
            // the state's products, and in between y
            bf16x8 bo[2][2][2];  // step, part, tile
            auto read_b = [&](int i) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k) bo[i & 1][p][k] = sh.B[i / (NT / 2)][p][2 * (i % (NT / 2)) + k][lane];
            };
            read_b(0);
            const auto yb = buffer((const char *)a.y + (int64_t)(u.begin + t) * yrow + u.ch0 * 2, (rem - 1) * yrow + 64);
            uint32_t yo = 16 * q * yrow + 4 * r;
            asm volatile("" : "+v"(yo));
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int hh = i / (NT / 2), nt = 2 * (i % (NT / 2));
                if (i + 1 < NT) read_b(i + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int p = kTwo; p < 6; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int c = 0; c < 2; ++c) acc[nt + k][c] = mfma(bo[i & 1][kTerm[p][0]][k], v[kTerm[p][1]][c][hh], acc[nt + k][c]);
#pragma unroll
                for (int j = i * 16 / NT; j < (i + 1) * 16 / NT; ++j) {
                    __builtin_amdgcn_raw_buffer_store_b32(
                        __builtin_bit_cast(uint32_t, bf16x2{(__bf16)Y[j / 4][0][j % 4], (__bf16)Y[j / 4][1][j % 4]}), yb, yo, 0, 0);
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
            if (!more) break;
            // Issued since the barrier before: the next chunk's C, G and decays, then the
            // 16 stores of y, which may stay in flight (accesses complete in order).
            asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
            lds_barrier();  // they are in LDS, and every wave is done with B and M
            stage_b(t + kQ);
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

// Workgroups of walk A per segment.
int64_t segment_units(int64_t H, int64_t P, int64_t G) { return G * ((H / G * (P / 64) + kBlocksA - 1) / kBlocksA); }

// Tokens per segment, the least of them where the device chooses: at most 4
// rounds of 512 workgroups of walk A whatever the lengths are, (rows + seqs (seg -
// 1)) / seg segments in the worst case, for the workspace and the launches. One
// sequence: the length that costs least over 1 to 8 rounds, a round costing a
// segment's chunks and about two more (16384 tokens of 80 heads in one round 386
// us, in two 409).
int64_t segment_tokens(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G) {
    const int64_t units = segment_units(H, P, G);
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

// The segments that the workspace holds: at least as many as the length above gives,
// and never fewer for more rows or sequences, although that length goes by steps; so
// that a workspace made for the largest batch serves any smaller one.
//
// One sequence in k rounds of m_k workgroups has m_k + 1 at most. k rounds are
// chosen before the first j that fit only if k (c / m_k + 2) < j (c / m_j + 3), c =
// rows / 64, which for large c stays true once it is; then m_k counts. Several
// sequences: the length is above (rows - seqs) / (most - seqs) wherever it is not
// 2048, and so rows / seg is below most - seqs + seqs / 64.
int64_t most_segments(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G) {
    const int64_t units = segment_units(H, P, G), chunks = rows / kQ + 1;
    int64_t one = 1, j = 0, mj = 0;
    for (int64_t k = 1; k <= 8; ++k) {
        const int64_t m = 512 * k / units;
        if (m < 1) continue;
        if (j == 0) {
            j = k, one = mj = m;
            continue;
        }
        const int64_t gain = j * m - k * mj, cost = (2 * k - 3 * j) * mj * m;
        if ((gain > 0 ? chunks * gain > cost : cost < 0) && m > one) one = m;
    }
    int64_t n = one + 1;
    if (seqs > 1) {
        const int64_t most = 512 * 4 / units + seqs / kQ + 1, whole = rows / 2048 + seqs;
        n = n > most ? n : most;
        n = n > whole ? n : whole;
    }
    const int64_t all = rows / kQ + seqs;
    return n < all ? n : all;
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
    a.ws_frag = take(chunks * a.G * frag_bytes(N));
    a.ws_head = (float *)take(chunks * a.H * kHead * 4);
    a.ws_w = (float *)take(chunks * a.H * kQ * 4 + 1024);  // read four heads at a time
    a.ws_dec = (float *)take(chunks * a.H * 4);
    a.ws_bad = (int32_t *)take(chunks * (a.H * a.P / 32) * 4);
    a.ws_x = take(chunks * (a.H * a.P / 32) * 8192);
    const size_t most = (size_t)most_segments(a.seqs, a.rows, a.H, a.P, a.G);
    a.ws_state = (float *)take(most * a.H * a.P * N * 4);
    a.ws_segdec = (float *)take(most * a.H * 4);
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
