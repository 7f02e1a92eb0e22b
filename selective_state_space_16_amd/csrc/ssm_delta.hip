// The gated delta rule over packed prompts, on a cache of states (gfx950):
// sequences of different lengths lie one behind the other in one array of rows,
// each starts from zero or from the state in its cache slot, and leaves it there.
//
//   q' = q scale / sqrt(|q|^2 + eps),  k' = k / sqrt(|k|^2 + eps)
//   a  = exp(softplus(dt_raw + dt_bias) A),  beta = 1 / (1 + exp(-beta_raw))
//   u[p]    = beta (v[p] - a sum_n S[p][n] k'[n])
//   S[p][n] = a S[p][n] + u[p] k'[n],   y[p] = sum_n S[p][n] q'[n]
//
// Every sequence is cut into chunks of 64 tokens. With G_i the summed log decay from
// the chunk's start through token i, S the state that enters it and
//
//   A_ij = beta_i e^(G_i - G_j) k'_i.k'_j  (j < i),   T = (I + A)^-1
//   M_ij = e^(G_i - G_j) q'_i.k'_j  (j <= i)
//
// a chunk's updates solve (I + A) U = diag(beta) (V - diag(e^G) K' S^T), and
//
//   U  = T diag(beta) (V - diag(e^G) K' S^T)
//   y  = diag(e^G) Q' S^T + M U
//   S^T <- e^(G_last) S^T + (diag(e^(G_last - G)) K')^T U
//
// T and M depend on keys, queries and gates alone: the first kernel forms them for
// all chunks at once, the second walks the chunks of a sequence in order.
//
// The walk keeps everything that one chunk hands to the next in one wave's registers.
// A column of S^T (a row p of the state) never meets another, so a wave takes 16 of
// them and all of N and of the 64 tokens (a call that leaves most of the chip idle so
// has each 16 columns shared by N / 32 waves instead: delta_team_kernel). The matrix
// cores leave a result with its rows in a lane's registers and its columns across 16
// lanes, and take their right operand with the summed index in a lane's registers: the
// result of one product is the next one's right operand as it stands, once its rows are
// numbered so that the two tiles of 16 rows hold, lane for lane, the eight consecutive
// indexes of the operand (tile_row). Keys, queries, T, M and the transposed keys are left
// operands, shared by the waves of a workgroup through LDS, laid out there (and by
// the first kernel in the workspace) as a wave loads them.
//
// Precision. Keys and queries are bfloat16 as they come; their lengths, the gates and
// the decays are factors per token, applied in float32 to what they multiply. The
// other operands (S, T, M, beta (V - ..), U) are sums of three bfloat16, 8 bits a part,
// which hold a float32 whole: the state and y, before its one rounding, come out as a
// float32 recurrence leaves them, also where large terms of y cancel. (With two parts in
// the products for y the walk of eight prompts of 4096 tokens took 525 us instead of 610.)
// Sums are float32, the summed log decays float64.
//
// Where an update is not finite, because an input is not, zeros of T and M no longer
// keep a token from those before it: such a chunk is taken a token at a time instead,
// from the state that entered it. A state that is not finite stays so, and with it the
// sequence's later chunks are taken so too: 0.9 us a token in the walk, where the whole
// workgroup waits for one wave's column, 1.8 us in a team (eight prompts of 4096 tokens
// with a NaN in the middle of the first 0.85 -> 2.7 ms, one of 16384 tokens 0.86 -> 15.5).
//
// Measured (us): 16384 tokens of 32 heads of 128 x 128, 140 ahead of the chunks and 725
// for them (2.8 a chunk); eight prompts of 4096 tokens, 275 and 620; one chunk of 24
// heads 9.5 and 7. The first kernel takes four workgroups of 36 KB a CU (three of 53 KB
// took 165 and 300); a wave waits there for the keys' tiles that it loads one after the
// other, for T's chain of substitutions and products and at five barriers. The chunks are
// bound by the instructions of a wave: 863 vector instructions a chunk, 216 of them
// products, the matrix cores busy for 34 % of the time.
#include "ssm_delta_device.h"
#include "ssm_packed.h"

namespace ssm {

namespace {

constexpr int kQ = 64;  // tokens per chunk
constexpr int kPrepThreads = 256;
// T and M as left operands: (tile of 16 rows, 32 of the columns) where the columns
// are not wholly above the diagonal, a register of 16 bytes of each lane per part.
constexpr int kTri = 6, kParts = 3;
constexpr int kFragTM = kTri * (kParts + kParts - 1);  // pieces of 1 KiB per (chunk, head): T, and M but for its last part
// behind them one of factors per token, e^G / |k|, beta, e^(G_last - G) / |k|, scale e^G / |q|, then M's last part
constexpr int kFactors = kFragTM, kLastM = kFactors + 1, kHeadPieces = kLastM + kTri;
constexpr int piece_t(int tri, int part) { return kParts * tri + part; }
constexpr int piece_m(int tri, int part) { return part < 2 ? kTri * kParts + 2 * tri + part : kLastM + tri; }
constexpr int pieces_kt(int N) { return 2 * N / 16; }  // of the transposed keys per (chunk, group)

__device__ __forceinline__ int tri_index(int tile, int half) { return tile < 2 ? tile : 2 * tile - 2 + half; }  // (tiles 0, 1: half 0 alone)

// The index, within 64 tokens or N keys' elements, of row m of tile t: two tiles share
// 32 indexes, of which lane group m / 4 holds eight consecutive ones.
__device__ __forceinline__ int tile_row(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// The first of the two tiles that the three groups of products with T and M take; the
// last group's columns are the second half.
constexpr int kTile[3] = {0, 2, 2};

// In what order the compiler places what stands ahead: READS reads of LDS; or COUNT
// products with VALU other instructions behind each.
template <int READS>
__device__ __forceinline__ void interleave_reads() {
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
}
template <int COUNT, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, VALU, 0);
    }
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Eight bfloat16 as floats.
__device__ __forceinline__ void ld8(const uint16_t *p, float *v) {
    const u32x4 u = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// An index that every lane shares.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// v summed over the four lanes that hold the same place of a tile's 16.
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// -------------------------------------------------------------------- prepare

template <int N>
struct PrepShared {
    static constexpr int R = kQ + 4, RK = N + 8;
    alignas(16) float A[kQ][R];  // then M
    union {
        alignas(16) float T[kQ][R];
        alignas(16) uint16_t K[kQ][RK];
    };
    double cum[kQ];
    float beta[kQ], rk[kQ], rq[kQ];
};

// Which slot a sequence owns, -1 for none.
__device__ __forceinline__ void own_slot(const DeltaArgs &a, int64_t s) {
    const int32_t slot = a.slots[s];
    bool dead = slot < 0 || slot >= a.num_slots;
    if (!dead) {
        bool same = false;
        for (int64_t i = threadIdx.x; i < s; i += kPrepThreads) same |= a.slots[i] == slot;
        dead = __syncthreads_or(same);
    }
    if (threadIdx.x == 0) a.ws_slot[s] = dead ? -1 : slot;
}

// One (chunk, head): T and M, the factors per token, and for the first head of a group
// the transposed keys. Wave w takes tile w of 16 rows (tokens 16 w ..).
template <int N>
__global__ __launch_bounds__(kPrepThreads) void delta_prepare_kernel(DeltaArgs a) {
    __shared__ PrepShared<N> sh;
    constexpr int KB = N / 32;
    uint32_t blk = blockIdx.x;
    if (blk < a.seqs) {
        own_slot(a, blk);
        return;
    }
    blk -= (uint32_t)a.seqs;
    const uint32_t H = (uint32_t)a.H, id = blk / H, h = blk % H, per = H / (uint32_t)a.G, g = h / per;
    const int s = find_seq(a, id, kQ);
    if (s < 0) return;
    const uint32_t begin = seq_begin(a, s), len = seq_length(a, s, begin), piece = id - (begin / kQ + s);
    if (piece >= (len + kQ - 1) / kQ) return;
    const uint32_t row = begin + piece * kQ;
    const int rem = len - piece * kQ < kQ ? (int)(len - piece * kQ) : kQ;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, grp = lane >> 4;
    const bool keys = h % per == 0;

    // operands: row `16 j + m` of the keys, elements 32 b + 8 grp ..
    auto load = [&](const void *base, int64_t stride, int tile, bf16x8 (&f)[KB]) {
        const int t = 16 * tile + m;
        const uint16_t *p = (const uint16_t *)base + (int64_t)(row + (t < rem ? t : 0)) * stride + g * N + 8 * grp;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            u32x4 u = *(const u32x4 *)(p + 32 * b);
            if (t >= rem) u = u32x4{0, 0, 0, 0};
            f[b] = __builtin_bit_cast(bf16x8, u);
        }
    };
    auto squares = [&](const bf16x8 (&f)[KB]) {
        float v = 0.0f;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) v = __builtin_fmaf((float)f[b][e], (float)f[b][e], v);
        return sum_groups(v);
    };
    bf16x8 kw[KB], qw[KB];
    load(a.k, a.k_stride, wave, kw);
    load(a.q, a.q_stride, wave, qw);
    if (wave == 0) {  // the gates, a lane per token
        const int64_t t = row + (lane < rem ? lane : rem - 1);
        const float dt = softplus(ld_act((const uint16_t *)a.dt_raw, t * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
        const float beta = delta_gate(ld_act((const uint16_t *)a.beta_raw, t * a.beta_stride + h));
        // A decay of 2^-256 leaves nothing of a float32 state: no more than that.
        double step = lane < rem ? (double)dt * ((double)a.A[h] * 1.4426950408889634) : 0.0;
        step = step < -256.0 ? -256.0 : step;
        sh.cum[lane] = wave_prefix_sum(step);
        sh.beta[lane] = lane < rem ? beta : 0.0f;
    }
    {
        const float kk = squares(kw), qq = squares(qw);
        if (grp == 0) {  // zeros behind the last token: with norm_eps = 0 its zeros would have infinite factors
            const bool in = 16 * wave + m < rem;
            sh.rk[16 * wave + m] = in ? unit_scale(kk, a.norm_eps) : 0.0f;
            sh.rq[16 * wave + m] = in ? unit_scale(qq, a.norm_eps) * a.scale : 0.0f;
        }
        if (keys)
#pragma unroll
            for (int b = 0; b < KB; ++b) *(bf16x8 *)&sh.K[16 * wave + m][32 * b + 8 * grp] = kw[b];
    }
    f32x4 kk[4] = {}, qk[4] = {};
    for (int j = 0; j <= wave; ++j) {
        bf16x8 kj[KB];
        load(a.k, a.k_stride, j, kj);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            x = mfma(kw[b], kj[b], x);
            y = mfma(qw[b], kj[b], y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == j) kk[i] = x, qk[i] = y;
    }
    __syncthreads();
    const int64_t at = (int64_t)id * H + h;
    if (wave == 0) {
        const double cum = sh.cum[lane], total = sh.cum[kQ - 1];
        const float grow = fast_exp2((float)cum), rk = sh.rk[lane];
        float *o = (float *)((char *)a.ws_tm + (at * kHeadPieces + kFactors) * 1024);
        o[lane] = grow * rk;
        o[kQ + lane] = sh.beta[lane];
        o[2 * kQ + lane] = fast_exp2((float)(total - cum)) * rk;
        o[3 * kQ + lane] = grow * sh.rq[lane];
        if (lane == kQ - 1) a.ws_decay[at] = grow;
    }
    // A and M from the products: rows 16 wave + 4 grp + r, column 16 j + m
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j > (wave | 1)) break;  // above the diagonal of 32
        const int col = 16 * j + m;
        const double cc = sh.cum[col];
        const float rk = sh.rk[col];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * wave + 4 * grp + r;
            float av = 0.0f, mv = 0.0f;
            if (col <= i) {
                const float d = fast_exp2((float)(sh.cum[i] - cc)) * rk;
                mv = d * sh.rq[i] * qk[j][r];
                if (col < i) av = d * sh.rk[i] * sh.beta[i] * kk[j][r];
            }
            sh.A[i][col] = av;
            qk[j][r] = mv;  // M, once A is done with
        }
    }
    if (keys) {  // the transposed keys as left operands: row tile_row(t, m), tokens 32 half + 8 grp ..
        char *o = (char *)a.ws_kt + ((int64_t)id * a.G + g) * pieces_kt(N) * 1024;
        for (int f = wave; f < pieces_kt(N); f += 4) {
            const int n = tile_row(f >> 1, m), t0 = 32 * (f & 1) + 8 * grp;
            u32x4 u;
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = (uint32_t)sh.K[t0 + 2 * e][n] | (uint32_t)sh.K[t0 + 2 * e + 1][n] << 16;
            *(u32x4 *)(o + f * 1024 + lane * 16) = u;
        }
    }
    __syncthreads();
    // T's diagonal block of the wave: column m by substitution, x_i = (i == m) - sum_j<i A_ij x_j
    const int d0 = 16 * wave;
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == m ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) v = __builtin_fmaf(-sh.A[d0 + i][d0 + j], x[j], v);
            x[i] = v;
        }
        if (grp == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) sh.T[d0 + i][d0 + m] = x[i];
        if ((wave & 1) == 0 && grp == 1)
#pragma unroll
            for (int i = 0; i < 16; ++i) sh.T[d0 + i][d0 + 16 + m] = 0.0f;
    }
    __syncthreads();
    // The blocks below in column `wave`, from the top: T_ij = -T_ii sum_l A_il T_lj (j <= l < i),
    // on the float32 matrix cores, whose summed index is taken as 4 grp + r.
    {
        f32x4 t[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) t[0][r] = sh.T[d0 + 4 * grp + r][d0 + m];
        for (int i = wave + 1; i < 4; ++i) {
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f}, out = sum;
#pragma unroll
            for (int l = 0; l < 3; ++l) {
                if (wave + l >= i) break;
                const f32x4 al = *(const f32x4 *)&sh.A[16 * i + m][16 * (wave + l) + 4 * grp];
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = mfma_f32(al[r], t[l][r], sum);
            }
            const f32x4 ti = *(const f32x4 *)&sh.T[16 * i + m][16 * i + 4 * grp];
#pragma unroll
            for (int r = 0; r < 4; ++r) out = mfma_f32(ti[r], -sum[r], out);
#pragma unroll
            for (int l = 1; l < 4; ++l)
                if (wave + l == i) t[l] = out;
#pragma unroll
            for (int r = 0; r < 4; ++r) sh.T[16 * i + 4 * grp + r][d0 + m] = out[r];
        }
    }
    __syncthreads();
    // T and M as left operands: row tile_row(tile, m), columns 32 half + 8 grp ..
    char *o = (char *)a.ws_tm + at * kHeadPieces * 1024;
    auto write = [&](const float (&src)[kQ][PrepShared<N>::R], int tri, auto piece) {
        const int tile = tri < 2 ? tri : tri < 4 ? 2 : 3, half = tri < 2 ? 0 : tri & 1;
        const float *p = src[tile_row(tile, m)] + 32 * half + 8 * grp;
        float v[8];
        *(f32x4 *)v = *(const f32x4 *)p;
        *(f32x4 *)(v + 4) = *(const f32x4 *)(p + 4);
        bf16x8 part[kParts];
        split<kParts>(v, part);
#pragma unroll
        for (int k = 0; k < kParts; ++k) *(bf16x8 *)(o + piece(tri, k) * 1024 + lane * 16) = part[k];
    };
    for (int tri = wave; tri < kTri; tri += 4) write(sh.T, tri, piece_t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j > (wave | 1)) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) sh.A[16 * wave + 4 * grp + r][16 * j + m] = qk[j][r];
    }
    __syncthreads();
    for (int tri = 3 - wave; tri < kTri; tri += 4) write(sh.A, tri, piece_m);
}

// ----------------------------------------------------------------------- walk

// What the walk reads of one chunk: pieces of 1 KiB, a register of 16 bytes of each lane.
template <int N>
struct Chunk {
    static constexpr int KB = N / 32, kHead = kFactors + 1, kPieces = 8 * KB + pieces_kt(N) + kHead;
    static constexpr int kK = 0, kQ_ = 4 * KB, kKt = 8 * KB, kTM = kKt + pieces_kt(N);
};

// One head of one sequence, WAVES x 16 columns p of it.
template <int N, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void delta_walk_kernel(DeltaArgs a) {
    using C = Chunk<N>;
    constexpr int KB = N / 32, NT = N / 16;
    __shared__ __align__(16) char sh[2][C::kPieces][1024];  // this chunk's and the next one's
    // Workgroups go round the eight XCDs: those of a group of heads, which share its keys and
    // queries, are 8 apart, so that they meet in one XCD's cache.
    const uint32_t H = (uint32_t)a.H, G = (uint32_t)a.G, per = H / G, nb = (uint32_t)a.P / (16 * WAVES);
    const uint32_t lin = blockIdx.x, one = lin / 8 % (per * nb), unit = lin / 8 / (per * nb) * 8 + lin % 8;
    if (unit >= G * (uint32_t)a.seqs) return;
    const uint32_t s = unit / G, g = unit % G, h = g * per + one / nb, pb = one % nb;
    const int wave = uniform((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63, m = lane & 15, grp = lane >> 4;
    const uint32_t begin = uniform(seq_begin(a, s)), len = uniform(seq_length(a, s, begin));
    const int64_t pw = (int64_t)(pb * WAVES + wave) * 16, p0 = pw + m;
    const int64_t y_stride = a.H * a.P;
    uint16_t *yb = (uint16_t *)a.y + (int64_t)begin * y_stride + h * a.P + pw;
    const int32_t slot = uniform(a.ws_slot[s]);
    if (slot < 0) {
        for (uint32_t t = grp; t < len; t += 4) yb[t * y_stride + m] = 0;
        return;
    }
    const bool resume = a.resume && a.resume[s] != 0;
    float *cache = a.state_cache + (((int64_t)slot * H + h) * a.P + p0) * N + 8 * grp;
    f32x4 S[NT];  // n = tile_row(t, 4 grp + r), column p0
#pragma unroll
    for (int t = 0; t < NT; ++t)
        S[t] = resume ? *(const f32x4 *)(cache + 32 * (t >> 1) + 4 * (t & 1)) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t chunks = (len + kQ - 1) / kQ, id0 = begin / kQ + s;
    const uint16_t *qb = (const uint16_t *)a.q + (int64_t)begin * a.q_stride + g * N;
    const uint16_t *kb = (const uint16_t *)a.k + (int64_t)begin * a.k_stride + g * N;
    const uint16_t *vb = (const uint16_t *)a.v + (int64_t)begin * a.v_stride + h * a.P + pw;
    const uint32_t lds0 = lds_addr(sh);
    // Chunk c into LDS. Keys and queries as operands: a wave takes tiles of 16 tokens; tokens
    // behind the last repeat it (their updates are zero).
    auto fetch = [&](uint32_t chunk) {
        const uint32_t c = uniform((int)chunk), to = lds0 + (c & 1) * C::kPieces * 1024, left = len - c * kQ - 1;
#pragma unroll
        for (int i = 0; i < 8 / WAVES; ++i) {
            const int tile = (wave + i * WAVES) & 3;
            const bool keys = wave + i * WAVES < 4;
            const int64_t stride = keys ? a.k_stride : a.q_stride;
            const uint16_t *base = (keys ? kb : qb) + (int64_t)c * kQ * stride;
            uint32_t t = tile_row(tile, m);
            t = t < left ? t : left;
            const uint32_t off = t * (uint32_t)stride * 2 + 16 * grp;
#pragma unroll
            for (int b = 0; b < KB; ++b) dma16_s(base + 32 * b, off, to + ((keys ? C::kK : C::kQ_) + tile * KB + b) * 1024);
        }
        const char *tm = (const char *)a.ws_tm + ((int64_t)(id0 + c) * H + h) * kHeadPieces * 1024;
        const char *kt = (const char *)a.ws_kt + ((int64_t)(id0 + c) * a.G + g) * pieces_kt(N) * 1024;
#pragma unroll
        for (int i = 0; i < (C::kHead + WAVES - 1) / WAVES; ++i) {
            const int f = wave + i * WAVES;
            if (f < C::kHead) dma16_s(tm + f * 1024, lane * 16, to + (C::kTM + f) * 1024);
        }
#pragma unroll
        for (int i = 0; i < pieces_kt(N) / WAVES; ++i) {
            const int f = wave + i * WAVES;
            dma16_s(kt + f * 1024, lane * 16, to + (C::kKt + f) * 1024);
        }
    };
    // The values of chunk c: column p0, tokens tile_row(tile, 4 grp + r); behind the last
    // token zeros.
    uint32_t v[4][4];
    const uint32_t v_row = (uint32_t)a.v_stride * 2, y_row = (uint32_t)y_stride * 2;
    auto fetch_v = [&](uint32_t c) {
        const uint16_t *base = vb + (int64_t)c * kQ * a.v_stride;
        const uint32_t left = len - c * kQ, lane_at = 8 * grp * v_row + 2 * m;
        const auto rows = buffer(base, (left < kQ ? left - 1 : kQ - 1) * v_row + 32);
#pragma unroll
        for (int tile = 0; tile < 4; ++tile)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = lane_at + tile_row(tile, r) * v_row;
                v[tile][r] = __builtin_amdgcn_raw_buffer_load_b16(rows, at, 0, 0);
            }
    };
    auto frag = [&](const char *p) { return *(const bf16x8 *)(p + lane * 16); };

    if (chunks > 0) {
        fetch(0);
        fetch_v(0);
    }
    // y of chunk c, a chunk later: a wait for loads waits for the stores before them too. What
    // lies behind the last token is dropped.
    uint16_t out[4][4];
    auto store_y = [&](uint32_t chunk) {
        const uint32_t c = uniform((int)chunk), left = len - c * kQ, lane_at = 8 * grp * y_row + 2 * m;
        const auto rows = buffer(yb + (int64_t)c * kQ * y_stride, (left < kQ ? left - 1 : kQ - 1) * y_row + 32);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = lane_at + tile_row(t, r) * y_row;
                __builtin_amdgcn_raw_buffer_store_b16(out[t][r], rows, at, 0, 0);
            }
    };
    uint32_t c = 0;
    for (; c < chunks; ++c) {
        vm_wait();
        lds_barrier();  // this chunk is there, the one before is done with
        // M's last part comes by registers: two chunks of it would not fit into LDS beside the
        // rest. (Loaded ahead of the products with T, the walk above took 640 us.)
        bf16x8 last[kTri];
        {
            const char *p = (const char *)a.ws_tm + (((int64_t)(id0 + c) * H + h) * kHeadPieces + kLastM) * 1024;
#pragma unroll
            for (int i = 0; i < kTri; ++i) last[i] = *(const bf16x8 *)(p + i * 1024 + lane * 16);
        }
        if (c > 0) store_y(c - 1);
        // The values are there as well, but the compiler would wait for them where they
        // are used, and with them for the loads that it does not know of: here it waits for none.
#pragma unroll
        for (int t = 0; t < 4; ++t) asm volatile("" : "+v"(v[t][0]), "+v"(v[t][1]), "+v"(v[t][2]), "+v"(v[t][3]));
        if (c + 1 < chunks) fetch(c + 1);
        const float decay = *(cf32_ptr)(a.ws_decay + uniform64((int64_t)(id0 + c) * H + h));
        const char(*in)[1024] = sh[c & 1];
        const float *sc = (const float *)in[C::kTM + kFactors];

        // K S^T and Q S^T. Operands are read from LDS a group of products ahead, and the
        // next 32 of n are split between the products.
        f32x4 ks[4], ys[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = ys[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto split_state = [&](int b, bf16x8 (&sp)[3]) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = S[2 * b][e], x[4 + e] = S[2 * b + 1][e];
            split<3>(x, sp);
        };
        bf16x8 sp[2][3], kf[2], qf[2];
        kf[0] = frag(in[C::kK]), qf[0] = frag(in[C::kQ_]);
        split_state(0, sp[0]);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int next = 4 * b + t + 1, tn = next & 3, bn = next >> 2;
                if (next < 4 * KB) kf[next & 1] = frag(in[C::kK + tn * KB + bn]), qf[next & 1] = frag(in[C::kQ_ + tn * KB + bn]);
#pragma unroll
                for (int part = 2; part >= 0; --part) {
                    ks[t] = mfma(kf[t & 1], sp[b & 1][part], ks[t]);
                    ys[t] = mfma(qf[t & 1], sp[b & 1][part], ys[t]);
                }
            }
            if (b + 1 < KB) split_state(b + 1, sp[(b + 1) & 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                interleave_reads<2>();
                interleave<6, 3>();
            }
            __builtin_amdgcn_sched_barrier(0);
        }

        // beta (V - diag(..) K S^T), in three parts
        bf16x8 rp[2][3], tf[2][2][3];
        auto read_t = [&](int i) {  // two tiles
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int part = 0; part < 3; ++part)
                    tf[i & 1][k][part] = frag(in[C::kTM + piece_t(tri_index(kTile[i] + k, i >> 1), part)]);
        };
        read_t(0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = 2 * half + k, at = 32 * half + 8 * grp + 4 * k;
                const f32x4 gk = *(const f32x4 *)(sc + at), be = *(const f32x4 *)(sc + kQ + at), gq = *(const f32x4 *)(sc + 3 * kQ + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float val = __uint_as_float(v[t][r] << 16);
                    x[4 * k + r] = be[r] * __builtin_fmaf(-gk[r], ks[t][r], val);
                    ys[t][r] *= gq[r];
                }
            }
            split<3>(x, rp[half]);
        }
        if (c + 1 < chunks) fetch_v(c + 1);
        __builtin_amdgcn_sched_barrier(0);

        // U = T times that; the first half's parts are formed between the second's products
        f32x4 u[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        bf16x8 um[2][3], us[2][3];  // of U for y, of diag(..) U for the state
        auto split_update = [&](int half) {
            float x[8], w[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4 tk = *(const f32x4 *)(sc + 2 * kQ + 32 * half + 8 * grp + 4 * k);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[4 * k + r] = u[2 * half + k][r];
                    w[4 * k + r] = x[4 * k + r] * tk[r];
                }
            }
            split<3>(x, um[half]);
            split<3>(w, us[half]);
        };
        float odd = 0.0f;  // NaN where an update is not finite
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (i < 2) read_t(i + 1);
#pragma unroll
            for (int k = 0; k < 6; ++k)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    u[kTile[i] + t] = mfma(tf[i & 1][t][kTerm[k][0]], rp[i >> 1][kTerm[k][1]], u[kTile[i] + t]);
            if (i == 0) {
                interleave_reads<6>();
                __builtin_amdgcn_sched_barrier(0);
                split_update(0);
            }
        }
        interleave_reads<6>();
        interleave<24, 5>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) odd = __builtin_fmaf(u[t][r], 0.0f, odd);
        if (uniform(__any(odd != odd))) break;

        // M U for y, two tiles at a time, and K^T (diag(..) U) for the state, two of the tiles of n
        bf16x8 mf[2][2][3], tk[3][2];
        auto read_m = [&](int i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int tri = tri_index(kTile[i] + k, i >> 1);
#pragma unroll
                for (int part = 0; part < 2; ++part) mf[i & 1][k][part] = frag(in[C::kTM + piece_m(tri, part)]);
                mf[i & 1][k][2] = last[tri];
            }
        };
        auto read_k = [&](int i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) tk[i % 3][k] = frag(in[C::kKt + 2 * (2 * (i % (NT / 2)) + k) + i / (NT / 2)]);
        };
        read_m(0);
        read_m(1);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int k = 0; k < 6; ++k)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    ys[kTile[i] + t] = mfma(mf[i & 1][t][kTerm[k][0]], um[i >> 1][kTerm[k][1]], ys[kTile[i] + t]);
            if (i == 0) {
                read_m(2);
                split_update(1);
            }
            if (i == 1) read_k(0);
            if (i == 2) read_k(1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) S[n] *= decay;
        interleave<36, 4>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int half = i / (NT / 2), n = 2 * (i % (NT / 2));
            if (i + 2 < NT) read_k(i + 2);
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int k = 0; k < 2; ++k) S[n + k] = mfma(tk[i % 3][k], us[half][part], S[n + k]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) out[t][r] = bf16_bits(ys[t][r]);
    }
    if (c > 0) store_y(c - 1);
    // What an update that is not finite leaves, a token at a time; the other waves go on, so
    // this one still fetches its share of each chunk.
    for (c = uniform((int)c); c < chunks; ++c) {
        const uint32_t left = len - c * kQ;
        const int rem = left < kQ ? (int)left : kQ;
        for (int i = 0; i < rem; ++i) {
            const int64_t t = (int64_t)c * kQ + i, row = begin + t;
            const float dt = softplus(ld_act((const uint16_t *)a.dt_raw, row * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
            const float beta = delta_gate(ld_act((const uint16_t *)a.beta_raw, row * a.beta_stride + h));
            const float one = fast_exp2(dt * a.A[h] * kLog2e);
            float kv[KB][8], qv[KB][8], kk = 0.0f, qq = 0.0f, sk = 0.0f, sq = 0.0f;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                ld8(kb + t * a.k_stride + 32 * b + 8 * grp, kv[b]);
                ld8(qb + t * a.q_stride + 32 * b + 8 * grp, qv[b]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    kk = __builtin_fmaf(kv[b][e], kv[b][e], kk);
                    qq = __builtin_fmaf(qv[b][e], qv[b][e], qq);
                }
            }
            const float rk = unit_scale(sum_groups(kk), a.norm_eps), rq = unit_scale(sum_groups(qq), a.norm_eps) * a.scale;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    S[n][r] *= one;
                    sk = __builtin_fmaf(S[n][r], kv[n >> 1][4 * (n & 1) + r], sk);
                }
            const float up = beta * __builtin_fmaf(-rk, sum_groups(sk), ld_act(vb + m, t * a.v_stride)) * rk;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    S[n][r] = __builtin_fmaf(up, kv[n >> 1][4 * (n & 1) + r], S[n][r]);
                    sq = __builtin_fmaf(S[n][r], qv[n >> 1][4 * (n & 1) + r], sq);
                }
            const float out = sum_groups(sq) * rq;
            if (grp == 0) st_act(yb + m, t * y_stride, out);
        }
        if (c + 1 >= chunks) break;
        vm_wait();
        lds_barrier();
        if (c + 2 < chunks) fetch(c + 2);
    }
    if (len > 0 || !resume)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            *(f32x4 *)(cache + 32 * (t >> 1) + 4 * (t & 1)) = S[t];
}

// ---------------------------------------------------------- walk, shared by waves

// LDS of a workgroup, in pieces of 1 KiB (16 bytes per lane): what the waves hand each other.
template <int N>
struct TeamShared {
    static constexpr int NW = N / 32;  // waves: 32 of n each
    union {
        alignas(16) char part[2][4][NW - 1][1024];  // of K S^T and Q S^T: (tile of tokens, from another wave)
        float sums[2][NW][16];                      // where a chunk is taken a token at a time
    };
    alignas(16) char r[2][3][1024];                   // beta (V - ..), as right operands
    alignas(16) char us[2][3][1024], um[2][3][1024];  // diag(..) U and U, as right operands
};

// One head of one sequence, 16 columns p of it, by N / 32 waves: wave w holds the
// columns' elements n = 32 w .. 32 w + 31, and takes TW of the chunk's four tiles of tokens.
template <int N>
__global__ __launch_bounds__(2 * N, N == 128 ? 2 : 1) void delta_team_kernel(DeltaArgs a) {
    constexpr int NW = N / 32, TW = 4 / NW, KB = N / 32;
    __shared__ TeamShared<N> sh;
    // Workgroups go round the eight XCDs: those of a group of heads, which share its keys and
    // queries, are 8 apart, so that they meet in one XCD's cache.
    const uint32_t H = (uint32_t)a.H, G = (uint32_t)a.G, per = H / G, nb = (uint32_t)a.P / 16;
    const uint32_t lin = blockIdx.x, one = lin / 8 % (per * nb), unit = lin / 8 / (per * nb) * 8 + lin % 8;
    if (unit >= G * (uint32_t)a.seqs) return;
    const uint32_t s = unit / G, g = unit % G, h = g * per + one / nb, pb = one % nb;
    const int wave = uniform((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63, m = lane & 15, grp = lane >> 4;
    const uint32_t begin = uniform(seq_begin(a, s)), len = uniform(seq_length(a, s, begin));
    const int64_t pw = (int64_t)pb * 16, p0 = pw + m;
    const int64_t y_stride = a.H * a.P;
    uint16_t *yb = (uint16_t *)a.y + (int64_t)begin * y_stride + h * a.P + pw;
    const int32_t slot = uniform(a.ws_slot[s]);
    if (slot < 0) {
        for (uint32_t t = 4 * wave + grp; t < len; t += 4 * NW) yb[t * y_stride + m] = 0;
        return;
    }
    const bool resume = a.resume && a.resume[s] != 0;
    float *cache = a.state_cache + (((int64_t)slot * H + h) * a.P + p0) * N + 32 * wave + 8 * grp;
    f32x4 S[2];  // n = 32 wave + 8 grp + 4 k + r, column p0
#pragma unroll
    for (int k = 0; k < 2; ++k)
        S[k] = resume ? *(const f32x4 *)(cache + 4 * k) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t chunks = (len + kQ - 1) / kQ, id0 = begin / kQ + s;
    const uint16_t *qb = (const uint16_t *)a.q + (int64_t)begin * a.q_stride + g * N;
    const uint16_t *kb = (const uint16_t *)a.k + (int64_t)begin * a.k_stride + g * N;
    const uint16_t *vb = (const uint16_t *)a.v + (int64_t)begin * a.v_stride + h * a.P + pw;
    const uint32_t v_row = (uint32_t)a.v_stride * 2, y_row = (uint32_t)y_stride * 2;

    // What a chunk reads, loaded a chunk ahead, each as soon as the one before is used. The
    // last chunk loads itself once more. Keys and queries behind the last token repeat it
    // (their updates are zero), values are zeros there.
    bf16x8 kf[4], qf[4], tf[TW][2][3], mf[TW][2][3], tk[2][2];
    f32x4 fk[TW], fb[TW], fd[TW], fq[TW];
    uint32_t v[TW][4];
    float decay;
    auto load_kq = [&](uint32_t c) {
        const uint32_t left = len - c * kQ - 1;
        const char *k0 = (const char *)(kb + (int64_t)c * kQ * a.k_stride + 32 * wave);
        const char *q0 = (const char *)(qb + (int64_t)c * kQ * a.q_stride + 32 * wave);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t i = tile_row(t, m);
            i = i < left ? i : left;
            kf[t] = *(const bf16x8 *)(k0 + (i * (uint32_t)a.k_stride * 2 + 16 * grp));
            qf[t] = *(const bf16x8 *)(q0 + (i * (uint32_t)a.q_stride * 2 + 16 * grp));
        }
    };
    auto head = [&](uint32_t c) { return (const char *)a.ws_tm + ((int64_t)(id0 + c) * H + h) * kHeadPieces * 1024; };
    auto load_v = [&](uint32_t c) {
        const uint32_t left = len - c * kQ, lane_at = 8 * grp * v_row + 2 * m;
        const auto rows = buffer(vb + (int64_t)c * kQ * a.v_stride, (left < kQ ? left - 1 : kQ - 1) * v_row + 32);
        const float *f = (const float *)(head(c) + kFactors * 1024) + 8 * grp;
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = wave * TW + i, at = 32 * (t >> 1) + 4 * (t & 1);
            fk[i] = *(const f32x4 *)(f + at), fb[i] = *(const f32x4 *)(f + kQ + at);
            fd[i] = *(const f32x4 *)(f + 2 * kQ + at), fq[i] = *(const f32x4 *)(f + 3 * kQ + at);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t o = lane_at + (at + r) * v_row;
                v[i][r] = __builtin_amdgcn_raw_buffer_load_b16(rows, o, 0, 0);
            }
        }
        decay = *(cf32_ptr)(a.ws_decay + uniform64((int64_t)(id0 + c) * H + h));
    };
    auto load_t = [&](uint32_t c) {
#pragma unroll
        for (int i = 0; i < TW; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int part = 0; part < 3; ++part)
                    tf[i][half][part] = *(const bf16x8 *)(head(c) + piece_t(tri_index(wave * TW + i, half), part) * 1024 + lane * 16);
    };
    auto load_m = [&](uint32_t c) {
        const char *kt = (const char *)a.ws_kt + ((int64_t)(id0 + c) * a.G + g) * pieces_kt(N) * 1024;
#pragma unroll
        for (int i = 0; i < TW; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int part = 0; part < 3; ++part)
                    mf[i][half][part] = *(const bf16x8 *)(head(c) + piece_m(tri_index(wave * TW + i, half), part) * 1024 + lane * 16);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) tk[k][half] = *(const bf16x8 *)(kt + (2 * (2 * wave + k) + half) * 1024 + lane * 16);
    };
    auto frag = [&](const char *p) { return *(const bf16x8 *)(p + lane * 16); };
    // the partial sums of tile t from wave w, for the wave that takes the tile
    auto slot_of = [&](int t, int w) { return w < t / TW ? w : w - 1; };

    if (chunks > 0) {
        load_kq(0);
        load_v(0);
        load_t(0);
        load_m(0);
    }
    // The state's loads are waited for here: the compiler may else wait for them at the head
    // of the loop, and for the next chunk's in every round of it (16384 tokens: 727 us, and 843 without this).
    asm volatile("" : "+v"(S[0]), "+v"(S[1]));
    for (uint32_t c = 0; c < chunks; ++c) {
        const uint32_t next = c + 1 < chunks ? c + 1 : c, left = len - c * kQ;
        // K S^T and Q S^T over the wave's n, for all tokens
        f32x4 ks[4], ys[4];
        {
            bf16x8 sp[3];
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = S[0][e], x[4 + e] = S[1][e];
            split<3>(x, sp);
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int t = 0; t < 4; ++t) ks[t] = mfma(kf[t], sp[part], part == 2 ? zero : ks[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t / TW != wave)
                    *(f32x4 *)(sh.part[0][t][slot_of(t, wave)] + lane * 16) = ks[t];
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int t = 0; t < 4; ++t) ys[t] = mfma(qf[t], sp[part], part == 2 ? zero : ys[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t / TW != wave)
                    *(f32x4 *)(sh.part[1][t][slot_of(t, wave)] + lane * 16) = ys[t];
        }
        load_kq(next);
        lds_barrier();
        // the waves' sums of the wave's tokens, and beta (V - diag(..) K S^T) in three parts
        f32x4 out[TW];
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = wave * TW + i;
            f32x4 sum = ks[0], rest = ys[0];
#pragma unroll
            for (int k = 1; k < 4; ++k) sum = t == k ? ks[k] : sum, rest = t == k ? ys[k] : rest;
#pragma unroll
            for (int w = 0; w < NW - 1; ++w) {
                sum += *(const f32x4 *)(sh.part[0][t][w] + lane * 16);
                rest += *(const f32x4 *)(sh.part[1][t][w] + lane * 16);
            }
            out[i] = rest * fq[i];
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float val = __uint_as_float(v[i][r] << 16);
                x[r] = fb[i][r] * __builtin_fmaf(-fk[i][r], sum[r], val);
            }
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                uint2 u;
                u.x = bf16_pair(x[0], x[1]);
                u.y = bf16_pair(x[2], x[3]);
                *(uint2 *)(sh.r[t >> 1][part] + lane * 16 + 8 * (t & 1)) = u;
            }
        }
        lds_barrier();
        // U = T times that
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = wave * TW + i;
            f32x4 u[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half == 0 || t >= 2) {
                    bf16x8 rp[3];
#pragma unroll
                    for (int part = 0; part < 3; ++part) rp[part] = frag(sh.r[half][part]);
#pragma unroll
                    for (int k = 0; k < 6; ++k) u[half] = mfma(tf[i][half][kTerm[k][0]], rp[kTerm[k][1]], u[half]);
                }
            float x[4], w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = u[0][r] + u[1][r];
                w[r] = x[r] * fd[i][r];
            }
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                uint2 o;
                o.x = bf16_pair(w[0], w[1]);
                o.y = bf16_pair(w[2], w[3]);
                *(uint2 *)(sh.us[t >> 1][part] + lane * 16 + 8 * (t & 1)) = o;
            }
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                uint2 o;
                o.x = bf16_pair(x[0], x[1]);
                o.y = bf16_pair(x[2], x[3]);
                *(uint2 *)(sh.um[t >> 1][part] + lane * 16 + 8 * (t & 1)) = o;
            }
        }
        load_t(next);
        lds_barrier();
        // All waves read all of diag(..) U, and so agree where an update is not finite.
        bf16x8 up[2][3];
        float odd = 0.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int part = 0; part < 3; ++part) up[half][part] = frag(sh.us[half][part]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const bf16x2 two = {up[half][0][e], up[half][0][e + 1]};
                odd = __builtin_amdgcn_fdot2_f32_bf16(two, bf16x2{(__bf16)0.0f, (__bf16)0.0f}, odd, false);
            }
        if (uniform(__any(odd != odd))) {
            // a token at a time; the barriers pass each token's sums over n from wave to wave
            const int rem = left < kQ ? (int)left : kQ;
            for (int i = 0; i < rem; ++i) {
                const int64_t t = (int64_t)c * kQ + i, row = begin + t;
                const float dt = softplus(ld_act((const uint16_t *)a.dt_raw, row * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f));
                const float beta = delta_gate(ld_act((const uint16_t *)a.beta_raw, row * a.beta_stride + h));
                const float keep = fast_exp2(dt * a.A[h] * kLog2e);
                float kv[8], qv[8], kk = 0.0f, qq = 0.0f;
                for (int b = 0; b < KB; ++b) {
                    const int n = 32 * ((b + wave + 1) % KB) + 8 * grp;  // the wave's own block last
                    ld8(kb + t * a.k_stride + n, kv);
                    ld8(qb + t * a.q_stride + n, qv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        kk = __builtin_fmaf(kv[e], kv[e], kk);
                        qq = __builtin_fmaf(qv[e], qv[e], qq);
                    }
                }
                const float rk = unit_scale(sum_groups(kk), a.norm_eps), rq = unit_scale(sum_groups(qq), a.norm_eps) * a.scale;
                float sk = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    S[e >> 2][e & 3] *= keep;
                    sk = __builtin_fmaf(S[e >> 2][e & 3], kv[e], sk);
                }
                sh.sums[0][wave][m] = sum_groups(sk);
                __syncthreads();
                float all = 0.0f, sq = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) all += sh.sums[0][w][m];
                const float up = beta * __builtin_fmaf(-rk, all, ld_act(vb + m, t * a.v_stride)) * rk;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    S[e >> 2][e & 3] = __builtin_fmaf(up, kv[e], S[e >> 2][e & 3]);
                    sq = __builtin_fmaf(S[e >> 2][e & 3], qv[e], sq);
                }
                sh.sums[1][wave][m] = sum_groups(sq);
                __syncthreads();
                if (wave == 0 && grp == 0) {
                    float out = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) out += sh.sums[1][w][m];
                    st_act(yb + m, t * y_stride, out * rq);
                }
            }
            __syncthreads();  // the next chunk's partial sums lie where the last token's were read
        } else {
        // S^T <- decay S^T + K^T (diag(..) U) over the wave's n
        f32x4 more[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int k = 0; k < 2; ++k) more[k] = mfma(tk[k][half], up[half][part], more[k]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[k][r] = __builtin_fmaf(S[k][r], decay, more[k][r]);
        // y = diag(..) Q S^T + M U of the wave's tokens; what lies behind the last is dropped
        const uint32_t y_lane = 8 * grp * y_row + 2 * m;
        const auto rows = buffer(yb + (int64_t)c * kQ * y_stride, (left < kQ ? left - 1 : kQ - 1) * y_row + 32);
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = wave * TW + i;
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half == 0 || t >= 2) {
                    bf16x8 uf[3];
#pragma unroll
                    for (int part = 0; part < 3; ++part) uf[part] = frag(sh.um[half][part]);
#pragma unroll
                    for (int k = 0; k < 6; ++k) out[i] = mfma(mf[i][half][kTerm[k][0]], uf[kTerm[k][1]], out[i]);
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = y_lane + (32 * (t >> 1) + 4 * (t & 1) + r) * y_row;
                __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(out[i][r]), rows, at, 0, 0);
            }
        }
        }
        load_m(next);
        load_v(next);
    }
    if (len > 0 || !resume)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            *(f32x4 *)(cache + 4 * k) = S[k];
}

template <int N>
hipError_t team(const DeltaArgs &a, hipStream_t s) {
    const int64_t blocks = (a.G * a.seqs + 7) / 8 * 8 * (a.H / a.G) * (a.P / 16);
    hipLaunchKernelGGL((delta_team_kernel<N>), dim3((unsigned)blocks), dim3(2 * N), 0, s, a);
    return hipGetLastError();
}

int64_t chunk_ids(int64_t seqs, int64_t rows) { return rows / kQ + seqs; }

template <int N, int WAVES>
hipError_t walk(const DeltaArgs &a, hipStream_t s) {
    const int64_t blocks = (a.G * a.seqs + 7) / 8 * 8 * (a.H / a.G) * (a.P / (16 * WAVES));
    hipLaunchKernelGGL((delta_walk_kernel<N, WAVES>), dim3((unsigned)blocks), dim3(64 * WAVES), 0, s, a);
    return hipGetLastError();
}

template <int N>
hipError_t delta(const DeltaArgs &a, hipStream_t s) {
    const int64_t blocks = a.seqs + chunk_ids(a.seqs, a.rows) * a.H;
    hipLaunchKernelGGL((delta_prepare_kernel<N>), dim3((unsigned)blocks), dim3(kPrepThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // A wave of the walk keeps all of N and fills the chip with less work in all; a team of
    // waves takes a chunk of 16 columns in less time. Teams are for calls whose workgroups all
    // run at once: two on each of 256 CUs. Whole calls (us), walk / team, by teams:
    //   N = 128   256: 397 / 243    384: 372 / 307, 447 / 407    512: 1054 / 720, 460 / 320, 498 / 456
    //             576: 422 / 496    640: 525 / 626    768: 1127 / 1098, 527 / 515    1024: 1196 / 1388, 557 / 649
    //   N = 64    256: 297 / 255    384: 285 / 247, 343 / 322    512: 823 / 616, 360 / 250, 387 / 372
    //             576: 305 / 449    768: 881 / 1011, 389 / 459    1024: 940 / 1095, 429 / 510
    //   2048 (8 prompts of 4096 tokens)  829 / 1369, N = 64: 640 / 1103    48 prompts of 64 tokens  119 / 219
    // That is for equal lengths. The host does not know them: a call with one long sequence among
    // short ones pays the walk's longer chain (13 ragged prompts 168 / 140 us, 16384 tokens beside
    // forty prompts of one token 1962 / 927).
    if (a.H * a.seqs * a.P / 16 <= 512) return team<N>(a, s);
    return a.P % 128 == 0 ? walk<N, 8>(a, s) : walk<N, 4>(a, s);
}

}  // namespace

size_t delta_workspace(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N) {
    DeltaArgs a{};
    a.seqs = seqs;
    a.rows = rows;
    a.H = H;
    a.G = G;
    return delta_layout(a, N, nullptr);
}

// Places the workspace's arrays and returns its size.
size_t delta_layout(DeltaArgs &a, int64_t N, void *workspace) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        void *p = (char *)workspace + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const size_t ids = (size_t)chunk_ids(a.seqs, a.rows), heads = ids * (size_t)a.H;
    a.ws_slot = (int32_t *)take((size_t)a.seqs * 4);
    a.ws_decay = (float *)take(heads * 4);
    a.ws_tm = take(heads * kHeadPieces * 1024);
    a.ws_kt = take(ids * (size_t)a.G * pieces_kt((int)N) * 1024);
    return at;
}

hipError_t launch_delta(DeltaArgs a, int N, void *workspace, hipStream_t s) {
    delta_layout(a, N, workspace);
    return N == 64 ? delta<64>(a, s) : delta<128>(a, s);
}

}  // namespace ssm
