// Device building blocks of the norms: rows by 16-byte accesses at any alignment,
// sums over the lanes that share a row, column sums over a workgroup's rows.
#pragma once

#include <type_traits>

#include "ssm_common.h"
#include "ssm_packed.h"

namespace ssm {

typedef float f32x4n __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4n __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8n __attribute__((ext_vector_type(8)));
typedef f32x4n f32x4u __attribute__((aligned(4)));  // at an element's alignment
typedef u32x4n u32x4u __attribute__((aligned(2)));
typedef bf16x8n bf16x8u __attribute__((aligned(2)));

constexpr int kVec = 8;

// kVec consecutive elements as floats. ODD: the row's length or stride is not
// whole 16-byte pieces; the accesses are as wide, at the elements' own alignment
// (the hardware takes any address), and a row's last elements, `left` of them,
// are taken one by one, zeros behind them. Against one element per lane and
// access (us, rows of 84 MB of bfloat16 in all): add norm of 1001 channels
// forward 131 -> 106, backward 371 -> 164, gate norm of 4095 122 -> 69 and
// 366 -> 165; as many rows of 1000 take 95 and 126, 41 and 92.
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void ld_vec(const float *p, int left, float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
        return;
    }
    using Piece = std::conditional_t<ODD, f32x4u, f32x4n>;
    const Piece *q = (const Piece *)p;
    const f32x4n a = STREAM ? __builtin_nontemporal_load(q) : q[0];
    const f32x4n b = STREAM ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void ld_vec(const uint16_t *p, int left, float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? ld_act(p, i) : 0.0f;
        return;
    }
    using Piece = std::conditional_t<ODD, u32x4u, u32x4n>;
    const u32x4n a = STREAM ? __builtin_nontemporal_load((const Piece *)p) : *(const Piece *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void st_vec(float *p, int left, const float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
        return;
    }
    using Piece = std::conditional_t<ODD, f32x4u, f32x4n>;
    const f32x4n a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    Piece *q = (Piece *)p;
    if constexpr (STREAM) {
        __builtin_nontemporal_store(a, q);
        __builtin_nontemporal_store(b, q + 1);
    } else {
        q[0] = a;
        q[1] = b;
    }
}
template <bool ODD, bool STREAM = false>
__device__ __forceinline__ void st_vec(uint16_t *p, int left, const float (&v)[8]) {
    if (ODD && left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) st_act(p, i, v[i]);
        return;
    }
    using Piece = std::conditional_t<ODD, bf16x8u, bf16x8n>;
    bf16x8n o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
    if constexpr (STREAM) __builtin_nontemporal_store(o, (Piece *)p);
    else *(Piece *)p = o;
}

// Sums of NV values over the TPR lanes that share a row, in every one of them.
// A wave adds by lane exchanges; more waves meet through LDS (two buffers in
// turn, so that one barrier per row is enough). In double precision: what rounds
// in the last steps of a tree is a whole row's error, and no other row averages it
// (two rows of 3088 channels, 40 seeds: at most 6.0e-8 of y, 8.0e-8 with float32
// sums and the hardware's root as it is; 1 % of the time of large batches).
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(const float (&part)[NV], double (&v)[NV], double (*sh)[16][NV], int &turn) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = (double)part[i];
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m *= 2)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], m);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i) sh[turn][w][i] = v[i];
        __syncthreads();
        if constexpr (TPR <= 512) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = 0.0;
#pragma unroll
                for (int k = 0; k < TPR / 64; ++k) v[i] += sh[turn][k][i];
            }
        } else {  // a lane per wave, four times over: 16 pairs at once cost registers that a workgroup of 16 waves has not
            const int k = threadIdx.x & 15;
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = k < TPR / 64 ? sh[turn][k][i] : 0.0;
#pragma unroll
            for (int m = 1; m < 16; m *= 2)
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], m);
        }
        turn ^= 1;
    }
}

// (sum / n + eps)^-1/2 rounded once: its error is a whole row's. The hardware's
// reciprocal root and one step of Newton's in double precision, four
// instructions per row.
__device__ __forceinline__ float inv_rms(double sum, double inv, float eps) {
    const double v = __builtin_fma(sum, inv, (double)eps);
    const double r = (double)rsqrtf((float)v);
    const float rstd = (float)__builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
    return finite(rstd) ? rstd : (float)r;  // of zero, infinity and NaN
}

constexpr int block_threads(int TPR) { return TPR < 256 ? 256 : TPR; }

// Adds a workgroup's column sums (one set per row-sharing group of lanes) in
// the order of the groups and writes them as one partial row of D columns.
template <int TPR, bool ODD, int ITER>
__device__ __forceinline__ void write_partial(const float (&acc)[ITER][kVec], float *sh, float *part, int64_t D) {
    constexpr int RPB = block_threads(TPR) / TPR;
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    for (int w = 0; w < RPB; ++w) {
        if (RPB > 1) __syncthreads();
        if (mine != w) continue;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * TPR + lane) * kVec, left = (int)D - c;
            if (left <= 0) continue;
            if (RPB == 1) {
                st_vec<ODD>(part + c, left, acc[k]);
            } else {
                float t[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    t[i] = w == 0 ? acc[k][i] : sh[c + i] + acc[k][i];
                    sh[c + i] = t[i];
                }
                if (w == RPB - 1) st_vec<ODD>(part + c, left, t);
            }
        }
    }
    if (RPB > 1) __syncthreads();
}

struct ColumnSums {
    float *p[3];  // up to three sums, NULL behind the last
};
// out[c] = sum over the partial rows, in order: 64 columns per workgroup, 16
// slices of the rows, whose sums are added in the order of the slices.
static __global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *part, int64_t nblk, int64_t D, ColumnSums out) {
    __shared__ float sh[16][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int s = threadIdx.x >> 6;
    const float *p = part + (int64_t)blockIdx.y * nblk * D;
    const int64_t per = (nblk + 15) / 16, lo = s * per, hi = lo + per < nblk ? lo + per : nblk;
    float v = 0.0f;
    if (c < D)
#pragma unroll 8
        for (int64_t i = lo; i < hi; ++i) v += p[i * D + c];
    sh[s][threadIdx.x & 63] = v;
    __syncthreads();
    if (s == 0 && c < D) {
#pragma unroll
        for (int k = 1; k < 16; ++k) v += sh[k][threadIdx.x & 63];
        out.p[blockIdx.y][c] = v;
    }
}

// Lanes per row and elements per lane by the row's length: a wave per row as
// long as it holds at most 24 elements per lane (1536 channels), then a
// workgroup of as many waves as give each lane 8. Short rows share a wave (rows of
// 24 channels, a wave each: add norm 423 us forward and 1146 backward, three
// lanes each: 102 and 195).
//
// Both sides at rows of 84 MB of bfloat16 (float32 residual), us: add norm
// forward / backward, gate norm forward / backward,
//   1536   a wave, 24 per lane       99 133  42  96     3 waves, 8 per lane    97 144  40 135
//   2048   a wave, 32 per lane      103 134  49  98     4 waves                94 132  42 102
//   2560   a wave, 40 per lane      103 137  44 102     5 waves                94 134  40  98
//   4096   4 waves, 16 per lane      94 136  43 107     8 waves                90 133  42  92
//   5120   4 waves, 24 per lane      98 141  44 120     10 waves               93 141  48  93
//   8192   4 waves, 32 per lane     100 138  42 105     16 waves               95 137  41  97
// Only the gate norm's forward pass keeps 4 waves for rows above 4096 (FEW):
// 32768 rows of 5120 channels take 173 us so and 182 with 10 waves.
#define SSM_NORM_ROWS(n, ODD, FEW, CALL)             \
    do {                                             \
        if (n <= 64) return CALL(8, ODD, 1);         \
        if (n <= 128) return CALL(16, ODD, 1);       \
        if (n <= 256) return CALL(32, ODD, 1);       \
        if (n <= 512) return CALL(64, ODD, 1);       \
        if (n <= 1024) return CALL(64, ODD, 2);      \
        if (n <= 1536) return CALL(64, ODD, 3);      \
        if (n <= 2048) return CALL(256, ODD, 1);     \
        if (n <= 2560) return CALL(320, ODD, 1);     \
        if (n <= 4096) return CALL(512, ODD, 1);     \
        if (n > 8192) return CALL(1024, ODD, 2);     \
        if constexpr (FEW) {                         \
            if (n <= 6144) return CALL(256, ODD, 3); \
            return CALL(256, ODD, 4);                \
        } else {                                     \
            if (n <= 5120) return CALL(640, ODD, 1); \
            if (n <= 6144) return CALL(768, ODD, 1); \
            return CALL(1024, ODD, 1);               \
        }                                            \
    } while (0)
#define SSM_NORM_DISPATCH(LEN, EVEN, FEW, CALL)         \
    do {                                                \
        const int64_t n_ = (LEN);                       \
        if (EVEN) SSM_NORM_ROWS(n_, false, FEW, CALL);  \
        else SSM_NORM_ROWS(n_, true, FEW, CALL);        \
    } while (0)

static inline unsigned norm_grid(int64_t rows, int tpr, int64_t cap) {
    const int64_t rpb = tpr < 256 ? 256 / tpr : 1, b = (rows + rpb - 1) / rpb;
    return (unsigned)(b < cap ? b : cap);
}

static inline hipError_t launch_reduce(const float *part, int64_t nblk, int64_t D, const ColumnSums &out, hipStream_t s) {
    const unsigned sums = out.p[2] ? 3 : out.p[1] ? 2 : 1;
    hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((D + 63) / 64), sums), dim3(1024), 0, s, part, nblk, D, out);
    return hipGetLastError();
}

}  // namespace ssm
