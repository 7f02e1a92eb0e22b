// Device building blocks of the operators on packed sequences: operands of the
// matrix products as sums of bfloat16, buffer accesses, prefix sums over a wave,
// and the sequences' rows from their offsets. `Args` is any argument struct with
// seqs, rows and cu_seqlens.
#pragma once

#include "ssm_device.h"

namespace ssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
// The product of two operands of three parts each, as six, the small ones first;
// the last three are that of two parts each.
constexpr int kTerm[6][2] = {{2, 0}, {0, 2}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};
constexpr int kTwo = 3;
// Buffer accesses: bytes from a wave-uniform base, a range that the hardware
// checks (loads outside it give 0, stores outside it are dropped).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// v plus the value of another lane (0 where DPP control CTRL gives none, or in the
// rows that ROWS leaves out).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Inclusive prefix sum over the 64 lanes: within rows of 16 (shifts by 1, 2, 4 and
// 8), then row 0 to row 1 and 2 to 3, then the lower half to the upper.
__device__ __forceinline__ double wave_prefix_sum(double v) {
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    return dpp_add<0x143, 0xC>(v);
}

// The rows of sequence s, kept inside [0, rows] whatever the offsets hold.
template <typename Args>
__device__ __forceinline__ uint32_t seq_begin(const Args &a, uint32_t s) {
    const int32_t lo = a.cu_seqlens[s], rows = (int32_t)a.rows;
    return lo < 0 ? 0 : lo > rows ? rows : lo;
}
template <typename Args>
__device__ __forceinline__ uint32_t seq_length(const Args &a, uint32_t s, uint32_t begin) {
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
template <typename Args>
__device__ __forceinline__ int find_seq(const Args &a, uint32_t id, uint32_t unit) {
    if (a.seqs == 1) return 0;
    return find(id, (uint32_t)a.seqs, [&](uint32_t s) { return seq_begin(a, s) / unit + s; });
}

}  // namespace ssm
