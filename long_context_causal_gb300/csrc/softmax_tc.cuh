// softmax_tc.cuh -- the softmax thread's part of a tcgen05 attention forward: one
// query row of 128 scores in TMEM, its maximum, and its probabilities written back
// over the scores as the bf16 A operand of the product with V.
#pragma once

#include <cmath>

#include "ptx.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr uint32_t kMinusInf = 0xff800000u;

// Column c of a tile is visible iff (c >= lo or c < ns) and c < lim.
struct Mask {
    int lo, lim, ns;
    int lo0, lim0, more;   // lo and lim of the warp's first row; its last row's are `more` larger
    // The warp's rows and columns [c, c + 32): none visible, all visible.
    __device__ __forceinline__ bool none(int c) const { return lim0 + more <= c || (lo0 >= c + 32 && ns <= c); }
    __device__ __forceinline__ bool all(int c) const { return lo0 + more <= c && lim0 >= c + 32; }
    // bit e: column c + e
    __device__ __forceinline__ uint32_t bits(int c) const {
        return (~low_bits(lo - c) | low_bits(ns - c)) & low_bits(lim - c);
    }
};

// The warp's P so far is in TMEM.
__device__ __forceinline__ void hand_over(uint64_t* bar, int lane) {
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void max32(float (&m)[4], const uint32_t (&u)[32]) {
#pragma unroll
    for (int e = 0; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(u[e]));
}
// P = exp2(s * c2 - m) of 32 columns as bf16 pairs to tP; acc: sums of the unrounded P
// of the even and of the odd columns.  Two columns per instruction where there is one:
// the softmax warps' instructions are on the chain (32K tokens, D = 128: window 4096 1342 -> 1320 us,
// 128 180 -> 175; D = 64 1170 -> 1160 and 164 -> 156).
__device__ __forceinline__ void exp32(uint64_t& acc, const uint32_t (&u)[32], float c2, float m, uint32_t tP) {
    uint32_t pk[16];
    const uint64_t cc = pack_f32x2(c2, c2), mm = pack_f32x2(-m, -m);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 x =
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), cc, mm));
        const float p0 = ex2(x.x), p1 = ex2(x.y);
        acc = add_f32x2(acc, pack_f32x2(p0, p1));
        pk[e] = pack_bf16(p0, p1);
    }
    tmem_st16(tP, pk);
}

// A tile that every row of the block sees whole: row max of this thread's 128
// scores in TMEM.  Each piece's load runs under the arithmetic of the one before
// it (here and in row_exp: 32K tokens, window 4096 1433 -> 1343 us).
__device__ __forceinline__ float row_max(uint32_t tS) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    uint32_t a[32], b[32];
    tmem_ld32_async(tS, a);
    tmem_wait_ld32(a);
    tmem_ld32_async(tS + 32, b);
    max32(m, a);
    tmem_wait_ld32(b);
    tmem_ld32_async(tS + 64, a);
    max32(m, b);
    tmem_wait_ld32(a);
    tmem_ld32_async(tS + 96, b);
    max32(m, a);
    tmem_wait_ld32(b);
    max32(m, b);
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// Its P, written as bf16 pairs over S (behind the columns still to be read);
// `most` is told when 96 columns are there.  Returns the row sum of the unrounded P.
template <bool TWICE>
__device__ __forceinline__ float row_exp(uint32_t tS, float c2, float m, uint64_t* most, int lane) {
    uint64_t acc = pack_f32x2(0.f, 0.f);
    uint32_t a[32], b[32];
    tmem_ld32_async(tS, a);
    tmem_wait_ld32(a);
    tmem_ld32_async(tS + 32, b);
    exp32(acc, a, c2, m, tS);
    tmem_wait_ld32(b);
    tmem_ld32_async(tS + 64, a);
    exp32(acc, b, c2, m, tS + 16);
    tmem_wait_ld32(a);
    tmem_ld32_async(tS + 96, b);
    exp32(acc, a, c2, m, tS + 32);
    if (TWICE) hand_over(most, lane);
    tmem_wait_ld32(b);
    exp32(acc, b, c2, m, tS + 48);
    return sum_f32x2(acc);
}

// The same two for the first 32 * chunks columns under a mask.
__device__ __forceinline__ float row_max_masked(uint32_t tS, int chunks, const Mask& k) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        if (k.none(c * 32)) continue;
        uint32_t u[32];
        tmem_ld32(tS + c * 32, u);
        if (!k.all(c * 32)) {
            const uint32_t see = k.bits(c * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = see >> e & 1 ? u[e] : kMinusInf;
        }
        max32(m, u);
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <bool TWICE>
__device__ __forceinline__ float row_exp_masked(uint32_t tS, int chunks, const Mask& k, float c2, float m, uint64_t* most,
                                                int lane) {
    uint64_t acc = pack_f32x2(0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        if (k.none(c * 32)) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0;
            tmem_st16(tS + c * 16, pk);
        } else {
            uint32_t u[32];
            tmem_ld32(tS + c * 32, u);
            const uint32_t see = k.bits(c * 32);          // a branch around it, as above, costs more than it saves
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = see >> e & 1 ? u[e] : kMinusInf;   // P = 0: the scale is positive
            exp32(acc, u, c2, m, tS + c * 16);
        }
        if (TWICE && c == 2) hand_over(most, lane);
    }
    if (TWICE && chunks < 3) hand_over(most, lane);
    return sum_f32x2(acc);
}

}  // namespace
}  // namespace dfa
