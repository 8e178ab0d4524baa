// sink_decode.cu -- the single-token form of windowed attention with sinks:
// one new query per sequence over a cache of keys and values.
//
// Sequence b holds n = kv_len[b] tokens; its query stands at position n - 1 and
// sees key j iff j < n and (j > n - 1 - W or j < N).  Every visible key and
// value is read once for every 16 of the G query heads of its key/value head (once
// in all up to G = 16) and used by all of those, a few operations per byte: the
// kernel is bound by HBM, and what matters is to keep every SM's loads in flight
// and to give every SM the same share.
//
// Split.  The visible keys of every (sequence, key/value head, block of 16
// query heads) -- a segment -- are cut into tiles of 64, and all tiles of all
// segments, in order, are dealt to the CTAs in equal contiguous ranges.  The
// lengths live on the device, so every CTA sums them up itself.  A segment
// that one CTA covers is finished there; the others leave fp32 partials (max,
// sum, unnormalised output), at most two per CTA, which a second kernel joins
// in the order of the keys.  No atomics: the same bits on every call.
//
// Few short segments (CLUSTER; rule at launch()): a cluster of eight CTAs takes a
// segment, an eighth of its tiles each, and joins the parts through distributed
// shared memory: one launch instead of two (1 sequence of 1501 tokens, 32 heads of 8
// kv heads, window 1024: 5.6 us, by the two kernels 7.1; calls in a stream 7.9 to 8.7
// and 9.6).
//
// Per CTA: one producer warp streams K and V tiles by TMA into a ring; eight
// consumer warps in two groups take the tiles in turn, each warp 16 keys of
// its tile.  S = Q K^T and O += P V run as m16n8k16 bf16 MMAs on registers,
// rows = the 16 query heads (those beyond G are zero): with so few rows the
// 128-row tcgen05 tile would be 7/8 padding and need P in shared memory, and
// either unit is idle most of the time.  Operand fragments come straight from
// the swizzled tiles with 16-byte loads: the order of the head dimension is
// permuted alike in Q and K, and V's rows are paired with byte permutes, so no
// transposing load is needed.  Each warp keeps its own running maximum and
// sum in fp32; the probabilities are rounded to bf16 for the second product.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr int KT = 64;                         // keys per tile
constexpr int MH = 16;                         // query heads per segment (MMA M)
constexpr int kConsumers = 8;                  // warps; two groups of four
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kCluster = 8;                    // CTAs of a segment's cluster
constexpr int kClusterTiles = 8 * kCluster;    // segments of more tiles are spread over all SMs (rule at launch())
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
    static constexpr int kHalf = KT * D * 2;                   // K or V of one tile
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = D == 128 ? 4 : 8;           // 128 KB in flight
    static constexpr int kMerge = kConsumers * MH * D * 4;     // the warps' outputs, fp32
    static constexpr int kOffMerge = kStages * kStage;
    static constexpr int kOffStat = kOffMerge + kMerge;        // [8][16] max, [8][16] sum
    static constexpr int kOffBar = kOffStat + 2 * kConsumers * MH * 4;
    static constexpr int kOffPrefix = kOffBar + 256;           // [B + 1] tiles before each sequence
};

struct Args {
    int B, H, Hkv, G, HB;         // G = H / Hkv heads per kv head in HB blocks of 16
    int S, window, n_sink;
    const int32_t* kv_len;
    const __nv_bfloat16* q;       // [B, H, D]
    __nv_bfloat16* O;             // [B, H, D]
    float* lse;                   // [B, H]
    float scale_log2;
    int* prefix;                  // [B + 1], for the joining kernel
    float* part;                  // [2 * n CTAs][MH][D + 2]: unnormalised O, max, sum
    int* err;
};

// The visible keys of a sequence as tiles: the sinks' tiles, if the window has
// moved off them, then the window's.
struct Seen {
    int n, lo, sink_tiles, tiles;
};
__device__ __forceinline__ Seen seen(const Args& a, int b) {
    Seen x;
    x.n = min(max(a.kv_len[b], 0), a.S);
    x.lo = max(x.n - a.window, 0);
    x.sink_tiles = 0;
    if (x.lo <= a.n_sink) x.lo = 0;
    else x.sink_tiles = (a.n_sink + KT - 1) / KT;
    x.tiles = x.sink_tiles + (x.n - x.lo + KT - 1) / KT;
    return x;
}
// First key and number of keys of a sequence's k-th tile.
__device__ __forceinline__ void tile_keys(const Seen& x, int n_sink, int k, int& key, int& n) {
    if (k < x.sink_tiles) {
        key = k * KT;
        n = min(n_sink - key, KT);
    } else {
        key = x.lo + (k - x.sink_tiles) * KT;
        n = min(x.n - key, KT);
    }
}

// m16n8k16, bf16 in, fp32 accumulate.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Cursor over a CTA's range of tiles.
struct Cursor {
    int b, r, k;        // sequence, segment of the sequence, tile of the segment
    Seen s;
};

// Finds tile x (0 <= x < total): prefix[b] <= x < prefix[b + 1].
__device__ __forceinline__ Cursor find(const Args& a, const int* prefix, int x) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (prefix[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    Cursor c;
    c.b = lo;
    c.s = seen(a, lo);
    const int at = x - prefix[lo];
    c.r = at / c.s.tiles;
    c.k = at % c.s.tiles;
    return c;
}
// The segment after the cursor's (the caller knows that there is one).
__device__ __forceinline__ void next_segment(const Args& a, Cursor& c) {
    c.k = 0;
    if (++c.r == a.Hkv * a.HB) {
        c.r = 0;
        do c.s = seen(a, ++c.b);
        while (c.s.tiles == 0);
    }
}

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {            // the swizzled tiles need a 1 KB aligned base
        if (threadIdx.x == 0 && a.err) atomicExch(a.err, 2);
        return;
    }
    float* s_merge = reinterpret_cast<float*>(smem + C::kOffMerge);
    float* s_max = reinterpret_cast<float*>(smem + C::kOffStat);
    float* s_sum = s_max + kConsumers * MH;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);   // [kStages]
    uint64_t* empty = full + C::kStages;                               // [kStages]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
    int* prefix = reinterpret_cast<int*>(smem + C::kOffPrefix);
    int* s_scan = reinterpret_cast<int*>(smem + C::kOffBar + 192);     // [9]

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);         // the four warps of the tile's group
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        prefix[0] = 0;
    }
    Cursor c;
    int begin, end;
    const int R = a.Hkv * a.HB, rank = blockIdx.x % kCluster;
    if constexpr (CLUSTER) {
        const int segment = blockIdx.x / kCluster;
        c.b = segment / R;
        c.r = segment % R;
        c.s = seen(a, c.b);
        begin = c.k = c.s.tiles * rank / kCluster;
        end = c.s.tiles * (rank + 1) / kCluster;
        __syncthreads();
    } else {
        // Tiles before each sequence, all segments counted.
        int carry = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + (int)threadIdx.x;
            int x = b < a.B ? seen(a, b).tiles * R : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            for (int w = 0; w < warp; ++w) x += s_scan[w];
            if (b < a.B) prefix[b + 1] = carry + x;
            int all = 0;
            for (int w = 0; w < kThreads / 32; ++w) all += s_scan[w];
            carry += all;
            __syncthreads();
        }
        __syncthreads();
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b <= a.B; b += kThreads) a.prefix[b] = prefix[b];
        const int total = prefix[a.B];
        const int n_ctas = min((int)gridDim.x, total);   // every one of them has a tile
        if ((int)blockIdx.x >= n_ctas) return;
        begin = (int)((int64_t)total * blockIdx.x / n_ctas);
        end = (int)((int64_t)total * (blockIdx.x + 1) / n_ctas);
        c = find(a, prefix, begin);
    }
    if (warp == kConsumers) {
        // ------------------------------------------------------------ TMA producer
        bool ok = true;
        int x = begin;
        for (; x < end && ok; ++x) {
            const int i = x - begin, slot = i % C::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&empty[slot], ((i / C::kStages) & 1) ^ 1, abort_flag, a.err, nullptr));
            if (!ok) break;
            int key, n;
            tile_keys(c.s, a.n_sink, c.k, key, n);
            if (lane == 0) {
                uint8_t* dst = smem + slot * C::kStage;
                const int g = c.r / a.HB;
                mbar_arrive_expect_tx(&full[slot], C::kStage);
                for (int blk = 0; blk < D / 64; ++blk) {
                    tma_load_4d(dst + blk * KT * 128, &tmK, &full[slot], blk * 64, g, key, c.b);
                    tma_load_4d(dst + C::kHalf + blk * KT * 128, &tmV, &full[slot], blk * 64, g, key, c.b);
                }
            }
            __syncwarp();
            if (++c.k == c.s.tiles && x + 1 < end) next_segment(a, c);
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            for (int i = max(x - begin - C::kStages, 0); i < x - begin; ++i)
                mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, &dummy, nullptr);
        }
        __syncwarp();
        if constexpr (CLUSTER) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    // ---------------------------------------------------------------- consumers
    // Lane (g, t) = (lane / 4, lane % 4).  Column n of an 8-key score tile is key
    // row(n) = (n / 2) + 4 (n % 2), and column n of an output tile j of a block of 64
    // is dim 8 row(n) + j: with these orders the 16-byte loads of a quarter warp
    // fall on distinct banks of the swizzled tiles.
    const int g = lane / 4, t = lane % 4, grp = warp / 4, w16 = (warp % 4) * 16;
    const int rn = (g >> 1) | ((g & 1) << 2);
    bool ok = true;
    float4 mine[2];                      // CLUSTER: this CTA's part of at most two groups of four dims
    float2 mine_ml[2];
    mine_ml[0] = mine_ml[1] = make_float2(-INFINITY, 0.f);
    mine[0] = mine[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = begin; x < end && ok;) {
        // One segment, or the part of it in this CTA's range.
        const int k0 = c.k, k1 = min(c.s.tiles, k0 + end - x);
        const int gq = c.r / a.HB, hb = c.r % a.HB;
        const int h0 = gq * a.G + hb * MH, nh = min(a.G - hb * MH, MH);
        uint4 qa[D / 32], qb[D / 32];        // dims [32 p + 8 t, + 8) of heads g and g + 8
        {
            const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)c.b * a.H + h0) * D) + t;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int p = 0; p < D / 32; ++p) {
                qa[p] = g < nh ? src[g * (D / 8) + 4 * p] : zero;
                qb[p] = g + 8 < nh ? src[(g + 8) * (D / 8) + 4 * p] : zero;
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads g, g + 8; l: this lane's columns
        for (int k = k0; k < k1; ++k, ++x) {
            const int i = x - begin;
            if ((i & 1) != grp) continue;
            const int slot = i % C::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&full[slot], (i / C::kStages) & 1, abort_flag, a.err, nullptr));
            if (!ok) break;
            int key, n;
            tile_keys(c.s, a.n_sink, k, key, n);
            n -= w16;                        // keys of this warp's 16 that are visible (may be <= 0)
            const uint8_t* sk = smem + slot * C::kStage + w16 * 128;
            const uint8_t* sv = sk + C::kHalf;
            if (n > 0) {
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int p = 0; p < D / 32; ++p) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int row = z * 8 + rn, chunk = (p & 1) * 4 + t;
                        const uint4 u = *reinterpret_cast<const uint4*>(sk + (p / 2) * KT * 128 + row * 128 +
                                                                        ((chunk ^ (row & 7)) * 16));
                        mma16816(s[z], qa[p].x, qb[p].x, qa[p].y, qb[p].y, u.x, u.y);
                        mma16816(s[z], qa[p].z, qb[p].z, qa[p].w, qb[p].w, u.z, u.w);
                    }
                }
                // columns 2t, 2t + 1 of tile z are keys 8 z + t and 8 z + t + 4
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[z][e] *= a.scale_log2;
                        if (8 * z + t + 4 * (e & 1) >= n) s[z][e] = -INFINITY;
                    }
                float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                    const float y0 = fmaxf(m0, x0), y1 = fmaxf(m1, x1);   // finite: key 0 of the 16 is visible
                    const float a0 = ex2(m0 - y0), a1 = ex2(m1 - y1);     // 0 at first
                    m0 = y0; m1 = y1;
                    l0 *= a0; l1 *= a1;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][0] *= a0; o[j][1] *= a0;
                        o[j][2] *= a1; o[j][3] *= a1;
                    }
                }
                uint32_t pa[4];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float p0 = ex2(s[z][0] - m0), p1 = ex2(s[z][1] - m0);
                    const float p2 = ex2(s[z][2] - m1), p3 = ex2(s[z][3] - m1);
                    l0 += p0 + p1;
                    l1 += p2 + p3;
                    pa[2 * z] = pack_bf16(p0, p1);
                    pa[2 * z + 1] = pack_bf16(p2, p3);
                }
                const bool ragged = n < 16;
#pragma unroll
                for (int blk = 0; blk < D / 64; ++blk) {
                    uint4 u[4];              // keys t, t + 4, t + 8, t + 12
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int row = t + 4 * y;
                        u[y] = *reinterpret_cast<const uint4*>(sv + blk * KT * 128 + row * 128 + ((rn ^ (row & 7)) * 16));
                        // rows that are not visible may hold anything: 0 times an infinity is not 0
                        if (ragged && row >= n) u[y] = make_uint4(0, 0, 0, 0);
                    }
                    const uint32_t* v0 = &u[0].x;
                    const uint32_t* v1 = &u[1].x;
                    const uint32_t* v2 = &u[2].x;
                    const uint32_t* v3 = &u[3].x;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        mma16816(o[blk * 8 + 2 * y], pa[0], pa[1], pa[2], pa[3], __byte_perm(v0[y], v1[y], 0x5410),
                                 __byte_perm(v2[y], v3[y], 0x5410));
                        mma16816(o[blk * 8 + 2 * y + 1], pa[0], pa[1], pa[2], pa[3], __byte_perm(v0[y], v1[y], 0x7632),
                                 __byte_perm(v2[y], v3[y], 0x7632));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }
        // ---- the eight warps' states become one
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (t == 0) {
            s_max[warp * MH + g] = m0;
            s_max[warp * MH + g + 8] = m1;
            s_sum[warp * MH + g] = l0;
            s_sum[warp * MH + g + 8] = l1;
        }
        {
            // o[blk * 8 + j][0]: dim 64 blk + 8 t + j of head g, [1]: 32 dims further; [2], [3]: head g + 8
            float* dst = s_merge + (warp * MH + g) * D + 8 * t;
#pragma unroll
            for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float* p = dst + (e >> 1) * 8 * D + blk * 64 + (e & 1) * 32;
                    *reinterpret_cast<float4*>(p) = make_float4(o[blk * 8 + 0][e], o[blk * 8 + 1][e], o[blk * 8 + 2][e], o[blk * 8 + 3][e]);
                    *reinterpret_cast<float4*>(p + 4) = make_float4(o[blk * 8 + 4][e], o[blk * 8 + 5][e], o[blk * 8 + 6][e], o[blk * 8 + 7][e]);
                }
        }
        ok = named_bar_and(1, kConsumers * 32, ok);
        if (!ok) break;
        const bool whole = k0 == 0 && k1 == c.s.tiles;
        float* part = a.part + (int64_t)(2 * blockIdx.x + (k0 == 0)) * MH * (D + 2);
        for (int y = threadIdx.x; y < nh * (D / 4); y += kConsumers * 32) {
            const int h = y / (D / 4), d = y % (D / 4) * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, s_max[w * MH + h]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
                const float f = ex2(s_max[w * MH + h] - m);      // a warp without keys: max -inf, factor 0
                const float4 v = *reinterpret_cast<const float4*>(s_merge + (w * MH + h) * D + d);
                l = fmaf(f, s_sum[w * MH + h], l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if constexpr (CLUSTER) {
                const bool second = y >= kConsumers * 32;
                mine[second] = acc;
                mine_ml[second] = make_float2(m, l);
            } else if (whole) {
                const float inv = 1.f / l;
                const int64_t row = (int64_t)c.b * a.H + h0 + h;
                *reinterpret_cast<uint2*>(a.O + row * D + d) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                if (d == 0) a.lse[row] = (m + __log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float2*>(part + h * (D + 2) + d) = make_float2(acc.x, acc.y);
                *reinterpret_cast<float2*>(part + h * (D + 2) + d + 2) = make_float2(acc.z, acc.w);
                if (d == 0) *reinterpret_cast<float2*>(part + h * (D + 2) + D) = make_float2(m, l);
            }
        }
        if constexpr (CLUSTER) break;
        named_bar_sync(1, kConsumers * 32);  // the merge buffer is read before the next segment fills it
        if (x < end) next_segment(a, c);
    }
    if constexpr (CLUSTER) {
        // Parts [rank][head][D + 4] (unnormalised output, maximum, sum) in rank 0's ring, which it no longer needs.
        const int h0 = c.r / a.HB * a.G + c.r % a.HB * MH, nh = min(a.G - c.r % a.HB * MH, MH);
        constexpr int kRow = D + 4;
        static_assert(kCluster * MH * kRow * 4 <= C::kOffMerge, "parts");
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int y = threadIdx.x + z * kConsumers * 32, h = y / (D / 4), d = y % (D / 4) * 4;
            if (h >= nh) continue;
            const uint32_t dst = map_to_rank(smem_u32(smem) + (uint32_t)((rank * MH + h) * kRow + d) * 4, 0);
            st_cluster_v4(dst, mine[z]);
            if (d == 0) st_cluster_v2(dst + D * 4, mine_ml[z]);
        }
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int y = threadIdx.x + z * kConsumers * 32, h = y / (D / 4), d = y % (D / 4) * 4;
            if (h >= nh) continue;
            const float* part = reinterpret_cast<const float*>(smem) + h * kRow;
            float m = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int p = 0; p < kCluster; ++p) m = fmaxf(m, part[p * MH * kRow + D]);
#pragma unroll
            for (int p = 0; p < kCluster; ++p) {
                const float* q = part + p * MH * kRow;
                if (q[D] == -INFINITY && q[D + 1] == 0.f) continue;   // a part without keys
                const float f = ex2(q[D] - m);
                const float4 v = *reinterpret_cast<const float4*>(q + d);
                l = fmaf(f, q[D + 1], l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;          // no tiles: an empty sequence
            const int64_t row = (int64_t)c.b * a.H + h0 + h;
            *reinterpret_cast<uint2*>(a.O + row * D + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            if (d == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
        }
    }
}

// Joins a segment's partials: blocks (segment, 256 pairs of dims of its heads),
// one thread per pair.  Eight partials are loaded at a time, so that a segment cut
// into many waits for memory a few times and not once per piece (one sequence of
// 1501 tokens, 8 segments of 17 pieces: the step takes 7.1 us, 9.3 with one at a time).
constexpr int kJoinThreads = 256, kJoinAhead = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const Args a, int grid) {
    wait_for_previous_kernel();      // its partials
    const int R = a.Hkv * a.HB, b = blockIdx.x / R, r = blockIdx.x % R;
    const int hb = r % a.HB, h0 = r / a.HB * a.G + hb * MH, nh = min(a.G - hb * MH, MH);
    const int y = blockIdx.y * kJoinThreads + threadIdx.x, h = y / (D / 2), d = y % (D / 2) * 2;
    if (h >= nh) return;
    const int64_t total = a.prefix[a.B], n_ctas = min((int64_t)grid, total);
    const int before = a.prefix[b], tiles = (a.prefix[b + 1] - before) / R;
    int c0 = 0, c1 = -1;
    if (tiles > 0) {
        // the CTA that holds tile x is the last one whose range begins at or before it
        const int64_t first = before + (int64_t)r * tiles, last = first + tiles - 1;
        c0 = (int)(((first + 1) * n_ctas - 1) / total);
        c1 = (int)(((last + 1) * n_ctas - 1) / total);
        if (c0 == c1) return;            // finished by the CTA itself
    }
    float m = -INFINITY, l = 0.f;
    float2 acc = make_float2(0.f, 0.f);
    for (int c = c0; c <= c1; c += kJoinAhead) {
        float2 st[kJoinAhead], v[kJoinAhead];
#pragma unroll
        for (int e = 0; e < kJoinAhead; ++e) {
            st[e] = make_float2(-INFINITY, 0.f);
            v[e] = make_float2(0.f, 0.f);
            if (c + e <= c1) {           // the first piece is its CTA's last one, the others are their CTAs' first
                const float* p = a.part + ((int64_t)(2 * (c + e) + (c + e == c0)) * MH + h) * (D + 2);
                st[e] = *reinterpret_cast<const float2*>(p + D);
                v[e] = *reinterpret_cast<const float2*>(p + d);
            }
        }
        float n = m;
#pragma unroll
        for (int e = 0; e < kJoinAhead; ++e) n = fmaxf(n, st[e].x);
        const float f = ex2(m - n);      // 0 at first: every piece has a visible key
        m = n;
        l *= f;
        acc.x *= f;
        acc.y *= f;
#pragma unroll
        for (int e = 0; e < kJoinAhead; ++e) {
            const float g = ex2(st[e].x - n);
            l = fmaf(st[e].y, g, l);
            acc.x = fmaf(v[e].x, g, acc.x);
            acc.y = fmaf(v[e].y, g, acc.y);
        }
    }
    const int64_t row = (int64_t)b * a.H + h0 + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // no tiles: an empty sequence
    *reinterpret_cast<uint32_t*>(a.O + row * D + d) = pack_bf16(acc.x * inv, acc.y * inv);
    if (d == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
dfa_status launch(const DecodeProblem& p, const void* q, const void* k, const void* v, const int32_t* kv_len, void* O,
                  float* lse, void* ws, cudaStream_t s) {
    using C = Cfg<D>;
    CUtensorMap mk, mv;
    if (!make_tmap_bshd(&mk, k, p.B, p.S, p.Hkv, D, p.kv_sb, p.kv_ss, p.kv_sh, KT) ||
        !make_tmap_bshd(&mv, v, p.B, p.S, p.Hkv, D, p.kv_sb, p.kv_ss, p.kv_sh, KT))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    Args a{};
    a.B = p.B; a.H = p.H; a.Hkv = p.Hkv; a.G = p.H / p.Hkv; a.HB = (a.G + MH - 1) / MH;
    a.S = p.S; a.window = p.window; a.n_sink = p.n_sink;
    a.kv_len = kv_len;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.lse = lse;
    a.scale_log2 = p.scale * kLog2e;
    a.prefix = static_cast<int*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + align256(sizeof(int) * ((size_t)p.B + 1)));
    a.err = device_error_flag();
    const int segments = p.B * a.Hkv * a.HB;
    const int64_t tiles = (int64_t)segments * decode_tiles(p);
    const int n = (int)std::min<int64_t>(num_sms(), tiles);
    const int smem = C::kOffPrefix + (int)sizeof(int) * (p.B + 1);
    static std::atomic<uint64_t> seen{0};
    static std::atomic<int> clusters{0};             // that run at a time
    auto spread = decode_kernel<D, false>;
    auto clustered = decode_kernel<D, true>;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)kCluster);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = C::kOffPrefix + 16;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (first_on_device(seen)) {
        constexpr int most = C::kOffPrefix + (int)sizeof(int) * (kMaxDecodeBatch + 1);
        static_assert(most <= 232448, "shared memory");
        int k = 0;
        if (cudaFuncSetAttribute(spread, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaFuncSetAttribute(clustered, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&k, clustered, &cfg) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "decode: kernel attributes");
        clusters.store(k);
        mark_on_device(seen);
    }
    // One round of clusters, each with tiles enough for its share of the SMs: 4096 keys of 8 kv
    // heads 8.2 us, spread over all SMs 8.9; 8192 keys 12.1 and 10.8; 262 keys 4.2 and 6.0.
    if (segments <= clusters.load() && decode_tiles(p) <= kClusterTiles) {
        cfg.gridDim = dim3((unsigned)(segments * kCluster));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, clustered, mk, mv, a);
        if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
        count_launch(DFA_KERNEL_FWD);
        return DFA_OK;
    }
    spread<<<n, kThreads, smem, s>>>(mk, mv, a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
    e = launch_overlapped(join_kernel<D>, dim3(segments, (std::min(a.G, MH) * (D / 2) + kJoinThreads - 1) / kJoinThreads),
                          kJoinThreads, 0, s, a, n);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode join launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_FWD);
    count_launch(DFA_KERNEL_MERGE);
    return DFA_OK;
}

}  // namespace

int64_t decode_tiles(const DecodeProblem& p) {
    const int64_t keys = std::min(p.window, p.S);
    return (keys + KT - 1) / KT + (p.window < p.S ? (p.n_sink + KT - 1) / KT : 0);
}

size_t decode_workspace(const DecodeProblem& p) {
    return align256(align256(sizeof(int) * ((size_t)p.B + 1)) +
                    sizeof(float) * 2 * (size_t)num_sms() * MH * (p.D + 2));
}

dfa_status sink_decode(const DecodeProblem& p, const void* q, const void* k, const void* v, const int32_t* kv_len,
                       void* O, float* lse, void* ws, cudaStream_t s) {
    return p.D == 128 ? launch<128>(p, q, k, v, kv_len, O, lse, ws, s) : launch<64>(p, q, k, v, kv_len, O, lse, ws, s);
}

}  // namespace dfa
