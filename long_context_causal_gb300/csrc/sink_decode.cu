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
//
// With masses (kMass).  A key's weight needs its heads' log-sum-exps, which are known
// at the end only: the consumers write the scores down, 4 bytes a head beside the 512
// of a key and value (D = 128; 3% more at 4 heads a group), and the launch that joins
// the outputs turns them into weights.  K and V are loaded to make room first, so the
// scores are still in the L2 then: 32 sequences of up to 16384 keys, 32/8 heads, 178 to 183 us
// a call (1.10 GB at 6000 to 6140 GB/s, 91% of the copy rate; D = 64 136, 4.1 TB/s), of which 165 are the cache and
// 11 the masses; 195 before the cache policy and with 1024 keys a block, 219 with a
// launch of its own for the masses and short sequences counted by their tiles alone.
// In a cluster (one sequence of 1501 keys) the scores stay in shared memory and the CTA
// that has them forms the weights: 6.3 to 6.5 us of GPU time, 8.9 to 9.3 by two launches.
//
// Behind a shared prefix (kParts, kSolo).  The same kernel over the sequences' own keys,
// started beside prefix_decode.cu's and leaving fp32 parts, which prefix_join_kernel adds
// to the prefix's: 128 sequences of up to 1024 own keys, 64/8 heads, behind 16384: 117 us
// a call (prefix 48, own keys 52 at 5.1 TB/s, join 10).  A segment costs a CTA 2 us beside
// its tiles (queries, the eight warps' states made one), so short sequences count for more
// than their keys when the tiles are dealt: with tiles alone the CTA of the shortest ones
// ran 123 us, the others 46.  Where the own keys are few (at most four tiles, a segment per
// SM at most) a CTA takes a segment and adds the prefix's parts itself: 4 sequences behind
// 1000 keys 7.5 to 7.8 us of GPU time; 10.7 with the launch that joins, 9.0 with a part's place
// worked out once the prefix is there and four parts asked for at a time.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
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
    float* part;                  // [2 * n CTAs][MH][row_floats]: unnormalised O, max, sum
    int* err;
    // MASS: the scores times log2 e of the visible keys, [B * H][stride] in the order of the tiles
    float* score;
    int stride;                   // 64 * the most tiles of a segment
    const float* mass;            // [B, Hkv, S], null: zero
    float* mass_out;              // [B, Hkv, S]; may be `mass`
    int fused;                    // CLUSTER: the scores stay in shared memory and the cluster forms the masses
    // PARTS: a segment that one CTA covers leaves its rows' parts here, [B * H][row_floats]
    float* own;
    PrefixPlan p;                 // PARTS, SOLO: the prefix's parts
    const float* p_part;
    const float2* p_stat;
};
// Plain; with masses; behind a prefix: leaving parts, or (SOLO) a CTA per segment, which adds the prefix's.
enum Mode { kPlain, kMass, kParts, kSolo };
// Units that a segment counts for beside its tiles when the tiles are dealt: it costs a CTA 2 us beside
// 0.7 to 0.9 us per tile.  (The plain step deals tiles alone.)
template <bool CLUSTER, Mode MODE>
constexpr int kUnits = CLUSTER || MODE == kPlain || MODE == kSolo ? 0 : kDecodeUnits;
// Floats of a head's partial: unnormalised O, max, sum.
template <int D, Mode MODE>
constexpr int row_floats() { return MODE == kPlain ? D + 2 : D + 4; }

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

// What a head's weights relative to 2^m, whose sum is l, make of its output and its log-sum-exp (times log2 e).  l = 0:
// there is no key, or the scores are -inf in 32 bits one and all; nothing is drawn then, O = 0 and lse = -inf, however
// the keys were cut.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log2_sum(float m, float l) { return l == 0.f ? -INFINITY : m + __log2f(l); }
// What a key's score is taken from for its weight: 2^(-inf - 0) is 0, 2^(-inf + inf) is not.
__device__ __forceinline__ float weight_base(float lse) { return lse == -INFINITY ? 0.f : lse; }

// Floats of a head's scores in shared memory: eight tiles of a cluster's CTA, rows on different banks.
constexpr int kScoreRow = kClusterTiles / kCluster * KT + 4;
constexpr int kScoreBytes = MH * kScoreRow * 4;
__device__ __forceinline__ void store4(float* at, const float (&x)[4]) {
    *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
}

// Cursor over a CTA's range.  A segment counts for W units more than its tiles, which
// stand before them: what its beginning and end cost a CTA.
struct Cursor {
    int b, r, v;        // sequence, segment of the sequence, unit of the segment
    Seen s;
};

// Finds unit x (0 <= x < total): prefix[b] <= x < prefix[b + 1].
template <int W>
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
    c.r = at / (c.s.tiles + W);
    c.v = at % (c.s.tiles + W);
    return c;
}
// The segment after the cursor's (the caller knows that there is one).
__device__ __forceinline__ void next_segment(const Args& a, Cursor& c) {
    c.v = 0;
    if (++c.r == a.Hkv * a.HB) {
        c.r = 0;
        do c.s = seen(a, ++c.b);
        while (c.s.tiles == 0);
    }
}

// The CTAs that hold units [x, x + n) of a list of `total` dealt to n_ctas in equal
// ranges: the last ones whose ranges begin at or before them.
__device__ __forceinline__ void ctas_of(int64_t x, int64_t n, int64_t total, int n_ctas, int& c0, int& c1) {
    if (total < (1 << 23)) {             // 32 bits: n_ctas is below 2^9
        c0 = (int)((((uint32_t)x + 1) * (uint32_t)n_ctas - 1) / (uint32_t)total);
        c1 = (int)((((uint32_t)x + (uint32_t)n) * (uint32_t)n_ctas - 1) / (uint32_t)total);
    } else {
        c0 = (int)(((x + 1) * n_ctas - 1) / total);
        c1 = (int)(((x + n) * n_ctas - 1) / total);
    }
}
// Brings a segment's queries (at most 16 rows) to the L1.
template <int D>
__device__ __forceinline__ void prefetch_rows(const Args& a, const Cursor& c, int lane) {
    const int hb = c.r % a.HB, h0 = c.r / a.HB * a.G + hb * MH, nh = min(a.G - hb * MH, MH);
    const char* rows = reinterpret_cast<const char*>(a.q + ((int64_t)c.b * a.H + h0) * D);
    if (lane < nh * D * 2 / 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(rows + lane * 128));
}

// Where the prefix's parts of the heads of a group are, in the order of the keys.
struct PrefixParts {
    int b, c0, count;             // sequence; first CTA, number of pieces
    int s, z, r, n;               // of a head: segment, tile of the pair, row; parts
    bool alone;
    int g;
    __device__ __forceinline__ PrefixParts(const Args& a, int sequence, int group) : b(sequence), c0(0), count(0), s(-1), n(0), g(group) {}
    __device__ __forceinline__ void head(const Args& a, int gi) {
        if (a.p.grid == 0) return;
        const int at = b * a.G + gi, tile = at / 128, seg = g * a.p.n_pairs + tile / 2;
        if (seg != s) {
            s = seg;
            int c1;
            ctas_of((int64_t)s * a.p.n_kt, a.p.n_kt, a.p.steps, a.p.grid, c0, c1);
            count = c1 - c0 + 1;
        }
        r = at % 128;
        z = tile & 1;
        alone = (tile & ~1) * 128 + 128 >= a.p.rows;         // the pair has this tile only: two parts a piece
        n = count << alone;
    }
    __device__ __forceinline__ int64_t at(const Args& a, int i) const {
        return (alone ? 2 * (int64_t)(s + c0) + i : 2 * (int64_t)(s + c0 + i) + z) * a.p.row_stride + r;
    }
};

template <int D, bool CLUSTER, Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args a) {
    using C = Cfg<D>;
    constexpr int W = kUnits<CLUSTER, MODE>, kRow = row_floats<D, MODE>();
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
    float* s_score = reinterpret_cast<float*>(smem + C::kOffPrefix);   // CLUSTER, MASS: in its place
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
    if (MODE == kMass) wait_for_previous_kernel();
    Cursor c;
    int begin, end;
    const int R = a.Hkv * a.HB, rank = blockIdx.x % kCluster;
    if constexpr (CLUSTER) {
        const int segment = blockIdx.x / kCluster;
        c.b = segment / R;
        c.r = segment % R;
        c.s = seen(a, c.b);
        begin = c.v = c.s.tiles * rank / kCluster;
        end = c.s.tiles * (rank + 1) / kCluster;
        __syncthreads();
    } else if constexpr (MODE == kSolo) {
        c.b = blockIdx.x / R;
        c.r = blockIdx.x % R;
        c.s = seen(a, c.b);
        begin = c.v = 0;
        end = c.s.tiles;
        __syncthreads();
    } else {
        // Units before each sequence, all segments counted.
        int carry = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + (int)threadIdx.x;
            int x = b < a.B ? seen(a, b).tiles : 0;
            x = x > 0 ? (x + W) * R : 0;
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
        const int n_ctas = min((int)gridDim.x, total);   // every one of them has a unit
        if ((int)blockIdx.x >= n_ctas) {
            if (MODE == kParts && blockIdx.x == 0) wait_for_previous_kernel();
            return;
        }
        begin = (int)((int64_t)total * blockIdx.x / n_ctas);
        end = (int)((int64_t)total * (blockIdx.x + 1) / n_ctas);
        c = find<W>(a, prefix, begin);
    }
    if (warp == kConsumers) {
        // ------------------------------------------------------------ TMA producer
        bool ok = true;
        int i = 0;
        const uint64_t once = MODE == kMass ? l2_evict_first() : 0;
        for (int x = begin; x < end && ok;) {
            const int v1 = min(c.s.tiles + W, c.v + end - x), k1 = v1 - W;
            for (int k = max(c.v - W, 0); k < k1; ++k, ++i) {
                const int slot = i % C::kStages;
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&empty[slot], ((i / C::kStages) & 1) ^ 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                int key, n;
                tile_keys(c.s, a.n_sink, k, key, n);
                if (lane == 0) {
                    uint8_t* dst = smem + slot * C::kStage;
                    const int g = c.r / a.HB;
                    mbar_arrive_expect_tx(&full[slot], C::kStage);
                    for (int blk = 0; blk < D / 64; ++blk) {
                        if (MODE == kMass) {         // read once: the scores are to stay in the L2
                            tma_load_4d_once(dst + blk * KT * 128, &tmK, &full[slot], blk * 64, g, key, c.b, once);
                            tma_load_4d_once(dst + C::kHalf + blk * KT * 128, &tmV, &full[slot], blk * 64, g, key, c.b, once);
                        } else {
                            tma_load_4d(dst + blk * KT * 128, &tmK, &full[slot], blk * 64, g, key, c.b);
                            tma_load_4d(dst + C::kHalf + blk * KT * 128, &tmV, &full[slot], blk * 64, g, key, c.b);
                        }
                    }
                }
                __syncwarp();
            }
            x += v1 - c.v;
            if (x < end) {
                next_segment(a, c);
                // its queries are on their way while the consumers are still at the ring's tiles
                if (MODE != kPlain) prefetch_rows<D>(a, c, lane);
            }
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            for (int m = max(i - C::kStages, 0); m < i; ++m)
                mbar_wait(&full[m % C::kStages], (m / C::kStages) & 1, &dummy, nullptr);
        }
        __syncwarp();
        // PARTS: started beside the prefix's kernel.  What joins the parts waits for this
        // one to end, and through its first CTA for that one.
        if (MODE == kParts && blockIdx.x == 0) wait_for_previous_kernel();
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
    float4 mine[2];                      // CLUSTER, SOLO: this CTA's part of at most two groups of four dims
    float2 mine_ml[2];
    mine_ml[0] = mine_ml[1] = make_float2(-INFINITY, 0.f);
    mine[0] = mine[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    int i = 0;
    for (int x = begin; x < end && ok;) {
        // One segment, or the part of it in this CTA's range.
        const int v1 = min(c.s.tiles + W, c.v + end - x), k0 = max(c.v - W, 0), k1 = v1 - W;
        x += v1 - c.v;
        if (k1 <= k0) {                      // nothing but what stands before the tiles (or an empty share)
            if constexpr (CLUSTER || MODE == kSolo) break;
            if (x < end) next_segment(a, c);
            continue;
        }
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
        // heads g, g + 8; l: this lane's columns.  The maxima begin at the lowest number, so that a score that is
        // -inf in 32 bits counts for nothing wherever it stands.
        float m0 = -FLT_MAX, m1 = -FLT_MAX, l0 = 0.f, l1 = 0.f;
        for (int k = k0; k < k1; ++k, ++i) {
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
                if constexpr (MODE == kMass) {
                    // keys 4 m + t of a head's 16 in lane t become 4 t .. 4 t + 3
                    const bool here = CLUSTER && a.fused;
                    float* to = here ? s_score + g * kScoreRow + i * KT : a.score + ((int64_t)c.b * a.H + h0 + g) * a.stride + k * KT;
                    to += w16 + 4 * t;
                    float lo[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
                    quad_transpose(lo, lane);
                    if (g < nh) store4(to, lo);
                    if (nh > 8) {
                        float hi[4] = {s[0][2], s[0][3], s[1][2], s[1][3]};
                        quad_transpose(hi, lane);
                        if (g + 8 < nh) store4(to + 8 * (here ? kScoreRow : a.stride), hi);
                    }
                }
                float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                    const float y0 = fmaxf(m0, x0), y1 = fmaxf(m1, x1);
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
        float* part = a.part + (int64_t)(2 * blockIdx.x + (k0 == 0)) * MH * kRow;
        if (MODE == kParts && whole) part = a.own + ((int64_t)c.b * a.H + h0) * kRow;
        for (int y = threadIdx.x; y < nh * (D / 4); y += kConsumers * 32) {
            const int h = y / (D / 4), d = y % (D / 4) * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, s_max[w * MH + h]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
                const float f = ex2(s_max[w * MH + h] - m);      // a warp without keys: sum and outputs 0
                const float4 v = *reinterpret_cast<const float4*>(s_merge + (w * MH + h) * D + d);
                l = fmaf(f, s_sum[w * MH + h], l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if constexpr (CLUSTER || MODE == kSolo) {
                const bool second = y >= kConsumers * 32;
                mine[second] = acc;
                mine_ml[second] = make_float2(m, l);
            } else if (MODE != kParts && whole) {
                const float inv = reciprocal(l);
                const int64_t row = (int64_t)c.b * a.H + h0 + h;
                *reinterpret_cast<uint2*>(a.O + row * D + d) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                if (d == 0) a.lse[row] = log2_sum(m, l) * kLn2;
            } else {
                *reinterpret_cast<float2*>(part + h * kRow + d) = make_float2(acc.x, acc.y);
                *reinterpret_cast<float2*>(part + h * kRow + d + 2) = make_float2(acc.z, acc.w);
                if (d == 0) *reinterpret_cast<float2*>(part + h * kRow + D) = make_float2(m, l);
            }
        }
        if constexpr (CLUSTER || MODE == kSolo) break;
        named_bar_sync(1, kConsumers * 32);  // the merge buffer is read before the next segment fills it
        if (x < end) next_segment(a, c);
    }
    if constexpr (CLUSTER) {
        // Parts [rank][head][D + 4] (unnormalised output, maximum, sum) in rank 0's ring, which it no longer needs.
        const int h0 = c.r / a.HB * a.G + c.r % a.HB * MH, nh = min(a.G - c.r % a.HB * MH, MH);
        constexpr int kRow = D + 4;          // unnormalised output, maximum, sum
        static_assert(kCluster * MH * kRow * 4 <= C::kOffMerge, "parts");
        const bool masses = MODE == kMass && a.fused;
        // The masses of this CTA's keys so far, and their place; -1: none.
        constexpr int kEach = kClusterTiles / kCluster * KT / (kConsumers * 32);
        float before[kEach];
        int64_t at[kEach];
        if (masses) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int y = threadIdx.x + e * kConsumers * 32;
                at[e] = -1;
                before[e] = 0.f;
                if (y >= (end - begin) * KT) continue;
                int key, n;
                tile_keys(c.s, a.n_sink, begin + y / KT, key, n);
                if (y % KT >= n) continue;
                at[e] = ((int64_t)c.b * a.Hkv + c.r) * a.S + key + y % KT;
                if (a.mass) before[e] = a.mass[at[e]];
            }
        }
        __syncwarp();
        cluster_sync();
        // Maxima and sums go to every CTA where each one forms the masses of its keys ([rank][head], in the merge buffer).
        if (masses && (int)threadIdx.x < nh) {
            const int h = threadIdx.x;
            float m = -INFINITY, l = 0.f;
            if (end > begin) {
                for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, s_max[w * MH + h]);
                for (int w = 0; w < kConsumers; ++w) l = fmaf(ex2(s_max[w * MH + h] - m), s_sum[w * MH + h], l);
            }
            for (int r = 0; r < kCluster; ++r)
                st_cluster_v2(map_to_rank(smem_u32(smem) + C::kOffMerge + (uint32_t)(rank * MH + h) * 8, r), make_float2(m, l));
        }
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
        if (masses) {
            if ((int)threadIdx.x < nh) {
                const float2* st = reinterpret_cast<const float2*>(smem + C::kOffMerge) + threadIdx.x;
                float m = -INFINITY, l = 0.f;
                for (int r = 0; r < kCluster; ++r) m = fmaxf(m, st[r * MH].x);
                for (int r = 0; r < kCluster; ++r) l += st[r * MH].y == 0.f ? 0.f : ex2(st[r * MH].x - m) * st[r * MH].y;   // a NaN stays
                s_max[threadIdx.x] = weight_base(log2_sum(m, l));
            }
            named_bar_sync(1, kConsumers * 32);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (at[e] < 0) continue;
                const float* score = s_score + threadIdx.x + e * kConsumers * 32;
                float w = 0.f;
                for (int h = 0; h < nh; ++h) w += ex2(score[h * kScoreRow] - s_max[h]);
                a.mass_out[at[e]] = before[e] + w;
            }
            // the keys that the query does not see, an eighth of them each
            const int64_t row = ((int64_t)c.b * a.Hkv + c.r) * a.S;
            const int j1 = (int)((int64_t)a.S * (rank + 1) / kCluster);
            for (int j = (int)((int64_t)a.S * rank / kCluster) + threadIdx.x; j < j1; j += kConsumers * 32)
                if (j >= c.s.n || (j < c.s.lo && j >= a.n_sink)) a.mass_out[row + j] = a.mass && j < c.s.n ? a.mass[row + j] : 0.f;
        }
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
            const float inv = reciprocal(l);
            const int64_t row = (int64_t)c.b * a.H + h0 + h;
            *reinterpret_cast<uint2*>(a.O + row * D + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            if (d == 0) a.lse[row] = log2_sum(m, l) * kLn2;
        }
    }
    if constexpr (MODE == kSolo) {
        if (!ok) return;
        const int gq = c.r / a.HB, hb = c.r % a.HB, nh = min(a.G - hb * MH, MH);
        // Where the parts are is known before they are there.
        PrefixParts pieces(a, c.b, gq);
        int parts[2];
        int64_t first[2], step[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int h = (threadIdx.x + z * kConsumers * 32) / (D / 4);
            parts[z] = 0;
            if (h >= nh) continue;
            pieces.head(a, hb * MH + h);
            parts[z] = pieces.n;
            first[z] = pieces.at(a, 0);
            step[z] = pieces.at(a, 1) - first[z];
        }
        wait_for_previous_kernel();          // the prefix's parts
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int y = threadIdx.x + z * kConsumers * 32, h = y / (D / 4), d = y % (D / 4) * 4;
            if (h >= nh) continue;
            constexpr int kAhead = 8;
            float m = mine_ml[z].x, l = mine_ml[z].y;
            float4 acc = mine[z];
#pragma unroll 1
            for (int e0 = 0; e0 < parts[z]; e0 += kAhead) {
                float2 st[kAhead];
                float4 v[kAhead];
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    st[e] = make_float2(-INFINITY, 0.f);
                    v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (e0 + e < parts[z]) {
                        const int64_t at = first[z] + (e0 + e) * step[z];
                        st[e] = a.p_stat[at];
                        v[e] = *reinterpret_cast<const float4*>(a.p_part + at * D + d);
                    }
                }
                float top = m;
#pragma unroll
                for (int e = 0; e < kAhead; ++e) top = fmaxf(top, st[e].x);
                const float base = top == -INFINITY ? 0.f : top;
                const float f = ex2(m - base);
                m = top;
                l *= f;
                acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    if (st[e].y == 0.f) continue;                // nothing else was written
                    const float w = ex2(st[e].x - base);
                    l = fmaf(w, st[e].y, l);
                    acc.x = fmaf(w, v[e].x, acc.x);
                    acc.y = fmaf(w, v[e].y, acc.y);
                    acc.z = fmaf(w, v[e].z, acc.z);
                    acc.w = fmaf(w, v[e].w, acc.w);
                }
            }
            const float inv = reciprocal(l);
            const int64_t row = (int64_t)c.b * a.H + gq * a.G + hb * MH + h;
            *reinterpret_cast<uint2*>(a.O + row * D + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            if (d == 0) a.lse[row] = log2_sum(m, l) * kLn2;
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
    const float inv = reciprocal(l);
    *reinterpret_cast<uint32_t*>(a.O + row * D + d) = pack_bf16(acc.x * inv, acc.y * inv);
    if (d == 0) a.lse[row] = log2_sum(m, l) * kLn2;
}

// Those of the tiles of a segment of sequence b; none: c1 < c0.
__device__ __forceinline__ void own_ctas(const Args& a, int b, int r, int W, int grid, int& c0, int& c1) {
    const int total = a.prefix[a.B], before = a.prefix[b], units = (a.prefix[b + 1] - before) / (a.Hkv * a.HB);
    c0 = 0, c1 = -1;
    if (units > 0) ctas_of((int64_t)before + (int64_t)r * units + W, units - W, total, min(grid, total), c0, c1);
}

// Parts of a row (sequence b, head h) joined by a warp: of the prefix, if there is
// one, then of the own keys, in the order of the keys, 32 at a time: a lane reads a
// part's maximum and sum, the warp adds the outputs up with the lanes' factors.
template <int D, Mode MODE>
__device__ __forceinline__ void join_row(const Args& a, int grid, int64_t row) {
    constexpr int V = D / 32, kRow = row_floats<D, MODE>(), kAhead = 8;
    const int lane = threadIdx.x % 32, b = (int)(row / a.H), h = (int)row - b * a.H, g = h / a.G, gi = h - g * a.G;
    int c0, c1;
    own_ctas(a, b, g * a.HB + gi / MH, kUnits<false, MODE>, grid, c0, c1);
    if (MODE == kMass && c0 == c1) return;       // finished by the CTA itself
    PrefixParts pieces(a, b, g);
    if (MODE == kParts) pieces.head(a, gi);
    const int n_prefix = pieces.n;
    const int n = n_prefix + c1 - c0 + 1;
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int base = 0; base < n; base += 32) {
        const int i = base + lane;
        const float* src = nullptr;
        float2 st = make_float2(-INFINITY, 0.f);
        if (i < n_prefix) {
            const int64_t z = pieces.at(a, i);
            st = a.p_stat[z];
            src = a.p_part + z * D;
        } else if (i < n) {
            const int c = c0 + i - n_prefix;
            src = c0 == c1 ? a.own + row * kRow : a.part + ((int64_t)(2 * c + (c == c0)) * MH + gi % MH) * kRow;
            st = *reinterpret_cast<const float2*>(src + D);
        }
        float top = st.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        const float old = top == -INFINITY ? 1.f : ex2(m - top);
        const float f = st.y > 0.f ? ex2(st.x - top) : 0.f;      // sum 0: no key in the part, nothing else was written
        float sum = f * st.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        m = top;
        l = fmaf(l, old, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= old;
        const int count = min(n - base, 32);
        for (int e = 0; e < count; e += kAhead) {
            float x[kAhead][V], w[kAhead];
#pragma unroll
            for (int z = 0; z < kAhead; ++z) {
                const float* from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), (e + z) & 31));
                w[z] = e + z < count ? __shfl_sync(0xffffffffu, f, (e + z) & 31) : 0.f;
                if (w[z] > 0.f) {
                    if constexpr (V == 4) {
                        const float4 y = *reinterpret_cast<const float4*>(from + lane * 4);
                        x[z][0] = y.x, x[z][1] = y.y, x[z][2] = y.z, x[z][3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2*>(from + lane * 2);
                        x[z][0] = y.x, x[z][1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) x[z][v] = 0.f;
                }
            }
#pragma unroll
            for (int z = 0; z < kAhead; ++z)
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(w[z], x[z][v], acc[v]);
        }
    }
    const float inv = reciprocal(l);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.O + row * D + lane * V);
    if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    else *dst = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (lane == 0) a.lse[row] = log2_sum(m, l) * kLn2;
}

// Joins the parts of a shared prefix and of the sequences' own keys, a warp per row.
constexpr int kFinishThreads = 256, kFinishWarps = kFinishThreads / 32;
template <int D>
__global__ void __launch_bounds__(kFinishThreads, 4)
prefix_join_kernel(const Args a, int grid) {
    wait_for_previous_kernel();
    const int64_t row = (int64_t)blockIdx.x * kFinishWarps + threadIdx.x / 32;
    if (row < (int64_t)a.B * a.H) join_row<D, kParts>(a, grid, row);
}

// The masses of a step, and the outputs of the segments that several CTAs share.
//   mass_out = mass + each visible key's 2^(score - lse log2 e), summed over the heads
//   of its group in their order; 0 behind the sequence.
// Blocks [0, joins): a warp per row.  The others: 4096 keys of a (sequence, key/value
// head) each, four of a thread at a time, once the block knows the heads' log-sum-exps:
// of the rows that are still being joined it adds up the parts' sums itself.  grid 0: every row
// has been finished.
constexpr int kMassRounds = 4, kMassKeys = kMassRounds * 4 * kFinishThreads, kMassHeads = 32;
template <int D>
__global__ void __launch_bounds__(kFinishThreads)
mass_kernel(const Args a, int grid, int joins, int blocks) {
    wait_for_previous_kernel();
    if ((int)blockIdx.x < joins) {
        const int64_t row = (int64_t)blockIdx.x * kFinishWarps + threadIdx.x / 32;
        if (row < (int64_t)a.B * a.H) join_row<D, kMass>(a, grid, row);
        return;
    }
    constexpr int kRow = row_floats<D, kMass>();
    __shared__ float s_lse[kMassHeads];              // times log2 e
    const int id = blockIdx.x - joins, r = id / blocks, b = r / a.Hkv, g = r - b * a.Hkv, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int first = (id - r * blocks) * kMassKeys, end = min(first + kMassKeys, a.S);
    const Seen x = seen(a, b);
    const float* mass = a.mass + (int64_t)r * a.S;
    float* out = a.mass_out + (int64_t)r * a.S;
    for (int j = max(first, x.n) + threadIdx.x; j < end; j += kFinishThreads) out[j] = 0.f;
    const int last = min(end, x.n);
    if (first >= last) return;
    for (int h0 = 0; h0 < a.G; h0 += kMassHeads) {
        const int heads = min(a.G - h0, kMassHeads);
        const int64_t row0 = (int64_t)b * a.H + g * a.G + h0;
        __syncthreads();                             // the last heads' have been read
        for (int h = warp; h < heads; h += kFinishWarps) {
            int c0 = 0, c1 = 0;
            if (grid > 0) own_ctas(a, b, g * a.HB + (h0 + h) / MH, kUnits<false, kMass>, grid, c0, c1);
            float m, l = 1.f;
            if (c0 == c1) {
                m = a.lse[row0 + h] * kLog2e;
            } else {
                float2 st = make_float2(-INFINITY, 0.f);
                for (int c = c0 + lane; c <= c1; c += 32) {
                    const float2 y = *reinterpret_cast<const float2*>(a.part + ((int64_t)(2 * c + (c == c0)) * MH + (h0 + h) % MH) * kRow + D);
                    const float t = fmaxf(st.x, y.x);
                    st = make_float2(t, st.y * ex2(st.x - t) + y.y * ex2(y.x - t));
                }
                m = st.x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                l = st.y * ex2(st.x - m);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            }
            if (lane == 0) s_lse[h] = weight_base(log2_sum(m, l));
        }
        __syncthreads();
        const float* score = a.score + row0 * a.stride;
        for (int j0 = first + threadIdx.x; j0 < last; j0 += 4 * kFinishThreads) {
            float before[4], w[4] = {0.f, 0.f, 0.f, 0.f};
            int key[4];                              // the key's place among the scores; -1: not seen
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + e * kFinishThreads;
                before[e] = j >= last ? 0.f : h0 > 0 ? out[j] : a.mass ? mass[j] : 0.f;
                key[e] = j >= last ? -1 : j >= x.lo ? x.sink_tiles * KT + j - x.lo : j < a.n_sink ? j : -1;
            }
#pragma unroll 4
            for (int h = 0; h < heads; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key[e] >= 0) w[e] += ex2(score[(int64_t)h * a.stride + key[e]] - s_lse[h]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + e * kFinishThreads;
                if (j < last) out[j] = before[e] + w[e];
            }
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t prefix_bytes(const DecodeProblem& p) { return align256(sizeof(int) * ((size_t)p.B + 1)); }
size_t own_bytes(const DecodeProblem& p) { return align256(sizeof(float) * (size_t)p.B * p.H * (p.D + 4)); }
size_t stat_bytes(const PrefixPlan& x) { return align256(sizeof(float2) * 2 * (size_t)x.slabs * x.row_stride); }
size_t part_bytes(const DecodeProblem& p) { return align256(sizeof(float) * 2 * (size_t)num_sms() * MH * (p.D + 4)); }

// grid: CTAs of the step's kernel, 0 if it has finished every row.
template <int D>
dfa_status launch_mass(const Args& a, int grid, cudaStream_t s) {
    const int blocks = (a.S + kMassKeys - 1) / kMassKeys, joins = grid > 0 ? (int)(((int64_t)a.B * a.H + kFinishWarps - 1) / kFinishWarps) : 0;
    const cudaError_t e = launch_overlapped(mass_kernel<D>, dim3((unsigned)(joins + a.B * a.Hkv * blocks)), kFinishThreads, 0, s, a, grid,
                                            joins, blocks);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode mass launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_MASS);
    return DFA_OK;
}

template <int D>
Args make_args(const DecodeProblem& p, const void* q, const int32_t* kv_len, void* O, float* lse, void* ws) {
    Args a{};
    a.B = p.B; a.H = p.H; a.Hkv = p.Hkv; a.G = p.H / p.Hkv; a.HB = (a.G + MH - 1) / MH;
    a.S = p.S; a.window = p.window; a.n_sink = p.n_sink;
    a.kv_len = kv_len;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.lse = lse;
    a.scale_log2 = p.scale * kLog2e;
    a.prefix = static_cast<int*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + prefix_bytes(p));
    a.err = device_error_flag();
    return a;
}

template <int D>
dfa_status make_maps(const DecodeProblem& p, const void* k, const void* v, CUtensorMap* mk, CUtensorMap* mv) {
    if (!make_tmap_bshd(mk, k, p.B, p.S, p.Hkv, D, p.kv_sb, p.kv_ss, p.kv_sh, KT) ||
        !make_tmap_bshd(mv, v, p.B, p.S, p.Hkv, D, p.kv_sb, p.kv_ss, p.kv_sh, KT))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    return DFA_OK;
}

template <int D>
constexpr int most_smem() {
    constexpr int most = Cfg<D>::kOffPrefix + (int)sizeof(int) * (kMaxDecodeBatch + 1);
    static_assert(most <= 232448, "shared memory");
    return most;
}

// The prefix's part, the own keys' part beside it, and the join; or a CTA per segment of own keys that joins as well.
// The second while the caches have room for at most four tiles (the host does not know the lengths) and an SM takes a
// segment at most.  GPU time by it and by the first, 4 sequences, 32/8 heads, behind 1000 keys: 64 own keys 7.7 and 10.5
// us, 256 7.7 and 12.3; 16 sequences of 256 11.4 and 16.1; behind 16000 19.3 and 26.8; D = 64 6.8 and 9.6, 6.8 and 11.3.
// With more room the second was still ahead, by less for each tile: 4 x 512 own keys 8.6 and 13.7, 4 x 1024 12.1 and 14.8.
constexpr int kSoloTiles = 4;
template <int D>
dfa_status launch_prefix(const DecodeProblem& p, int P, const void* q, const void* kp, const void* vp, int64_t ss, int64_t sh,
                         const void* k, const void* v, const int32_t* kv_len, void* O, float* lse, void* ws, cudaStream_t s) {
    CUtensorMap mk, mv;
    dfa_status st = make_maps<D>(p, k, v, &mk, &mv);
    if (st) return st;
    Args a = make_args<D>(p, q, kv_len, O, lse, ws);
    const PrefixPlan plan = prefix_plan(p.B, a.G, p.Hkv, P, num_sms());
    char* at = static_cast<char*>(ws) + prefix_bytes(p) + part_bytes(p);
    a.own = reinterpret_cast<float*>(at);
    at += own_bytes(p);
    float2* stat = reinterpret_cast<float2*>(at);
    float* part = reinterpret_cast<float*>(at + stat_bytes(plan));
    a.p = plan;
    a.p_stat = stat;
    a.p_part = part;
    auto own = decode_kernel<D, false, kParts>;
    auto solo = decode_kernel<D, false, kSolo>;
    static std::atomic<uint64_t> seen{0};
    if (first_on_device(seen)) {
        if (cudaFuncSetAttribute(own, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem<D>()) != cudaSuccess ||
            cudaFuncSetAttribute(solo, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem<D>()) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "decode: kernel attributes");
        mark_on_device(seen);
    }
    if (plan.grid > 0 && (st = tc_prefix(p, plan, q, kp, vp, ss, sh, part, stat, s))) return st;
    // Beside the prefix's kernel, on SMs that it leaves or does not need: it starts when that one has, which is after all
    // work before the call.  Without a prefix it is launched as any other.
    auto launch_own = [&](auto kernel, int grid, size_t smem) {
        if (plan.grid > 0) return launch_overlapped(kernel, dim3((unsigned)grid), kThreads, smem, s, mk, mv, a);
        kernel<<<grid, kThreads, smem, s>>>(mk, mv, a);
        return cudaGetLastError();
    };
    const int64_t segments = (int64_t)p.B * a.Hkv * a.HB, tiles = decode_tiles(p);
    cudaError_t e;
    if (tiles <= kSoloTiles && segments <= num_sms()) {
        e = launch_own(solo, (int)segments, Cfg<D>::kOffPrefix + 16);
        if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
        count_launch(DFA_KERNEL_FWD);
        return DFA_OK;
    }
    const int n = (int)std::min<int64_t>(num_sms(), segments * tiles);
    e = launch_own(own, n, Cfg<D>::kOffPrefix + sizeof(int) * (p.B + 1));
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
    e = launch_overlapped(prefix_join_kernel<D>, dim3((unsigned)(((int64_t)p.B * p.H + kFinishWarps - 1) / kFinishWarps)), kFinishThreads,
                          0, s, a, n);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "prefix join launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_FWD);
    count_launch(DFA_KERNEL_MERGE);
    return DFA_OK;
}

template <int D, Mode MODE>
dfa_status launch(const DecodeProblem& p, const void* q, const void* k, const void* v, const int32_t* kv_len, void* O,
                  float* lse, const float* mass, float* mass_out, void* ws, cudaStream_t s) {
    using C = Cfg<D>;
    constexpr bool MASS = MODE == kMass;
    CUtensorMap mk, mv;
    const dfa_status st = make_maps<D>(p, k, v, &mk, &mv);
    if (st) return st;
    Args a = make_args<D>(p, q, kv_len, O, lse, ws);
    if (MASS) {
        a.score = reinterpret_cast<float*>(static_cast<char*>(ws) + prefix_bytes(p) + part_bytes(p));
        a.stride = (int)(KT * decode_tiles(p));
        a.mass = mass;
        a.mass_out = mass_out;
    }
    const int segments = p.B * a.Hkv * a.HB;
    const int64_t tiles = (int64_t)segments * decode_tiles(p);
    const int n = (int)std::min<int64_t>(num_sms(), tiles);
    const int smem = C::kOffPrefix + (int)sizeof(int) * (p.B + 1);
    static std::atomic<uint64_t> seen{0};
    static std::atomic<int> clusters{0};             // that run at a time
    auto spread = decode_kernel<D, false, MODE>;
    auto clustered = decode_kernel<D, true, MODE>;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)kCluster);
    cfg.blockDim = dim3((unsigned)kThreads);
    a.fused = MASS && a.HB == 1;             // the heads of a group in one segment
    constexpr int cluster_smem = C::kOffPrefix + (MASS ? kScoreBytes : 16);
    static_assert(cluster_smem <= 232448, "shared memory");
    cfg.dynamicSmemBytes = cluster_smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (first_on_device(seen)) {
        constexpr int most = most_smem<D>();
        int k = 0;
        if (cudaFuncSetAttribute(spread, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaFuncSetAttribute(clustered, cudaFuncAttributeMaxDynamicSharedMemorySize, std::max(most, cluster_smem)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&k, clustered, &cfg) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "decode: kernel attributes");
        clusters.store(k);
        mark_on_device(seen);
    }
    // One round of clusters, each with tiles enough for its share of the SMs: 4096 keys of 8 kv
    // heads 8.2 us, spread over all SMs 8.9; 8192 keys 12.1 and 10.8; 262 keys 4.2 and 6.0.  With masses, GPU time: 262
    // keys 5.4 and 7.7, 1501 6.5 and 8.9, 4096 9.1 and 11.9 (D = 64 7.6 and 13.7); 4096 of one kv head 8.8 and 12.6.
    if (segments <= clusters.load() && decode_tiles(p) <= kClusterTiles) {
        cfg.gridDim = dim3((unsigned)(segments * kCluster));
        if (MASS) cfg.numAttrs = 2;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, clustered, mk, mv, a);
        if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
        count_launch(DFA_KERNEL_FWD);
        return MASS && !a.fused ? launch_mass<D>(a, 0, s) : DFA_OK;
    }
    cudaError_t e;
    if (MASS) {
        e = launch_overlapped(spread, dim3((unsigned)n), kThreads, (size_t)smem, s, mk, mv, a);
    } else {
        spread<<<n, kThreads, smem, s>>>(mk, mv, a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_FWD);
    if (MASS) return launch_mass<D>(a, n, s);
    e = launch_overlapped(join_kernel<D>, dim3(segments, (std::min(a.G, MH) * (D / 2) + kJoinThreads - 1) / kJoinThreads),
                          kJoinThreads, 0, s, a, n);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "decode join launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_MERGE);
    return DFA_OK;
}

}  // namespace

int64_t decode_tiles(const DecodeProblem& p) {
    const int64_t keys = std::min(p.window, p.S);
    return (keys + KT - 1) / KT + (p.window < p.S ? (p.n_sink + KT - 1) / KT : 0);
}

size_t decode_workspace(const DecodeProblem& p, bool mass) {
    return prefix_bytes(p) + part_bytes(p) + (mass ? sizeof(float) * (size_t)p.B * p.H * KT * decode_tiles(p) : 0);
}

dfa_status sink_decode(const DecodeProblem& p, const void* q, const void* k, const void* v, const int32_t* kv_len,
                       void* O, float* lse, const float* mass, float* mass_out, void* ws, cudaStream_t s) {
    if (mass_out)
        return p.D == 128 ? launch<128, kMass>(p, q, k, v, kv_len, O, lse, mass, mass_out, ws, s)
                          : launch<64, kMass>(p, q, k, v, kv_len, O, lse, mass, mass_out, ws, s);
    return p.D == 128 ? launch<128, kPlain>(p, q, k, v, kv_len, O, lse, nullptr, nullptr, ws, s)
                      : launch<64, kPlain>(p, q, k, v, kv_len, O, lse, nullptr, nullptr, ws, s);
}

size_t prefix_workspace(const DecodeProblem& p, int P) {
    const PrefixPlan x = prefix_plan(p.B, p.H / p.Hkv, p.Hkv, P, num_sms());
    return prefix_bytes(p) + part_bytes(p) + own_bytes(p) + stat_bytes(x) + sizeof(float) * 2 * (size_t)x.slabs * x.row_stride * p.D;
}

dfa_status prefix_decode(const DecodeProblem& p, int P, const void* q, const void* kp, const void* vp, int64_t ss, int64_t sh,
                         const void* k, const void* v, const int32_t* kv_len, void* O, float* lse, void* ws, cudaStream_t s) {
    return p.D == 128 ? launch_prefix<128>(p, P, q, kp, vp, ss, sh, k, v, kv_len, O, lse, ws, s)
                      : launch_prefix<64>(p, P, q, kp, vp, ss, sh, k, v, kv_len, O, lse, ws, s);
}

}  // namespace dfa
