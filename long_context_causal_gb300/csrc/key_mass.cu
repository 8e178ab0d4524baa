// key_mass.cu -- attention weight gathered per key over a prompt, for sm_103a.
//
// mass[b, g, j] = sum over the heads h of group g and the queries i >= S - n_last
// that see key j of exp(scale <q_ih, k_j> - lse_ih), with the window and sinks of
// sink_fwd_tc.cu: the column sums of the softmax that the forward never forms.
//
// One product per pair, S^T = K Q^T, keys in the rows: an accumulator row is a
// key's, so a thread adds up its key's weights in a register and no sum crosses
// threads.  A CTA holds a block of 512 keys (four tiles of 128) in shared memory
// and sweeps the heads of the group and the tiles of 128 queries that see it; each
// query tile is loaded once for the four key tiles (16 bytes a cycle, a quarter of
// what one key tile at a time would ask of the L2).  TMEM holds the four tiles'
// scores, one warpgroup for each: while a warpgroup forms its weights the tensor
// cores run the other three products.
//
// What bounds it: the warpgroups' arithmetic.  128 x 128 scores are 512 cycles of the
// exponential unit and 512 of the tensor cores.  The arithmetic around the exponentials
// alone lets a sub-partition do a tile's 32 rows in 632 cycles with four warps; in the
// kernel a step of four tiles takes 3030 (tensor cores 66% busy, exponentials 66%, issue
// slots 52%), set by the sub-partition that also has the issuing warp.  32K tokens, 32/8
// heads, D = 128, window 4096, 4 sinks: 827 to 862 us (1200 to 1250 TFLOP/s); 2 x 5003
// tokens causal, 16/2 heads, 80 to 83 us (1240).  At D = 64 the products are half and the
// exponentials the same: 721 and 75 us, exponentials 70% busy, tensor cores 35%, issue slots
// 55% (the exponentials alone would take 400 and 40 us at the highest clock).  With three quarters of the products left
// out 720 us, without the loads of the queries' log-sum-exps 792, with half of the
// exponentials 779: no unit alone.  Measured and not kept: two warpgroups that hold a
// tile's 128 scores each 974 (too few warps to hide the latencies); scores loaded ahead
// across a loop's end 1960 to 2080; the warpgroups' waits by polling 876, the issuing
// warp's by suspending 878; a region handed back at half of the arithmetic instead of
// three quarters 853; log-sum-exps loaded 8 bytes at a time instead of 16 no change.
//
// Roles (640 threads, one CTA per SM): warp 0 TMA producer of K and Q, warp 1 MMA
// issuer, warp 2 TMEM owner, warp 3 the queries' -lse log2 e (-inf for rows past
// the end: weight 0), warps 4-19 four warpgroups.
//
// Split.  A block's sweep is a list of steps (head, query tile); the steps of all
// blocks, in order, are dealt to the CTAs in equal contiguous ranges.  How many
// steps lie before a block is a sum of three linear pieces, so a CTA finds its
// first step without a table.  A block that one CTA sweeps whole is written there;
// of the others each CTA leaves 512 sums, which a second kernel adds up in the
// order of the steps.  No atomics: the same bits on every call.  With few blocks (rule at
// launch()) a cluster shares a block's steps instead, in one launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr int kThreads = 640;
constexpr int BT = 128;                    // keys or queries per tile
constexpr int kTiles = 4;                  // key tiles per block, and regions of TMEM
constexpr int kBlock = kTiles * BT;
constexpr int kNSlots = 4;                 // query tiles whose lse are at hand
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
    static constexpr int kTileBytes = BT * D * 2;
    static constexpr int kQSlots = D == 128 ? 3 : 4;
    static constexpr int kOffQ = kTiles * kTileBytes;
    static constexpr int kOffN = kOffQ + kQSlots * kTileBytes;
    static constexpr int kOffBar = kOffN + kNSlots * BT * 4;
    static constexpr int kSmem = kOffBar + 256;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Args {
    int H, Hkv, G, S;
    int window, n_sink;    // window <= S; n_sink 0 when the window covers every key
    int q0, n_qt;          // first query; tiles of 128 from it on
    int n_kb;              // key blocks per (batch, kv head)
    int64_t steps;         // of all blocks, one per (head of the group, query tile)
    int e1, c0;            // block kb is seen by tiles [max(0, 4 kb - c0), min(n_qt, 4 kb + e1))
    float scale_log2;
    const float* lse;      // [B, H, S]
    float* mass;           // [B, Hkv, S]
    float* part;           // [2 * CTAs][kBlock]
    int* err;
};

// sum over k < K of max(0, 4 k + c)
__host__ __device__ inline int64_t ramp(int64_t K, int64_t c) {
    const int64_t k0 = c > 0 ? 0 : -c / 4 + 1;          // the first k with 4 k + c > 0
    return K > k0 ? (K - k0) * (c + 2 * (k0 + K - 1)) : 0;
}
// Query tiles that see the blocks before K, all counted.
__host__ __device__ inline int64_t tiles_before(const Args& a, int64_t K) {
    int64_t x = ramp(K, a.e1) - ramp(K, a.e1 - a.n_qt) - ramp(K, -a.c0);
    if (K > 0 && a.n_sink > 0) x += a.n_qt - min(a.n_qt, max(a.e1, 0));     // all of them see block 0
    return x;
}
// The tiles that see a block: [first, last).
__host__ __device__ inline void tiles_of(const Args& a, int kb, int& first, int& last) {
    first = max(0, 4 * kb - a.c0);
    last = kb == 0 && a.n_sink > 0 ? a.n_qt : min(a.n_qt, 4 * kb + a.e1);
}

// Position in the list of steps: block kb of row r = b * Hkv + g, head h of the group, query tile t.
struct Cursor {
    int r, kb, h, t, first, last;
    __device__ __forceinline__ void find(const Args& a, int64_t x) {
        const int64_t per_row = tiles_before(a, a.n_kb) * a.G;
        r = (int)(x / per_row);
        x -= r * per_row;
        int lo = 0, hi = a.n_kb - 1;                    // the last block that begins at or before x and is not empty
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (tiles_before(a, mid) * a.G <= x) lo = mid;
            else hi = mid - 1;
        }
        kb = lo;
        tiles_of(a, kb, first, last);
        const int at = (int)(x - tiles_before(a, kb) * a.G);
        h = at / (last - first);
        t = first + at % (last - first);
    }
    // To the next step; the caller knows that there is one.  True if it is another block's.
    __device__ __forceinline__ bool next(const Args& a) {
        if (++t < last) return false;
        t = first;
        if (++h < a.G) return false;
        h = 0;
        do {
            if (++kb == a.n_kb) kb = 0, ++r;
            tiles_of(a, kb, first, last);
        } while (last <= first);
        t = first;
        return true;
    }
    __device__ __forceinline__ int row0(const Args& a) const { return a.q0 + t * BT; }
    // Whether a key tile has a pair that is visible in this step.
    __device__ __forceinline__ bool sees(const Args& a, int w) const {
        const int k0 = kb * kBlock + w * BT, i0 = row0(a);
        return k0 < a.S && min(i0 + BT, a.S) > k0 && (i0 - k0 < BT + a.window - 1 || k0 < a.n_sink);
    }
    // The first query tile from t on that does not see a key tile whole (or has rows past the end); t if it is one.
    __device__ __forceinline__ int whole_until(const Args& a, int w) const {
        const int k0 = kb * kBlock + w * BT, i0 = row0(a);
        if (i0 < k0 + BT - 1) return t;
        // i0 + 127 - k0 < window and i0 + 128 <= S
        return t + max(min(min(a.window - (i0 - k0), a.S - i0) / BT, last - t), 0);
    }
    // 32 columns each that hold queries
    __device__ __forceinline__ int chunks(const Args& a) const { return min(4, (a.S - row0(a) + 31) / 32); }
};

// Weights of 32 queries for this thread's key: 2^(s c + n), n the queries' -lse log2 e;
// see: the queries that see the key.  The others' weights are 0 whatever their scores and n are (a NaN
// among them): the mask comes behind both.
template <bool MASKED = false>
__device__ __forceinline__ void add32(uint64_t (&acc)[4], const uint32_t (&u)[32], float c, const float* n, uint32_t see = 0xffffffffu) {
    const uint64_t cc = pack_f32x2(c, c);
    uint64_t x[16];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float4 m = *reinterpret_cast<const float4*>(n + 2 * e);
        x[e] = fma_f32x2(pack_f32x2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), cc, pack_f32x2(m.x, m.y));
        x[e + 1] = fma_f32x2(pack_f32x2(__uint_as_float(u[2 * e + 2]), __uint_as_float(u[2 * e + 3])), cc, pack_f32x2(m.z, m.w));
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float2 y = unpack_f32x2(x[e]);
        if (MASKED) {
            y.x = see >> (2 * e) & 1 ? y.x : -INFINITY;
            y.y = see >> (2 * e + 1) & 1 ? y.y : -INFINITY;
        }
        x[e] = pack_f32x2(ex2(y.x), ex2(y.y));
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e & 3] = add_f32x2(acc[e & 3], x[e]);
}
// Bit e: query i0 + e sees key j, i.e. j <= i and (i < j + window or j < n_sink).  Rows past the end are zeros and
// see nothing: times a key's infinity they would be NaN.
__device__ __forceinline__ uint32_t see32(int key, int i0, int S, int window, int n_sink) {
    return ~low_bits(key - i0) & low_bits(S - i0) & (key < n_sink ? 0xffffffffu : low_bits(key - i0 + window));
}
__device__ __forceinline__ float sum4(const uint64_t (&acc)[4]) {
    return sum_f32x2(add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3])));
}
// Those of 128 queries, all of which see it: each piece's load runs under the arithmetic of the one before.
__device__ __forceinline__ void add128(uint64_t (&acc)[4], uint32_t tS, float c, const float* n) {
    uint32_t x[32], y[32];
    tmem_ld32_async(tS, x);
    tmem_wait_ld32(x);
    tmem_ld32_async(tS + 32, y);
    add32(acc, x, c, n);
    tmem_wait_ld32(y);
    tmem_ld32_async(tS + 64, x);
    add32(acc, y, c, n + 32);
    tmem_wait_ld32(x);
    tmem_ld32_async(tS + 96, y);
    add32(acc, x, c, n + 64);
    tmem_wait_ld32(y);
    add32(acc, y, c, n + 96);
}
// CLUSTER: a block's steps are shared by a cluster of eight CTAs, an eighth each, whose sums
// meet in the first one's shared memory: one launch.
constexpr int kCluster = 8, kJoinSteps = 4;
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
key_mass_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const Args a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {            // the swizzled tiles need a 1 KB aligned base
        if (threadIdx.x == 0 && a.err) atomicExch(a.err, 2);
        return;
    }
    uint8_t *sK = smem, *sQ = smem + C::kOffQ;
    float* sN = reinterpret_cast<float*>(smem + C::kOffN);                // [kNSlots][128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* k_full = bars + 0;             // [kTiles]
    uint64_t* k_empty = bars + 4;            // one for the block
    uint64_t* s_full = bars + 5;             // [kTiles]
    uint64_t* s_free = bars + 9;             // [kTiles]
    uint64_t* q_full = bars + 13;            // [kQSlots]
    uint64_t* q_empty = bars + 17;
    uint64_t* n_full = bars + 21;            // [kNSlots]
    uint64_t* n_empty = bars + 25;
    uint64_t* done = bars + 29;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 30);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 31);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kTiles; ++w) {
            mbar_init(&k_full[w], 1);
            mbar_init(&s_full[w], 1);
            mbar_init(&s_free[w], 4);
        }
        mbar_init(k_empty, 1);
        for (int s = 0; s < C::kQSlots; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
        }
        for (int s = 0; s < kNSlots; ++s) {
            mbar_init(&n_full[s], 1);
            mbar_init(&n_empty[s], 4 * kTiles);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_previous_kernel();
    const uint32_t tmem = *tmem_slot;
    Cursor c;
    int n, rank = 0;
    float total = 0.f;                       // of a key's weights, in the threads that add them up
    if constexpr (CLUSTER) {
        rank = blockIdx.x % kCluster;
        c.r = blockIdx.x / kCluster / a.n_kb;
        c.kb = blockIdx.x / kCluster % a.n_kb;
        tiles_of(a, c.kb, c.first, c.last);
        const int per = max(c.last - c.first, 0), all = per * a.G, from = all * rank / kCluster;
        n = all * (rank + 1) / kCluster - from;
        c.h = per ? from / per : 0;
        c.t = c.first + (per ? from % per : 0);
    } else {
        const int64_t begin = a.steps * blockIdx.x / gridDim.x, end = a.steps * (blockIdx.x + 1) / gridDim.x;
        n = (int)(end - begin);              // at least one: the grid is no larger than the list
        c.find(a, begin);
    }

    if (CLUSTER && n == 0) {
        // nothing to sweep
    } else if (warp == 0) {
        // ------------------------------------------------------------ TMA producer of K and Q
        uint32_t blocks = 0;
        bool ok = true, fresh = true;
        int i = 0;
        for (; i < n && ok; ++i) {
            if (fresh) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(k_empty, (blocks & 1) ^ 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                if (lane == 0) {
                    for (int w = 0; w < kTiles; ++w) {
                        const int k0 = c.kb * kBlock + w * BT;
                        if (k0 >= a.S) {
                            mbar_arrive(&k_full[w]);
                            continue;
                        }
                        mbar_arrive_expect_tx(&k_full[w], C::kTileBytes);
                        for (int blk = 0; blk < D / 64; ++blk)
                            tma_load_4d(sK + w * C::kTileBytes + blk * 16384, &tmK, &k_full[w], blk * 64, c.r % a.Hkv, k0,
                                        c.r / a.Hkv);
                    }
                }
                __syncwarp();
                ++blocks;
            }
            const int slot = i % C::kQSlots;
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&q_empty[slot], ((i / C::kQSlots) & 1) ^ 1, abort_flag, a.err, nullptr));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&q_full[slot], C::kTileBytes);
                for (int blk = 0; blk < D / 64; ++blk)
                    tma_load_4d(sQ + slot * C::kTileBytes + blk * 16384, &tmQ, &q_full[slot], blk * 64,
                                c.r % a.Hkv * a.G + c.h, c.row0(a), c.r / a.Hkv);
            }
            __syncwarp();
            fresh = i + 1 < n && c.next(a);
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            if (blocks > 0)
                for (int w = 0; w < kTiles; ++w) mbar_wait(&k_full[w], (blocks - 1) & 1, &dummy, nullptr);
            for (int m = max(i - C::kQSlots, 0); m < i; ++m)
                mbar_wait(&q_full[m % C::kQSlots], (m / C::kQSlots) & 1, &dummy, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one lane of a converged warp)
        const uint32_t lead = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);      // uniform
        const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
        constexpr uint64_t kStep = C::kTileBytes >> 4;
        uint32_t blocks = 0, used[kTiles] = {0, 0, 0, 0};
        bool ok = true, fresh = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && mbar_wait_spin(bar, parity, abort_flag, a.err);
            if (ok) tc_fence_after();
            return ok;
        };
        for (int i = 0; i < n && ok; ++i) {
            const int slot = i % C::kQSlots;
            if (!wait(&q_full[slot], (i / C::kQSlots) & 1)) break;
            const uint32_t id = idesc_bf16_f32(BT, 32 * c.chunks(a), false, false);
#pragma unroll
            for (int w = 0; w < kTiles; ++w) {
                if (fresh && !wait(&k_full[w], blocks & 1)) break;
                if (!c.sees(a, w)) continue;
                if (!wait(&s_free[w], (used[w] & 1) ^ 1)) break;
                ++used[w];
                const uint64_t a0 = dK + w * kStep, b0 = dQ + slot * kStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss_lead(lead, tm + w * BT, a0 + off, b0 + off, id, kk > 0);
                }
                mma_commit_lead(lead, &s_full[w]);
            }
            if (!ok) break;
            mma_commit_lead(lead, &q_empty[slot]);
            if (fresh) ++blocks;
            fresh = i + 1 < n && c.next(a);
            if (fresh) mma_commit_lead(lead, k_empty);
        }
        // Drain: every MMA issued here has finished before TMEM is freed.
        mma_commit_lead(lead, done);
        int dummy = 0;
        mbar_wait(done, 0, &dummy, a.err);
    } else if (warp == 3) {
        // ------------------------------------------------------------ -lse log2 e of the queries
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int slot = i % kNSlots;
            float x[4];
            const float* lse = a.lse + ((int64_t)(c.r / a.Hkv) * a.H + c.r % a.Hkv * a.G + c.h) * a.S;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = c.row0(a) + e * 32 + lane;
                const float l = row < a.S ? lse[row] : -INFINITY;
                x[e] = l == -INFINITY ? l : -l * kLog2e;      // no such query, or one that sees nothing: weight 0
            }
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&n_empty[slot], ((i / kNSlots) & 1) ^ 1, abort_flag, a.err, nullptr));
            if (!ok) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) sN[slot * BT + e * 32 + lane] = x[e];
            __syncwarp();
            if (lane == 0) mbar_arrive(&n_full[slot]);
            if (i + 1 < n) c.next(a);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ weights: a warpgroup per key tile, a thread per key
        const int w = (warp - 4) / 4, row = w * BT + (warp % 4) * 32 + lane;
        const uint32_t tS = tmem + ((uint32_t)((warp % 4) * 32) << 16) + w * BT;
        uint32_t used = 0;
        bool from_start = c.h == 0 && c.t == c.first;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            // Steps whose 128 queries see all keys of the tile, up to the head's last one or the first that does not.
            const int whole = c.whole_until(a, w) - c.t;
            if (whole > 0) {
                const int end_i = min(i + whole, n);
                c.t += end_i - i - 1;
#pragma unroll 1
                for (;; ++i) {
                    const int slot = i % kNSlots;
                    const float* nl = sN + slot * BT;
                    ok = mbar_wait_acc(&n_full[slot], (i / kNSlots) & 1, abort_flag, a.err, nullptr) &&
                         mbar_wait_acc(&s_full[w], used++ & 1, abort_flag, a.err, nullptr);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
                    uint64_t acc[4] = {0, 0, 0, 0};
                    uint32_t x[32], y[32];
                    tmem_ld32_async(tS, x);
                    tmem_wait_ld32(x);
                    tmem_ld32_async(tS + 32, y);
                    add32(acc, x, a.scale_log2, nl);
                    tmem_wait_ld32(y);
                    tmem_ld32_async(tS + 64, x);
                    add32(acc, y, a.scale_log2, nl + 32);
                    tmem_wait_ld32(x);
                    tmem_ld32_async(tS + 96, y);
                    add32(acc, x, a.scale_log2, nl + 64);
                    tmem_wait_ld32(y);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[w]);
                    add32(acc, y, a.scale_log2, nl + 96);
                    total += sum4(acc);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&n_empty[slot]);
                    if (i + 1 == end_i) break;
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            } else {
                const int slot = i % kNSlots;
                const bool sees = c.sees(a, w);
                ok = mbar_wait_acc(&n_full[slot], (i / kNSlots) & 1, abort_flag, a.err, nullptr);
                if (sees) ok = ok && mbar_wait_acc(&s_full[w], used & 1, abort_flag, a.err, nullptr);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (sees) {
                    ++used;
                    tc_fence_after();
                    const float* nl = sN + slot * BT;
                    const int i0 = c.row0(a), key = c.kb * kBlock + row, chunks = c.chunks(a);
                    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
                    for (int q = 0; q < chunks; ++q) {
                        uint32_t x[32];
                        tmem_ld32(tS + q * 32, x);
                        add32<true>(acc, x, a.scale_log2, nl + q * 32, see32(key, i0 + q * 32, a.S, a.window, a.n_sink));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[w]);
                    total += sum4(acc);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&n_empty[slot]);
            }
            const int r = c.r, key = c.kb * kBlock + row;
            const bool last_step = c.h == a.G - 1 && c.t == c.last - 1;
            if (!CLUSTER && (last_step || i + 1 == n)) {
                if (last_step && from_start) {
                    if (key < a.S) a.mass[(int64_t)r * a.S + key] = total;
                } else {
                    a.part[(int64_t)(2 * blockIdx.x + from_start) * kBlock + row] = total;
                }
                total = 0.f;
                from_start = true;
            }
            if (i + 1 < n) c.next(a);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
    if constexpr (CLUSTER) {
        // [rank][key] in the first CTA's key tiles, which nothing reads any more
        __syncwarp();
        cluster_sync();
        const int at = threadIdx.x - 128;
        if (at >= 0) st_cluster_f32(map_to_rank(smem_u32(smem) + (uint32_t)(rank * kBlock + at) * 4, 0), total);
        __syncwarp();
        cluster_sync();
        const int key = c.kb * kBlock + at;
        if (rank != 0 || at < 0 || key >= a.S) return;
        float sum = 0.f;
        for (int r = 0; r < kCluster; ++r) sum += reinterpret_cast<const float*>(smem)[r * kBlock + at];
        a.mass[(int64_t)c.r * a.S + key] = sum;
    }
}

// A block per key block: what no query sees is 0, what several CTAs swept is added up.
__global__ void __launch_bounds__(kBlock)
join_kernel(const Args a, int grid) {
    wait_for_previous_kernel();
    const int r = blockIdx.x / a.n_kb, kb = blockIdx.x % a.n_kb, key = kb * kBlock + threadIdx.x;
    int first, last;
    tiles_of(a, kb, first, last);
    float sum = 0.f;
    if (last > first) {
        const int64_t x0 = (r * tiles_before(a, a.n_kb) + tiles_before(a, kb)) * a.G, x1 = x0 + (int64_t)(last - first) * a.G - 1;
        // the CTA that holds step x is the last one whose range begins at or before it
        const int c0 = (int)(((x0 + 1) * grid - 1) / a.steps), c1 = (int)(((x1 + 1) * grid - 1) / a.steps);
        if (c0 == c1) return;                  // written by the CTA itself
        for (int c = c0; c <= c1; ++c) sum += a.part[(int64_t)(2 * c + (c == c0)) * kBlock + threadIdx.x];
    }
    if (key < a.S) a.mass[(int64_t)r * a.S + key] = sum;
}

// ---------------------------------------------------------------- few queries
// An observation window: the last queries of a group's heads, each head's padded to a
// multiple of 32, are at most 512 rows.  They stay in shared memory as the B operand,
// in P groups of 128, and the tiles of 128 keys stream through a ring: every key is
// read once and its mass is finished there, in one launch.  A tile's P products go to
// P of the four TMEM regions, so 4 / P tiles are in work at a time; a warpgroup adds
// up a region, and the P sums of a key meet in shared memory, in their order.
//
// The last 64 queries of 32K tokens, 32/8 heads, D = 128: 19.4 to 20.1 us a call (68.7 MB at 3.4
// to 3.5 TB/s, half of the copy rate; 42 by blocks of 512 keys as above; D = 64 18.7).  A tile of keys takes
// 1770 cycles where HBM would bring one in 1400: as above, the arithmetic of the weights
// (1024 cycles of exponentials).  The 14 tiles of a CTA are 12.5 us of it, 4 us pass
// until the first tile of keys is there.  Measured and not kept: the queries by plain loads
// of the waiting warps, so that the keys are asked for first, 20.0 us; fewer tiles in flight
// at first 19.6; regions handed back at three quarters of the arithmetic 19.8.
constexpr int kMostCols = 512;

template <int D, int P>
struct TailCfg {
    static constexpr int kTileBytes = BT * D * 2;
    static constexpr int kSlots = D == 128 ? 6 - P : 8;
    static constexpr int kOffK = P * kTileBytes;
    static constexpr int kOffN = kOffK + kSlots * kTileBytes;
    static constexpr int kOffPart = kOffN + 2 * P * BT * 4;
    static constexpr int kOffBar = kOffPart + 2 * kTiles * BT * 4;
    static constexpr int kSmem = kOffBar + 512;
    static_assert(kSmem <= 232448, "shared memory");
};

struct TailArgs {
    int H, Hkv, G, S;
    int window, n_sink;
    int q0, pad, cols;     // first query; rows of a head, of a group
    int jt, sink;          // first key tile of the window; 1: tile 0 before it, for the sinks
    int n_tiles;           // tiles of a row (batch, key/value head)
    int rows;
    float scale_log2;
    const float* lse;
    float* mass;
    int* err;
};

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1)
tail_mass_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const TailArgs a) {
    using C = TailCfg<D, P>;
    constexpr int kTeams = kTiles / P;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {            // the swizzled tiles need a 1 KB aligned base
        if (threadIdx.x == 0 && a.err) atomicExch(a.err, 2);
        return;
    }
    uint8_t *sQ = smem, *sK = smem + C::kOffK;
    float* sN = reinterpret_cast<float*>(smem + C::kOffN);                // [2][P * 128]
    float* sPart = reinterpret_cast<float*>(smem + C::kOffPart);          // [team][2][P][128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* q_full = bars + 0;
    uint64_t* q_empty = bars + 1;
    uint64_t* n_full = bars + 2;             // [2]
    uint64_t* n_empty = bars + 4;            // [2]
    uint64_t* s_full = bars + 6;             // [kTiles]
    uint64_t* s_free = bars + 10;            // [kTiles]
    uint64_t* done = bars + 14;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);
    uint64_t* k_full = bars + 20;            // [kSlots]
    uint64_t* k_empty = k_full + C::kSlots;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&n_full[i], 1);
            mbar_init(&n_empty[i], 4 * kTiles);
        }
        for (int w = 0; w < kTiles; ++w) {
            mbar_init(&s_full[w], 1);
            mbar_init(&s_free[w], 4);
        }
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_previous_kernel();
    const uint32_t tmem = *tmem_slot;
    const int64_t steps = (int64_t)a.rows * a.n_tiles, begin = steps * blockIdx.x / gridDim.x, end = steps * (blockIdx.x + 1) / gridDim.x;
    const int n = (int)(end - begin);        // at least one: the grid is no larger than the list
    int r = (int)(begin / a.n_tiles), k = (int)(begin - (int64_t)r * a.n_tiles);
    // The tile's first key; to the next tile: true if it is another row's.
    auto key0 = [&] { return (a.sink ? (k == 0 ? 0 : a.jt + k - 1) : a.jt + k) * BT; };
    auto next = [&] {
        if (++k < a.n_tiles) return false;
        k = 0;
        ++r;
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer of Q and K
        bool ok = true, fresh = true;
        uint32_t row = 0;
        int i = 0;
        for (; i < n && ok; ++i) {
            if (fresh) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(q_empty, (row & 1) ^ 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (uint32_t)(a.cols * D * 2));
                    for (int c = 0; c < a.cols; c += 32)
                        for (int blk = 0; blk < D / 64; ++blk)
                            tma_load_4d(sQ + c / BT * C::kTileBytes + blk * 16384 + c % BT * 128, &tmQ, q_full, blk * 64,
                                        r % a.Hkv * a.G + c / a.pad, a.q0 + c % a.pad, r / a.Hkv);
                }
                __syncwarp();
                ++row;
            }
            const int slot = i % C::kSlots;
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&k_empty[slot], ((i / C::kSlots) & 1) ^ 1, abort_flag, a.err, nullptr));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&k_full[slot], C::kTileBytes);
                for (int blk = 0; blk < D / 64; ++blk)
                    tma_load_4d(sK + slot * C::kTileBytes + blk * 16384, &tmK, &k_full[slot], blk * 64, r % a.Hkv, key0(), r / a.Hkv);
            }
            __syncwarp();
            fresh = i + 1 < n && next();
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            if (row > 0) mbar_wait(q_full, (row - 1) & 1, &dummy, nullptr);
            for (int m = max(i - C::kSlots, 0); m < i; ++m) mbar_wait(&k_full[m % C::kSlots], (m / C::kSlots) & 1, &dummy, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one lane of a converged warp)
        const uint32_t lead = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);      // uniform
        const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
        constexpr uint64_t kStep = C::kTileBytes >> 4;
        bool ok = true, fresh = true;
        uint32_t row = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && mbar_wait_spin(bar, parity, abort_flag, a.err);
            if (ok) tc_fence_after();
            return ok;
        };
        for (int i = 0; i < n && ok; ++i) {
            const int slot = i % C::kSlots, team = i % kTeams;
            if (fresh && !wait(q_full, row++ & 1)) break;
            if (!wait(&k_full[slot], (i / C::kSlots) & 1)) break;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int w = team * P + q;
                if (!wait(&s_free[w], ((i / kTeams) & 1) ^ 1)) break;
                const int cols = min(a.cols - q * BT, BT);
                if (cols > 0) {                  // 257 to 384 columns leave the last group without any
                    const uint32_t id = idesc_bf16_f32(BT, cols, false, false);
                    const uint64_t a0 = dK + slot * kStep, b0 = dQ + q * kStep;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                        mma_ss_lead(lead, tm + w * BT, a0 + off, b0 + off, id, kk > 0);
                    }
                }
                mma_commit_lead(lead, &s_full[w]);
            }
            if (!ok) break;
            mma_commit_lead(lead, &k_empty[slot]);
            fresh = i + 1 < n && next();
            if (fresh) mma_commit_lead(lead, q_empty);
        }
        // Drain: every MMA issued here has finished before TMEM is freed.
        mma_commit_lead(lead, done);
        int dummy = 0;
        mbar_wait(done, 0, &dummy, a.err);
    } else if (warp == 2) {
        // ------------------------------------------------------------ keys that no query sees
        const int from = a.sink * BT, len = a.jt * BT - from;
        const int z0 = (int)((int64_t)len * blockIdx.x / gridDim.x), z1 = (int)((int64_t)len * (blockIdx.x + 1) / gridDim.x);
        for (int y = 0; y < a.rows; ++y)
            for (int z = z0 + lane; z < z1; z += 32) a.mass[(int64_t)y * a.S + from + z] = 0.f;
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ -lse log2 e of the queries, once per row
        const int last = (int)((end - 1) / a.n_tiles);
        for (int row = 0; r <= last; ++r, ++row) {
            if (!__all_sync(0xffffffffu, mbar_wait_acc(&n_empty[row & 1], ((row >> 1) & 1) ^ 1, abort_flag, a.err, nullptr))) break;
            const float* lse = a.lse + ((int64_t)(r / a.Hkv) * a.H + r % a.Hkv * a.G) * a.S;
            float x[P * 4];
#pragma unroll
            for (int e = 0; e < P * 4; ++e) {
                const int c = e * 32 + lane, h = e * 32 / a.pad, i = a.q0 + c - h * a.pad;   // 32 columns are one head's
                const float l = c < a.cols && i < a.S ? lse[(int64_t)h * a.S + i] : -INFINITY;
                x[e] = l == -INFINITY ? l : -l * kLog2e;      // no such query, or one that sees nothing
            }
#pragma unroll
            for (int e = 0; e < P * 4; ++e) sN[(row & 1) * P * BT + e * 32 + lane] = x[e];
            __syncwarp();
            if (lane == 0) mbar_arrive(&n_full[row & 1]);
        }
    } else {
        // ------------------------------------------------------------ weights: a warpgroup per region, a thread per key
        const int w = (warp - 4) / 4, team = w / P, q = w % P, row = (warp % 4) * 32 + lane;
        const uint32_t tS = tmem + ((uint32_t)((warp % 4) * 32) << 16) + w * BT;
        const int chunks = max(min(a.cols - q * BT, BT), 0) / 32, per = a.pad / 32;     // of 32 columns: here, per head
        float* part = sPart + team * 2 * P * BT;
        bool ok = true, fresh = true;
        int seen_rows = 0;
        uint32_t used = 0;
        for (int i = 0; i < n; ++i) {
            // A warp whose wait gave up still comes to its team's next barrier: the others may be waiting there.
            if (fresh) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_acc(&n_full[seen_rows & 1], (seen_rows >> 1) & 1, abort_flag, a.err, nullptr));
                ++seen_rows;
            }
            if (i % kTeams == team) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_acc(&s_full[w], used & 1, abort_flag, a.err, nullptr));
                float sum = 0.f;
                const int k0 = key0(), key = k0 + row;
                if (ok) {
                    tc_fence_after();
                    const float* nl = sN + ((seen_rows - 1) & 1) * P * BT + q * BT;
                    uint64_t acc[4] = {0, 0, 0, 0};
                    const bool whole = k0 + BT - 1 <= a.q0 && a.S - 1 - k0 < a.window;      // every query sees all keys
                    if (whole && chunks == 4 && a.q0 + a.pad == a.S) {
                        add128(acc, tS, a.scale_log2, nl);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < chunks; ++c) {
                            const int i0 = a.q0 + (q * 4 + c) % per * 32;
                            uint32_t x[32];
                            tmem_ld32(tS + c * 32, x);
                            if (whole && i0 + 32 <= a.S) add32(acc, x, a.scale_log2, nl + c * 32);
                            else add32<true>(acc, x, a.scale_log2, nl + c * 32, see32(key, i0, a.S, a.window, a.n_sink));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[w]);
                    sum = sum4(acc);
                }
                if constexpr (P > 1) {
                    // the parts of two tiles in turn: a buffer is written again only behind the barrier that comes
                    // after it was read
                    float* buf = part + (used & 1) * P * BT;
                    if (q > 0) buf[q * BT + row] = sum;
                    ok = named_bar_and(1 + team, P * BT, ok);
                    if (q == 0)
#pragma unroll
                        for (int z = 1; z < P; ++z) sum += buf[z * BT + row];
                }
                if (!ok) break;
                if (q == 0 && key < a.S) a.mass[(int64_t)r * a.S + key] = sum;
                ++used;
            }
            fresh = i + 1 < n && next();
            if (fresh || i + 1 == n) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&n_empty[(seen_rows - 1) & 1]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D, int P>
dfa_status launch_tail(const SinkProblem& p, const TailArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, cudaStream_t s) {
    static std::atomic<uint64_t> seen{0};
    auto kernel = tail_mass_kernel<D, P>;
    constexpr int smem = TailCfg<D, P>::kSmem;
    if (first_on_device(seen)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "key_mass: kernel attributes");
        mark_on_device(seen);
    }
    const cudaError_t e = launch_overlapped(kernel, dim3((unsigned)std::min<int64_t>(num_sms(), (int64_t)a.rows * a.n_tiles)), kThreads, smem, s, mq, mk, a);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "key_mass launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_MASS);
    return DFA_OK;
}

template <int D>
dfa_status launch_tail(const SinkProblem& p, int n_last, const void* q, const void* k, const float* lse, float* mass, cudaStream_t s) {
    CUtensorMap mq, mk;
    if (!make_tmap_bshd(&mq, q, p.B, p.S, p.H, D, (int64_t)p.S * p.H * D, (int64_t)p.H * D, D, 32) ||
        !make_tmap_bshd(&mk, k, p.B, p.S, p.Hkv, D, (int64_t)p.S * p.Hkv * D, (int64_t)p.Hkv * D, D))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    TailArgs a{};
    a.H = p.H; a.Hkv = p.Hkv; a.G = p.H / p.Hkv; a.S = p.S;
    a.window = p.window; a.n_sink = p.n_sink;
    a.q0 = p.S - n_last;
    a.pad = (n_last + 31) / 32 * 32;
    a.cols = a.G * a.pad;
    a.jt = std::max(a.q0 - p.window + 1, 0) / BT;
    a.sink = p.n_sink > 0 && a.jt > 0;
    a.n_tiles = (p.S + BT - 1) / BT - a.jt + a.sink;
    a.rows = p.B * p.Hkv;
    a.scale_log2 = p.scale * kLog2e;
    a.lse = lse; a.mass = mass;
    a.err = device_error_flag();
    if (a.cols <= BT) return launch_tail<D, 1>(p, a, mq, mk, s);
    if (a.cols <= 2 * BT) return launch_tail<D, 2>(p, a, mq, mk, s);
    return launch_tail<D, 4>(p, a, mq, mk, s);
}

template <int D>
dfa_status launch(const SinkProblem& p, int n_last, const void* q, const void* k, const float* lse, float* mass, void* ws,
                  cudaStream_t s) {
    CUtensorMap mq, mk;
    if (!make_tmap_bshd(&mq, q, p.B, p.S, p.H, D, (int64_t)p.S * p.H * D, (int64_t)p.H * D, D) ||
        !make_tmap_bshd(&mk, k, p.B, p.S, p.Hkv, D, (int64_t)p.S * p.Hkv * D, (int64_t)p.Hkv * D, D))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    Args a{};
    a.H = p.H; a.Hkv = p.Hkv; a.G = p.H / p.Hkv; a.S = p.S;
    a.window = p.window; a.n_sink = p.n_sink;
    a.q0 = p.S - n_last;
    a.n_qt = (n_last + BT - 1) / BT;
    a.n_kb = (p.S + kBlock - 1) / kBlock;
    a.c0 = (a.q0 + BT - 1) / BT;
    // the last tile that sees key 512 kb + 511: the last t with q0 + 128 t <= that + window - 1
    const int64_t x = (int64_t)kBlock - 2 + p.window - a.q0;
    a.e1 = (int)(x >= 0 ? x / BT : -((-x + BT - 1) / BT)) + 1;
    a.steps = (int64_t)p.B * p.Hkv * tiles_before(a, a.n_kb) * a.G;
    a.scale_log2 = p.scale * kLog2e;
    a.lse = lse; a.mass = mass;
    a.part = static_cast<float*>(ws);
    a.err = device_error_flag();
    static std::atomic<uint64_t> seen{0};
    static std::atomic<int> clusters{0};             // that run at a time
    auto kernel = key_mass_kernel<D, false>;
    auto clustered = key_mass_kernel<D, true>;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)kCluster);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (first_on_device(seen)) {
        int k = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(clustered, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&k, clustered, &cfg) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "key_mass: kernel attributes");
        clusters.store(k);
        mark_on_device(seen);
    }
    // One round of clusters, if the longest of their shares is not longer than an equal share of all SMs and the second
    // launch (kJoinSteps).  GPU time by clusters and by all SMs: 2 x 301 tokens, 8/4 heads, 6.0 and 7.7 us (D = 64 5.5 and
    // 7.3); 700 tokens, 8/8 heads, 8.9 both; 1000 tokens, 8/2 heads, the longest shares that the rule lets through, 11.3
    // and 10.3; 2000 tokens, left to all SMs, 16.9 and 14.0.
    const int64_t segments = (int64_t)p.B * p.Hkv * a.n_kb;
    int64_t longest = 0;
    if (segments <= clusters.load())
        for (int kb = 0; kb < a.n_kb; ++kb) longest = std::max(longest, (tiles_before(a, kb + 1) - tiles_before(a, kb)) * a.G);
    if (segments <= clusters.load() && (longest + kCluster - 1) / kCluster <= (a.steps + num_sms() - 1) / num_sms() + kJoinSteps) {
        cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * a.n_kb * kCluster));
        cfg.numAttrs = 2;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, clustered, mq, mk, a);
        if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "key_mass launch: %s", cudaGetErrorString(e));
        count_launch(DFA_KERNEL_MASS);
        return DFA_OK;
    }
    const int grid = (int)std::min<int64_t>(num_sms(), a.steps);
    cudaError_t e = launch_overlapped(kernel, dim3((unsigned)grid), kThreads, Cfg<D>::kSmem, s, mq, mk, a);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "key_mass launch: %s", cudaGetErrorString(e));
    e = launch_overlapped(join_kernel, dim3((unsigned)(p.B * p.Hkv * a.n_kb)), kBlock, 0, s, a, grid);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "key_mass join launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_MASS, 2);
    return DFA_OK;
}

}  // namespace

size_t key_mass_workspace() { return sizeof(float) * 2 * (size_t)num_sms() * kBlock; }

dfa_status tc_key_mass(const SinkProblem& p, int n_last, const void* q, const void* k, const float* lse, float* mass, void* ws,
                       cudaStream_t s) {
    if ((int64_t)(p.H / p.Hkv) * ((n_last + 31) / 32 * 32) <= kMostCols)
        return p.D == 128 ? launch_tail<128>(p, n_last, q, k, lse, mass, s) : launch_tail<64>(p, n_last, q, k, lse, mass, s);
    return p.D == 128 ? launch<128>(p, n_last, q, k, lse, mass, ws, s) : launch<64>(p, n_last, q, k, lse, mass, ws, s);
}

}  // namespace dfa
