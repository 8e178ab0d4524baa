// sink_fwd_tc.cu -- tcgen05 forward of causal attention with a sliding window
// of tokens and a few first tokens that stay visible (sinks), for sm_103a.
//
// Row i sees key j iff j <= i and (j > i - W or j < N):
//   s_ij = scale <q_i, k_j>,  lse_i = ln sum_j exp(s_ij),  O_i = sum_j exp(s_ij - lse_i) v_j.
// One pass over the visible keys with a running maximum, running sum and
// unnormalised output per row (the online-normalizer rule DISTFLASHATTN §3.2
// merges chunk partials with), fp32 throughout; the probabilities are rounded
// to bf16 as the tensor cores' A operand, the row sum adds them unrounded.
//
// Layout of the work.  A CTA owns a block of 256 query rows of one head, two
// 128-row tiles that ping-pong: while one warpgroup runs its tile's softmax
// the tensor cores run the other tile's MMAs (as fwd_tc.cu).  What differs is
// the list of key tiles: the sink tile first, when the window has moved off
// it, then the band.  Each of the two query tiles takes part only in the key
// tiles it can see -- the first skips the band's last tile, the second its
// first -- so a window of a multiple of 128 tokens costs each query tile
// W / 128 + 1 tiles, not W / 128 + 2.  The sink tile's MMAs are as wide as the
// sinks, rounded up to 16 columns: N = 4 costs an eighth of a tile.
//
// What bounds it.  A query tile's steps form a chain: S (550 cycles at D = 128),
// the softmax of its row (1350), barriers (500), P V (550, of which three quarters
// run under the softmax).  The two chains of a CTA overlap, and the tensor cores
// work for 2200 of a step's 2550 cycles.  The softmax is bound by latency (two
// warps on a sub-partition; issue slots 41% busy, MUFU 33%): exponentials moved to
// the FMA pipe made it slower, fewer instructions and loads under arithmetic
// faster; two threads a row (four softmax warpgroups, maxima exchanged) took 1724 us
// for 1312: too few registers, and five warps beside the issuing one.  A block's
// ends -- masked tiles, the sink tile's step, the epilogue -- cost another 4 us of
// chain, so the lists of a CTA's blocks run on into one another (issuer),
// 32-column pieces of a masked tile that no row sees are skipped (Mask), and the
// output leaves in 64-byte pieces.  Measured back to back (the same
// tensors each time; 1424 us where they change from call to call), 32K tokens, 32 heads of
// 8 kv heads, 4 sinks: window 4096 1320 us (D = 128; 1560 TFLOP/s, 82% of the cuBLAS
// rate), window 1024 499; D = 64 1160 and 443; without sinks, window 128 175 and
// window 1 105 (D = 128; 100 at the memory's rate).
//
// Schedule.  No work list: costs never fall from a block to the next one of
// its head, so the blocks in the order last to first of all heads are sorted
// by cost, and dealing them to the persistent CTAs in a snake (0..n-1, then
// n-1..0, ...) balances them to within one block.  Nothing is uploaded and
// there is no workspace, so a call is one launch and can be captured.  With few
// blocks a block would leave most SMs without work: then the blocks, or those
// behind the last full round, are shared by clusters of two or four CTAs, each
// with a piece of the key list, and joined through distributed shared memory
// (make_plan weighs the shorter lists against the join: 1500 tokens of 8 heads,
// D = 128, causal: 21.5 us, whole blocks 24.2; 4000 tokens 44 and 55; 16000 tokens
// of one head 71 and 193; 700 tokens of 4 heads stay whole, 14.9 and 16.9).
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer of K and V, warp 1 MMA
// issuer (one lane issues), warp 2 TMEM owner, warp 3 TMA producer of Q, warps 4-11
// two softmax warpgroups, one query row per thread.  TMEM columns: S_0 [0,128)
// S_1 [128,256) O_0 [256,256+D) O_1 [384,384+D); P_w (bf16 pairs) overwrites the
// first 64 columns of S_w.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "softmax_tc.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int BM = 128;            // query rows per tile (MMA M)
constexpr int BN = 128;            // key rows per tile
constexpr int kBlockRows = 2 * BM;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMost = 6;           // steps of 16 keys in the first part of P that is handed over
constexpr float kRescaleThreshold = 8.0f;   // log2 units: rescale O only when the max grows by > 2^8

template <int D>
struct Cfg {
    static constexpr int kTileBytes = BN * D * 2;
    static constexpr int kSlots = 4;                           // K/V ring depth (6 and 8 gain nothing at D = 64)
    static constexpr bool kTwice = D == 128;                   // P is handed over in two parts (rule at p_most)
    static constexpr int kQBytes = 2 * kTileBytes;
    static constexpr int kSmem = kQBytes + kSlots * kTileBytes + 1024 /*barriers*/ + 1024 /*align*/;
};

// n / d for 0 <= n < 2^31 by a multiplication: with 2^(l-1) < d <= 2^l and
// m = floor(2^(31 + l) / d) + 1, m d exceeds 2^(31 + l) by at most d <= 2^l, so
// n m / 2^(31 + l) exceeds n / d by less than 1 / d (Granlund and Montgomery 1994).
// A block's start divides five times; the divisions took 1700 cycles of it.
struct Divider {
    uint32_t d, m, shift;
    Divider(int x = 1) : d((uint32_t)x), shift(31) {
        while ((uint64_t{1} << (shift - 31)) < d) ++shift;
        m = (uint32_t)((uint64_t{1} << shift) / d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return (int)((uint64_t)(uint32_t)n * m >> shift); }
};

struct Args {
    Divider rows;          // B * H
    Divider H, G;          // G = H / H_kv
    int S;
    int window, n_sink;    // window <= S; n_sink <= 128, 0 when the window covers every key
    int n_units, n_items;  // 256-row blocks per head; rows * n_units
    int n_whole, log_p;    // SPLIT: the first n_whole blocks are whole CTAs', the others of clusters of 2^log_p
    float scale_log2;      // scale * log2(e)
    __nv_bfloat16* O;      // [B, S, H, D]
    float* lse;            // [B, H, S]
    int* err;
};

// A block's list of key tiles: the sink tile, when the window has moved off it, then the band.
struct Block {
    int b, h, g, q0;
    int j0;                // first key tile of the band
    int n;                 // key tiles in the list
    int lead;              // 1: the list starts with tile 0 as a sink tile
    int from;              // n tiles from here on are this CTA's piece of a split block's list
    bool split;
    // k-th key tile of the list
    __device__ __forceinline__ int tile(int k) const { return lead && k + from == 0 ? 0 : j0 + k + from - lead; }
};

__device__ __forceinline__ Block decode(const Args& a, int it) {
    Block x;
    const int u = a.rows.div(it), row = it - u * (int)a.rows.d, unit = a.n_units - 1 - u;
    x.b = a.H.div(row);
    x.h = row - x.b * (int)a.H.d;
    x.g = a.G.div(x.h);
    x.q0 = unit * kBlockRows;
    x.j0 = max(x.q0 - a.window + 1, 0) / BN;
    const bool two = x.q0 + BM < a.S;                     // the second query tile has rows
    x.lead = a.n_sink > 0 && x.j0 > 0;
    x.n = x.lead + (x.q0 / BN + two - x.j0 + 1);
    x.from = 0;
    x.split = false;
    return x;
}

// A CTA's blocks in order: first whole ones, then (SPLIT) its pieces of the
// blocks that its cluster shares, which may be empty.
template <bool SPLIT>
struct Deal {
    const Args& a;
    int n_whole, rank, cluster, n_clusters, rounds;
    __device__ __forceinline__ explicit Deal(const Args& args) : a(args), rank(0), cluster(0), n_clusters(0) {
        rounds = n_whole = snake_count(SPLIT ? a.n_whole : a.n_items, blockIdx.x, gridDim.x);
        if (SPLIT) {
            rank = blockIdx.x & ((1 << a.log_p) - 1);
            cluster = blockIdx.x >> a.log_p;
            n_clusters = gridDim.x >> a.log_p;
            rounds += snake_count(a.n_items - a.n_whole, cluster, n_clusters);
        }
    }
    __device__ __forceinline__ Block operator()(int i) const {
        if (!SPLIT || i < n_whole) return decode(a, snake_item(i, blockIdx.x, gridDim.x));
        Block x = decode(a, a.n_whole + snake_item(i - n_whole, cluster, n_clusters));
        x.from = x.n * rank >> a.log_p;
        x.n = (x.n * (rank + 1) >> a.log_p) - x.from;
        x.split = true;
        return x;
    }
};

// How a block's query tile takes part in its list: in the band's positions
// [b0, b1], none if b1 < b0, and in the first one's sink columns if its own band
// starts behind that tile.
struct Run {
    int b0, b1;
    int sink;              // 0, or -1: no sink tile
    int piece_last;        // split blocks: the last position that it takes part in, -1: none
    template <bool SPLIT>
    __device__ __forceinline__ int last() const { return SPLIT ? piece_last : b1; }
    // 0 not at all, 1 the sink columns only, 2 the whole tile.
    __device__ __forceinline__ int part(int k) const { return k == sink ? 1 : (k >= b0 && k <= b1) ? 2 : 0; }
};
template <bool SPLIT>
__device__ __forceinline__ Run run(const Args& a, const Block& x, int w) {
    const int f = x.q0 + w * BM;
    if (f >= a.S) return Run{0, -1, -1, -1};              // no rows
    const int lo = max(f - a.window + 1, 0) / BN, at = x.lead - x.j0;
    Run u{lo + at, f / BN + at, a.n_sink > 0 && lo > 0 ? 0 : -1, f / BN + at};
    if (SPLIT && x.split) {
        u.b0 = max(u.b0 - x.from, 0);
        u.b1 = min(u.b1 - x.from, x.n - 1);
        if (x.from > 0 || x.n == 0) u.sink = -1;
        u.piece_last = u.b1 >= u.b0 ? u.b1 : u.sink;
    }
    return u;
}

// A softmax thread's part in joining a split block: row `row` of 256, whose
// unnormalised output over this CTA's piece is in TMEM at tO (if `some`), with
// reference maximum m and sum l.  o: the row's output, null if it is past the
// end.  Out of line, so that its registers are not the softmax loop's.
template <int D>
__device__ __noinline__ bool join(int log_p, int rank, uint32_t phase, int row, int lane, bool some, float m, float l,
                                  uint32_t tO, uint8_t* buf, uint64_t* ready, uint64_t* landed,
                                  volatile int* abort_flag, int* err, __nv_bfloat16* o, float* lse) {
    const int P = 1 << log_p, per_log = (D == 128 ? 5 : 4) - log_p, per = 1 << per_log;   // 16-byte groups per CTA
    const uint32_t ring = smem_u32(buf), slot = per * 4096;
    if (lane == 0)
        for (int d = 0; d < P; ++d)
            if (d != rank) cluster_arrive(smem_u32(ready), d);
    if (!__all_sync(0xffffffffu, mbar_wait_acc(ready, phase, abort_flag, err, nullptr))) return false;
    fence_cluster();
    // [sender][group][row] in the ring of the CTA that finishes the group
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
        const int at = c * 4, d = at >> per_log;
        if (d == rank) continue;
        uint32_t u[16];
        if (some) {
            tmem_ld16_async(tO + c * 16, u);
            tmem_wait_ld16(u);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = 0;
        }
        const uint32_t dst = map_to_rank(ring + rank * slot + ((at & (per - 1)) * 256 + row) * 16, d);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            st_cluster_v4(dst + e * 4096, make_float4(__uint_as_float(u[4 * e]), __uint_as_float(u[4 * e + 1]),
                                                      __uint_as_float(u[4 * e + 2]), __uint_as_float(u[4 * e + 3])));
    }
    // maxima and sums: in the slot that the receiver's own output does not need
    for (int d = 0; d < P; ++d)
        if (d != rank) st_cluster_v2(map_to_rank(ring + d * slot + (rank * 256 + row) * 8, d), make_float2(m, l));
    __syncwarp();
    if (lane == 0)
        for (int d = 0; d < P; ++d)
            if (d != rank) cluster_arrive(smem_u32(landed), d);
    if (!__all_sync(0xffffffffu, mbar_wait_acc(landed, phase, abort_flag, err, nullptr))) return false;
    fence_cluster();
    const float2* stat = reinterpret_cast<const float2*>(buf + rank * slot) + row;
    float top = m, sum = 0.f;
    for (int d = 0; d < P; ++d)
        if (d != rank) top = fmaxf(top, stat[d * 256].x);
    for (int d = 0; d < P; ++d) {
        const float2 z = d == rank ? make_float2(m, l) : stat[d * 256];
        sum += ex2(z.x - top) * z.y;                  // no visible key in the piece: 0 * 0
    }
    const float inv = 1.f / sum;
#pragma unroll 1
    for (int g = 0; g < per; g += 4) {
        float acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        for (int d = 0; d < P; ++d) {
            if (d == rank) {
                if (!some) continue;
                const float f = ex2(m - top) * inv;
                uint32_t u[16];
                tmem_ld16_async(tO + (rank * per + g) * 4, u);
                tmem_wait_ld16(u);
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[e] = fmaf(f, __uint_as_float(u[e]), acc[e]);
            } else {
                const float f = ex2(stat[d * 256].x - top) * inv;
                const float4* src = reinterpret_cast<const float4*>(buf + d * slot) + g * 256 + row;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 v = src[e * 256];
                    acc[4 * e + 0] = fmaf(f, v.x, acc[4 * e + 0]);
                    acc[4 * e + 1] = fmaf(f, v.y, acc[4 * e + 1]);
                    acc[4 * e + 2] = fmaf(f, v.z, acc[4 * e + 2]);
                    acc[4 * e + 3] = fmaf(f, v.w, acc[4 * e + 3]);
                }
            }
        }
        if (o) {
            uint4* dst = reinterpret_cast<uint4*>(o + (rank * per + g) * 4);
            dst[0] = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                                pack_bf16(acc[6], acc[7]));
            dst[1] = make_uint4(pack_bf16(acc[8], acc[9]), pack_bf16(acc[10], acc[11]), pack_bf16(acc[12], acc[13]),
                                pack_bf16(acc[14], acc[15]));
        }
    }
    tc_fence_before();
    if (o && rank == 0) *lse = (top + __log2f(sum)) * kLn2;
    return true;
}

// SPLIT: launched in clusters of 2^log_p CTAs.  For the last blocks each CTA of a
// cluster takes a piece of the block's key list; then every CTA sends the others
// its unnormalised output (the columns that they finish), maxima and sums through
// distributed shared memory, into the ring that the pieces' tiles have left, and
// finishes D / 2^log_p columns of the 256 rows, pieces in the order of the keys.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
sink_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Args a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;                                   // 2 tiles
    uint8_t* sKV = smem + C::kQBytes;                     // ring: K and V tiles alternate
    uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + C::kSlots * C::kTileBytes);
    uint64_t* q_full = bars + 0;          // [2], as all of these one per query tile
    uint64_t* q_empty = bars + 2;
    uint64_t* s_full = bars + 4;
    // The first 96 columns of P: the product with V starts on them while the softmax works on
    // the others (32K tokens, D = 128, window 4096 1320 us, 1342 without; 5003 tokens, window
    // 1000 82.7 and 84.7; with 64 columns 1300 and 84.5).  At D = 64 the product is half as
    // long and the second wait costs more than it gives: 1204 us, 1160 without.
    uint64_t* p_most = bars + 8;
    uint64_t* p_full = bars + 10;
    uint64_t* o_full = bars + 12;
    uint64_t* done = bars + 14;
    // SPLIT: the other CTAs' rings may be written; what they sent is here; it has been used
    uint64_t* ready = bars + 34;
    uint64_t* landed = bars + 35;
    uint64_t* merged = bars + 36;
    uint64_t* kv_full = bars + 16;        // [kSlots]
    uint64_t* kv_empty = bars + 16 + C::kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 33);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Deal<SPLIT> deal(a);
    const int rounds = deal.rounds, P = SPLIT ? 1 << a.log_p : 1;

    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            mbar_init(&q_full[w], 1);
            mbar_init(&q_empty[w], 1);
            mbar_init(&s_full[w], 1);
            mbar_init(&p_most[w], 4);
            mbar_init(&p_full[w], 4);
            mbar_init(&o_full[w], 1);
        }
        mbar_init(done, 1);
        if (SPLIT) {
            mbar_init(ready, (P - 1) * 8);
            mbar_init(landed, (P - 1) * 8);
            mbar_init(merged, 8);
        }
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_sync();      // every CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer of K and V
        uint32_t ld = 0;
        bool ok = true;
        for (int r = 0; r < rounds && ok; ++r) {
            const Block x = deal(r);
            // the ring carries the outputs of a split block until they are joined
            if (SPLIT && r > deal.n_whole) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(merged, (r - deal.n_whole - 1) & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
            }
            for (int k = 0; k < x.n && ok; ++k) {
                const int j = x.tile(k);
                for (int which = 0; which < 2; ++which, ++ld) {
                    const int slot = ld % C::kSlots;
                    ok = __all_sync(0xffffffffu, mbar_wait_acc(&kv_empty[slot], ((ld / C::kSlots) & 1) ^ 1, abort_flag,
                                                               a.err, nullptr));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&kv_full[slot], C::kTileBytes);
                        for (int blk = 0; blk < D / 64; ++blk)
                            tma_load_4d(sKV + slot * C::kTileBytes + blk * 16384, which ? &tmV : &tmK, &kv_full[slot],
                                        blk * 64, x.g, j * BN, x.b);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            for (uint32_t s = 0; s < (uint32_t)C::kSlots && s < ld; ++s) {
                const uint32_t last = s + C::kSlots * ((ld - 1 - s) / C::kSlots);
                mbar_wait(&kv_full[s], (last / C::kSlots) & 1, &dummy, nullptr);
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ TMA producer of Q: a warp of its own, for
        // the other one would not load the next block's first keys before a query tile's buffer is free
        uint32_t qi = 0;
        bool ok = true;
        for (int r = 0; r < rounds && ok; ++r) {
            const Block x = deal(r);
            if (SPLIT && x.n == 0) continue;
            for (int w = 0; w < 2 && ok; ++w) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&q_empty[w], ((qi >> 1) & 1) ^ 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                ++qi;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[w], C::kTileBytes);
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_4d(sQ + w * C::kTileBytes + blk * 16384, &tmQ, &q_full[w], blk * 64, x.h, x.q0 + w * BM,
                                    x.b);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            int dummy = 0;
            for (uint32_t m = qi > 1 ? qi - 2 : 0; m < qi; ++m) mbar_wait(&q_full[m & 1], (m >> 1) & 1, &dummy, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one lane of a converged warp)
        const uint32_t lead = elect_one();
        const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);   // uniform
        const uint32_t idS = idesc_bf16_f32(BM, BN, false, false);
        const uint32_t idO = idesc_bf16_f32(BM, D, false, true);
        const int ns16 = (a.n_sink + 15) / 16;                              // sink columns / 16
        const uint32_t idSink = idesc_bf16_f32(BM, 16 * ns16, false, false);
        const uint64_t dQk = sdesc_sw128(smem_u32(sQ), 16, 1024);          // Q, K-major
        const uint64_t dKk = sdesc_sw128(smem_u32(sKV), 16, 1024);         // K slots, K-major
        const uint64_t dVn = sdesc_sw128(smem_u32(sKV), 16384, 1024);      // V slots, N-major
        constexpr uint64_t kSlotStep = C::kTileBytes >> 4;
        uint32_t cons = 0, t[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && mbar_wait_issuer(bar, parity, abort_flag, a.err);
            if (ok) tc_fence_after();
            return ok;
        };
        auto issue_S = [&](int w, uint32_t slot, uint32_t id) {
            const uint64_t a0 = dQk + w * kSlotStep, b0 = dKk + slot * kSlotStep;
            const uint32_t d = tmem + w * 128;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                mma_ss_lead(lead, d, a0 + off, b0 + off, id, kk > 0);
            }
            mma_commit_lead(lead, &s_full[w]);
        };
        // O_w += P_w V, most of the keys as soon as their P is there
        auto issue_PV = [&](int w, uint32_t slot, uint32_t par, uint32_t acc) {
            const uint64_t b0 = dVn + slot * kSlotStep;
            const uint32_t d = tmem + 256 + w * 128, p = tmem + w * 128;
            if (!wait(C::kTwice ? &p_most[w] : &p_full[w], par)) return;
            mma_ts_lead(lead, d, p, b0, idO, acc);
#pragma unroll
            for (int kk = 1; kk < kMost; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, 1u);
            if (C::kTwice && !wait(&p_full[w], par)) return;
#pragma unroll
            for (int kk = kMost; kk < BN / 16; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, 1u);
        };
        auto issue_PV_sink = [&](int w, uint32_t slot, uint32_t par, uint32_t acc) {
            const uint64_t b0 = dVn + slot * kSlotStep;
            const uint32_t d = tmem + 256 + w * 128, p = tmem + w * 128;
            if ((C::kTwice && !wait(&p_most[w], par)) || !wait(&p_full[w], par)) return;
#pragma unroll 1
            for (int kk = 0; kk < ns16; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, kk > 0 ? 1u : acc);
        };
        // The blocks' lists run on into one another: at a block's last key tile the next block's
        // first S is issued where its next S would be, so that neither warpgroup waits for the
        // other one's end or for its own epilogue.  Block -1 is empty.
        uint32_t now[2] = {0, 0}, first[2] = {1, 1};
        Block x{}, y{};
        Run u0{0, -1, -1, -1}, u1 = u0, v0 = u0, v1 = u0;
        int k = -1, r = -1, dealt = 0;
        // y: the next block that has key tiles
        auto fetch = [&]() {
            while (dealt < rounds) {
                y = deal(dealt++);
                if (SPLIT && y.n == 0) continue;
                v0 = run<SPLIT>(a, y, 0);
                v1 = run<SPLIT>(a, y, 1);
                return true;
            }
            return false;
        };
        bool have_y = fetch();
        for (;;) {
            // Steps in which both query tiles take both key tiles whole run without looking at the bands.
            const int hot = u0.b1;
            if (now[0] == 2 && now[1] == 2 && k < hot) {
                uint32_t a0 = 1u - first[0], a1 = 1u - first[1];
                first[0] = first[1] = 0;
                for (; k < hot; ++k) {
                    const uint32_t slotV = cons % C::kSlots;
                    if (!wait(&kv_full[slotV], (cons / C::kSlots) & 1)) break;
                    issue_PV(0, slotV, t[0]++ & 1, a0);
                    if (!ok) break;
                    const uint32_t slotK = (cons + 1) % C::kSlots;
                    if (!wait(&kv_full[slotK], ((cons + 1) / C::kSlots) & 1)) break;
                    issue_S(0, slotK, idS);
                    issue_PV(1, slotV, t[1]++ & 1, a1);
                    if (!ok) break;
                    mma_commit_lead(lead, &kv_empty[slotV]);
                    issue_S(1, slotK, idS);
                    mma_commit_lead(lead, &kv_empty[slotK]);
                    cons += 2;
                    a0 = a1 = 1u;
                }
                if (!ok) break;
                // The first query tile's last product is issued; the second one's band goes one tile
                // further, unless a piece ends here.
                mma_commit_lead(lead, &q_empty[0]);
                if (SPLIT && u1.piece_last == hot) mma_commit_lead(lead, &q_empty[1]);
            }
            const bool end = k + 1 == x.n, more = !end || (SPLIT ? have_y : r + 1 < rounds);
            const int kn = end ? 0 : k + 1, rn = end ? r + 1 : r;
            const uint32_t slotV = cons % C::kSlots;
            if (k >= 0) {
                if (!wait(&kv_full[slotV], (cons / C::kSlots) & 1)) break;
                ++cons;
            }
            const uint32_t slotK = cons % C::kSlots;
            bool have_k = false;
            // a query tile that skips this key tile goes first: it does not wait for the other one
            const int swap = now[1] == 0 && now[0] != 0;
            // The ring takes the next piece's keys only behind the join of the split block before it,
            // which waits for this block's products: those first.
            const bool apart = SPLIT && end && have_y && dealt - 1 > deal.n_whole;
#pragma unroll 1
            for (int i = 0; i < (apart ? 4 : 2); ++i) {
                const int w = (i & 1) ^ swap;
                if (i < 2 && (w ? now[1] : now[0])) {
                    const uint32_t acc = 1u - (w ? first[1] : first[0]), par = (w ? t[1] : t[0]) & 1;
                    if ((w ? now[1] : now[0]) == 2) issue_PV(w, slotV, par, acc);
                    else issue_PV_sink(w, slotV, par, acc);
                    if (!ok) break;
                    if (w) ++t[1];
                    else ++t[0];
                    if (w) first[1] = 0;
                    else first[0] = 0;
                    if (k == (w ? u1 : u0).template last<SPLIT>()) mma_commit_lead(lead, &o_full[w]);
                }
                if (i == 1 && k >= 0) mma_commit_lead(lead, &kv_empty[slotV]);
                if (!more || (apart && i < 2)) continue;
                // S of the next key tile
                const Run u = end ? (w ? v1 : v0) : (w ? u1 : u0);
                if (kn == 0 && !wait(&q_full[w], rn & 1)) break;
                const int part = u.part(kn);
                if (part) {
                    if (!have_k && !wait(&kv_full[slotK], (cons / C::kSlots) & 1)) break;
                    have_k = true;
                    issue_S(w, slotK, part == 1 ? idSink : idS);
                }
                if (w) now[1] = part;
                else now[0] = part;
                // behind the query tile's last product its buffer is free for the next block's
                if (kn == max(u.template last<SPLIT>(), 0)) mma_commit_lead(lead, &q_empty[w]);
            }
            if (!ok || !more) break;
            mma_commit_lead(lead, &kv_empty[slotK]);
            ++cons;
            k = kn;
            if (end) {
                r = rn;
                x = y;
                u0 = v0;
                u1 = v1;
                first[0] = first[1] = 1;
                have_y = fetch();
            }
        }
        // Drain: every MMA issued here has finished before TMEM is freed.
        mma_commit_lead(lead, done);
        int dummy = 0;
        mbar_wait(done, 0, &dummy, a.err);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax warpgroups
        const int w = (warp - 4) / 4;                 // which query tile
        const int r = (warp % 4) * 32 + lane;         // row within the tile == TMEM lane
        const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tmem + lane_base + w * 128;
        const uint32_t tO = tmem + lane_base + 256 + w * 128;
        const float c2 = a.scale_log2;
        uint32_t t = 0, qi = 0;
        bool ok = true;
        Block x = deal(0), y = x;
        for (int rd = 0; rd < rounds && ok; ++rd, x = y) {
            const int f = x.q0 + w * BM, row = f + r;
            const Run u = run<SPLIT>(a, x, w);
            if (u.template last<SPLIT>() < 0 && !(SPLIT && x.split)) {             // no row of the sequence in this tile
                if (rd + 1 < rounds) y = deal(rd + 1);
                continue;
            }
            const int row0 = __shfl_sync(0xffffffffu, row, 0);
            const int lo_row = row - a.window + 1, lo_last = f + BM - a.window;   // lowest visible keys
            float m_run = -INFINITY, l = 0.f;
            bool started = false;
            for (int k = 0; k < x.n; ++k) {
                const int j = x.tile(k), part = u.part(k);
                if (!part) continue;
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&s_full[w], t & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                ++t;
                tc_fence_after();
                const int kv0 = j * BN;
                Mask mk{0, BN, 0, 0, BN, 0};
                int chunks = BN / 32;
                bool masked = true;
                if (part == 1) {
                    mk.lim = mk.lim0 = a.n_sink;
                    chunks = (a.n_sink + 31) / 32;
                } else {
                    masked = kv0 + BN > f || kv0 < lo_last;   // the diagonal tile (and the ragged end) or the window's edge
                    if (masked) {
                        mk.lo = lo_row - kv0;
                        mk.lim = row - kv0 + 1;
                        mk.lo0 = row0 - a.window + 1 - kv0;
                        mk.lim0 = row0 + 1 - kv0;
                        mk.more = 31;
                        mk.ns = j == 0 ? a.n_sink : 0;
                    }
                }
                const float mx = masked ? row_max_masked(tS, chunks, mk) : row_max(tS);
                const float mx2 = mx * c2;
                // Lazy rescale: this row's reference max moves only when the tile max
                // exceeds it by more than 2^8; tcgen05.ld/st are warp-collective, so O is
                // rescaled for the warp when any row needs it (alpha = 1 elsewhere).
                float alpha = 1.f;
                bool resc = false;
                if (mx2 > m_run + kRescaleThreshold) {
                    if (m_run != -INFINITY) {
                        alpha = ex2(m_run - mx2);
                        l *= alpha;
                        resc = true;
                    }
                    m_run = mx2;
                }
                if (started && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t u[32];
                        tmem_ld32(tO + c * 32, u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
                        tmem_st32(tO + c * 32, u);
                    }
                }
                started = true;
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                l += masked ? row_exp_masked<C::kTwice>(tS, chunks, mk, c2, m_use, &p_most[w], lane)
                            : row_exp<C::kTwice>(tS, c2, m_use, &p_most[w], lane);
                hand_over(&p_full[w], lane);
            }
            if (!ok) break;
            // ---- epilogue: O = O_acc / l, lse = ln(sum exp(s)); every row sees itself, so l > 0
            if (rd + 1 < rounds) y = deal(rd + 1);
            if (!SPLIT || started) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&o_full[w], qi & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                tc_fence_after();
                ++qi;
            }
            const bool valid = row < a.S;
            if (SPLIT && x.split) {
                ok = join<D>(a.log_p, deal.rank, (rd - deal.n_whole) & 1, w * BM + r, lane, started, m_run, l, tO, sKV, ready,
                             landed, abort_flag, a.err,
                             valid ? a.O + (((int64_t)x.b * a.S + row) * a.H.d + x.h) * D : nullptr,
                             a.lse + ((int64_t)x.b * (int)a.H.d + x.h) * a.S + row);
                if (!ok) break;
                fence_proxy_async_smem();             // the next loads into the ring come behind its reads
                __syncwarp();
                if (lane == 0) mbar_arrive(merged);
                continue;
            }
            const float inv = 1.f / l;
            // A lane holds a row: stored as it stands, every 16 bytes would go to a line of their own.
            // Four lanes exchange theirs and each store writes 64 contiguous bytes of eight rows.
            const int row4 = row & ~3;
            uint4* dst = reinterpret_cast<uint4*>(a.O + (((int64_t)x.b * a.S + row4) * a.H.d + x.h) * D) + (lane & 3);
            const int64_t step = (int64_t)a.H.d * (D / 8);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t u[32];
                tmem_ld32(tO + c * 32, u);
                uint32_t o[4][4];                         // [word][16 bytes of the row's 64]
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e % 4][e / 4] = pack_bf16(__uint_as_float(u[2 * e]) * inv, __uint_as_float(u[2 * e + 1]) * inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) quad_transpose(o[e], lane);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row4 + e < a.S) dst[c * 4 + e * step] = make_uint4(o[0][e], o[1][e], o[2][e], o[3][e]);
            }
            tc_fence_before();
            if (valid) a.lse[((int64_t)x.b * (int)a.H.d + x.h) * a.S + row] = (m_run + __log2f(l)) * kLn2;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_sync();      // no CTA leaves while another one may still write to it
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

// How a problem's blocks are dealt: whole ones first, the others split over
// clusters of 2^log_p CTAs.
struct Plan {
    int log_p, n_whole, grid;
};

// Costs in steps of a key tile (1.4 us at D = 128): kBlockSteps for a block's
// ends, kJoinSteps for joining the pieces of one (5 us).
constexpr int kBlockSteps = 3, kJoinSteps = 4;

cudaLaunchConfig_t cluster_config(int grid, int cluster, size_t smem, cudaStream_t s, cudaLaunchAttribute* at) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}

Plan make_plan(const Args& a, int sms, int clusters4) {
    Plan best{0, a.n_items, std::min(sms, a.n_items)};
    const int rows = (int)a.rows.d;
    auto tiles = [&](int it) {
        const int q0 = (a.n_units - 1 - it / rows) * kBlockRows, j0 = std::max(q0 - a.window + 1, 0) / BN;
        return (a.n_sink > 0 && j0 > 0) + q0 / BN + (q0 + BM < a.S) - j0 + 1;
    };
    // With many blocks per CTA the deal is even enough; short lists are not worth a join.
    const int longest = tiles(0);
    if (a.n_items > 2 * sms || longest - (longest + 3) / 4 <= kJoinSteps) return best;
    int load[1024], least = 1 << 30;
    for (int log_p = 0; log_p < 3; ++log_p) {
        const int n = log_p == 0 ? sms : log_p == 1 ? sms / 2 : clusters4, grid = n << log_p;
        if (grid < 1 || grid > 1024) continue;
        for (int whole = log_p == 0 ? a.n_items : 0; whole <= a.n_items; whole += grid) {
            std::fill(load, load + grid, 0);
            for (int i = 0, c = 0, step = 1; i < whole; ++i) {
                load[c] += tiles(i) + kBlockSteps;
                if ((step > 0 ? c == grid - 1 : c == 0)) step = -step;
                else c += step;
            }
            for (int i = whole, c = 0, step = 1; i < a.n_items; ++i) {
                const int cost = ((tiles(i) + (1 << log_p) - 1) >> log_p) + kBlockSteps + kJoinSteps;
                for (int e = 0; e < 1 << log_p; ++e) load[(c << log_p) + e] += cost;
                if ((step > 0 ? c == n - 1 : c == 0)) step = -step;
                else c += step;
            }
            const int most = *std::max_element(load, load + grid);
            if (most < least) {
                least = most;
                if (log_p > 0) best = Plan{log_p, whole, whole > 0 ? grid : std::min(n, a.n_items) << log_p};
            }
        }
    }
    return best;
}

template <int D>
dfa_status launch(const SinkProblem& p, const void* q, const void* k, const void* v, void* O, float* lse,
                  cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    const int64_t kv_sb = (int64_t)p.S * p.Hkv * D, kv_ss = (int64_t)p.Hkv * D;
    if (!make_tmap_bshd(&mq, q, p.B, p.S, p.H, D, (int64_t)p.S * p.H * D, (int64_t)p.H * D, D) ||
        !make_tmap_bshd(&mk, k, p.B, p.S, p.Hkv, D, kv_sb, kv_ss, D) ||
        !make_tmap_bshd(&mv, v, p.B, p.S, p.Hkv, D, kv_sb, kv_ss, D))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    Args a{};
    a.rows = Divider(p.B * p.H);
    a.H = Divider(p.H); a.G = Divider(p.H / p.Hkv); a.S = p.S;
    a.window = p.window; a.n_sink = p.n_sink;
    a.n_units = (p.S + kBlockRows - 1) / kBlockRows;
    a.n_items = p.B * p.H * a.n_units;
    a.scale_log2 = p.scale * kLog2e;
    a.O = static_cast<__nv_bfloat16*>(O); a.lse = lse;
    a.err = device_error_flag();
    const int smem = Cfg<D>::kSmem;
    static std::atomic<uint64_t> seen{0};
    static std::atomic<int> clusters4{0};            // clusters of four that run at a time
    auto whole = sink_fwd_kernel<D, false>;
    auto split = sink_fwd_kernel<D, true>;
    if (first_on_device(seen)) {
        int n = 0;
        cudaLaunchAttribute at[1];
        const cudaLaunchConfig_t cfg = cluster_config(4, 4, smem, s, at);
        if (cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, split, &cfg) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "sink_fwd: kernel attributes");
        clusters4.store(n);
        mark_on_device(seen);
    }
    const Plan plan = make_plan(a, num_sms(), clusters4.load());
    a.log_p = plan.log_p;
    a.n_whole = plan.n_whole;
    cudaError_t e;
    if (plan.log_p == 0) {
        whole<<<plan.grid, kThreads, smem, s>>>(mq, mk, mv, a);
        e = cudaGetLastError();
    } else {
        cudaLaunchAttribute at[1];
        const cudaLaunchConfig_t cfg = cluster_config(plan.grid, 1 << plan.log_p, smem, s, at);
        e = cudaLaunchKernelEx(&cfg, split, mq, mk, mv, a);
    }
    return e == cudaSuccess ? DFA_OK : fail(DFA_ERR_CUDA, "sink_fwd launch: %s", cudaGetErrorString(e));
}

}  // namespace

dfa_status tc_sink_fwd(const SinkProblem& p, const void* q, const void* k, const void* v, void* O, float* lse,
                       cudaStream_t s) {
    return p.D == 128 ? launch<128>(p, q, k, v, O, lse, s) : launch<64>(p, q, k, v, O, lse, s);
}

}  // namespace dfa
