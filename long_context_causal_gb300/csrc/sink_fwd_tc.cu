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
// Schedule.  No work list: costs never fall from a block to the next one of
// its head, so the blocks in the order last to first of all heads are sorted
// by cost, and dealing them to the persistent CTAs in a snake (0..n-1, then
// n-1..0, ...) balances them to within one block.  Nothing is uploaded and
// there is no workspace, so a call is one launch and can be captured.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer
// (one lane issues), warp 2 TMEM owner, warps 4-11 two softmax warpgroups, one
// query row per thread.  TMEM columns: S_0 [0,128) S_1 [128,256) O_0 [256,256+D)
// O_1 [384,384+D); P_w (bf16 pairs) overwrites the first 64 columns of S_w.
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

constexpr int kThreads = 384;
constexpr int BM = 128;            // query rows per tile (MMA M)
constexpr int BN = 128;            // key rows per tile
constexpr int kBlockRows = 2 * BM;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: rescale O only when the max grows by > 2^8

template <int D>
struct Cfg {
    static constexpr int kTileBytes = BN * D * 2;
    static constexpr int kSlots = D == 128 ? 4 : 6;            // K/V ring depth
    static constexpr int kQBytes = 2 * kTileBytes;
    static constexpr int kSmem = kQBytes + kSlots * kTileBytes + 1024 /*barriers*/ + 1024 /*align*/;
};

struct Args {
    int rows;              // B * H
    int H, G, S;           // G = H / H_kv
    int window, n_sink;    // window <= S; n_sink <= 128, 0 when the window covers every key
    int n_units, n_items;  // 256-row blocks per head; rows * n_units
    float scale_log2;      // scale * log2(e)
    __nv_bfloat16* O;      // [B, S, H, D]
    float* lse;            // [B, H, S]
    int* err;
};

// Band of the 128-row query tile whose first row is f: key tiles [lo, hi], none if f is past the end.
struct Band {
    int lo, hi;
    // How the tile takes part in key tile j: 0 not at all, 1 the sink columns only, 2 the whole tile.
    __device__ __forceinline__ int part(int j, int n_sink) const {
        if (j > hi) return 0;
        if (j >= lo) return 2;
        return j == 0 && n_sink > 0 ? 1 : 0;
    }
};
__device__ __forceinline__ Band band(const Args& a, int f) {
    return Band{max(f - a.window + 1, 0) / BN, f < a.S ? f / BN : -1};
}

struct Block {
    int b, h, g, q0;
    int j0;                // first key tile of the band
    int n;                 // key tiles in the list
    int sink0;             // 1: the list starts with tile 0 as a sink tile
    // k-th key tile of the list
    __device__ __forceinline__ int tile(int k) const { return (sink0 && k == 0) ? 0 : j0 + k - sink0; }
};

__device__ __forceinline__ Block decode(const Args& a, int it) {
    Block x;
    const int row = it % a.rows, unit = a.n_units - 1 - it / a.rows;
    x.b = row / a.H;
    x.h = row % a.H;
    x.g = x.h / a.G;
    x.q0 = unit * kBlockRows;
    const Band lo = band(a, x.q0), hi = band(a, x.q0 + BM);
    x.j0 = lo.lo;
    x.sink0 = a.n_sink > 0 && x.j0 > 0;
    x.n = max(lo.hi, hi.hi) - x.j0 + 1 + x.sink0;
    return x;
}

// Column c of a tile is visible iff (c >= lo or c < ns) and c < lim.
struct Mask {
    int lo, lim, ns;
    // bit e: column c + e
    __device__ __forceinline__ uint32_t bits(int c) const {
        return (~low_bits(lo - c) | low_bits(ns - c)) & low_bits(lim - c);
    }
};

// Row max of the first 32 * chunks scores of this thread's row in TMEM.
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t tS, int chunks, Mask k) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const uint32_t see = MASK ? k.bits(c * 32) : 0u;
        if (MASK && !__any_sync(0xffffffffu, see)) continue;   // no row of the warp sees the 32 columns
        uint32_t u[32];
        tmem_ld32(tS + c * 32, u);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float x = __uint_as_float(u[e]);
            m[e & 3] = fmaxf(m[e & 3], (!MASK || (see >> e & 1)) ? x : -INFINITY);
        }
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P = exp2(s * c2 - m) of the same columns, written as bf16 pairs over S (behind
// the columns still to be read).  Returns the row sum of the unrounded P.
template <bool MASK>
__device__ __forceinline__ float row_exp(uint32_t tS, int chunks, Mask k, float c2, float m) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        uint32_t pk[16];
        const uint32_t see = MASK ? k.bits(c * 32) : 0u;
        if (MASK && !__any_sync(0xffffffffu, see)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0;
            tmem_st16(tS + c * 16, pk);
            continue;
        }
        uint32_t u[32];
        tmem_ld32(tS + c * 32, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float p0 = ex2(fmaf(__uint_as_float(u[2 * e]), c2, -m));
            float p1 = ex2(fmaf(__uint_as_float(u[2 * e + 1]), c2, -m));
            if (MASK) {
                p0 = see >> (2 * e) & 1 ? p0 : 0.f;
                p1 = see >> (2 * e + 1) & 1 ? p1 : 0.f;
            }
            acc[e & 3] += p0 + p1;
            pk[e] = pack_bf16(p0, p1);
        }
        tmem_st16(tS + c * 16, pk);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

template <int D>
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
    uint64_t* p_full = bars + 6;
    uint64_t* o_full = bars + 8;
    uint64_t* done = bars + 10;
    uint64_t* kv_full = bars + 16;        // [kSlots]
    uint64_t* kv_empty = bars + 16 + C::kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 33);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rounds = snake_count(a.n_items, blockIdx.x, gridDim.x);

    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            mbar_init(&q_full[w], 1);
            mbar_init(&q_empty[w], 1);
            mbar_init(&s_full[w], 1);
            mbar_init(&p_full[w], BM);
            mbar_init(&o_full[w], 1);
        }
        mbar_init(done, 1);
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
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        uint32_t ld = 0, qi = 0;
        bool ok = true;
        for (int r = 0; r < rounds && ok; ++r) {
            const Block x = decode(a, snake_item(r, blockIdx.x, gridDim.x));
            for (int w = 0; w < 2 && ok; ++w) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&q_empty[w], (r & 1) ^ 1, abort_flag, a.err, nullptr));
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
            if (!ok) break;
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
        auto issue_PV = [&](int w, uint32_t slot, uint32_t acc) {
            const uint64_t b0 = dVn + slot * kSlotStep;
            const uint32_t d = tmem + 256 + w * 128, p = tmem + w * 128;
            mma_ts_lead(lead, d, p, b0, idO, acc);
#pragma unroll
            for (int kk = 1; kk < BN / 16; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, 1u);
        };
        auto issue_PV_sink = [&](int w, uint32_t slot, uint32_t acc) {
            const uint64_t b0 = dVn + slot * kSlotStep;
            const uint32_t d = tmem + 256 + w * 128, p = tmem + w * 128;
#pragma unroll 1
            for (int kk = 0; kk < ns16; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, kk > 0 ? 1u : acc);
        };
        for (int r = 0; r < rounds && ok; ++r) {
            const Block x = decode(a, snake_item(r, blockIdx.x, gridDim.x));
            const Band bd[2] = {band(a, x.q0), band(a, x.q0 + BM)};
            uint32_t slotK = cons % C::kSlots;
            if (!wait(&kv_full[slotK], (cons / C::kSlots) & 1)) break;
            ++cons;
            int now[2], first[2] = {1, 1};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!wait(&q_full[w], r & 1)) break;
                now[w] = bd[w].part(x.tile(0), a.n_sink);
                if (now[w]) issue_S(w, slotK, now[w] == 1 ? idSink : idS);
                // The query tile's last product is the one with the band's last tile; its buffer
                // is then free for the next block's.  A tile past the end has none.
                if (x.tile(0) >= bd[w].hi) mma_commit_lead(lead, &q_empty[w]);
            }
            if (!ok) break;
            mma_commit_lead(lead, &kv_empty[slotK]);
            // Steps in which both query tiles take both key tiles whole run without looking at the bands.
            const int hot = bd[0].hi - x.j0 + x.sink0;       // the first query tile's last key tile in the list
            int k = 0;
            while (k < x.n) {
                if (now[0] == 2 && now[1] == 2 && k < hot) {
                    const uint32_t acc0 = 1u - first[0], acc1 = 1u - first[1];
                    first[0] = first[1] = 0;
                    uint32_t a0 = acc0, a1 = acc1;
                    for (; k < hot; ++k) {
                        const uint32_t slotV = cons % C::kSlots;
                        if (!wait(&kv_full[slotV], (cons / C::kSlots) & 1)) break;
                        if (!wait(&p_full[0], t[0] & 1)) break;
                        ++t[0];
                        issue_PV(0, slotV, a0);
                        slotK = (cons + 1) % C::kSlots;
                        if (!wait(&kv_full[slotK], ((cons + 1) / C::kSlots) & 1)) break;
                        issue_S(0, slotK, idS);
                        if (!wait(&p_full[1], t[1] & 1)) break;
                        ++t[1];
                        issue_PV(1, slotV, a1);
                        mma_commit_lead(lead, &kv_empty[slotV]);
                        issue_S(1, slotK, idS);
                        mma_commit_lead(lead, &kv_empty[slotK]);
                        cons += 2;
                        a0 = a1 = 1u;
                    }
                    if (!ok) break;
                    mma_commit_lead(lead, &q_empty[0]);   // its last product is issued; the second query tile has one more
                }
                const bool more = k + 1 < x.n;
                const uint32_t slotV = cons % C::kSlots;
                if (!wait(&kv_full[slotV], (cons / C::kSlots) & 1)) break;
                slotK = (cons + 1) % C::kSlots;
                bool have_k = false;
                const int jn = x.tile(k + 1);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int next = more ? bd[w].part(jn, a.n_sink) : 0;
                    if (now[w]) {
                        if (!wait(&p_full[w], t[w] & 1)) break;
                        ++t[w];
                        if (now[w] == 2) issue_PV(w, slotV, first[w] ? 0u : 1u);
                        else issue_PV_sink(w, slotV, first[w] ? 0u : 1u);
                        first[w] = 0;
                    }
                    if (w == 1) mma_commit_lead(lead, &kv_empty[slotV]);
                    // a query tile takes part in an unbroken run of the list, sinks apart: it has ended
                    // when the tile after this one lies beyond its band
                    if (now[w] && (!more || jn > bd[w].hi)) mma_commit_lead(lead, &o_full[w]);
                    if (next) {
                        if (!have_k) {
                            if (!wait(&kv_full[slotK], ((cons + 1) / C::kSlots) & 1)) break;
                            have_k = true;
                        }
                        issue_S(w, slotK, next == 1 ? idSink : idS);
                        if (jn == bd[w].hi) mma_commit_lead(lead, &q_empty[w]);
                    }
                    if (w == 1 && more) mma_commit_lead(lead, &kv_empty[slotK]);
                    now[w] = next;
                }
                if (!ok) break;
                cons += more ? 2 : 1;
                ++k;
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
        for (int rd = 0; rd < rounds && ok; ++rd) {
            const Block x = decode(a, snake_item(rd, blockIdx.x, gridDim.x));
            const int f = x.q0 + w * BM, row = f + r;
            if (f >= a.S) continue;                   // no row of the sequence in this tile
            const Band bd = band(a, f);
            const int lo_row = row - a.window + 1, lo_last = f + BM - a.window;   // lowest visible keys
            float m_run = -INFINITY, l = 0.f;
            bool started = false;
            for (int k = 0; k < x.n; ++k) {
                const int j = x.tile(k), part = bd.part(j, a.n_sink);
                if (!part) continue;
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&s_full[w], t & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                ++t;
                tc_fence_after();
                const int kv0 = j * BN;
                Mask mk{0, BN, 0};
                int chunks = BN / 32;
                bool masked = true;
                if (part == 1) {
                    mk.lim = a.n_sink;
                    chunks = (a.n_sink + 31) / 32;
                } else {
                    masked = kv0 + BN > f || kv0 < lo_last;   // the diagonal tile (and the ragged end) or the window's edge
                    if (masked) {
                        mk.lo = max(lo_row - kv0, 0);
                        mk.lim = min(row - kv0 + 1, BN);
                        mk.ns = j == 0 ? a.n_sink : 0;
                    }
                }
                const float mx = masked ? row_max<true>(tS, chunks, mk) : row_max<false>(tS, chunks, mk);
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
                l += masked ? row_exp<true>(tS, chunks, mk, c2, m_use) : row_exp<false>(tS, chunks, mk, c2, m_use);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[w]);
            }
            if (!ok) break;
            // ---- epilogue: O = O_acc / l, lse = ln(sum exp(s)); every row sees itself, so l > 0
            ok = __all_sync(0xffffffffu, mbar_wait_acc(&o_full[w], qi & 1, abort_flag, a.err, nullptr));
            if (!ok) break;
            tc_fence_after();
            ++qi;
            const bool valid = row < a.S;
            const float inv = 1.f / l;
            uint4* dst = reinterpret_cast<uint4*>(a.O + (((int64_t)x.b * a.S + row) * a.H + x.h) * D);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t u[32];
                tmem_ld32(tO + c * 32, u);
                if (valid) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 o;
                        o.x = pack_bf16(__uint_as_float(u[8 * e + 0]) * inv, __uint_as_float(u[8 * e + 1]) * inv);
                        o.y = pack_bf16(__uint_as_float(u[8 * e + 2]) * inv, __uint_as_float(u[8 * e + 3]) * inv);
                        o.z = pack_bf16(__uint_as_float(u[8 * e + 4]) * inv, __uint_as_float(u[8 * e + 5]) * inv);
                        o.w = pack_bf16(__uint_as_float(u[8 * e + 6]) * inv, __uint_as_float(u[8 * e + 7]) * inv);
                        dst[c * 4 + e] = o;
                    }
                }
            }
            tc_fence_before();
            if (valid) a.lse[((int64_t)x.b * a.H + x.h) * a.S + row] = (m_run + __log2f(l)) * kLn2;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D>
dfa_status launch(const SinkProblem& p, const void* q, const void* k, const void* v, void* O, float* lse,
                  cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!make_tmap_bshd(&mq, q, p.B, p.S, p.H, D, (int64_t)p.S * p.H * D, (int64_t)p.H * D, D) ||
        !make_tmap_bshd(&mk, k, p.B, p.S, p.Hkv, D, (int64_t)p.S * p.Hkv * D, (int64_t)p.Hkv * D, D) ||
        !make_tmap_bshd(&mv, v, p.B, p.S, p.Hkv, D, (int64_t)p.S * p.Hkv * D, (int64_t)p.Hkv * D, D))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    Args a{};
    a.rows = p.B * p.H;
    a.H = p.H; a.G = p.H / p.Hkv; a.S = p.S;
    a.window = p.window; a.n_sink = p.n_sink;
    a.n_units = (p.S + kBlockRows - 1) / kBlockRows;
    a.n_items = a.rows * a.n_units;
    a.scale_log2 = p.scale * kLog2e;
    a.O = static_cast<__nv_bfloat16*>(O); a.lse = lse;
    a.err = device_error_flag();
    const int smem = Cfg<D>::kSmem;
    auto kern = sink_fwd_kernel<D>;
    static std::atomic<uint64_t> seen{0};
    if (first_on_device(seen)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "sink_fwd: shared memory attribute");
        mark_on_device(seen);
    }
    kern<<<std::min(num_sms(), a.n_items), kThreads, smem, s>>>(mq, mk, mv, a);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DFA_OK : fail(DFA_ERR_CUDA, "sink_fwd launch: %s", cudaGetErrorString(e));
}

}  // namespace

dfa_status tc_sink_fwd(const SinkProblem& p, const void* q, const void* k, const void* v, void* O, float* lse,
                       cudaStream_t s) {
    return p.D == 128 ? launch<128>(p, q, k, v, O, lse, s) : launch<64>(p, q, k, v, O, lse, s);
}

}  // namespace dfa
