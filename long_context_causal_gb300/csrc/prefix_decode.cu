// prefix_decode.cu -- single tokens of a batch whose sequences share their first
// keys and values: the prefix's part, on tcgen05, for sm_103a.
//
// The queries of all B sequences and of the G heads of a group see the same P keys,
// so for each key/value head they are the rows of one matrix of R = B G rows, and
// the prefix is attended to as a forward without a mask: the keys are read once per
// 256 rows and not once per sequence.  Each CTA leaves an unnormalised fp32 output
// with its maximum and sum per row; the kernel that joins the sequences' own keys'
// parts (sink_decode.cu) adds these to them.
//
// A segment is a pair of 128-row tiles of a head.  As in sink_fwd_tc.cu two
// warpgroups take a query tile each and ping-pong on the tensor cores.  Where the
// pair has one tile only (R <= 128, or an odd number of tiles), both warpgroups take
// it, with every other key tile each, and leave two parts: the chain S -> softmax ->
// P V of one key tile runs under the other one's, as before, and the loads of K and
// V keep coming.  The key tiles of all segments, in order, are dealt to the CTAs in
// equal contiguous ranges; a part is numbered by segment + CTA, which no two pieces
// share.
//
// What bounds it: HBM (the prefix is read once) up to about 256 rows a head, above that
// the softmax chain as in the forward.  48 sequences of 4 heads a group (192 rows) behind
// 32768 keys, 8 kv heads, D = 128: 28 to 30 us (134 MB, 4.6 TB/s); 128 sequences of 8 heads
// a group (1024 rows) behind 16384: 48 us (1430 TFLOP/s; tensor cores 47% busy under cold
// caches; at D = 64 29%, as busy as the exponentials: the chain of product, softmax, product).
// Waits of the issuing warp by polling: 1% slower on both.
//
// The kernel of the own keys is let go at once (launch_dependents) and takes the SMs as
// this one leaves them.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer of K and V, warp 1 MMA
// issuer, warp 2 TMEM owner, warps 4-11 two softmax warpgroups, one row per thread,
// which also bring their rows of Q to shared memory.
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

constexpr int kThreads = 384;
constexpr int BM = 128, BN = 128;            // rows and keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMost = 6;                     // steps of 16 keys in the first part of P that is handed over
constexpr float kRescaleThreshold = 8.0f;    // log2 units: rescale O only when the max grows by > 2^8

template <int D>
struct Cfg {
    static constexpr int kTileBytes = BN * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 10;
    static constexpr bool kTwice = D == 128;
    static constexpr int kOffKV = 2 * kTileBytes;
    static constexpr int kOffBar = kOffKV + kSlots * kTileBytes;
    static constexpr int kSmem = kOffBar + 512;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Args {
    PrefixPlan p;
    int H, Hkv, G;
    const __nv_bfloat16* q;       // [B, H, D]
    float scale_log2;
    float* part;                  // [slabs][2][row_stride][D]
    float2* stat;                 // [slabs][2][row_stride]
    int* err;
};

// A CTA's piece of a segment: its key tiles [k, k + n).
struct Piece {
    int s, k, n;
    int g, row0;                  // key/value head, first row
    bool both;                    // two query tiles; else one, for both warpgroups
};
__device__ __forceinline__ Piece piece_at(const Args& a, int64_t x, int64_t end) {
    Piece c;
    c.s = (int)(x / a.p.n_kt);
    c.k = (int)(x - (int64_t)c.s * a.p.n_kt);
    c.n = (int)min((int64_t)(a.p.n_kt - c.k), end - x);
    c.g = c.s / a.p.n_pairs;
    c.row0 = (c.s - c.g * a.p.n_pairs) * 2 * BM;
    c.both = c.row0 + BM < a.p.rows;
    return c;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {            // the swizzled tiles need a 1 KB aligned base
        if (threadIdx.x == 0 && a.err) atomicExch(a.err, 2);
        return;
    }
    uint8_t *sQ = smem, *sKV = smem + C::kOffKV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* q_full = bars + 0;          // [2], as all of these one per warpgroup
    uint64_t* s_full = bars + 2;
    uint64_t* p_most = bars + 4;
    uint64_t* p_full = bars + 6;
    uint64_t* o_full = bars + 8;
    uint64_t* done = bars + 10;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 11);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 12);
    uint64_t* kv_full = bars + 16;        // [kSlots]
    uint64_t* kv_empty = bars + 16 + C::kSlots;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            mbar_init(&q_full[w], 4);
            mbar_init(&s_full[w], 1);
            mbar_init(&p_most[w], 4);
            mbar_init(&p_full[w], 4);
            mbar_init(&o_full[w], 1);
        }
        mbar_init(done, 1);
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
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
    wait_for_previous_kernel();
    launch_dependents();                  // the sequences' own keys need nothing of this
    const uint32_t tmem = *tmem_slot;
    const int64_t steps = a.p.steps, begin = steps * blockIdx.x / gridDim.x, end = steps * (blockIdx.x + 1) / gridDim.x;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer of K and V
        uint32_t ld = 0;
        bool ok = true;
        for (int64_t x = begin; x < end && ok;) {
            const Piece c = piece_at(a, x, end);
            for (int k = c.k; k < c.k + c.n && ok; ++k)
                for (int which = 0; which < 2; ++which, ++ld) {
                    const int slot = ld % C::kSlots;
                    ok = __all_sync(0xffffffffu, mbar_wait_acc(&kv_empty[slot], ((ld / C::kSlots) & 1) ^ 1, abort_flag, a.err, nullptr));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&kv_full[slot], C::kTileBytes);
                        for (int blk = 0; blk < D / 64; ++blk)
                            tma_load_4d(sKV + slot * C::kTileBytes + blk * 16384, which ? &tmV : &tmK, &kv_full[slot], blk * 64,
                                        c.g, k * BN, 0);
                    }
                    __syncwarp();
                }
            x += c.n;
        }
        if (!ok && lane == 0) {
            // Aborted: let the copies already issued land before the CTA exits.
            int dummy = 0;
            for (uint32_t m = ld > (uint32_t)C::kSlots ? ld - C::kSlots : 0; m < ld; ++m)
                mbar_wait(&kv_full[m % C::kSlots], (m / C::kSlots) & 1, &dummy, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one lane of a converged warp)
        const uint32_t lead = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);       // uniform
        const uint32_t idS = idesc_bf16_f32(BM, BN, false, false), idO = idesc_bf16_f32(BM, D, false, true);
        const uint64_t dQk = sdesc_sw128(smem_u32(sQ), 16, 1024);          // Q, K-major
        const uint64_t dKk = sdesc_sw128(smem_u32(sKV), 16, 1024);         // K slots, K-major
        const uint64_t dVn = sdesc_sw128(smem_u32(sKV), 16384, 1024);      // V slots, N-major
        constexpr uint64_t kSlotStep = C::kTileBytes >> 4;
        uint32_t cons = 0, t[2] = {0, 0}, qi[2] = {0, 0};                  // K of a CTA's m-th tile is load 2 m, its V 2 m + 1
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && mbar_wait_issuer(bar, parity, abort_flag, a.err);
            if (ok) tc_fence_after();
            return ok;
        };
        auto wait_load = [&](uint32_t m) { return wait(&kv_full[m % C::kSlots], (m / C::kSlots) & 1); };
        auto release = [&](uint32_t m) { mma_commit_lead(lead, &kv_empty[m % C::kSlots]); };
        // S_w = Q_tile K^T
        auto issue_S = [&](int w, int tile, uint32_t m) {
            const uint64_t a0 = dQk + tile * kSlotStep, b0 = dKk + (m % C::kSlots) * kSlotStep;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                mma_ss_lead(lead, tm + w * 128, a0 + off, b0 + off, idS, kk > 0);
            }
            mma_commit_lead(lead, &s_full[w]);
        };
        // O_w += P_w V, most of the keys as soon as their P is there
        auto issue_PV = [&](int w, uint32_t m, uint32_t acc) {
            const uint64_t b0 = dVn + (m % C::kSlots) * kSlotStep;
            const uint32_t d = tm + 256 + w * 128, p = tm + w * 128, par = (w ? t[1]++ : t[0]++) & 1;
            if (!wait(C::kTwice ? &p_most[w] : &p_full[w], par)) return;
            mma_ts_lead(lead, d, p, b0, idO, acc);
#pragma unroll
            for (int kk = 1; kk < kMost; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, 1u);
            if (C::kTwice && !wait(&p_full[w], par)) return;
#pragma unroll
            for (int kk = kMost; kk < BN / 16; ++kk) mma_ts_lead(lead, d, p + kk * 8, b0 + kk * (2048 >> 4), idO, 1u);
        };
        for (int64_t x = begin; x < end && ok;) {
            const Piece c = piece_at(a, x, end);
            x += c.n;
            if (!wait(&q_full[0], qi[0]++ & 1)) break;
            if (c.both) {
                if (!wait(&q_full[1], qi[1]++ & 1) || !wait_load(cons)) break;
                issue_S(0, 0, cons);
                issue_S(1, 1, cons);
                release(cons);
                for (int j = 0; j < c.n && ok; ++j, cons += 2) {
                    const bool more = j + 1 < c.n;
                    if (!wait_load(cons + 1)) break;
                    issue_PV(0, cons + 1, j > 0);
                    if (!ok) break;
                    if (more) {
                        if (!wait_load(cons + 2)) break;
                        issue_S(0, 0, cons + 2);
                    } else {
                        mma_commit_lead(lead, &o_full[0]);
                    }
                    issue_PV(1, cons + 1, j > 0);
                    if (!ok) break;
                    release(cons + 1);
                    if (more) {
                        issue_S(1, 1, cons + 2);
                        release(cons + 2);
                    } else {
                        mma_commit_lead(lead, &o_full[1]);
                    }
                }
            } else {
                for (int j = 0; j < 2 && j < c.n; ++j) {
                    if (!wait_load(cons + 2 * j)) break;
                    issue_S(j, 0, cons + 2 * j);
                    release(cons + 2 * j);
                }
                for (int j = 0; j < c.n && ok; ++j, cons += 2) {
                    const int w = j & 1;
                    if (!wait_load(cons + 1)) break;
                    issue_PV(w, cons + 1, j > 1);
                    if (!ok) break;
                    release(cons + 1);
                    if (j + 2 < c.n) {
                        if (!wait_load(cons + 4)) break;
                        issue_S(w, 0, cons + 4);
                        release(cons + 4);
                    } else {
                        mma_commit_lead(lead, &o_full[w]);
                    }
                }
            }
        }
        // Drain: every MMA issued here has finished before TMEM is freed.
        mma_commit_lead(lead, done);
        int dummy = 0;
        mbar_wait(done, 0, &dummy, a.err);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax warpgroups
        const int w = (warp - 4) / 4, r = (warp % 4) * 32 + lane;      // row within the tile == TMEM lane
        const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tmem + lane_base + w * 128, tO = tmem + lane_base + 256 + w * 128;
        const float c2 = a.scale_log2;
        uint32_t t = 0, oi = 0;
        bool ok = true;
        for (int64_t x = begin; x < end && ok;) {
            const Piece c = piece_at(a, x, end);
            x += c.n;
            const int tile = c.both ? w : 0, row = c.row0 + tile * BM + r;
            if (c.both || w == 0) {
                // the products that read this buffer before are done: o_full of the last piece was committed behind them
                const int b = row / a.G;
                const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.H + c.g * a.G + (row - b * a.G)) * D);
                uint4 u[D / 8];
#pragma unroll
                for (int e = 0; e < D / 8; ++e) u[e] = row < a.p.rows ? src[e] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < D / 8; ++e)
                    *reinterpret_cast<uint4*>(sQ + tile * C::kTileBytes + (e / 8) * 16384 + sw128_offset(r, (e % 8) * 8)) = u[e];
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[tile]);
            }
            float m_run = -INFINITY, l = 0.f;
            bool started = false;
            for (int j = c.both ? 0 : w; j < c.n; j += c.both ? 1 : 2) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&s_full[w], t & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                ++t;
                tc_fence_after();
                const int left = a.p.P - (c.k + j) * BN;
                const Mask mk{0, left, 0, 0, left, 0};
                const bool masked = left < BN;
                const float mx2 = (masked ? row_max_masked(tS, BN / 32, mk) : row_max(tS)) * c2;
                // lazy rescale, for the warp when any row needs it (sink_fwd_tc.cu)
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
                    for (int e = 0; e < D / 32; ++e) {
                        uint32_t u[32];
                        tmem_ld32(tO + e * 32, u);
#pragma unroll
                        for (int f = 0; f < 32; ++f) u[f] = __float_as_uint(__uint_as_float(u[f]) * alpha);
                        tmem_st32(tO + e * 32, u);
                    }
                }
                started = true;
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                l += masked ? row_exp_masked<C::kTwice>(tS, BN / 32, mk, c2, m_use, &p_most[w], lane)
                            : row_exp<C::kTwice>(tS, c2, m_use, &p_most[w], lane);
                hand_over(&p_full[w], lane);
            }
            if (!ok) break;
            // ---- this piece's part: what no tile came to has sum 0
            if (started) {
                ok = __all_sync(0xffffffffu, mbar_wait_acc(&o_full[w], oi & 1, abort_flag, a.err, nullptr));
                if (!ok) break;
                ++oi;
                tc_fence_after();
            }
            const int64_t slab = (int64_t)(c.s + (int)blockIdx.x) * 2 + w;
            if (r < a.p.row_stride && row < a.p.rows) a.stat[slab * a.p.row_stride + r] = make_float2(m_run, l);
            if (!started) continue;
            // four lanes exchange their rows' 16 bytes, so that a store writes 64 contiguous bytes of eight rows
            const int r4 = r & ~3, left = min(a.p.row_stride, a.p.rows - (c.row0 + tile * BM)) - r4;
            float4* dst = reinterpret_cast<float4*>(a.part + (slab * a.p.row_stride + r4) * D) + (lane & 3);
#pragma unroll 1
            for (int e0 = 0; e0 < D / 16; e0 += 4) {
                uint32_t u[4][16];
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_ld16_async(tO + (e0 + e) * 16, u[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    tmem_wait_ld16(u[e]);
                    uint32_t o[4][4];                     // [word][16 bytes of the row's 64]
#pragma unroll
                    for (int f = 0; f < 16; ++f) o[f % 4][f / 4] = u[e][f];
#pragma unroll
                    for (int f = 0; f < 4; ++f) quad_transpose(o[f], lane);
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        if (f < left)
                            dst[f * (D / 4) + (e0 + e) * 4] = make_float4(__uint_as_float(o[0][f]), __uint_as_float(o[1][f]),
                                                                          __uint_as_float(o[2][f]), __uint_as_float(o[3][f]));
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D>
dfa_status launch(const DecodeProblem& p, const PrefixPlan& plan, const void* q, const void* kp, const void* vp, int64_t ss,
                  int64_t sh, float* part, float2* stat, cudaStream_t s) {
    CUtensorMap mk, mv;
    if (!make_tmap_bshd(&mk, kp, 1, plan.P, p.Hkv, D, 0, ss, sh) || !make_tmap_bshd(&mv, vp, 1, plan.P, p.Hkv, D, 0, ss, sh))
        return fail(DFA_ERR_CUDA, "tensor map encoding failed");
    Args a{};
    a.p = plan;
    a.H = p.H; a.Hkv = p.Hkv; a.G = p.H / p.Hkv;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.scale_log2 = p.scale * kLog2e;
    a.part = part; a.stat = stat;
    a.err = device_error_flag();
    static std::atomic<uint64_t> seen{0};
    auto kernel = prefix_kernel<D>;
    if (first_on_device(seen)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess)
            return fail(DFA_ERR_CUDA, "prefix: kernel attributes");
        mark_on_device(seen);
    }
    const cudaError_t e = launch_overlapped(kernel, dim3((unsigned)plan.grid), kThreads, Cfg<D>::kSmem, s, mk, mv, a);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "prefix launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_FWD);
    return DFA_OK;
}

}  // namespace

PrefixPlan prefix_plan(int B, int G, int Hkv, int P, int sms) {
    PrefixPlan p{};
    p.P = P;
    p.rows = B * G;
    p.row_stride = std::min(p.rows, BM);
    p.n_pairs = (p.rows + 2 * BM - 1) / (2 * BM);
    p.n_kt = (P + BN - 1) / BN;
    p.n_seg = Hkv * p.n_pairs;
    p.steps = (int64_t)p.n_seg * p.n_kt;
    // A multiple of the segments where that uses nine tenths of the SMs: no CTA has two pieces then.  Calls with it and
    // with all SMs: 10 segments on 150 CTAs 35.3 and 38.9 us (16384 keys, 128 rows a head; D = 64 22.4 and 25.6), 12 on 144
    // 41.3 and 46.1 (30.2 and 31.8), 24 on 144 39.9 and 41.5 (25.5 and 27.1), 4 on 144 42.2 both (34.1 and 33.8).  Fewer SMs
    // may pay or not: 32 segments on 128 78.7 and 81.7 us, at D = 64 64.2 and 61.6.
    p.grid = (int)std::min<int64_t>(sms, p.steps);
    const int even = sms / p.n_seg * p.n_seg;
    if (p.steps > even && even * 10 >= sms * 9) p.grid = even;
    p.slabs = p.grid > 0 ? p.n_seg + p.grid : 0;
    return p;
}

dfa_status tc_prefix(const DecodeProblem& p, const PrefixPlan& plan, const void* q, const void* kp, const void* vp, int64_t ss,
                     int64_t sh, float* part, float2* stat, cudaStream_t s) {
    return p.D == 128 ? launch<128>(p, plan, q, kp, vp, ss, sh, part, stat, s)
                      : launch<64>(p, plan, q, kp, vp, ss, sh, part, stat, s);
}

}  // namespace dfa
