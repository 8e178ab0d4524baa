// cache_evict.cu -- eviction from a key/value cache by gathered attention weight.
//
// Of the n = kv_len[b] keys of a sequence and key/value head, `keep` stay: the
// first n_first, the last n_recent, and of the others those with the greatest
// mass, ties to the lowest position.  They move, in their order, to the front of
// another cache.  Two launches.
//
// select_kernel finds the border: masses become unsigned integers of the same
// order, and a radix select of three digits (11, 11 and 10 bits) narrows down the
// integer T of the last one that stays, and how many of those equal to T do.
// Positions follow from counts: a warp owns a contiguous range of keys, counts
// what it keeps, and after one scan over all warps of the row writes its keys'
// positions in order.  A row is shared by a cluster of up to eight CTAs that add
// their histograms and counts through distributed shared memory.
//
// copy_kernel moves the rows: bound by HBM (each kept row read and written once).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;

struct Args {
    int Hkv, S, keep, cap, n_first, n_recent;
    const int32_t* kv_len;
    const float* mass;            // [B, Hkv, S]
    int32_t* len_out;             // [B]
    float* mass_out;              // [B, Hkv, cap]
    int32_t* kept;                // [B, Hkv, keep]
};

// Unsigned integers in the order of the numbers; -0 is 0, NaN stands below all.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
    return r;
}

// Inclusive sum over the threads before and including this one; all: of all threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* s_warp, uint32_t& all) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                 // the last scan's sums have been read
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    return x + (warp ? before : 0);
}

__global__ void __launch_bounds__(kThreads, 1)
select_kernel(const Args a, int log_c) {
    __shared__ uint32_t hist[2][kBins];
    __shared__ uint32_t s_scan[kWarps], s_count[kWarps + 1], s_found[2];
    const int C = 1 << log_c, rank = blockIdx.x & (C - 1), row = blockIdx.x >> log_c, b = row / a.Hkv;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n = min(max(a.kv_len[b], 0), a.S);
    const float* mass = a.mass + (int64_t)row * a.S;
    float* mass_out = a.mass_out + (int64_t)row * a.cap;
    int32_t* kept = a.kept + (int64_t)row * a.keep;
    if (row % a.Hkv == 0 && rank == 0 && tid == 0) a.len_out[b] = min(n, a.keep);
    // behind the kept keys
    for (int r = min(n, a.keep) + rank * kThreads + tid; r < a.cap; r += C * kThreads) {
        mass_out[r] = 0.f;
        if (r < a.keep) kept[r] = -1;
    }
    if (n <= a.keep) {
        for (int r = rank * kThreads + tid; r < n; r += C * kThreads) {
            mass_out[r] = mass[r];
            kept[r] = r;
        }
        return;
    }
    const int lo = a.n_first, hi = n - a.n_recent;      // the keys that compete
    const int want = a.keep - a.n_first - a.n_recent;   // so many of them stay; fewer than there are
    // a warp's keys: 32 * steps from `from` on
    const int steps = (n + 32 * C * kWarps - 1) / (32 * C * kWarps), from = (rank * kWarps + warp) * 32 * steps;
    uint32_t T = 0xffffffffu;       // what stays is above T, or equal to it and among the first E of those
    int E = 0;
    if (want > 0) {
        T = 0;
        E = want;
        int top = 32;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            uint32_t* h = hist[pass & 1];
            const int bits = pass == 2 ? 10 : 11, low = top - bits;
            for (int i = tid; i < kBins; i += kThreads) h[i] = 0;
            __syncthreads();
            for (int s = 0; s < steps; ++s) {
                const int j = from + s * 32 + lane;
                if (j < lo || j >= hi) continue;
                const uint32_t u = ordered(mass[j]);
                if (top == 32 || u >> top == T >> top) atomicAdd(&h[u >> low & ((1u << bits) - 1)], 1u);
            }
            __syncwarp();
            if (C > 1) cluster_sync();
            else __syncthreads();
            // bins in falling order, two of them a thread
            uint32_t c[2] = {0, 0};
            const int bin = kBins - 1 - 2 * tid;
            for (int r = 0; r < C; ++r) {
                c[0] += C > 1 ? ld_cluster_u32(&h[bin], r) : h[bin];
                c[1] += C > 1 ? ld_cluster_u32(&h[bin - 1], r) : h[bin - 1];
            }
            uint32_t all;
            const uint32_t upto = block_scan(c[0] + c[1], s_scan, all), before = upto - c[0] - c[1];
            if (before < (uint32_t)E && upto >= (uint32_t)E) {
                const bool second = before + c[0] < (uint32_t)E;
                s_found[0] = bin - second;
                s_found[1] = E - before - (second ? c[0] : 0);
            }
            __syncthreads();
            T |= s_found[0] << low;
            E = s_found[1];
            top = low;
        }
    }
    // what each warp keeps for certain (upper half), and its keys equal to T (lower half)
    uint32_t sure = 0, equal = 0;
    for (int s = 0; s < steps; ++s) {
        const int j = from + s * 32 + lane;
        const bool in = j < n, free = j >= lo && j < hi;
        const uint32_t u = in ? ordered(mass[j]) : 0;
        sure += __popc(__ballot_sync(0xffffffffu, in && (!free || u > T)));
        equal += __popc(__ballot_sync(0xffffffffu, in && free && u == T));
    }
    if (E == 0) equal = 0;           // want = 0: none of them stays
    // keys before this warp's: of the CTAs before, then of the warps before
    uint32_t all;
    const uint32_t upto_s = block_scan(lane == 0 ? sure : 0, s_scan, all);
    if (tid == 0) s_count[0] = all;
    const uint32_t upto_e = block_scan(lane == 0 ? equal : 0, s_scan, all);
    if (tid == 0) s_count[1] = all;
    uint32_t at_s = __shfl_sync(0xffffffffu, upto_s, 0) - sure, at_e = __shfl_sync(0xffffffffu, upto_e, 0) - equal;
    if (C > 1) {
        __syncwarp();
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            at_s += ld_cluster_u32(&s_count[0], r);
            at_e += ld_cluster_u32(&s_count[1], r);
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int s = 0; s < steps; ++s) {
        const int j = from + s * 32 + lane;
        const bool in = j < n, free = j >= lo && j < hi;
        const float x = in ? mass[j] : 0.f;
        const uint32_t u = ordered(x);
        const bool is_s = in && (!free || u > T), is_e = in && free && u == T && E > 0;
        const uint32_t ms = __ballot_sync(0xffffffffu, is_s), me = __ballot_sync(0xffffffffu, is_e);
        const uint32_t e = at_e + __popc(me & below);
        if (is_s || (is_e && e < (uint32_t)E)) {
            const int r = at_s + __popc(ms & below) + min(e, (uint32_t)E);
            kept[r] = j;
            mass_out[r] = x;
        }
        at_s += __popc(ms);
        at_e += __popc(me);
    }
    __syncwarp();
    if (C > 1) cluster_sync();       // no CTA leaves while another one may still read its counts
}

struct CopyArgs {
    int Hkv, S, keep, log_u;      // 16-byte units of a row: 2^log_u
    const int32_t* kv_len;
    const int32_t* kept;
    const uint4 *k, *v;
    uint4 *k_out, *v_out;
    int64_t in_sb, in_ss, in_sh, out_sb, out_ss, out_sh;   // units
};

constexpr int kCopyThreads = 256, kCopyAhead = 4;
// Block (x, b): units [x, x + 1) * kCopyThreads * kCopyAhead of sequence b's rows, heads
// within a row, units within a head.
__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const CopyArgs a, int blocks) {
    wait_for_previous_kernel();
    const int b = blockIdx.x / blocks;
    const int rows = min(min(max(a.kv_len[b], 0), a.S), a.keep);
    const int64_t units = (int64_t)rows * a.Hkv << a.log_u;
    const int64_t first = (int64_t)(blockIdx.x % blocks) * (kCopyThreads * kCopyAhead) + threadIdx.x;
    uint4 k[kCopyAhead], v[kCopyAhead];
    int64_t to[kCopyAhead];
#pragma unroll
    for (int e = 0; e < kCopyAhead; ++e) {
        const int64_t x = first + e * kCopyThreads;
        to[e] = -1;
        if (x >= units) continue;
        const int64_t rh = x >> a.log_u;
        const int c = (int)(x - (rh << a.log_u)), r = (int)(rh / a.Hkv), g = (int)(rh - (int64_t)r * a.Hkv);
        const int j = a.kept[((int64_t)b * a.Hkv + g) * a.keep + r];
        const int64_t at = b * a.in_sb + j * a.in_ss + g * a.in_sh + c;
        k[e] = a.k[at];
        v[e] = a.v[at];
        to[e] = b * a.out_sb + r * a.out_ss + g * a.out_sh + c;
    }
#pragma unroll
    for (int e = 0; e < kCopyAhead; ++e)
        if (to[e] >= 0) {
            a.k_out[to[e]] = k[e];
            a.v_out[to[e]] = v[e];
        }
}

}  // namespace

dfa_status cache_evict(const EvictProblem& p, const void* k, const void* v, const int32_t* kv_len, const float* mass,
                       void* k_out, void* v_out, int32_t* len_out, float* mass_out, int32_t* kept, cudaStream_t s) {
    const Args a{p.Hkv, p.S, p.keep, p.cap, p.n_first, p.n_recent, kv_len, mass, len_out, mass_out, kept};
    const int rows = p.B * p.Hkv;
    int log_c = 0;
    while ((1 << log_c) < kMaxCluster && p.S > (kThreads * 2 << log_c)) ++log_c;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1u << log_c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)rows << log_c);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, a, log_c);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "evict launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_EVICT);
    const int unit = 16 / p.elt;
    CopyArgs c{};
    c.Hkv = p.Hkv; c.S = p.S; c.keep = p.keep;
    while ((unit << c.log_u) < p.D) ++c.log_u;
    c.kv_len = kv_len;
    c.kept = kept;
    c.k = static_cast<const uint4*>(k); c.v = static_cast<const uint4*>(v);
    c.k_out = static_cast<uint4*>(k_out); c.v_out = static_cast<uint4*>(v_out);
    c.in_sb = p.in_sb / unit; c.in_ss = p.in_ss / unit; c.in_sh = p.in_sh / unit;
    c.out_sb = p.out_sb / unit; c.out_ss = p.out_ss / unit; c.out_sh = p.out_sh / unit;
    const int64_t units = (int64_t)std::min(p.keep, p.S) * p.Hkv << c.log_u;
    const int blocks = (int)((units + kCopyThreads * kCopyAhead - 1) / (kCopyThreads * kCopyAhead));
    e = launch_overlapped(copy_kernel, dim3((unsigned)(p.B * blocks)), kCopyThreads, 0, s, c, blocks);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "evict copy launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_EVICT);
    return DFA_OK;
}

}  // namespace dfa
