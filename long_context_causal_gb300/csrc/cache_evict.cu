// cache_evict.cu -- eviction from a key/value cache by gathered attention weight.
//
// Of the n = kv_len[b] keys of a sequence and key/value head, `keep` stay: the
// first n_first, the last n_recent, and of the others those with the greatest
// mass, ties to the lowest position.  They move, in their order, to the front of
// another cache.  Two launches, or one where the rows are short (kMoveUnits).
//
// select_kernel finds the border: masses become unsigned integers of the same
// order, and a radix select (digits of 11, 11 and 10 bits, or four of 8) narrows down
// the integer T of the last one that stays, and how many of those equal to T do; it
// ends early where a whole bin stays.  Positions follow from counts: a thread owns up to
// 16 consecutive keys, which it holds in registers, counts what it keeps of them,
// and after one scan over all threads of the row writes their positions in order.  A
// long row is shared by a cluster of up to eight CTAs that add their histograms and
// counts through distributed shared memory.
//
// copy_kernel moves the rows: bound by HBM (each kept row read and written once).
//
// What it takes: 8 x 8 rows of up to 16384 keys to 4096, D = 128, 50.3 to 50.5 us a call (265 MB,
// 5.3 TB/s, 78% of the copy rate; D = 64 32.7, 4.1 TB/s): 36 the copy, 9 the choice on 64 of the
// SMs -- latency of the dependent passes, 32 warps each with barriers between; one prompt of 131072
// keys to 16384 36.9 to 38.0 us (140 MB; D = 64 29): 19 and 15, of which three digits' exchanges
// through distributed shared memory are half.  The masses are read once while a row fits the threads.
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

struct Args {
    int Hkv, S, keep, cap, n_first, n_recent;
    const int32_t* kv_len;
    const float* mass;            // [B, Hkv, S]
    int32_t* len_out;             // [B]
    float* mass_out;              // [B, Hkv, cap]
    int32_t* kept;                // [B, Hkv, keep]
};

// Unsigned integers in the order of the numbers; -0 is 0, NaN stands below all (1).
// 0: no key that competes; kSure: stays in any case (above every number).
constexpr uint32_t kSure = 0xffffffffu;
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 1;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
    return r;
}

// Sum over the threads up to and including this one.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* s_warp) {
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
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    return x + (warp ? before : 0);
}

// A thread's keys at .. at + PER - 1 in their order; `at` is on 16 bytes and may be below 0.
template <int PER>
__device__ __forceinline__ void load(uint32_t (&u)[PER], const float* mass, int at, int n, int lo, int hi) {
    float x[PER];
#pragma unroll
    for (int s = 0; s < PER; s += 4) {
        if (at + s >= 0 && at + s + 3 < n) {
            const float4 y = *reinterpret_cast<const float4*>(mass + at + s);
            x[s] = y.x, x[s + 1] = y.y, x[s + 2] = y.z, x[s + 3] = y.w;
        } else {
#pragma unroll
            for (int e = s; e < s + 4; ++e) x[e] = at + e >= 0 && at + e < n ? mass[at + e] : 0.f;
        }
    }
#pragma unroll
    for (int s = 0; s < PER; ++s) u[s] = ordered(x[s]);
    if (at < lo || at + PER > hi) {
#pragma unroll
        for (int s = 0; s < PER; ++s)
            if (at + s < lo || at + s >= hi) u[s] = 0;
    }
}
// The keys that stay in any case, once the others have been counted.
template <int PER>
__device__ __forceinline__ void mark(uint32_t (&u)[PER], int at, int n, int lo, int hi) {
    if (at < lo || at + PER > hi) {
#pragma unroll
        for (int s = 0; s < PER; ++s) {
            const int j = at + s;
            if (j >= 0 && j < n && (j < lo || j >= hi)) u[s] = kSure;
        }
    }
}

struct CopyArgs {
    int Hkv, S, keep, log_u;      // 16-byte units of a row: 2^log_u
    const int32_t* kv_len;
    const int32_t* kept;
    const uint4 *k, *v;
    uint4 *k_out, *v_out;
    int64_t in_sb, in_ss, in_sh, out_sb, out_ss, out_sh;   // units
};

// Rows from(r) -> r of a (sequence, head)'s keys and values, r0 <= r < r1, by the CTA.
template <typename From>
__device__ __forceinline__ void copy_rows(const CopyArgs& c, int b, int g, int r0, int r1, From from) {
    constexpr int kAhead = 4;
    const int units = r1 << c.log_u;
    for (int y = (r0 << c.log_u) + threadIdx.x; y < units; y += kAhead * kThreads) {
        uint4 k[kAhead], v[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int x = y + e * kThreads;
            if (x >= units) break;
            const int64_t at = b * c.in_sb + from(x >> c.log_u) * c.in_ss + g * c.in_sh + (x & ((1 << c.log_u) - 1));
            k[e] = c.k[at];
            v[e] = c.v[at];
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int x = y + e * kThreads;
            if (x >= units) break;
            const int64_t at = b * c.out_sb + (x >> c.log_u) * c.out_ss + g * c.out_sh + (x & ((1 << c.log_u) - 1));
            c.k_out[at] = k[e];
            c.v_out[at] = v[e];
        }
    }
}

// MOVE: the rows are moved as well, those of each chunk behind its choice (one CTA per row).
template <int LOG_C, int PER, bool MOVE>
__global__ void __launch_bounds__(kThreads, 1)
select_kernel(const Args a, const CopyArgs copy) {
    constexpr int C = 1 << LOG_C;
    static_assert(!MOVE || C == 1, "one CTA per row");
    // Digits of 11 bits; where CTAs share a row, of 8, for all of them read all histograms (131072 keys: 9 bits the same,
    // 10 bits 1.3 us more; one CTA with 12 bits 0.6 us more).  One histogram per CTA: equal digits of a warp are added up
    // by the shared memory, copies of it only share its banks (8 of them: 2 us more).  A pass counts in one while it
    // clears the next one's; the one before may still be read by other CTAs.
    constexpr int kBits = C == 1 ? 11 : 8, kBins = 1 << kBits, kBufs = C == 1 ? 2 : 3;
    __shared__ union {
        uint32_t hist[kBufs][kBins];
        uint16_t list[kThreads * PER];       // what stays of a chunk
    } sm;
    __shared__ uint32_t s_scan[kWarps], s_count[2], s_found[3];
    const int rank = blockIdx.x % C, row = blockIdx.x / C, b = row / a.Hkv;
    const int tid = threadIdx.x, lane = tid % 32;
    wait_for_previous_kernel();
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
        if constexpr (MOVE) copy_rows(copy, b, row - b * a.Hkv, 0, n, [](int r) -> int64_t { return r; });
        return;
    }
    const int lo = a.n_first, hi = n - a.n_recent;      // the keys that compete
    // Rows of more than C * kThreads * PER keys are read in chunks of that many, again in each pass.
    constexpr int chunk = C * kThreads * PER;
    const int shift = (int)(reinterpret_cast<uintptr_t>(mass) / 4 % 4);
    const int from = (rank * kThreads + tid) * PER - shift, chunks = (n + shift + chunk - 1) / chunk;
    uint32_t u[PER];
    load(u, mass, from, n, lo, hi);
    // What stays is above T, or equal to it and among the first E of those: the digits of T, from above.
    uint32_t T = kSure - 1, E = a.keep - a.n_first - a.n_recent;
    int at = from;
    if (E > 0) {
        T = 0;
        for (int i = tid; i < kBins; i += kThreads) sm.hist[0][i] = 0;
        __syncthreads();
#pragma unroll 1
        for (int pass = 0, top = 32; top > 0; ++pass) {
            const int low = max(top - kBits, 0);
            uint32_t* mine = sm.hist[pass % kBufs];
#pragma unroll 1
            for (int ch = 0; ch < chunks; ++ch) {
                if (chunks > 1) load(u, mass, at = ch * chunk + from, n, lo, hi);
                if (pass == 0) {
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        if (u[s]) atomicAdd(&mine[u[s] >> (32 - kBits)], 1u);
                } else {
                    const uint32_t high = T >> top, digit = (1u << (top - low)) - 1;
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        if (u[s] >> top == high) atomicAdd(&mine[u[s] >> low & digit], 1u);
                }
            }
            for (int i = tid; i < kBins; i += kThreads) sm.hist[(pass + 1) % kBufs][i] = 0;
            __syncwarp();
            if (C > 1) cluster_sync();
            else __syncthreads();
            // the bin that holds the E-th one from above, and how many of it stay
            constexpr int kEach = kBins > kThreads ? kBins / kThreads : 1;      // bins of a thread, in falling order
            uint32_t c[kEach], sum = 0;
            const int bin = kBins - 1 - kEach * tid;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                c[e] = 0;
                if (bin < 0) continue;
                if constexpr (C == 1) {
                    c[e] = mine[bin - e];
                } else {
                    uint32_t part[C];
#pragma unroll
                    for (int r = 0; r < C; ++r) part[r] = ld_cluster_u32(&mine[bin - e], r);
#pragma unroll
                    for (int r = 0; r < C; ++r) c[e] += part[r];
                }
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e) sum += c[e];
            uint32_t before = block_scan(sum, s_scan) - sum;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (before < E && before + c[e] >= E) {
                    s_found[0] = bin - e;
                    s_found[1] = E - before;
                    s_found[2] = c[e];
                }
                before += c[e];
            }
            __syncthreads();
            T |= s_found[0] << low;
            E = s_found[1];
            top = low;
            if (E == s_found[2]) {   // the whole bin stays: everything above its lower end
                T -= 1;
                E = 0;
                break;
            }
        }
    }
    // Positions: what is above T (upper half of a count) and equal to it (lower half) before a key; both below 2^16 in a CTA.
    uint32_t base_s = 0, base_e = 0;                 // in the chunks before
#pragma unroll 1
    for (int ch = 0; ch < chunks; ++ch) {
        if (chunks > 1) load(u, mass, at = ch * chunk + from, n, lo, hi);
        mark(u, at, n, lo, hi);
        uint32_t mine = 0;
#pragma unroll
        for (int s = 0; s < PER; ++s) mine += u[s] > T ? 1u << 16 : u[s] == T ? 1u : 0u;
        const uint32_t upto = block_scan(mine, s_scan);
        if (tid == kThreads - 1) s_count[ch & 1] = upto;
        __syncwarp();
        if (C > 1) cluster_sync();
        else __syncthreads();
        uint32_t cta_s = base_s, cta_e = base_e, own = s_count[ch & 1];    // before this CTA's keys; its counts
        if constexpr (C > 1) {
            const uint32_t theirs = ld_cluster_u32(&s_count[ch & 1], lane % C);      // all at once
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const uint32_t c = __shfl_sync(0xffffffffu, theirs, r);
                if (r < rank) cta_s += c >> 16, cta_e += c & 0xffffu;
                base_s += c >> 16, base_e += c & 0xffffu;
            }
        } else {
            base_s += own >> 16, base_e += own & 0xffffu;
        }
        const int r0 = cta_s + min(cta_e, E), r1 = cta_s + (own >> 16) + min(cta_e + (own & 0xffffu), E);
        uint32_t at_s = cta_s + ((upto - mine) >> 16), at_e = cta_e + ((upto - mine) & 0xffffu);
        if (mine) {
#pragma unroll
            for (int s = 0; s < PER; ++s) {
                const bool sure = u[s] > T, equal = u[s] == T;
                if (sure || (equal && at_e < E)) sm.list[at_s + min(at_e, E) - r0] = (uint16_t)(tid * PER + s);
                at_s += sure;
                at_e += equal;
            }
        }
        __syncthreads();
        const int first = at - tid * PER;
        for (int r = r0 + tid; r < r1; r += kThreads) {
            const int j = first + sm.list[r - r0];
            kept[r] = j;
            mass_out[r] = mass[j];
        }
        if constexpr (MOVE) copy_rows(copy, b, row - b * a.Hkv, r0, r1, [&](int r) -> int64_t { return first + sm.list[r - r0]; });
        if (chunks > 1) __syncthreads();
    }
    __syncwarp();
    if (C > 1) cluster_sync();       // no CTA leaves while another one may still read its counts
}

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

// Rows of up to this many 16-byte units (keys; the values as many) are moved by the CTA that chose them: one launch.
// GPU time in one launch and in two: 2048 units a row, 8 rows of 501 keys 7.0 and 7.2 us, 256 rows of 4000 14.4 and
// 15.1; 4096 units 9.0 and 8.2, 17.8 and 18.9; 8192 units, 8 rows of 4000 11.6 and 8.2, 256 of them 30.4 and 31.3.
constexpr int kMoveUnits = 4096;

dfa_status cache_evict(const EvictProblem& p, const void* k, const void* v, const int32_t* kv_len, const float* mass,
                       void* k_out, void* v_out, int32_t* len_out, float* mass_out, int32_t* kept, cudaStream_t s) {
    const Args a{p.Hkv, p.S, p.keep, p.cap, p.n_first, p.n_recent, kv_len, mass, len_out, mass_out, kept};
    const int rows = p.B * p.Hkv;
    // A row to a CTA while its threads hold the keys, GPU time with the copy: 8 x 8 rows of up to 16384 keys 50.1 us, by
    // two CTAs each 53.7, by eight 95 (their barriers and 3.5 times as many CTAs as SMs); 8 rows of 16384 12.7 and 17.3.
    // Longer rows by as many as hold them: 8 rows of 32768 by one 25.3 (chunks), by two 17.6, by eight 19.4; of 131072 by
    // one 83, by four 50, by eight 34.7.  Four keys a thread while that holds a row: 501 keys, two launches 7.5, 16 a
    // thread 11.2.
    int log_c = 0;
    while ((1 << log_c) < kMaxCluster && p.S > (kThreads * 16 << log_c)) ++log_c;
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
    const int most = std::min(p.keep, p.S);
    const bool small = p.S <= kThreads * 4, move = small && (most << c.log_u) <= kMoveUnits;
    using Kernel = void (*)(const Args, const CopyArgs);
    const Kernel kernels[] = {small ? (move ? Kernel(select_kernel<0, 4, true>) : Kernel(select_kernel<0, 4, false>)) : Kernel(select_kernel<0, 16, false>),
                              select_kernel<1, 16, false>, select_kernel<2, 16, false>, select_kernel<3, 16, false>};
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1u << log_c;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)rows << log_c);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1 + (log_c > 0);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernels[log_c], a, c);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "evict launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_EVICT);
    if (move) return DFA_OK;
    const int64_t units = (int64_t)most * p.Hkv << c.log_u;
    const int blocks = (int)((units + kCopyThreads * kCopyAhead - 1) / (kCopyThreads * kCopyAhead));
    e = launch_overlapped(copy_kernel, dim3((unsigned)(p.B * blocks)), kCopyThreads, 0, s, c, blocks);
    if (e != cudaSuccess) return fail(DFA_ERR_CUDA, "evict copy launch: %s", cudaGetErrorString(e));
    count_launch(DFA_KERNEL_EVICT);
    return DFA_OK;
}

}  // namespace dfa
