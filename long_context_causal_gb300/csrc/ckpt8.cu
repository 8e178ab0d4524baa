// ckpt8.cu -- 8-bit attention checkpoints, and the streaming passes around the
// windowed backward.
//
// What a layer's attention saves for its backward is q, k, v, O and lse
// (DISTFLASHATTN §3.3: the backward reuses them and never re-runs the forward).
// Here q, k, v and O are held in 8 bits: each group of 32 elements of the head
// dimension shares an exponent e = max(floor(log2 max|x|) - 6, -120), and an
// element is the integer m nearest to x / 2^e (ties to even, |m| <= 127).  It
// stands for m 2^e.  Why this form and not 8-bit floats with a scale: the
// rounding error is 2^(e-1) at most, 0.4-0.8% of the group's largest element,
// against 3-6% of each element with three mantissa bits; and m 2^e has seven
// significant bits, so it is a bf16 number exactly -- the backward's tensor
// cores see what the checkpoint holds, with no second rounding.  8.25 bits per
// element.  The exponent byte is e + 127; 255 marks a group that held an
// infinity or NaN, all of which stands for NaN.
//
// Every kernel here is bound by HBM: 16-byte accesses, each byte moved once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "sink_bwd.cuh"

namespace dfa {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 32;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Two fp32 values that are bf16 numbers -> packed, `lo` in the low half (exact).
__device__ __forceinline__ uint32_t pack_exact(float lo, float hi) {
    return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}
__device__ __forceinline__ float exp_scale(uint32_t code) {   // 2^e of an exponent byte
    return code == 255u ? __uint_as_float(0x7fff0000u) : __uint_as_float(code << 23);
}
__device__ __forceinline__ float s8(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Eight int8 elements times 2^e.
__device__ __forceinline__ void dequant8(const uint2& u, float sc, float* x) {
#pragma unroll
    for (int z = 0; z < 8; ++z) x[z] = s8(z < 4 ? u.x : u.y, z & 3) * sc;
}

// A unit is eight elements: 16 bytes of bf16, 8 of the payload; four units make
// a group.  A block takes kPer * kThreads consecutive units of one tensor, each
// thread kPer of them kThreads apart, all loaded before the first is used: a
// warp's accesses are contiguous on both sides, and 2048 threads of an SM have
// 64 bytes each in flight.
constexpr int kPer = 4;
struct Tensors {
    const void* src[4];
    void* dst[4];
    int64_t units[4];
    int end[4];         // running count of the tensors' blocks
};
__device__ __forceinline__ int tensor_of(const Tensors& t, int block, int n) {
    int i = 0;
    for (int z = 0; z + 1 < n; ++z) i += block >= t.end[z];
    return i;
}

__global__ void __launch_bounds__(kThreads)
save_kernel(const __grid_constant__ Tensors t, uint8_t* __restrict__ ckpt, const __grid_constant__ Ckpt8Layout L) {
    const int i = tensor_of(t, blockIdx.x, 4);
    const int64_t u0 = (int64_t)(blockIdx.x - (i ? t.end[i - 1] : 0)) * (kPer * kThreads) + threadIdx.x, n = t.units[i];
    const uint4* src = static_cast<const uint4*>(t.src[i]);
    uint8_t* data = ckpt + L.data[i];
    uint8_t* exps = ckpt + L.exps[i];
    uint4 in[kPer];
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
        const int64_t u = u0 + y * kThreads;
        in[y] = u < n ? src[u] : make_uint4(0, 0, 0, 0);   // whole groups: n is a multiple of 4
    }
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
        const int64_t u = u0 + y * kThreads;
        const uint32_t w[4] = {in[y].x, in[y].y, in[y].z, in[y].w};
        // The largest magnitude as an integer: the order of the bits without the
        // sign is the order of the values, and an infinity or NaN is above all.
        uint32_t big = 0;
#pragma unroll
        for (int z = 0; z < 4; ++z) big = max(big, max(w[z] & 0x7fffu, (w[z] >> 16) & 0x7fffu));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const uint32_t ex = big >> 7;    // biased exponent of the largest
        // e + 127 = ex - 6, at least 7
        const uint32_t code = ex == 255u ? 255u : max((int)ex - 6, 7);
        const float down = __uint_as_float((254u - code) << 23);   // 2^-e (unused for code 255)
        uint32_t o[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t v = w[2 * z + e / 2];
                const int m = __float2int_rn((e & 1 ? bf_hi(v) : bf_lo(v)) * down);
                r |= (uint32_t)(uint8_t)max(-127, min(127, m)) << (8 * e);
            }
            o[z] = code == 255u ? 0u : r;
        }
        if (u < n) {
            *reinterpret_cast<uint2*>(data + 8 * u) = make_uint2(o[0], o[1]);
            if ((u & 3) == 0) exps[u / 4] = (uint8_t)code;
        }
    }
}

// kPer units of a thread from the checkpoint's section i to dst.
__device__ __forceinline__ void restore_units(const uint8_t* ckpt, const Ckpt8Layout& L, int i, int64_t u0, int64_t n,
                                              uint4* dst) {
    const uint2* data = reinterpret_cast<const uint2*>(ckpt + L.data[i]);
    const uint8_t* exps = ckpt + L.exps[i];
    uint2 in[kPer];
    uint32_t code[kPer];
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
        const int64_t u = min(u0 + y * kThreads, n - 1);
        in[y] = data[u];
        code[y] = exps[u / 4];
    }
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
        const int64_t u = u0 + y * kThreads;
        float x[8];
        dequant8(in[y], exp_scale(code[y]), x);
        if (u < n)
            dst[u] = make_uint4(pack_exact(x[0], x[1]), pack_exact(x[2], x[3]), pack_exact(x[4], x[5]),
                                pack_exact(x[6], x[7]));
    }
}

__global__ void __launch_bounds__(kThreads)
restore_kernel(const __grid_constant__ Tensors t, const uint8_t* __restrict__ ckpt,
               const __grid_constant__ Ckpt8Layout L) {
    const int i = tensor_of(t, blockIdx.x, 4);
    restore_units(ckpt, L, i, (int64_t)(blockIdx.x - (i ? t.end[i - 1] : 0)) * (kPer * kThreads) + threadIdx.x, t.units[i],
                  static_cast<uint4*>(t.dst[i]));
}

// ---------------------------------------------------------------- before the backward
struct PrepArgs {
    int H, S, S_pad;
    int row_blocks;                  // blocks that take query rows; the rest restore q, k, v
    const __nv_bfloat16* O;
    const uint4* dO;
    const float* lse;
    float p_shift;
    float *nlse2, *delta, *dq_acc;
    const uint8_t* ckpt;
};

// D / 8 threads take one row (b, i, h) of the padded range i < S_pad: Delta =
// <dO, O> and p_shift - lse log2 e (so that a score's base-2 exponent is
// one fused multiply-add), and the row's zeros in the head-major accumulator.
// The blocks behind those restore q, k and v.
template <int D, bool CKPT>
__global__ void __launch_bounds__(kThreads)
prep_kernel(const __grid_constant__ PrepArgs a, const __grid_constant__ Tensors t, const __grid_constant__ Ckpt8Layout L,
            int n_rows) {
    constexpr int T = D / 8;         // threads per row
    if (CKPT && (int)blockIdx.x >= a.row_blocks) {
        const int block = (int)blockIdx.x - a.row_blocks, i = tensor_of(t, block, 3);
        restore_units(a.ckpt, L, i, (int64_t)(block - (i ? t.end[i - 1] : 0)) * (kPer * kThreads) + threadIdx.x, t.units[i],
                      static_cast<uint4*>(t.dst[i]));
        return;
    }
    constexpr int R = 2;             // rows per thread, loaded before the first is used
    const int part = threadIdx.x % T;
    // rows are counted in 32 bits: 2^31 rows of 64 elements would not fit in the memory
    const uint32_t row0 = blockIdx.x * (uint32_t)(R * kThreads / T) + threadIdx.x / T;
    uint4 od[R], dd[R];
    uint32_t code[R];
    int64_t at[R], dst[R], src[R];
    bool on[R], real[R];
#pragma unroll
    for (int y = 0; y < R; ++y) {
        const uint32_t row = row0 + y * (kThreads / T);
        on[y] = row < (uint32_t)n_rows;
        const uint32_t h = row % a.H, bi = row / a.H;
        const int i = (int)(bi % a.S_pad);
        const int64_t b = bi / a.S_pad, bh = b * a.H + h;
        real[y] = on[y] && i < a.S;
        dst[y] = bh * a.S_pad + i;
        src[y] = bh * a.S + i;
        at[y] = ((b * a.S + i) * a.H + h) * T + part;   // unit
        if (real[y]) {
            dd[y] = a.dO[at[y]];
            if constexpr (CKPT) {
                const uint2 u = reinterpret_cast<const uint2*>(a.ckpt + L.data[3])[at[y]];
                od[y].x = u.x;
                od[y].y = u.y;
                code[y] = a.ckpt[L.exps[3] + at[y] / 4];
            } else {
                od[y] = reinterpret_cast<const uint4*>(a.O)[at[y]];
            }
        }
    }
#pragma unroll
    for (int y = 0; y < R; ++y) {
        float acc = 0.f;
        if (real[y]) {
            float o[8];
            if constexpr (CKPT) {
                dequant8(make_uint2(od[y].x, od[y].y), exp_scale(code[y]), o);
            } else {
                const uint32_t w[4] = {od[y].x, od[y].y, od[y].z, od[y].w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    o[2 * z] = bf_lo(w[z]);
                    o[2 * z + 1] = bf_hi(w[z]);
                }
            }
            const uint32_t w[4] = {dd[y].x, dd[y].y, dd[y].z, dd[y].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                acc = fmaf(o[2 * z], bf_lo(w[z]), acc);
                acc = fmaf(o[2 * z + 1], bf_hi(w[z]), acc);
            }
            float4* zero = reinterpret_cast<float4*>(a.dq_acc + src[y] * D);
            zero[part] = make_float4(0.f, 0.f, 0.f, 0.f);
            zero[T + part] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int o = T / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (on[y] && part == 0) {
            a.delta[dst[y]] = acc;
            a.nlse2[dst[y]] = real[y] ? fmaf(a.lse[src[y]], -1.4426950408889634f, a.p_shift) : 0.f;
        }
    }
}

// ---------------------------------------------------------------- after it
__device__ __forceinline__ uint4 pack8(const float4& a, const float4& b, float c) {
    __nv_bfloat162 r[4] = {__floats2bfloat162_rn(c * a.x, c * a.y), __floats2bfloat162_rn(c * a.z, c * a.w),
                           __floats2bfloat162_rn(c * b.x, c * b.y), __floats2bfloat162_rn(c * b.z, c * b.w)};
    return *reinterpret_cast<uint4*>(r);
}

// dQ: eight elements of [B, S, H, D] per thread from the head-major
// accumulator.  The blocks behind those sum the slabs of the key tiles whose
// lists were cut, eight elements per thread, in the pieces' order.
template <int D>
__global__ void __launch_bounds__(kThreads)
finish_kernel(int H, int Hkv, int S, const __grid_constant__ SinkBwdPlan p, float scale, int dq_blocks, int n_rows,
              const float* __restrict__ acc, const float* __restrict__ slabs, uint4* __restrict__ dQ,
              uint4* __restrict__ dK, uint4* __restrict__ dV) {
    constexpr int T = D / 8;
    ptx::wait_for_previous_kernel();
    if ((int)blockIdx.x < dq_blocks) {
        constexpr int R = 2;         // rows per thread, loaded before the first is used
        const int part = threadIdx.x % T;
        const uint32_t row0 = blockIdx.x * (uint32_t)(R * kThreads / T) + threadIdx.x / T;
        float4 a[R], b[R];
#pragma unroll
        for (int y = 0; y < R; ++y) {
            const uint32_t row = min(row0 + y * (kThreads / T), (uint32_t)n_rows - 1);
            const uint32_t h = row % H, bs = row / H, s = bs % S;
            const int64_t bb = bs / S;
            const float4* src = reinterpret_cast<const float4*>(acc + ((bb * H + h) * S + s) * D) + 2 * part;
            a[y] = src[0];
            b[y] = src[1];
        }
#pragma unroll
        for (int y = 0; y < R; ++y) {
            const uint32_t row = row0 + y * (kThreads / T);
            if (row < (uint32_t)n_rows) dQ[(int64_t)row * T + part] = pack8(a[y], b[y], scale);
        }
        return;
    }
    // (key tile, row, dK or dV, key, eight elements); the tensor and tile are the block's
    constexpr int kBlocks = 2 * 128 * T / kThreads;
    const int block = (int)blockIdx.x - dq_blocks, in = block % kBlocks * kThreads + threadIdx.x;
    const int row = block / kBlocks % p.rows, t = block / kBlocks / p.rows;
    const int first = p.cut_all ? p.first[t] : 0, pieces = p.cut_all ? p.first[t + 1] - first : p.pieces0;
    const int key = t * 128 + in / T % 128;
    if (pieces == 1 || key >= S) return;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
#pragma unroll 4
    for (int z = first; z < first + pieces; ++z) {
        const float4* src = reinterpret_cast<const float4*>(slabs + ((int64_t)z * p.rows + row) * 2 * 128 * D) + 2 * in;
        const float4 u = src[0], w = src[1];
        a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
        c.x += w.x; c.y += w.y; c.z += w.z; c.w += w.w;
    }
    const int b = row / Hkv, g = row % Hkv;
    (in < 128 * T ? dK : dV)[(((int64_t)b * S + key) * Hkv + g) * T + in % T] = pack8(a, c, 1.f);
}

dfa_status launched(const char* what) {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DFA_OK : fail(DFA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

int64_t blocks_for(int64_t n) { return (n + kThreads - 1) / kThreads; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

Ckpt8Layout ckpt8_layout(int B, int H, int Hkv, int S, int D) {
    Ckpt8Layout L{};
    const int heads[4] = {H, Hkv, Hkv, H};
    size_t off = 0;
    for (int i = 0; i < 4; ++i) {
        L.n[i] = (int64_t)B * S * heads[i] * D;
        L.data[i] = off;
        off = align256(off + (size_t)L.n[i]);
    }
    for (int i = 0; i < 4; ++i) {
        L.exps[i] = off;
        off = align256(off + (size_t)(L.n[i] / kGroup));
    }
    L.total = off;
    return L;
}

namespace {
// Blocks for the first n tensors of a checkpoint; returns how many there are.
int split_blocks(const Ckpt8Layout& L, int n, Tensors* t) {
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) {
        t->units[i] = L.n[i] / 8;
        blocks += (t->units[i] + kPer * kThreads - 1) / (kPer * kThreads);
        t->end[i] = (int)blocks;     // B * S * H * D < 2^44 / 8192 elements by the callers' checks
    }
    return (int)blocks;
}
}  // namespace

dfa_status launch_ckpt8_save(const Ckpt8Layout& L, const void* const src[4], void* ckpt, cudaStream_t s) {
    Tensors t{};
    for (int i = 0; i < 4; ++i) t.src[i] = src[i];
    const int blocks = split_blocks(L, 4, &t);
    save_kernel<<<blocks, kThreads, 0, s>>>(t, static_cast<uint8_t*>(ckpt), L);
    return launched("checkpoint save");
}

dfa_status launch_ckpt8_restore(const Ckpt8Layout& L, const void* ckpt, void* const dst[4], cudaStream_t s) {
    Tensors t{};
    for (int i = 0; i < 4; ++i) t.dst[i] = dst[i];
    const int blocks = split_blocks(L, 4, &t);
    restore_kernel<<<blocks, kThreads, 0, s>>>(t, static_cast<const uint8_t*>(ckpt), L);
    return launched("checkpoint restore");
}

dfa_status launch_sink_prep(const SinkProblem& p, int S_pad, const void* O, const void* dO, const float* lse,
                            float* nlse2, float* delta, float* dq_acc, const void* ckpt, const Ckpt8Layout* L,
                            void* const qkv[3], cudaStream_t s) {
    PrepArgs a{};
    a.H = p.H; a.S = p.S; a.S_pad = S_pad;
    a.O = static_cast<const __nv_bfloat16*>(O);
    a.dO = static_cast<const uint4*>(dO);
    a.lse = lse; a.p_shift = (float)p.p_shift; a.nlse2 = nlse2; a.delta = delta; a.dq_acc = dq_acc;
    a.ckpt = static_cast<const uint8_t*>(ckpt);
    const int n_rows = p.B * S_pad * p.H, per = 2 * kThreads / (p.D / 8);
    a.row_blocks = (n_rows - 1) / per + 1;
    Tensors t{};
    int more = 0;
    if (ckpt) {
        for (int i = 0; i < 3; ++i) t.dst[i] = qkv[i];
        more = split_blocks(*L, 3, &t);
    }
    const unsigned grid = (unsigned)(a.row_blocks + more);
    const Ckpt8Layout none{};
    const Ckpt8Layout& l = ckpt ? *L : none;
    if (p.D == 128) {
        if (ckpt) prep_kernel<128, true><<<grid, kThreads, 0, s>>>(a, t, l, n_rows);
        else prep_kernel<128, false><<<grid, kThreads, 0, s>>>(a, t, l, n_rows);
    } else {
        if (ckpt) prep_kernel<64, true><<<grid, kThreads, 0, s>>>(a, t, l, n_rows);
        else prep_kernel<64, false><<<grid, kThreads, 0, s>>>(a, t, l, n_rows);
    }
    return launched("windowed backward preparation");
}

dfa_status launch_sink_finish(const SinkProblem& p, const SinkBwdPlan& plan, const float* dq_acc, const float* slabs,
                              void* dQ, void* dK, void* dV, cudaStream_t s) {
    const int n_rows = p.B * p.S * p.H, per = 2 * kThreads / (p.D / 8);
    const int dq_blocks = (n_rows - 1) / per + 1;
    const float scale = p.scale / (1 << p.p_shift);
    const int tiles = plan.cut_all ? plan.n_q : plan.pieces0 > 1;
    const unsigned grid = (unsigned)(dq_blocks + tiles * plan.rows * (2 * 128 * (p.D / 8) / kThreads));
    auto kern = p.D == 128 ? finish_kernel<128> : finish_kernel<64>;
    const cudaError_t e = launch_overlapped(kern, (int)grid, kThreads, 0, s, p.H, p.Hkv, p.S, plan, scale, dq_blocks, n_rows,
                                            dq_acc, slabs, static_cast<uint4*>(dQ), static_cast<uint4*>(dK),
                                            static_cast<uint4*>(dV));
    return e == cudaSuccess ? DFA_OK : fail(DFA_ERR_CUDA, "windowed backward finish launch: %s", cudaGetErrorString(e));
}

// The time of a plan is estimated in query tiles (about 2.4 us): an item costs
// its tiles (FINE ones kFine each; 1.6 and 1.9 give the same times to 1%, 2.2 up to 7% more) and kItem more (loads, pipeline fill,
// epilogue); a CTA has up to four items of one size in whole rounds, and more
// or mixed ones within half an item of the mean; each slab, written and read
// at the memory's rate, costs the GPU 0.013 of a tile on top of one for the
// summing.
constexpr double kFine = 1.9, kItem = 2.5;

SinkBwdPlan sink_bwd_plan(const SinkProblem& p, int sms) {
    SinkBwdPlan x{};
    sms = std::max(sms, 2);          // key tile 0 has CTAs of its own
    x.rows = p.B * p.Hkv;
    x.G = p.H / p.Hkv;
    x.n_q = (p.S + 127) / 128;
    x.window_tiles = std::min(x.n_q, (p.window + 126) / 128 + 1);   // a tile's last key is seen by window - 1 more queries
    x.n_sink = p.n_sink;
    if (x.rows == 0 || x.n_q == 0) return x;                        // an empty batch: no items
    const int longest = x.G * sink_range(x, 0), ordinary = x.G * x.window_tiles;
    const int tail = std::min(x.n_q, x.window_tiles);               // the last tiles' ranges shrink to 1
    const double rest = (double)x.rows * x.G *                      // tiles of the lists behind the first
                        ((double)(x.n_q - tail) * x.window_tiles + tail * (tail + 1.) / 2 - x.window_tiles);
    const double tiles = rest + (double)x.rows * longest;

    auto spread = [&](int64_t n, int ctas, int len, double work, bool even) {
        if (n == 0) return 0.0;
        if (n <= ctas || (even && n <= 4 * (int64_t)ctas)) return (double)((n + ctas - 1) / ctas) * (len + kItem);
        return (work + kItem * n) / ctas + 0.5 * len;
    };
    // Time of n items of up to len tiles, the first n0 of them key tile 0's, and the CTAs for those.
    auto time_of = [&](int64_t n, int64_t n0, int len, int len0, bool even, int* fine_ctas) {
        *fine_ctas = 0;
        if (!p.fine) return spread(n, sms, len, tiles, even);
        const double one = kFine * len0 + kItem;
        if (n <= sms || n == n0) {
            *fine_ctas = (int)std::min<int64_t>(n0, sms);
            return std::max((double)((n0 + *fine_ctas - 1) / *fine_ctas) * one, n > n0 ? len + kItem : 0.0);
        }
        // Key tile 0 in r rounds of f CTAs, from the most CTAs down until those are what takes longest.
        double least = 1e30;
        for (int f = sms - 1; f > 0; --f) {
            const int64_t r = (n0 + f - 1) / f;
            f = (int)((n0 + r - 1) / r);
            const double t = std::max(r * one, spread(n - n0, sms - f, len, rest, even));
            if (t < least) least = t, *fine_ctas = f;
            if (r * one >= t) break;
        }
        return least;
    };

    auto slab_time = [](int64_t n) { return n ? 1 + 0.013 * n : 0.0; };

    // Key tile 0 alone cut: pieces about as long as an ordinary key tile's list, or
    // shorter where that ends earlier; 8 tiles pay for the piece's K and V loads and
    // its slab.
    x.piece = longest;
    x.pieces0 = 1;
    double uncut = time_of((int64_t)x.rows * x.n_q, x.rows, std::max(ordinary, 1), longest, false, &x.fine_ctas);
    for (int k = 0; k < 4 && p.n_sink > 0; ++k) {
        const int len = std::max(std::max(x.G * std::max(x.window_tiles, 8) >> k, 8), (longest + 255) / 256);
        const int64_t n0 = (longest + len - 1) / len;
        if (len >= longest) continue;
        int f;
        const double t = time_of(x.rows * (x.n_q - 1 + n0), x.rows * n0, std::max(ordinary, 1), len, false, &f) +
                         slab_time(x.rows * n0);
        if (t < uncut) uncut = t, x.piece = len, x.pieces0 = (int)n0, x.fine_ctas = f;
    }
    x.n_items = x.rows * (x.n_q - 1 + x.pieces0);
    x.n_slabs = x.pieces0 > 1 ? x.pieces0 * x.rows : 0;
    // Cut every list while the SMs' even share is less than a few of them.
    if (x.n_q <= kPlanTiles && longest > 1 && tiles < 4.0 * sms * std::max(x.piece, ordinary)) {
        double least = 0.95 * uncut;
        int best = 0, fine = 0;
        for (int len = 2; len < longest; len += 1 + longest / 64) {
            const int64_t n0 = (int64_t)x.rows * ((longest + len - 1) / len);
            int64_t n = 0;
            for (int t = std::max(x.n_q - tail, 1); t < x.n_q; ++t) n += (x.G * (x.n_q - t) + len - 1) / len;
            n += (int64_t)std::max(x.n_q - tail - 1, 0) * ((ordinary + len - 1) / len);
            n = n * x.rows + n0;
            if (n > (int64_t)sms * kPlanItems) continue;
            int f;
            const double t = time_of(n, n0, len, len, true, &f) + slab_time(n);
            if (t < least) least = t, best = len, fine = f;
        }
        if (best > 0) {
            x.cut_all = 1;
            x.piece = best;
            x.fine_ctas = fine;
            int n = 0;
            for (int t = 0; t < x.n_q; ++t) {
                x.first[t] = (uint16_t)n;
                n += (x.G * sink_range(x, t) + best - 1) / best;
            }
            x.first[x.n_q] = (uint16_t)n;
            x.pieces0 = x.first[1];
            x.n_items = x.n_slabs = n * x.rows;
        }
    }
    x.grid = std::min(sms, x.n_items);
    return x;
}

}  // namespace dfa
