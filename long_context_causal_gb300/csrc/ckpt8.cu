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

// Sixteen int8 elements (one 16-byte word) times 2^e.
__device__ __forceinline__ void dequant16(const uint4& u, float sc, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int z = 0; z < 16; ++z) x[z] = s8(w[z / 4], z % 4) * sc;
}

struct Tensors {
    const void* src[4];
    void* dst[4];
    int64_t end[4];     // running count of 16-element units
};

// 16 elements of one tensor per thread; two threads make a group.
__global__ void __launch_bounds__(kThreads)
save_kernel(const Tensors t, uint8_t* __restrict__ ckpt, const Ckpt8Layout L) {
    int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool on = u < t.end[3];    // the same for both threads of a group: there is an even number of units
    if (!on) u = u & 1;              // stays for the shuffle, stores nothing
    int i = 0;
#pragma unroll
    for (int z = 0; z < 3; ++z) i += u >= t.end[z];
    const int64_t at = u - (i ? t.end[i - 1] : 0);
    const uint4* src = static_cast<const uint4*>(t.src[i]) + 2 * at;
    const uint4 a = src[0], b = src[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    // The largest magnitude as an integer: the order of the bits without the
    // sign is the order of the values, and an infinity or NaN is above all.
    uint32_t big = 0;
#pragma unroll
    for (int z = 0; z < 8; ++z) big = max(big, max(w[z] & 0x7fffu, (w[z] >> 16) & 0x7fffu));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    const uint32_t ex = big >> 7;    // biased exponent of the largest
    // e + 127 = ex - 6, at least 7
    const uint32_t code = ex == 255u ? 255u : max((int)ex - 6, 7);
    const float down = __uint_as_float((254u - code) << 23);   // 2^-e (unused for code 255)
    uint32_t o[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        uint32_t r = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint32_t v = w[2 * z + y / 2];
            const int m = __float2int_rn((y & 1 ? bf_hi(v) : bf_lo(v)) * down);
            r |= (uint32_t)(uint8_t)max(-127, min(127, m)) << (8 * y);
        }
        o[z] = code == 255u ? 0u : r;
    }
    if (!on) return;
    *reinterpret_cast<uint4*>(ckpt + L.data[i] + 16 * at) = make_uint4(o[0], o[1], o[2], o[3]);
    if ((at & 1) == 0) ckpt[L.exps[i] + at / 2] = (uint8_t)code;
}

__device__ __forceinline__ void restore_unit(const uint8_t* ckpt, const Ckpt8Layout& L, int i, int64_t at, uint4* dst) {
    const uint4 d = *reinterpret_cast<const uint4*>(ckpt + L.data[i] + 16 * at);
    float x[16];
    dequant16(d, exp_scale(ckpt[L.exps[i] + at / 2]), x);
    dst[0] = make_uint4(pack_exact(x[0], x[1]), pack_exact(x[2], x[3]), pack_exact(x[4], x[5]), pack_exact(x[6], x[7]));
    dst[1] = make_uint4(pack_exact(x[8], x[9]), pack_exact(x[10], x[11]), pack_exact(x[12], x[13]),
                        pack_exact(x[14], x[15]));
}

__global__ void __launch_bounds__(kThreads)
restore_kernel(const Tensors t, const uint8_t* __restrict__ ckpt, const Ckpt8Layout L) {
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= t.end[3]) return;
    int i = 0;
#pragma unroll
    for (int z = 0; z < 3; ++z) i += u >= t.end[z];
    const int64_t at = u - (i ? t.end[i - 1] : 0);
    restore_unit(ckpt, L, i, at, static_cast<uint4*>(t.dst[i]) + 2 * at);
}

// ---------------------------------------------------------------- before the backward
struct PrepArgs {
    int H, S, S_pad;
    int64_t row_blocks;              // blocks that take query rows; the rest restore q, k, v
    const __nv_bfloat16* O;
    const uint4* dO;
    const float* lse;
    float p_shift;
    float *nlse2, *delta, *dq_acc;
    const uint8_t* ckpt;
};

// D / 16 threads take one row (b, i, h) of the padded range i < S_pad: Delta =
// <dO, O> and p_shift - lse log2 e (so that a score's base-2 exponent is
// one fused multiply-add), and the row's zeros in the head-major accumulator.
template <int D, bool CKPT>
__global__ void __launch_bounds__(kThreads)
prep_kernel(const PrepArgs a, const Tensors t, const Ckpt8Layout L, int64_t n_rows) {
    constexpr int T = D / 16;        // threads per row
    if (CKPT && blockIdx.x >= a.row_blocks) {
        const int64_t u = ((int64_t)blockIdx.x - a.row_blocks) * kThreads + threadIdx.x;
        if (u >= t.end[2]) return;
        const int i = (u >= t.end[0]) + (u >= t.end[1]);
        const int64_t at = u - (i ? t.end[i - 1] : 0);
        restore_unit(a.ckpt, L, i, at, static_cast<uint4*>(t.dst[i]) + 2 * at);
        return;
    }
    const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / T;
    const int part = threadIdx.x % T;
    const bool on = row < n_rows;    // threads past the last row stay for the shuffles
    const int h = (int)(row % a.H);
    const int64_t bi = row / a.H;
    const int i = (int)(bi % a.S_pad);
    const int64_t b = bi / a.S_pad, bh = b * a.H + h, dst = bh * a.S_pad + i;
    float acc = 0.f;
    const bool real = on && i < a.S;
    if (real) {
        const int64_t at = ((b * a.S + i) * a.H + h) * T + part;   // 16-element unit
        float o[16];
        if constexpr (CKPT) {
            dequant16(*reinterpret_cast<const uint4*>(a.ckpt + L.data[3] + 16 * at),
                      exp_scale(a.ckpt[L.exps[3] + at / 2]), o);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(a.O) + 2 * at;
            const uint4 x = p[0], y = p[1];
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int z = 0; z < 8; ++z) {
                o[2 * z] = bf_lo(w[z]);
                o[2 * z + 1] = bf_hi(w[z]);
            }
        }
        const uint4 x = a.dO[2 * at], y = a.dO[2 * at + 1];
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            acc = fmaf(o[2 * z], bf_lo(w[z]), acc);
            acc = fmaf(o[2 * z + 1], bf_hi(w[z]), acc);
        }
        float4* zero = reinterpret_cast<float4*>(a.dq_acc + (bh * a.S + i) * D);
#pragma unroll
        for (int z = 0; z < 4; ++z) zero[z * T + part] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int o = T / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (on && part == 0) {
        a.delta[dst] = acc;
        a.nlse2[dst] = real ? fmaf(a.lse[bh * a.S + i], -1.4426950408889634f, a.p_shift) : 0.f;
    }
}

// ---------------------------------------------------------------- after it
__device__ __forceinline__ uint4 pack8(const float4& a, const float4& b, float c) {
    __nv_bfloat162 r[4] = {__floats2bfloat162_rn(c * a.x, c * a.y), __floats2bfloat162_rn(c * a.z, c * a.w),
                           __floats2bfloat162_rn(c * b.x, c * b.y), __floats2bfloat162_rn(c * b.z, c * b.w)};
    return *reinterpret_cast<uint4*>(r);
}

// dQ: eight elements of [B, S, H, D] per thread from the head-major
// accumulator.  The blocks behind those sum key tile 0's slabs, eight elements
// per thread, in the pieces' order.
template <int D>
__global__ void __launch_bounds__(kThreads)
finish_kernel(int H, int Hkv, int S, int rows, int n_pieces, float scale, int64_t dq_blocks, int64_t n8,
              const float* __restrict__ acc, const float* __restrict__ slabs, uint4* __restrict__ dQ,
              uint4* __restrict__ dK, uint4* __restrict__ dV) {
    constexpr int T = D / 8;
    if (blockIdx.x < dq_blocks) {
        const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        if (x >= n8) return;
        const int part = (int)(x % T);
        const int64_t r = x / T;
        const int h = (int)(r % H);
        const int64_t bs = r / H;
        const int s = (int)(bs % S);
        const int64_t b = bs / S;
        const float4* src = reinterpret_cast<const float4*>(acc + ((b * H + h) * S + s) * D) + 2 * part;
        dQ[x] = pack8(src[0], src[1], scale);
        return;
    }
    const int64_t x = ((int64_t)blockIdx.x - dq_blocks) * kThreads + threadIdx.x;   // (row, dK or dV, key, part)
    if (x >= (int64_t)rows * 2 * 128 * T) return;
    const int row = (int)(x / (2 * 128 * T)), in = (int)(x % (2 * 128 * T));
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
    for (int p = 0; p < n_pieces; ++p) {
        const float4* src = reinterpret_cast<const float4*>(slabs + ((int64_t)p * rows + row) * 2 * 128 * D) + 2 * in;
        const float4 u = src[0], w = src[1];
        a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
        c.x += w.x; c.y += w.y; c.z += w.z; c.w += w.w;
    }
    const int b = row / Hkv, g = row % Hkv, key = in / T % 128;   // S > 128 whenever there are pieces
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

dfa_status launch_ckpt8_save(const Ckpt8Layout& L, const void* const src[4], void* ckpt, cudaStream_t s) {
    Tensors t{};
    int64_t n = 0;
    for (int i = 0; i < 4; ++i) {
        t.src[i] = src[i];
        t.end[i] = n += L.n[i] / 16;
    }
    save_kernel<<<(unsigned)blocks_for(n), kThreads, 0, s>>>(t, static_cast<uint8_t*>(ckpt), L);
    return launched("checkpoint save");
}

dfa_status launch_ckpt8_restore(const Ckpt8Layout& L, const void* ckpt, void* const dst[4], cudaStream_t s) {
    Tensors t{};
    int64_t n = 0;
    for (int i = 0; i < 4; ++i) {
        t.dst[i] = dst[i];
        t.end[i] = n += L.n[i] / 16;
    }
    restore_kernel<<<(unsigned)blocks_for(n), kThreads, 0, s>>>(t, static_cast<const uint8_t*>(ckpt), L);
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
    const int64_t n_rows = (int64_t)p.B * S_pad * p.H;
    a.row_blocks = blocks_for(n_rows * (p.D / 16));
    Tensors t{};
    int64_t n = 0;
    if (ckpt)
        for (int i = 0; i < 3; ++i) {
            t.dst[i] = qkv[i];
            t.end[i] = n += L->n[i] / 16;
        }
    const Ckpt8Layout none{};
    const unsigned grid = (unsigned)(a.row_blocks + blocks_for(n));
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
    const int64_t n8 = (int64_t)p.B * p.S * p.H * p.D / 8, dq_blocks = blocks_for(n8);
    const int rows = p.B * p.Hkv;
    const float scale = p.scale / (1 << p.p_shift);
    const int64_t extra = plan.n_pieces > 1 ? blocks_for((int64_t)rows * 2 * 128 * p.D / 8) : 0;
    const unsigned grid = (unsigned)(dq_blocks + extra);
    if (p.D == 128)
        finish_kernel<128><<<grid, kThreads, 0, s>>>(p.H, p.Hkv, p.S, rows, plan.n_pieces, scale, dq_blocks, n8, dq_acc,
                                                     slabs, (uint4*)dQ, (uint4*)dK, (uint4*)dV);
    else
        finish_kernel<64><<<grid, kThreads, 0, s>>>(p.H, p.Hkv, p.S, rows, plan.n_pieces, scale, dq_blocks, n8, dq_acc,
                                                    slabs, (uint4*)dQ, (uint4*)dK, (uint4*)dV);
    return launched("windowed backward finish");
}

SinkBwdPlan sink_bwd_plan(const SinkProblem& p) {
    SinkBwdPlan x{};
    const int64_t rows = (int64_t)p.B * p.Hkv;
    x.n_q = (p.S + 127) / 128;
    x.piece_len = x.n_q;
    x.n_pieces = 1;
    if (p.n_sink > 0) {
        // Pieces about as long as an ordinary key tile's range, so that the snake's
        // order by cost holds; at least 8 tiles, which pay for the piece's K and V
        // loads and its 128 KB slab, and at most 64 pieces.
        const int wlen = std::min(x.n_q, (p.window + 126) / 128 + 1);
        const int len = std::max(std::max(wlen, 8), (x.n_q + 63) / 64);
        if (len < x.n_q) {
            x.piece_len = len;
            x.n_pieces = (x.n_q + len - 1) / len;
        }
    }
    x.n_items = rows * (x.n_q + x.n_pieces - 1);
    return x;
}

}  // namespace dfa
