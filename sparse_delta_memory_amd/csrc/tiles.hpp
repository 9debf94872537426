// What the chunked kernels over dense states share (the gated linear recurrence and the gated delta rule): operands
// of matrix products and their parts, tiles in LDS and how they are filled, a chunk's gate factors.
#pragma once

#include <hip/hip_runtime.h>

#include "mixer_device.hpp"

namespace sdm {
namespace {

constexpr int kL = 64;           // tokens of a chunk
constexpr float kGateMin = -10000.0f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One operand of a matrix-product tile: 8 inner indexes at the lane's row (or column).
template <typename T>
struct Frag;
template <>
struct Frag<bf16_t> {
    u32x4 w;
};
template <>
struct Frag<float> {
    float v[8];
};

// c += a b^T over 32 inner indexes: rows of a (lane % 16) down, rows of b across.
__device__ __forceinline__ void mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f32x4& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.w), __builtin_bit_cast(bf16x8, b.w), c, 0, 0, 0);
}
__device__ __forceinline__ void mma(const Frag<float>& a, const Frag<float>& b, f32x4& c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
}

// f x, but 0 where the factor f is 0, whatever x: a reset, or a decay past the smallest float32, leaves nothing of values
// that are not finite either. One instruction, the multiplication in which 0 times anything is 0.
extern "C" __device__ float sdm_decayed(float f, float x) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ f32x4 decayed(float f, f32x4 x) {
    return f32x4{sdm_decayed(f, x[0]), sdm_decayed(f, x[1]), sdm_decayed(f, x[2]), sdm_decayed(f, x[3])};
}
// f x + y in the same sense.
__device__ __forceinline__ float decay_add(float f, float x, float y) { return f == 0.0f ? y : fmaf(f, x, y); }

// The parts of 8 float32 values: NS bfloat16 words by truncation, or the floats themselves.
template <typename T, int NS>
struct Parts {
    Frag<T> p[NS];
};
template <int NS>
__device__ __forceinline__ void cut(const float (&x)[8], Parts<bf16_t, NS>& o) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e)   // the high halves of two words
            o.p[s].w[e] = __builtin_amdgcn_perm(__float_as_uint(r[2 * e + 1]), __float_as_uint(r[2 * e]), 0x07060302u);
        if (s + 1 < NS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] -= __uint_as_float(__float_as_uint(r[e]) & 0xFFFF0000u);
        }
    }
}
template <int NS>
__device__ __forceinline__ void cut(const float (&x)[8], Parts<float, NS>& o) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o.p[0].v[e] = x[e];
}
template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 1 : 3;

// LDS tiles [64][W]: the 16-byte piece c of a row lies at piece c ^ twist(row), which spreads 16 rows' reads of one piece
// and 4 rows' transposed reads over the banks. Counted, a row read still takes 8 cycles (4 at best: the lanes LDS serves
// together are not 16 in a row) and a transposed one 4. Twists from four row bits that bring them to 4 and 2 were measured
// too: the addresses' instructions cost more than that saves (8 x 4096 tokens x 16 heads of 128, forward 219 against 216 us,
// backward 749 against 730).
template <typename T, int W>
__device__ __forceinline__ int twist(int row) {
    constexpr int pieces = W * static_cast<int>(sizeof(T)) / 16;
    if constexpr (pieces == 8) return 4 * ((row >> 1) & 1) + ((row >> 2) & 3);
    else if constexpr (sizeof(T) == 2) return 4 * (row & 3) + ((row >> 2) & 3);
    else return row & (pieces == 32 ? 7 : 15);
}
template <typename T, int W>
__device__ __forceinline__ char* piece(T* tile, int row, int c) {
    return reinterpret_cast<char*>(tile) + row * (W * static_cast<int>(sizeof(T))) + ((c ^ twist<T, W>(row)) << 4);
}

// 8 consecutive columns 32 kb + 8 quarter + .. of one row.
template <int W>
__device__ __forceinline__ Frag<bf16_t> row_frag(bf16_t* tile, int row, int kb, int quarter) {
    return Frag<bf16_t>{*reinterpret_cast<const u32x4*>(piece<bf16_t, W>(tile, row, 4 * kb + quarter))};
}
template <int W>
__device__ __forceinline__ Frag<float> row_frag(float* tile, int row, int kb, int quarter) {
    Frag<float> f;
    const f32x4 a = *reinterpret_cast<const f32x4*>(piece<float, W>(tile, row, 8 * kb + 2 * quarter));
    const f32x4 b = *reinterpret_cast<const f32x4*>(piece<float, W>(tile, row, 8 * kb + 2 * quarter + 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) { f.v[e] = a[e]; f.v[4 + e] = b[e]; }
    return f;
}

// Tokens 32 jb + 4 quarter + {0..3} and 32 jb + 16 + 4 quarter + {0..3} at one column per lane: column
// base + i (STEP 4), or base + 8 (i / 4) + i % 4 (STEP 8: the state's row order), i = lane % 16.
template <int W, int STEP>
__device__ __forceinline__ Frag<bf16_t> col_frag(bf16_t* tile, int jb, int base, int i, int quarter) {
    Frag<bf16_t> f;
    const int col = base + STEP * (i & 3);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int row = 32 * jb + 16 * s + 4 * quarter + (i >> 2);
        char* p = piece<bf16_t, W>(tile, row, col >> 3) + 2 * (col & 7);
        const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
        const u32x2 w = __builtin_bit_cast(u32x2, r);
        f.w[2 * s] = w[0];
        f.w[2 * s + 1] = w[1];
    }
    return f;
}
template <int W, int STEP>
__device__ __forceinline__ Frag<float> col_frag(float* tile, int jb, int base, int i, int quarter) {
    Frag<float> f;
    const int col = STEP == 4 ? base + i : base + 8 * (i >> 2) + (i & 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int row = 32 * jb + 16 * (e >> 2) + 4 * quarter + (e & 3);
        f.v[e] = *reinterpret_cast<const float*>(piece<float, W>(tile, row, col >> 2) + 4 * (col & 3));
    }
    return f;
}

__device__ __forceinline__ void widen8(const Frag<bf16_t>& f, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(f.w[e] << 16);
        x[2 * e + 1] = __uint_as_float(f.w[e] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen8(const Frag<float>& f, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f.v[e];
}

// Whether the wave's two operands hold an infinity or NaN (seen by some lane): 0 times a finite value is 0. For bfloat16 a
// matrix product does the multiplications (4 vector instructions beside it; comparing the exponents takes 20).
__device__ __forceinline__ bool not_finite(const Frag<bf16_t>& f, const Frag<bf16_t>& g) {
    f32x4 c = {0, 0, 0, 0};
    const Frag<bf16_t> zero{u32x4{0, 0, 0, 0}};
    mma(f, zero, c);
    mma(g, zero, c);
    const float x = (c[0] + c[1]) + (c[2] + c[3]);
    return x != x;
}
__device__ __forceinline__ bool not_finite(const Frag<float>& f, const Frag<float>& g) {
    float x = 0.0f;   // 0 times a finite value is 0
#pragma unroll
    for (int e = 0; e < 8; ++e) x = fmaf(f.v[e], 0.0f, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x = fmaf(g.v[e], 0.0f, x);
    return x != x;
}
// The values with 0 in place of those that are not finite, and 1 in their places with 0 elsewhere.
__device__ __forceinline__ void split_finite(const Frag<bf16_t>& f, Frag<bf16_t>& finite, Frag<bf16_t>& mark) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool lo = (f.w[e] & 0x7F80u) == 0x7F80u, hi = (f.w[e] & 0x7F800000u) == 0x7F800000u;
        finite.w[e] = (lo ? 0u : f.w[e] & 0xFFFFu) | (hi ? 0u : f.w[e] & 0xFFFF0000u);
        mark.w[e] = (lo ? 0x3F80u : 0u) | (hi ? 0x3F800000u : 0u);
    }
}
__device__ __forceinline__ void split_finite(const Frag<float>& f, Frag<float>& finite, Frag<float>& mark) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool bad = (__float_as_uint(f.v[e]) & 0x7F800000u) == 0x7F800000u;
        finite.v[e] = bad ? 0.0f : f.v[e];
        mark.v[e] = bad ? 1.0f : 0.0f;
    }
}

// Rows of one operand: element (b, t, h / per) at p + ..., `width` of them contiguous.
struct Rows {
    const void* p;
    int64_t b, t, h;
    int width, per;
    int wide;      // 16-byte loads: aligned rows of whole 16-byte pieces that do not overlap, 64 of them within 2^30 bytes
};

// Four consecutive elements of a row; those from `left` on are 0.
template <typename T>
struct Four;
template <>
struct Four<bf16_t> {
    u32x2 w;
    __device__ __forceinline__ void load(const bf16_t* p, int left, int wide) {
        w = u32x2{0, 0};
        if (left <= 0) return;
        if (wide) {   // rows of whole 16-byte pieces: left is a multiple of 4
            w = *reinterpret_cast<const u32x2*>(p);
            return;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < left) w[r >> 1] |= static_cast<uint32_t>(p[r].bits) << (16 * (r & 1));
        }
    }
    __device__ __forceinline__ float at(int r) const { return __uint_as_float(r & 1 ? w[r >> 1] & 0xFFFF0000u : w[r >> 1] << 16); }
};
template <>
struct Four<float> {
    f32x4 w;
    __device__ __forceinline__ void load(const float* p, int left, int wide) {
        w = f32x4{0, 0, 0, 0};
        if (left <= 0) return;
        if (wide) {
            w = *reinterpret_cast<const f32x4*>(p);
            return;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < left) w[r] = p[r];
        }
    }
    __device__ __forceinline__ float at(int r) const { return w[r]; }
};

// A chunk's tile of one operand, global memory to LDS. Rows that take wide loads go there directly, 16
// bytes per lane, no registers between (the lanes' pieces lie in lane order in LDS, so the lane reads the
// piece that belongs there by the twist); others element by element. Zero past the row's length and the
// head's width: the loads' buffer descriptor ends with the chunk's last token, and what lies outside its
// range reads as zero. The range check covers the register offset, which holds all of it.
// 16 bytes per lane from the buffer's byte offset `off` to LDS at `to` (the wave's, uniform) + 16 lane. The wait for it is
// tile_barrier's: the compiler, which knows the builtin of this instruction but not whether a later LDS read meets its bytes,
// would wait for it before every such read. It has no result register, so nothing is in flight towards one.
__device__ __forceinline__ void to_lds16(u32x4 rsrc, char* to, uint32_t off) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass has no such registers
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)to));
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rsrc) : "memory", "m0");
#endif
}
__device__ __forceinline__ u32x4 buffer_of(const void* base, int bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32) & 0xFFFFu, static_cast<uint32_t>(bytes), 0x00027000u};
}

template <typename T, int W, int THREADS>
struct Stage {
    static constexpr int kPieces = W * static_cast<int>(sizeof(T)) / 16;       // per row
    static constexpr int kEach = kL * kPieces / THREADS;                        // per thread
    static constexpr int kElems = 16 / static_cast<int>(sizeof(T));
    static constexpr int kStep = THREADS / kPieces;                             // rows between a thread's pieces
    static_assert(kStep % 16 == 0 || (kStep % 8 == 0 && kPieces == 32), "a thread's rows have one twist");
    uint32_t off;      // of the thread's first piece from the chunk's first row, bytes; out of any range past the head's width

    __device__ __forceinline__ void init(const Rows& s) { init(s, static_cast<int>(threadIdx.x)); }
    __device__ __forceinline__ void init(const Rows& s, int tid) {
        const int row = tid / kPieces;
        const int c = (tid % kPieces) ^ twist<T, W>(row);
        off = c * kElems < s.width ? (static_cast<uint32_t>(row) * static_cast<uint32_t>(s.t) * static_cast<uint32_t>(sizeof(T)) + c * 16) : 0xC0000000u;
    }
    // base: the chunk's first row; left: its tokens. Complete after a wait for vector memory and a barrier.
    __device__ __forceinline__ void fill(const Rows& s, const T* base, int left, T* tile, int wave, int tid) const {
        const int tok = left < kL ? left : kL;
        if (s.wide) {
            const int bytes = ((tok - 1) * static_cast<int>(s.t) + s.width) * static_cast<int>(sizeof(T));
            const u32x4 rsrc = buffer_of(base, bytes);
            const uint32_t step = static_cast<uint32_t>(kStep * static_cast<int>(s.t) * static_cast<int>(sizeof(T)));
            char* to = reinterpret_cast<char*>(tile) + wave * (kWave * 16);
#pragma unroll
            for (int n = 0; n < kEach; ++n) to_lds16(rsrc, to + n * THREADS * 16, off + n * step);
            return;
        }
        for (int at = tid; at < kL * W; at += THREADS) {
            const int t = at / W, col = at % W;
            T v = narrow<T>(0.0f);
            if (t < tok && col < s.width) v = base[static_cast<int64_t>(t) * s.t + col];
            *reinterpret_cast<T*>(piece<T, W>(tile, t, col / kElems) + (col % kElems) * static_cast<int>(sizeof(T))) = v;
        }
    }
};

// Barrier after which every wave's tile loads are in LDS.
__device__ __forceinline__ void tile_barrier() { __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A chunk's gate factors (one wave computes them, a token per lane). Sums are in units of log 2.
struct Gates {
    float lhi[kL], llo[kL];   // the sum of gates since the start of the token's tile of 16, in two parts
    float up[kL];             // exp(G_i - G at the start of its tile)
    float down[kL];           // exp(G at the end of its tile - G_j)
    float f[kL], u[kL];       // factors of S^T x_i and of y_j z_j^T
    float tau[16];            // [it][jt]: exp(G at the start of tile max - G at the end of tile min)
    float all;                // exp(G_L)
    int gone;                 // whether a token's u is 0
    int odd;                  // set with the scores: whether one of a token with itself is not finite
    double sum;               // G_L
};

// x of the lane DPP names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_d(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xF, false));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xF, false));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// Inclusive sums over the wave's lanes: row shifts by 1, 2, 4, 8, then the row ends (row_bcast 15, 31).
__device__ __forceinline__ double scan_d(double x) {
    x += dpp_d<0x111, 0xF>(x);
    x += dpp_d<0x112, 0xF>(x);
    x += dpp_d<0x114, 0xF>(x);
    x += dpp_d<0x118, 0xF>(x);
    x += dpp_d<0x142, 0xA>(x);
    x += dpp_d<0x143, 0xC>(x);
    return x;
}
// x of one lane, the same for all.
__device__ __forceinline__ double uniform_d(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), lane));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// 2^x of a float64 exponent: the rounded part through the hardware exp2 (its results below 2^-126 are 0), the
// remainder to first order.
__device__ __forceinline__ float exp2_of(double x) {
    const float hi = static_cast<float>(x);
    const float lo = static_cast<float>(x - hi);
    const float e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e, lo * 0.69314718056f, e);
}

constexpr double kLog2E = 1.4426950408889634074;

template <bool REV>
__device__ __forceinline__ void gate_factors(float g, float m_o, float m_s, Gates& o, int l) {
    const double G = scan_d((g < kGateMin ? kGateMin : g) * kLog2E);   // NaN stays
    const double e0 = uniform_d(G, 15), e1 = uniform_d(G, 31), e2 = uniform_d(G, 47), last = uniform_d(G, 63);   // ends of the tiles of 16
    const int tile = l >> 4;
    const double before = tile == 1 ? e0 : tile == 2 ? e1 : e2, end = tile == 0 ? e0 : tile == 1 ? e1 : tile == 2 ? e2 : last;
    const double local = tile > 0 ? G - before : G;
    const float hi = static_cast<float>(local);
    o.lhi[l] = hi;
    o.llo[l] = static_cast<float>(local - hi);
    o.up[l] = exp2_of(local);
    o.down[l] = exp2_of(end - G);
    const float fwd = exp2_of(G), bwd = exp2_of(last - G);
    o.f[l] = (REV ? bwd : fwd) * m_o;
    const float u = (REV ? fwd : bwd) * m_s;
    o.u[l] = u;
    const bool gone = __ballot(u == 0.0f) != 0;
    if (l < 16) {   // tile it and jt: from the end of the lower to the start of the higher
        const int it = l >> 2, jt = l & 3, hi_t = it > jt ? it : jt, lo_t = it > jt ? jt : it;
        const double a = hi_t == 1 ? e0 : hi_t == 2 ? e1 : e2, b = lo_t == 0 ? e0 : lo_t == 1 ? e1 : e2;
        o.tau[l] = it == jt ? 1.0f : exp2_of(a - b);
    }
    if (l == 0) {
        o.all = exp2_of(last);
        o.gone = gone;
        o.odd = 0;
        o.sum = last;
    }
}

// The lanes [from, to) of a wave's 64 tokens, in pieces that no reset cuts: per piece its inclusive sums of x, which start
// afresh in each. cuts: the lanes that start a piece of their own. f(piece's first lane, its end, the lane's sum).
template <typename F>
__device__ __forceinline__ void pieces(uint64_t cuts, double x, int lane, F f) {
    for (int from = 0; from < kWave;) {
        const uint64_t rest = from + 1 < kWave ? cuts >> (from + 1) << (from + 1) : 0;
        const int to = rest != 0 ? __builtin_ctzll(rest) : kWave;
        f(from, to, scan_d(lane >= from && lane < to ? x : 0.0));
        from = to;
    }
}

// exp(g) of one gate as the chunks take it: 0 below 2^-126 (the gate resets); NaN stays.
__device__ __forceinline__ float gate_factor(float g) { return exp2_of(static_cast<double>(g < kGateMin ? kGateMin : g) * kLog2E); }
__device__ __forceinline__ bool resets(float g) { return gate_factor(g) == 0.0f; }
// The same for one token. expf goes on below 2^-126, where a state that is not finite would outlive the gate that resets it in a chunk.
__device__ __forceinline__ float token_factor(float g) { return resets(g) ? 0.0f : expf(g); }

// The score operands of a chunk, computed once and shared by the waves: pair n is (it, jb), the tiles of tokens
// 16 it across and 32 jb down; its two halves are the score tiles jt = 2 jb and 2 jb + 1. Of the 16 tiles the
// 6 pairs below hold all that the direction needs (and two that are zero).
template <bool REV>
struct Pairs {
    static constexpr int kIt[6] = {REV ? 0 : 0, REV ? 0 : 1, REV ? 1 : 2, REV ? 1 : 2, REV ? 2 : 3, REV ? 3 : 3};
    static constexpr int kJb[6] = {REV ? 0 : 0, REV ? 1 : 0, REV ? 0 : 0, REV ? 1 : 1, REV ? 1 : 0, REV ? 1 : 1};
};

int padded(int d) { return d <= 64 ? 64 : 128; }

Rows rows_of(const void* p, int64_t b, int64_t t, int64_t h, int width, int per, int es) {
    const int unit = 16 / es;
    Rows r{p, b, t, h, width, per, 0};
    r.wide = reinterpret_cast<uintptr_t>(p) % 16 == 0 && b % unit == 0 && t % unit == 0 && h % unit == 0 && width % unit == 0 &&
             t >= width && t < (int64_t(1) << 30) / (kL * es);
    return r;
}
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace
}  // namespace sdm
