// The gated linear recurrence with a dense state per head, forward and backward:
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = scale S_t^T q_t.
//
// In chunks of L = 64 tokens, with G_i the sum of the chunk's gates up to i and S the state before it,
//     o_i = scale (sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j + exp(G_i) S^T q_i),
//     S'  = exp(G_L) S + sum_j exp(G_L - G_j) k_j v_j^T,
// which are matrix products. One kernel body computes
//     out_i = m_p sum_j D_ij (x_i . y_j) z_j + m_o f_i S^T x_i,     S <- exp(G_L) S + m_s sum_j u_j y_j z_j^T
// over the chunks of a stream's head, forwards (D_ij for j <= i, f = exp(G_i), u = exp(G_L - G_j)) or
// backwards in time (j >= i, f and u exchanged), and it is every pass there is:
//     o  : x = q,   y = k,   z = v,    forwards on S;         dq : x = d_o, y = v,   z = k,  forwards on S^T;
//     dk : x = v,   y = d_o, z = q,    backwards on R^T;      dv : x = k,   y = q,   z = d_o, backwards on R,
// R the gradient of the state. A gate scales all that reaches t or a later token from before t, so
//     dg_t = sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <S_T, R_T>;
// q . dq and k . dk come from the float32 results before they are rounded, and the sums start afresh at
// every segment (below) from <S, R> there, so that what cancels is never longer than a segment.
//
// Layout. A block of four waves owns one (stream, head, segment); each wave owns VD/4 columns of z, out
// and the state, and keeps its part of the state in registers over all chunks as the accumulators of
// 16 x 16 matrix-product tiles (rows: the key dimension). The same registers, cut into bfloat16 parts, are
// directly the other operand of x S, and a score tile y x^T is directly the other operand of the product
// with z, because the accumulator layout (four rows at one column per lane) equals an operand's (some
// inner indexes at one row): the inner index is only permuted, and the matching operand is read in the
// same permutation. So neither scores nor state pass through LDS. The scores are computed by every wave
// (40 of its 200 to 270 matrix instructions per chunk), which costs less than a barrier and the trip
// through LDS. Tiles of x, y and z are staged in LDS with 16-byte pieces permuted per row such that row
// reads and transposed reads (ds_read_tr) are both free of bank conflicts; the next chunk's global loads
// are in flight during a chunk's products.
//
// Numbers. Products of bfloat16 inputs are exact; a float32 factor (decayed score, state, decayed z) is
// cut into bfloat16 parts by truncation and multiplied part by part: three parts hold all 24 bits. The
// state's update and everything a dg sums takes three; o and dv are rounded to bfloat16 in the end, so
// their scores and the state's use take two (16 bits, a 2^-16 relative error beside the 2^-9 of the
// result). float32 inputs go through the float32 matrix instructions. Gates are summed in float64 per
// chunk (one wave, one token per lane) and only differences of a chunk's sums are rounded to float32, so
// neither long rows nor a reset (a gate of -infinity counts as -10000) cost digits.
//
// Segments. With few streams and heads the time axis is cut: a first kernel sums each segment's own
// state, a second one walks the segments' states in order, and the main kernel starts every segment from
// the state before it.
#include <hip/hip_runtime.h>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"

namespace sdm {
namespace {

constexpr int kL = 64;           // tokens of a chunk
constexpr int kGlrThreads = 256;
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
template <typename T, int NS>
constexpr int kParts = sizeof(T) == 4 ? 1 : NS;

// LDS tiles [64][W]: the 16-byte piece c of a row lies at piece c ^ twist(row).
template <typename T, int W>
__device__ __forceinline__ int twist(int row) {
    constexpr int pieces = W * static_cast<int>(sizeof(T)) / 16;
    if constexpr (pieces == 8) return 4 * ((row >> 1) & 1) + ((row >> 2) & 3);
    else if constexpr (sizeof(T) == 2) return 4 * (row & 3) + ((row >> 2) & 3);
    else return row & 15;
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

// Rows of one operand: element (b, t, h / per) at p + ..., `width` of them contiguous.
struct Rows {
    const void* p;
    int64_t b, t, h;
    int width, per;
    int wide;      // 16-byte loads: aligned rows of whole 16-byte pieces
};

struct GlrPass {
    Rows x, y, z, w;          // w: the rows the results are dotted with (dot != NULL)
    const float* g;
    int64_t g_b, g_t, g_h;
    const int32_t* lens;
    int B, T, H;
    int nseg, seg;            // segments, and tokens of each (a multiple of 64)
    float m_p, m_o, m_s;
    // The state before a segment (in the pass's direction), [B H, nseg] states from s_in (NULL: zero), element (key, value)
    // at key * s_k + value * s_v; the state after the last segment to s_out, [B H] states (NULL: not kept).
    const float* s_in;
    float* s_out;
    int64_t s_k, s_v;
    // out rows: [B, T, H] with strides, narrowed to the input type, or float32 (fold)
    void* out;
    int64_t o_b, o_t, o_h;
    int out_wide;             // 4-element stores
    int out_f32;
    float* dot;               // [B H, T] row dots of w and the result
    // <state after the segment, the gradient of it>: [B H, nseg], from r_end (indexed like s_in: the gradient at the segment's end)
    const float* r_end;
    int64_t r_k, r_v;
    float* cross;
    // state-only pass
    float* seg_state;         // [B H, nseg] states [s_k, s_v]
    float* seg_decay;         // [B H, nseg]
};

__device__ __forceinline__ int row_len(const GlrPass& p, int b) {
    const int n = p.lens != nullptr ? p.lens[b] : p.T;
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// A chunk's tile in flight: 16-byte pieces per thread, zero past the row's length and the head's width.
template <typename T, int W>
struct Stage {
    static constexpr int kPieces = W * static_cast<int>(sizeof(T)) / 16;       // per row
    static constexpr int kEach = kL * kPieces / kGlrThreads;                    // per thread
    static constexpr int kElems = 16 / static_cast<int>(sizeof(T));
    u32x4 r[kEach];

    __device__ __forceinline__ void load(const Rows& s, const T* base, int t0, int len) {
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const int at = n * kGlrThreads + static_cast<int>(threadIdx.x), row = at / kPieces, c = at % kPieces;
            r[n] = u32x4{0, 0, 0, 0};
            const int left = s.width - c * kElems;
            if (t0 + row < len && left > 0) {
                const T* p = base + static_cast<int64_t>(t0 + row) * s.t + c * kElems;
                if (s.wide) {
                    r[n] = *reinterpret_cast<const u32x4*>(p);
                } else {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < kElems; ++e) {
                        if (e < left) {
                            if constexpr (sizeof(T) == 2) w[e / 2] |= static_cast<uint32_t>(p[e].bits) << (16 * (e & 1));
                            else w[e] = __float_as_uint(p[e]);
                        }
                    }
                    r[n] = u32x4{w[0], w[1], w[2], w[3]};
                }
            }
        }
    }
    __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
            const int at = n * kGlrThreads + static_cast<int>(threadIdx.x), row = at / kPieces, c = at % kPieces;
            *reinterpret_cast<u32x4*>(piece<T, W>(tile, row, c)) = r[n];
        }
    }
};

// A chunk's gate factors (one wave computes them, a token per lane).
struct Gates {
    float lhi[kL], llo[kL];   // the sum of gates since the start of the token's tile of 16, in two parts
    float up[kL];             // exp(G_i - G at the start of its tile)
    float down[kL];           // exp(G at the end of its tile - G_j)
    float f[kL], u[kL];       // factors of S^T x_i and of y_j z_j^T
    float tau[16];            // [it][jt]: exp(G at the start of tile max - G at the end of tile min)
    float all;                // exp(G_L)
    double sum;               // G_L
};

__device__ __forceinline__ double shfl_up_d(double x, int n) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const int src = (static_cast<int>(lane_id()) - n) << 2;
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(src, static_cast<int>(u)));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(src, static_cast<int>(u >> 32)));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double lane_d(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(lane << 2, static_cast<int>(u)));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(lane << 2, static_cast<int>(u >> 32)));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

template <bool REV>
__device__ __forceinline__ void gate_factors(float g, float m_o, float m_s, Gates& o) {
    const int l = static_cast<int>(lane_id());
    double G = g < kGateMin ? kGateMin : g;   // NaN stays
#pragma unroll
    for (int n = 1; n < kL; n *= 2) {
        const double below = shfl_up_d(G, n);
        if (l >= n) G += below;
    }
    const int tile = l & ~15;
    const double before = lane_d(G, (tile + 63) & 63), end = lane_d(G, tile + 15), last = lane_d(G, kL - 1);
    const double local = tile > 0 ? G - before : G;
    const float hi = static_cast<float>(local);
    o.lhi[l] = hi;
    o.llo[l] = static_cast<float>(local - hi);
    o.up[l] = expf(hi);
    o.down[l] = expf(static_cast<float>(end - G));
    const float fwd = expf(static_cast<float>(G)), bwd = expf(static_cast<float>(last - G));
    o.f[l] = (REV ? bwd : fwd) * m_o;
    o.u[l] = (REV ? fwd : bwd) * m_s;
    {
        const int it = (l >> 2) & 3, jt = l & 3, hi_t = it > jt ? it : jt, lo_t = it > jt ? jt : it;
        const double a = lane_d(G, (16 * hi_t + 63) & 63), b = lane_d(G, 16 * lo_t + 15);   // starts of tile hi_t, end of lo_t
        if (l < 16) o.tau[l] = it == jt ? 1.0f : expf(static_cast<float>(a - b));
    }
    if (l == 0) {
        o.all = expf(static_cast<float>(last));
        o.sum = last;
    }
}

// KD, VD: padded widths of x / y and of z (64 or 128). NS: parts of scores and of the state where it meets x.
template <typename T, int KD, int VD, bool REV, bool OUT, int NS>
__global__ __launch_bounds__(kGlrThreads) void glr_kernel(GlrPass p) {
    constexpr int KB = KD / 32, KT = KD / 16, NT = VD / 64;
    constexpr int P2 = kParts<T, NS>, P3 = kParts<T, 3>;
    constexpr bool kAhead = sizeof(T) == 2;   // float32 tiles are twice as wide: no registers for a chunk in flight
    extern __shared__ __align__(16) char lds[];
    T* xt = reinterpret_cast<T*>(lds);
    T* yt = xt + (OUT ? kL * KD : 0);
    T* zt = yt + kL * KD;
    Gates& gates = *reinterpret_cast<Gates*>(zt + kL * VD);
    float* dots = reinterpret_cast<float*>(&gates + 1);   // [4][64]

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int si = blk % p.nseg, bh = blk / p.nseg, b = bh / p.H, h = bh - b * p.H;
    const int lane = static_cast<int>(lane_id()), wave = static_cast<int>(threadIdx.x) / kWave;
    const int i16 = lane & 15, qd = lane >> 4;
    const int n0 = wave * 16 * NT;   // the wave's first column
    const int len = row_len(p, b);
    const int t_lo = si * p.seg, t_hi = min(p.T, t_lo + p.seg);   // the segment's tokens
    const int live = min(len, t_hi);
    const int chunks = live > t_lo ? (live - t_lo + kL - 1) / kL : 0;

    const T* xb = OUT ? static_cast<const T*>(p.x.p) + b * p.x.b + (h / p.x.per) * p.x.h : nullptr;
    const T* yb = static_cast<const T*>(p.y.p) + b * p.y.b + (h / p.y.per) * p.y.h;
    const T* zb = static_cast<const T*>(p.z.p) + b * p.z.b + (h / p.z.per) * p.z.h;
    const float* gb = p.g + b * p.g_b + h * p.g_h;
    const int kd = p.y.width, vd = p.z.width;
    const int64_t one = static_cast<int64_t>(kd) * vd;

    // The wave's state: tile d, rows 32 (d / 2) + 8 quarter + 4 (d % 2) + r, column n0 + 16 nt + lane % 16.
    f32x4 S[KT][NT];
#pragma unroll
    for (int d = 0; d < KT; ++d) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            S[d][nt] = f32x4{0, 0, 0, 0};
            if (OUT && p.s_in != nullptr) {
                const float* s = p.s_in + (static_cast<int64_t>(bh) * p.nseg + si) * one;
                const int n = n0 + 16 * nt + i16, k0 = 32 * (d >> 1) + 8 * qd + 4 * (d & 1);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (n < vd && k0 + r < kd) S[d][nt][r] = s[(k0 + r) * p.s_k + n * p.s_v];
                }
            }
        }
    }
    double decay = 0.0;   // state-only: the sum of the segment's gates

    Stage<T, KD> sx, sy;
    Stage<T, VD> sz;
    float gate = 0.0f;
    auto fetch = [&](int c) {
        const int t0 = t_lo + c * kL;
        if (OUT) sx.load(p.x, xb, t0, live);
        sy.load(p.y, yb, t0, live);
        sz.load(p.z, zb, t0, live);
        if (wave == 0) gate = t0 + lane < live ? gb[static_cast<int64_t>(t0 + lane) * p.g_t] : 0.0f;
    };
    if (kAhead && chunks > 0) fetch(REV ? chunks - 1 : 0);

    for (int cc = 0; cc < chunks; ++cc) {
        const int c = REV ? chunks - 1 - cc : cc, t0 = t_lo + c * kL;
        if (!kAhead) fetch(c);
        if (OUT) sx.store(xt);
        sy.store(yt);
        sz.store(zt);
        if (wave == 0) gate_factors<REV>(gate, p.m_o, p.m_s, gates);
        __syncthreads();
        if (kAhead && cc + 1 < chunks) fetch(REV ? c - 1 : c + 1);

        if constexpr (OUT) {
            f32x4 O[4][NT];   // tile it: columns n0 + 16 nt + 4 quarter + r down, token 16 it + lane % 16
#pragma unroll
            for (int it = 0; it < 4; ++it) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) O[it][nt] = f32x4{0, 0, 0, 0};
            }
            // S^T x
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Parts<T, P2> sp[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float s[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) { s[r] = S[2 * kb][nt][r]; s[4 + r] = S[2 * kb + 1][nt][r]; }
                    cut(s, sp[nt]);
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const Frag<T> xf = row_frag<KD>(xt, 16 * it + i16, kb, qd);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int s = P2 - 1; s >= 0; --s) mma(sp[nt].p[s], xf, O[it][nt]);
                    }
                }
            }
            // The chunk's own tokens.
            Frag<T> zf[2][NT];
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) zf[jb][nt] = col_frag<VD, 4>(zt, jb, n0 + 16 * nt, i16, qd);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float f = gates.f[16 * it + i16];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) O[it][nt] *= f;
                Frag<T> xf[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) xf[kb] = row_frag<KD>(xt, 16 * it + i16, kb, qd);
                const float own = (REV ? gates.down : gates.up)[16 * it + i16] * p.m_p;
                const float lhi = gates.lhi[16 * it + i16], llo = gates.llo[16 * it + i16];
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    if (REV ? 2 * jb + 1 < it : 2 * jb > it) continue;
                    float s[8];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int jt = 2 * jb + half;
                        if (REV ? jt < it : jt > it) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) s[4 * half + r] = 0.0f;
                            continue;
                        }
                        f32x4 a = {0, 0, 0, 0};   // token 16 jt + 4 quarter + r down, token 16 it + lane % 16 across
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) mma(row_frag<KD>(yt, 16 * jt + i16, kb, qd), xf[kb], a);
                        if (jt == it) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int j = 4 * qd + r;
                                const float dh = lhi - gates.lhi[16 * jt + j], dl = llo - gates.llo[16 * jt + j];
                                const float e = expf(REV ? -(dh + dl) : dh + dl);
                                s[4 * half + r] = (REV ? j >= i16 : j <= i16) ? a[r] * (e * p.m_p) : 0.0f;
                            }
                        } else {
                            const float ot = own * gates.tau[4 * it + jt];
                            const f32x4 d = *reinterpret_cast<const f32x4*>(&(REV ? gates.up : gates.down)[16 * jt + 4 * qd]);
#pragma unroll
                            for (int r = 0; r < 4; ++r) s[4 * half + r] = a[r] * (ot * d[r]);
                        }
                    }
                    Parts<T, P2> sp;
                    cut(s, sp);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int k = P2 - 1; k >= 0; --k) mma(zf[jb][nt], sp.p[k], O[it][nt]);
                    }
                }
                // Out.
                const int t = t0 + 16 * it + i16;
                float dot = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int n = n0 + 16 * nt + 4 * qd;
                    if (t >= live || n >= vd) continue;
                    const f32x4 v = O[it][nt];
                    if (p.dot != nullptr) {
                        const T* w = static_cast<const T*>(p.w.p) + b * p.w.b + static_cast<int64_t>(t) * p.w.t + (h / p.w.per) * p.w.h + n;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (n + r < vd) dot = fmaf(widen(w[r]), v[r], dot);
                        }
                    }
                    const int64_t at = b * p.o_b + t * p.o_t + h * p.o_h + n;
                    if (p.out_f32 || sizeof(T) == 4) {
                        float* o = static_cast<float*>(p.out) + at;
                        if (p.out_wide) {
                            *reinterpret_cast<f32x4*>(o) = v;
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                if (n + r < vd) o[r] = v[r];
                            }
                        }
                    } else {
                        bf16_t* o = static_cast<bf16_t*>(p.out) + at;
                        if (p.out_wide) {
                            *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                if (n + r < vd) o[r] = narrow<bf16_t>(v[r]);
                            }
                        }
                    }
                }
                if (p.dot != nullptr) {
                    dot += lane_xor_f<16>(dot);
                    dot += lane_xor_f<32>(dot);
                    if (qd == 0) dots[wave * kL + 16 * it + i16] = dot;
                }
            }
        } else {
            decay += gates.sum;
        }

        // The state. (The last chunk's is only needed where someone reads it.)
        const float all = gates.all;
#pragma unroll
        for (int d = 0; d < KT; ++d) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) S[d][nt] *= all;
        }
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            Parts<T, P3> zp[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float z[8];
                widen8(col_frag<VD, 4>(zt, jb, n0 + 16 * nt, i16, qd), z);
                const f32x4 ua = *reinterpret_cast<const f32x4*>(&gates.u[32 * jb + 4 * qd]);
                const f32x4 ub = *reinterpret_cast<const f32x4*>(&gates.u[32 * jb + 16 + 4 * qd]);
#pragma unroll
                for (int r = 0; r < 4; ++r) { z[r] *= ua[r]; z[4 + r] *= ub[r]; }
                cut(z, zp[nt]);
            }
#pragma unroll
            for (int d = 0; d < KT; ++d) {
                const Frag<T> yf = col_frag<KD, 8>(yt, jb, 32 * (d >> 1) + 4 * (d & 1), i16, qd);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int s = P3 - 1; s >= 0; --s) mma(yf, zp[nt].p[s], S[d][nt]);
                }
            }
        }
        __syncthreads();   // the tiles and factors may be overwritten; the dots are complete
        if (OUT && p.dot != nullptr && threadIdx.x < kL && t0 + static_cast<int>(threadIdx.x) < live) {
            const int i = threadIdx.x;
            p.dot[static_cast<int64_t>(bh) * p.T + t0 + i] = dots[i] + dots[kL + i] + dots[2 * kL + i] + dots[3 * kL + i];
        }
    }

    if constexpr (OUT) {
        // Tokens past the row's length.
        for (int64_t e = threadIdx.x; e < static_cast<int64_t>(t_hi - max(live, t_lo)) * vd; e += kGlrThreads) {
            const int t = max(live, t_lo) + static_cast<int>(e / vd), n = static_cast<int>(e % vd);
            const int64_t at = b * p.o_b + t * p.o_t + h * p.o_h + n;
            if (p.out_f32 || sizeof(T) == 4) static_cast<float*>(p.out)[at] = 0.0f;
            else static_cast<bf16_t*>(p.out)[at] = bf16_t{0};
        }
        if (p.dot != nullptr) {
            for (int t = max(live, t_lo) + static_cast<int>(threadIdx.x); t < t_hi; t += kGlrThreads)
                p.dot[static_cast<int64_t>(bh) * p.T + t] = 0.0f;
        }
        if (p.cross != nullptr) {
            // <S, R> at the segment's end.
            const float* r_ = p.r_end != nullptr ? p.r_end + (static_cast<int64_t>(bh) * p.nseg + si) * one : nullptr;
            float x = 0.0f;
            if (r_ != nullptr) {
#pragma unroll
                for (int d = 0; d < KT; ++d) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int n = n0 + 16 * nt + i16, k0 = 32 * (d >> 1) + 8 * qd + 4 * (d & 1);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (n < vd && k0 + r < kd) x = fmaf(S[d][nt][r], r_[(k0 + r) * p.r_k + n * p.r_v], x);
                        }
                    }
                }
            }
            x = group_sum<kWave>(x);
            __syncthreads();   // the last chunk's dots have been read
            if (lane == 0) dots[wave] = x;
            __syncthreads();
            if (threadIdx.x == 0) p.cross[static_cast<int64_t>(bh) * p.nseg + si] = dots[0] + dots[1] + dots[2] + dots[3];
        }
    } else if (threadIdx.x == 0) {
        p.seg_decay[static_cast<int64_t>(bh) * p.nseg + si] = expf(static_cast<float>(decay));
    }
    float* so = OUT ? (p.s_out != nullptr && si == (REV ? 0 : p.nseg - 1) ? p.s_out + bh * one : nullptr)
                    : p.seg_state + (static_cast<int64_t>(bh) * p.nseg + si) * one;
    if (so != nullptr) {
#pragma unroll
        for (int d = 0; d < KT; ++d) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int n = n0 + 16 * nt + i16, k0 = 32 * (d >> 1) + 8 * qd + 4 * (d & 1);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (n < vd && k0 + r < kd) so[(k0 + r) * p.s_k + n * p.s_v] = S[d][nt][r];
                }
            }
        }
    }
}

// The states before every segment, in place of the segments' own: s <- start, then s_seg, s <- decay s + own.
// Backwards the last segment comes first.
template <bool REV>
__global__ __launch_bounds__(256) void glr_chain_kernel(float* states, const float* decay, const float* start, int nseg, int64_t one,
                                                        int64_t total) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= total) return;
    const int64_t bh = e / one, at = e - bh * one;
    float s = start != nullptr ? start[e] : 0.0f;
    constexpr int kU = 8;   // segments in flight
    for (int n0 = 0; n0 < nseg; n0 += kU) {
        float own[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int n = REV ? nseg - 1 - (n0 + u) : n0 + u;
            own[u] = n0 + u < nseg ? states[(bh * nseg + n) * one + at] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (n0 + u < nseg) {
                const int n = REV ? nseg - 1 - (n0 + u) : n0 + u;
                states[(bh * nseg + n) * one + at] = s;
                s = fmaf(decay[bh * nseg + n], s, own[u]);
            }
        }
    }
}

// dg: one wave per (stream, head, segment), 64 tokens at a time from the segment's end, in float64.
__global__ __launch_bounds__(256) void glr_gate_grad_kernel(const float* dq_dot, const float* dk_dot, const float* cross,
                                                            const int32_t* lens, float* dg, int T, int H, int nseg, int seg,
                                                            int64_t waves) {
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kWave;
    if (id >= waves) return;
    const int lane = static_cast<int>(lane_id());
    const int si = static_cast<int>(id % nseg);
    const int64_t bh = id / nseg, b = bh / H, h = bh - b * H;
    int len = lens != nullptr ? lens[b] : T;
    len = len < 0 ? 0 : len > T ? T : len;
    const int t_lo = si * seg, t_hi = min(T, t_lo + seg);
    double carry = cross != nullptr ? cross[bh * nseg + si] : 0.0f;
    for (int t1 = t_hi; t1 > t_lo; t1 -= kWave) {   // lane l takes token t1 - 1 - l
        const int t = t1 - 1 - lane;
        double x = t >= t_lo ? static_cast<double>(dq_dot[bh * T + t]) - static_cast<double>(dk_dot[bh * T + t]) : 0.0;
#pragma unroll
        for (int n = 1; n < kWave; n *= 2) {
            const double below = shfl_up_d(x, n);
            if (lane >= n) x += below;
        }
        if (t >= t_lo) dg[(b * T + t) * H + h] = t < len ? static_cast<float>(carry + x) : 0.0f;
        carry += lane_d(x, kWave - 1);
    }
}

// The gradients of shared heads: the sum of `per` value heads' float32 rows, in head order.
template <typename T>
__global__ __launch_bounds__(256) void glr_fold_kernel(const float* in, T* out, int64_t total, int d, int per) {
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = e / d, c = e - row * d;
        float s = 0.0f;
        for (int r = 0; r < per; ++r) s += in[(row * per + r) * d + c];
        out[e] = narrow<T>(s);
    }
}

// ------------------------------------------------------------------------------------------ one token
//
// A block owns a tile of columns of one request's head: rows of the state are dealt to its lanes in
// 16-byte pieces, read, updated and written back at once, and each column's products with q are added
// across the block in LDS in a fixed order. Bound by the state's bytes, read once and written once.
struct GlrStep {
    sdm_glr_step_io io;
    int cols;        // columns of a tile
    int tiles;
};

template <typename T, int V>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStep a) {
    const sdm_glr_step_io& io = a.io;
    __shared__ float qk[2][128];
    __shared__ float part[256 * V];
    const int tile = static_cast<int>(blockIdx.x % a.tiles);
    const int64_t bh = blockIdx.x / a.tiles;
    const int b = static_cast<int>(bh / io.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * io.H), hk = h / (io.H / io.Hk);
    const int n0 = tile * a.cols, nc = min(a.cols, io.dv - n0);
    const int64_t row = io.slots != nullptr ? io.slots[b] : b;
    T* o = static_cast<T*>(io.o) + b * io.o_b + h * io.o_h;
    const int tid = static_cast<int>(threadIdx.x);
    if (row < 0 || row >= io.rows) {
        for (int n = tid; n < nc; n += 256) o[n0 + n] = narrow<T>(0.0f);
        return;
    }
    const int per_row = (nc + V - 1) / V, groups = 256 / per_row;
    const int rg = tid / per_row, c = tid - rg * per_row, n = n0 + c * V;
    const bool on = rg < groups;
    const int64_t base = (row * io.H + h) * static_cast<int64_t>(io.dk) * io.dv + n;
    float acc[V], v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        acc[e] = 0.0f;
        v[e] = on ? widen((static_cast<const T*>(io.v) + b * io.v_b + h * io.v_h)[n + e]) : 0.0f;
    }
    if (tid < io.dk) {
        qk[0][tid] = widen((static_cast<const T*>(io.q) + b * io.q_b + hk * io.q_h)[tid]);
    } else if (tid >= 128 && tid - 128 < io.dk) {
        qk[1][tid - 128] = widen((static_cast<const T*>(io.k) + b * io.k_b + hk * io.k_h)[tid - 128]);
    }
    const float ga = expf(io.g[b * io.g_b + h * io.g_h]);
    constexpr int kU = 8;   // rows in flight
    typedef float fv __attribute__((ext_vector_type(V)));
    for (int d0 = 0; d0 < io.dk; d0 += groups * kU) {   // the same trips for every lane: the barrier below is in it
        fv s[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = d0 + rg + u * groups;
            s[u] = fv(0.0f);
            if (on && d < io.dk) s[u] = *reinterpret_cast<const fv*>(io.state + base + static_cast<int64_t>(d) * io.dv);
        }
        if (d0 == 0) __syncthreads();   // q and k are in LDS; the first rows are in flight
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = d0 + rg + u * groups;
            if (on && d < io.dk) {
                const float qd = qk[0][d], kd = qk[1][d];
                fv x = s[u];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[e] = fmaf(kd, v[e], ga * x[e]);
                    acc[e] = fmaf(qd, x[e], acc[e]);
                }
                *reinterpret_cast<fv*>(io.new_state + base + static_cast<int64_t>(d) * io.dv) = x;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (on) part[(rg * per_row + c) * V + e] = acc[e];
    }
    __syncthreads();
    if (tid < nc) {
        float s = 0.0f;
        for (int r = 0; r < groups; ++r) s += part[r * per_row * V + tid];
        o[n0 + tid] = narrow<T>(s * io.scale);
    }
}

// --------------------------------------------------------------------------------------------- plans

int padded(int d) { return d <= 64 ? 64 : 128; }

Rows rows_of(const void* p, int64_t b, int64_t t, int64_t h, int width, int per, int es) {
    const int unit = 16 / es;
    Rows r{p, b, t, h, width, per, 0};
    r.wide = reinterpret_cast<uintptr_t>(p) % 16 == 0 && b % unit == 0 && t % unit == 0 && h % unit == 0 && width % unit == 0;
    return r;
}

// Segments of the time axis: enough that streams x heads x segments are kGlrBlocks blocks, each at least
// kGlrSegMin tokens long.
constexpr int kGlrBlocks = 512;
constexpr int kGlrSegMin = 256;
struct SegPlan {
    int nseg, seg;
};
SegPlan seg_plan(int64_t bh, int T) {
    int64_t want = (kGlrBlocks + bh - 1) / bh;
    const int64_t most = T / kGlrSegMin > 1 ? T / kGlrSegMin : 1;
    if (want > most) want = most;
    const int64_t chunks = (static_cast<int64_t>(T) + kL - 1) / kL;
    const int64_t per = want > 0 ? (chunks + want - 1) / want : 1;
    SegPlan s;
    s.seg = static_cast<int>((per < 1 ? 1 : per) * kL);
    s.nseg = static_cast<int>(chunks > 0 ? (chunks * kL + s.seg - 1) / s.seg : 1);
    return s;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Byte offsets in the workspace.
struct GlrLayout {
    size_t s, sd, r, rd, dqd, dkd, cross, fq, fk, total;
};
GlrLayout glr_layout(const sdm_glr_io* io, bool backward) {
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    const SegPlan sp = seg_plan(bh, io->T);
    const size_t states = up256(static_cast<size_t>(bh) * sp.nseg * io->dk * io->dv * 4), per_seg = up256(static_cast<size_t>(bh) * sp.nseg * 4);
    const size_t rows = static_cast<size_t>(bh) * io->T;
    GlrLayout l{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up256(n);
        return o;
    };
    const bool cut = sp.nseg > 1;
    if (cut) {
        l.s = take(states);
        l.sd = take(per_seg);
    }
    if (backward) {
        if (cut) {
            l.r = take(states);
            l.rd = take(per_seg);
        }
        l.dqd = take(rows * 4);
        l.dkd = take(rows * 4);
        l.cross = take(per_seg);
        if (io->H > io->Hk) {
            l.fq = take(rows * io->dk * 4);
            l.fk = take(rows * io->dk * 4);
        }
    }
    l.total = at;
    return l;
}

template <typename T, int KD, int VD>
size_t glr_lds(bool out) {
    return static_cast<size_t>(kL) * ((out ? 2 : 1) * KD + VD) * sizeof(T) + sizeof(Gates) + 4 * kL * sizeof(float);
}

template <typename T, int KD, int VD, bool REV, bool OUT, int NS>
hipError_t glr_go3(const GlrPass& p, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * p.nseg);
    glr_kernel<T, KD, VD, REV, OUT, NS><<<grid, kGlrThreads, glr_lds<T, KD, VD>(OUT), st>>>(p);
    return hipGetLastError();
}
template <typename T, bool REV, bool OUT, int NS>
hipError_t glr_go2(const GlrPass& p, hipStream_t st) {
    const int kd = padded(p.y.width), vd = padded(p.z.width);
    if (kd == 64) return vd == 64 ? glr_go3<T, 64, 64, REV, OUT, NS>(p, st) : glr_go3<T, 64, 128, REV, OUT, NS>(p, st);
    return vd == 64 ? glr_go3<T, 128, 64, REV, OUT, NS>(p, st) : glr_go3<T, 128, 128, REV, OUT, NS>(p, st);
}
template <bool REV, bool OUT, int NS>
hipError_t glr_go(const GlrPass& p, int dtype, hipStream_t st) {
    return dtype == SDM_BF16 ? glr_go2<bf16_t, REV, OUT, NS>(p, st) : glr_go2<float, REV, OUT, NS>(p, st);
}

template <bool REV>
hipError_t chain(float* states, const float* decay, const float* start, int nseg, int64_t one, int64_t bh, hipStream_t st) {
    const int64_t total = bh * one;
    glr_chain_kernel<REV><<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(states, decay, start, nseg, one, total);
    return hipGetLastError();
}

template <typename T, bool REV, bool OUT, int NS>
void list(const void** all, int& n) {
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 64, 64, REV, OUT, NS>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 64, 128, REV, OUT, NS>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 128, 64, REV, OUT, NS>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 128, 128, REV, OUT, NS>);
}
template <typename T>
void list_type(const void** all, int& n) {
    list<T, false, true, 2>(all, n);
    list<T, false, true, 3>(all, n);
    list<T, true, true, 2>(all, n);
    list<T, true, true, 3>(all, n);
    list<T, false, false, 3>(all, n);
    list<T, true, false, 3>(all, n);
}

// A pass over io's shape.
GlrPass base_pass(const sdm_glr_io* io, const SegPlan& sp) {
    GlrPass p{};
    p.g = io->g;
    p.g_b = io->g_b;
    p.g_t = io->g_t;
    p.g_h = io->g_h;
    p.lens = io->lens;
    p.B = io->B;
    p.T = io->T;
    p.H = io->H;
    p.nseg = sp.nseg;
    p.seg = sp.seg;
    p.m_p = p.m_o = p.m_s = 1.0f;
    return p;
}

}  // namespace

int glr_lds_kernels(const void** fns, int cap) {
    const void* all[64];
    int n = 0;
    list_type<bf16_t>(all, n);
    list_type<float>(all, n);
    int k = 0;
    for (; k < n && k < cap; ++k) fns[k] = all[k];
    return k;
}

size_t glr_workspace_bytes(const sdm_glr_io* io, bool backward) {
    return io->B < 1 ? 0 : glr_layout(io, backward).total;
}

hipError_t glr_forward_launch(const sdm_glr_io* io, hipStream_t st) {
    const int es = io->dtype == SDM_BF16 ? 2 : 4, per = io->H / io->Hk;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H, one = static_cast<int64_t>(io->dk) * io->dv;
    const SegPlan sp = seg_plan(bh, io->T);
    const GlrLayout l = glr_layout(io, false);
    char* ws = static_cast<char*>(io->workspace);
    GlrPass p = base_pass(io, sp);
    p.x = rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, es);
    p.y = rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, es);
    p.z = rows_of(io->v, io->v_b, io->v_t, io->v_h, io->dv, 1, es);
    p.s_k = io->dv;
    p.s_v = 1;
    hipError_t e = hipSuccess;
    if (sp.nseg > 1) {
        p.seg_state = reinterpret_cast<float*>(ws + l.s);
        p.seg_decay = reinterpret_cast<float*>(ws + l.sd);
        if ((e = glr_go<false, false, 3>(p, io->dtype, st)) != hipSuccess) return e;
        if ((e = chain<false>(p.seg_state, p.seg_decay, io->state, sp.nseg, one, bh, st)) != hipSuccess) return e;
        p.s_in = p.seg_state;
    } else {
        p.s_in = io->state;
    }
    p.s_out = io->last;
    p.m_p = p.m_o = io->scale;
    p.out = io->o;
    p.o_b = io->o_b;
    p.o_t = io->o_t;
    p.o_h = io->o_h;
    const int ou = 4;
    p.out_wide = reinterpret_cast<uintptr_t>(io->o) % (ou * es) == 0 && io->o_b % ou == 0 && io->o_t % ou == 0 && io->o_h % ou == 0 && io->dv % ou == 0;
    return glr_go<false, true, 2>(p, io->dtype, st);
}

hipError_t glr_backward_launch(const sdm_glr_io* io, const sdm_glr_grad* g, hipStream_t st) {
    const int es = io->dtype == SDM_BF16 ? 2 : 4, per = io->H / io->Hk;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H, one = static_cast<int64_t>(io->dk) * io->dv;
    const SegPlan sp = seg_plan(bh, io->T);
    const GlrLayout l = glr_layout(io, true);
    char* ws = static_cast<char*>(io->workspace);
    const Rows q = rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, es), k = rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, es),
               v = rows_of(io->v, io->v_b, io->v_t, io->v_h, io->dv, 1, es), d = rows_of(g->d_o, g->do_b, g->do_t, g->do_h, io->dv, 1, es);
    const GlrPass base = base_pass(io, sp);
    float *S = nullptr, *R = nullptr;
    hipError_t e = hipSuccess;
    if (sp.nseg > 1) {
        GlrPass p = base;   // the states before the segments, and the gradients of those after them
        S = reinterpret_cast<float*>(ws + l.s);
        R = reinterpret_cast<float*>(ws + l.r);
        p.s_k = io->dv;
        p.s_v = 1;
        p.y = k;
        p.z = v;
        p.seg_state = S;
        p.seg_decay = reinterpret_cast<float*>(ws + l.sd);
        if ((e = glr_go<false, false, 3>(p, io->dtype, st)) != hipSuccess) return e;
        if ((e = chain<false>(S, p.seg_decay, io->state, sp.nseg, one, bh, st)) != hipSuccess) return e;
        p.y = q;
        p.z = d;
        p.m_s = io->scale;
        p.seg_state = R;
        p.seg_decay = reinterpret_cast<float*>(ws + l.rd);
        if ((e = glr_go<true, false, 3>(p, io->dtype, st)) != hipSuccess) return e;
        if ((e = chain<true>(R, p.seg_decay, g->d_last, sp.nseg, one, bh, st)) != hipSuccess) return e;
    }
    const float* s_in = sp.nseg > 1 ? S : io->state;
    const float* r_in = sp.nseg > 1 ? R : g->d_last;
    const bool fold = per > 1;
    float* dqd = reinterpret_cast<float*>(ws + l.dqd);
    float* dkd = reinterpret_cast<float*>(ws + l.dkd);
    float* cross = reinterpret_cast<float*>(ws + l.cross);
    auto key_out = [&](GlrPass& p, void* out, size_t at) {   // [B, T, H or Hk, dk]
        p.out = fold ? static_cast<void*>(ws + at) : out;
        p.out_f32 = fold;
        p.o_h = io->dk;
        p.o_t = static_cast<int64_t>(io->H) * io->dk;
        p.o_b = p.o_t * io->T;
        p.out_wide = io->dk % 4 == 0;
    };
    {   // dq: keys and values exchanged, on the transposed state
        GlrPass p = base;
        p.x = d;
        p.y = v;
        p.z = k;
        p.w = q;
        p.m_p = p.m_o = io->scale;
        p.s_in = s_in;
        p.s_k = 1;
        p.s_v = io->dv;
        key_out(p, g->dq, l.fq);
        p.dot = dqd;
        p.r_end = r_in;
        p.r_k = 1;
        p.r_v = io->dv;
        p.cross = cross;
        if ((e = glr_go<false, true, 3>(p, io->dtype, st)) != hipSuccess) return e;
    }
    {   // dk: back in time on the transposed gradient of the state
        GlrPass p = base;
        p.x = v;
        p.y = d;
        p.z = q;
        p.w = k;
        p.m_p = p.m_s = io->scale;
        p.s_in = r_in;
        p.s_k = 1;
        p.s_v = io->dv;
        key_out(p, g->dk, l.fk);
        p.dot = dkd;
        if ((e = glr_go<true, true, 3>(p, io->dtype, st)) != hipSuccess) return e;
    }
    {   // dv
        GlrPass p = base;
        p.x = k;
        p.y = q;
        p.z = d;
        p.m_p = p.m_s = io->scale;
        p.s_in = r_in;
        p.s_out = g->d_state;
        p.s_k = io->dv;
        p.s_v = 1;
        p.out = g->dv;
        p.o_h = io->dv;
        p.o_t = static_cast<int64_t>(io->H) * io->dv;
        p.o_b = p.o_t * io->T;
        p.out_wide = io->dv % 4 == 0;
        if ((e = glr_go<true, true, 2>(p, io->dtype, st)) != hipSuccess) return e;
    }
    if (io->T == 0) return hipSuccess;
    const int64_t waves = bh * sp.nseg;
    glr_gate_grad_kernel<<<static_cast<unsigned>((waves * kWave + 255) / 256), 256, 0, st>>>(dqd, dkd, cross, io->lens, g->dg, io->T, io->H,
                                                                                             sp.nseg, sp.seg, waves);
    if ((e = hipGetLastError()) != hipSuccess || !fold) return e;
    const int64_t total = static_cast<int64_t>(io->B) * io->T * io->Hk * io->dk;
    const int64_t need = (total + 255) / 256;
    const unsigned blocks = static_cast<unsigned>(need < (1 << 20) ? need : 1 << 20);
    for (int i = 0; i < 2; ++i) {
        const float* in = reinterpret_cast<const float*>(ws + (i ? l.fk : l.fq));
        void* out = i ? g->dk : g->dq;
        if (io->dtype == SDM_BF16) glr_fold_kernel<bf16_t><<<blocks, 256, 0, st>>>(in, static_cast<bf16_t*>(out), total, io->dk, per);
        else glr_fold_kernel<float><<<blocks, 256, 0, st>>>(in, static_cast<float*>(out), total, io->dk, per);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t glr_step_launch(const sdm_glr_step_io* io, hipStream_t st) {
    GlrStep a{*io, io->dv, 1};
    // Narrower column tiles until there are four blocks for each compute unit (or 16 columns a tile).
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    a.cols = 128;
    while (a.cols > 16 && bh * ((io->dv + a.cols - 1) / a.cols) < 1024) a.cols /= 2;
    a.tiles = (io->dv + a.cols - 1) / a.cols;
    const unsigned grid = static_cast<unsigned>(bh * a.tiles);
    const bool vec = io->dv % 4 == 0;
    if (io->dtype == SDM_BF16) {
        if (vec) glr_step_kernel<bf16_t, 4><<<grid, 256, 0, st>>>(a);
        else glr_step_kernel<bf16_t, 1><<<grid, 256, 0, st>>>(a);
    } else {
        if (vec) glr_step_kernel<float, 4><<<grid, 256, 0, st>>>(a);
        else glr_step_kernel<float, 1><<<grid, 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace sdm
