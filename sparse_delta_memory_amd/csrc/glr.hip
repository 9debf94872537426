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
// every segment (below) from <S, R> there and at every reset from 0, so that what cancels is never longer than a segment.
//
// Layout. A block owns one (stream, head, segment); each of its waves owns 16 columns of z, out and the
// state (8 waves for widths past 64, else 4) and keeps its part of the state in registers over all chunks
// as the accumulators of 16 x 16 matrix-product tiles (rows: the key dimension). The same registers, cut
// into bfloat16 parts, are directly the other operand of x S: the accumulator layout (four rows at one
// column per lane) equals an operand's (some inner indexes at one row); the inner index is only permuted,
// and the matching operand is read in the same permutation. So is a score tile y x^T the other operand of
// the product with z; the twelve score tiles of a chunk are dealt to the waves and shared through LDS in
// that form. (Every wave computing all of them saves a barrier but took 309 us where this takes 253: 8 x
// 4096 tokens x 16 heads of 128, then at one block per compute unit.) The products are formed transposed,
// so that a lane holds four consecutive columns of a result row: 8-byte stores, and row dots that need two
// lane exchanges. Tiles of x, y and z go from global memory to LDS without registers between, 16-byte
// pieces permuted per row against bank conflicts; x's next tile is loaded once the scores are done, y's and
// z's at the chunk's end, and the second block of the compute unit works meanwhile. That takes 128 registers (205 with a chunk's loads
// held in registers and one block: 253 us; 151 so).
//
// Numbers. Products of bfloat16 inputs are exact; a float32 factor (decayed score, state, decayed z) is
// cut into three bfloat16 parts by truncation, which hold all 24 bits, and multiplied part by part. (For o and dv,
// which are rounded to bfloat16 in the end, two parts of the scores and of the state that meets x take 6 % less,
// 8 x 4096 x 16 forward 218 against 233 us, but sums that cancel show their error of up to 2^-15.) float32
// inputs go through the float32 matrix instructions. Gates are summed in float64 per chunk (one wave, one token
// per lane) and only differences of a chunk's sums are rounded to float32, so neither long rows nor a reset (a
// gate of -infinity counts as -10000) cost digits.
//
// What is not finite reaches what it is part of by the recurrence and nothing else: no token before it, nothing past a
// reset, although a tile product multiplies it by zeros there. Factors of 0 are applied by a multiplication
// whose 0 times anything is 0; z is looked over before its product with the scores, and a chunk with such a value
// goes another way; rows of y that a reset cuts off from the state are cleared. Looking costs 3 to 5 % (8 x 4096
// tokens x 16 heads of 128, forward 213 -> 220 us, backward 706 -> 720).
//
// Segments. With few streams and heads the time axis is cut: a first kernel sums each segment's own
// state, and the main kernel starts every segment from the state before it, made up of the start and the
// segments before (by itself when they are few, else a kernel chains them).
//
// What bounds it, 8 x 4096 tokens x 16 heads of 128 (bfloat16): o in 232 us, 2.4 TB/s of its 547 MB: about 165 us
// of main kernel and 65 of the segments' states, which read k and v once more. Counted per chunk and compute unit, the main
// kernel's 968 matrix instructions keep the matrix units busy for 3900 cycles, its 4980 other vector instructions
// (cutting states, scores and z into parts, scaling, addresses) take 5000 cycles of issue and LDS is busy for 4400 (1600 of
// them bank conflicts); a chunk passes in 11200. So the three overlap little: with two blocks per unit, each between
// the same barriers, they mostly follow each other. The backward (736 us) is three such passes and two of states; dq
// and dk read a fourth row for the dots, 215 us each beside 166 for dv.
#include <hip/hip_runtime.h>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"
#include "tiles.hpp"

namespace sdm {
namespace {

struct GlrPass {
    Rows x, y, z, w;          // w: the rows the results are dotted with (DOT)
    const float* g;
    int64_t g_b, g_t, g_h;
    const int32_t* lens;
    int B, T, H;
    int nseg, seg;            // segments, and tokens of each (a multiple of 64)
    float m_p, m_o, m_s;
    // States, element (key, value) at key * s_k + value * s_v. start: [B H] before the first segment in the pass's direction
    // (NULL: zero); segs: [B H, nseg] (NULL when nseg is 1), the segments' own states with their decays [B H, nseg], or,
    // chained, the states before the segments. last: [B H] after the last segment (NULL: not kept).
    const float* start;
    float* segs;
    float* decays;
    int chained;
    float* last;
    int s_k, s_v;
    // out rows: [B, T, H] with strides, narrowed to the input type, or float32 (shared heads, added up later)
    void* out;
    int64_t o_b, o_t, o_h;
    int out_wide;             // 4-element stores
    int out_f32;
    float* dot;               // [B H, T] row dots of w and the result (DOT)
    // DOT: <S, R> at the segment's end to cross [B H, nseg]; R's start, segs and decays like S's, backwards in time.
    float* cross;
    const float* r_start;
    const float* r_segs;
    const float* r_decays;
};

__device__ __forceinline__ int row_len(const GlrPass& p, int b) {
    const int n = p.lens != nullptr ? p.lens[b] : p.T;
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// out_i of a chunk is not finite in the columns where z_j is not, for every token i that j reaches (D_ij > 0): NaN there.
// Which ones is the product of the marks of such z_j with the marks of D_ij > 0.
template <typename T, int VD, bool REV>
__device__ __forceinline__ void stray_values(T* zc, const Gates& gates, int n0, int i16, int qd, f32x4 (&O)[4]) {
    f32x4 E[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) E[it] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
        Frag<T> mark, finite;
        split_finite(col_frag<VD, 4>(zc, jb, n0, i16, qd), finite, mark);
#pragma unroll
        for (int pr = 0; pr < 6; ++pr) {
            if (Pairs<REV>::kJb[pr] != jb) continue;
            const int it = Pairs<REV>::kIt[pr], i = 16 * it + i16;
            float reach[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int jt = 2 * jb + (e >> 2), jj = 4 * qd + (e & 3), j = 16 * jt + jj;
                float d = 0.0f;
                if (jt == it) {
                    const float x = (gates.lhi[i] - gates.lhi[j]) + (gates.llo[i] - gates.llo[j]);
                    if (REV ? jj >= i16 : jj <= i16) d = __builtin_amdgcn_exp2f(REV ? -x : x);
                } else if (REV ? jt > it : jt < it) {
                    d = (REV ? gates.down : gates.up)[i] * gates.tau[4 * it + jt] * (REV ? gates.up : gates.down)[j];
                }
                reach[e] = d > 0.0f ? 1.0f : 0.0f;
            }
            Parts<T, 1> to;
            cut(reach, to);
            mma(mark, to.p[0], E[it]);
        }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
#pragma unroll
        for (int r = 0; r < 4; ++r) O[it][r] = E[it][r] > 0.0f ? __builtin_nanf("") : O[it][r];
    }
}

// KD, VD: padded widths of x / y and of z (64 or 128).
// OUT: results (else the segments' own states alone). DOT: row dots of the results, and <S, R>. FOLD: float32 results
// of bfloat16 inputs.
template <typename T, int KD, int VD, bool REV, bool OUT, bool DOT, bool FOLD>
__global__ __launch_bounds__(4 * VD, sizeof(T) == 2 ? 4 : 1) void glr_kernel(GlrPass p) {
    constexpr int KB = KD / 32, KT = KD / 16, kThreads = 4 * VD, kWaves = VD / 16;
    constexpr int NP = kParts<T>;
    constexpr bool F32 = sizeof(T) == 4 || FOLD;
    // Without results two chunks' tiles fit beside each other (in bfloat16) and the next chunk's loads run under a chunk's
    // products; with them x's tile is free half way through a chunk, y's and z's at its end.
    constexpr int kBufs = !OUT && sizeof(T) == 2 ? 2 : 1;
    constexpr int kScoreWords = 8 * static_cast<int>(sizeof(T)) / 4;   // per lane and part
    extern __shared__ __align__(16) char lds[];
    T* xt = reinterpret_cast<T*>(lds);
    T* yt = xt + (OUT ? kL * KD : 0);
    T* zt = yt + kBufs * kL * KD;
    uint32_t* scores = reinterpret_cast<uint32_t*>(zt + kBufs * kL * VD);   // [6][NP][64 lanes][kScoreWords]
    Gates* gate_at = reinterpret_cast<Gates*>(scores + (OUT ? 6 * NP * kWave * kScoreWords : 0));   // two chunks
    float* dots = reinterpret_cast<float*>(gate_at + 2);   // [waves][64]

    const int nblk = OUT ? p.nseg : p.nseg - 1;   // the last segment's own state (in the pass's direction) is not needed
    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int bh = blk / nblk, si = blk - bh * nblk + (!OUT && REV ? 1 : 0), b = bh / p.H, h = bh - b * p.H;
    const int lane = static_cast<int>(lane_id()), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int n0 = wave * 16;   // the wave's first column
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

    // The wave's state: tile d, rows 32 (d / 2) + 8 quarter + 4 (d % 2) + r, column n0 + lane % 16.
    f32x4 S[KT];
    // Its elements are read and written through buffer descriptors of one state's range; the lanes' offsets past the
    // state's widths are out of it (read as zero, not written), so no branches cut the accumulators' registers apart.
    const uint32_t at0 = 4u * static_cast<uint32_t>((n0 + i16) * p.s_v + 8 * qd * p.s_k);
    auto state_at = [&](int d, int r) {
        const int k = 32 * (d >> 1) + 4 * (d & 1) + r;
        return static_cast<int>(n0 + i16 < vd && k + 8 * qd < kd ? at0 + 4u * static_cast<uint32_t>(k * p.s_k) : 0xC0000000u);
    };
    auto state_of = [&](const float* s) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(s), 0, static_cast<int>(one) * 4, 0x00027000);
    };
    auto state_read = [&](__amdgpu_buffer_rsrc_t s, int d, int r) {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(s, state_at(d, r), 0, 0));
    };
#pragma unroll
    for (int d = 0; d < KT; ++d) S[d] = f32x4{0, 0, 0, 0};
    if constexpr (OUT) {
        const bool whole = p.segs != nullptr && p.chained;
        const float* s0 = whole ? p.segs + (static_cast<int64_t>(bh) * p.nseg + si) * one : p.start != nullptr ? p.start + bh * one : nullptr;
        if (s0 != nullptr) {
            const auto s = state_of(s0);
#pragma unroll
            for (int d = 0; d < KT; ++d) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[d][r] = state_read(s, d, r);
            }
        }
        // The segments before this one, in order.
#pragma unroll 1
        for (int n = REV ? p.nseg - 1 : 0; !whole && n != si; n += REV ? -1 : 1) {
            const auto s = state_of(p.segs + (static_cast<int64_t>(bh) * p.nseg + n) * one);
            const float dec = p.decays[static_cast<int64_t>(bh) * p.nseg + n];
#pragma unroll
            for (int d = 0; d < KT; ++d) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[d][r] = decay_add(dec, S[d][r], state_read(s, d, r));
            }
        }
    }
    double decay = 0.0;   // state-only: the sum of the segment's gates

    Stage<T, KD, kThreads> sx, sy;
    Stage<T, VD, kThreads> sz;
    if (OUT) sx.init(p.x);
    sy.init(p.y);
    sz.init(p.z);
    auto fill_x = [&](int c, int tid) {
        const int t0 = t_lo + c * kL;
        if (OUT) sx.fill(p.x, xb + t0 * p.x.t, live - t0, xt, wave, tid);
    };
    auto fill_yz = [&](int c, int buf, int tid) {
        const int t0 = t_lo + c * kL;
        sy.fill(p.y, yb + t0 * p.y.t, live - t0, yt + buf * kL * KD, wave, tid);
        sz.fill(p.z, zb + t0 * p.z.t, live - t0, zt + buf * kL * VD, wave, tid);
    };
    // Chunk c's gates, one token per lane (c >= 0 has tokens; a lane past them loads the last one's, and drops it).
    auto gate_load = [&](int c, int lane) { return gb[static_cast<int64_t>(min(t_lo + max(c, 0) * kL + lane, live - 1)) * p.g_t]; };
    auto gate_of = [&](int c, float g, int lane) { return t_lo + c * kL + lane < live ? g : 0.0f; };
    float next_gate = 0.0f;
    if (chunks > 0) {
        const int c = REV ? chunks - 1 : 0;
        const float g = gate_load(c, lane);
        next_gate = gate_load(REV ? c - 1 : min(c + 1, chunks - 1), lane);
        fill_x(c, threadIdx.x);
        fill_yz(c, 0, threadIdx.x);
        if (wave == kWaves - 1) gate_factors<REV>(gate_of(c, g, lane), p.m_o, p.m_s, gate_at[0], lane);
    }

    for (int cc = 0; cc < chunks; ++cc) {
        const int c = REV ? chunks - 1 - cc : cc, t0 = t_lo + c * kL, left = live - t0;
        Gates& gates = gate_at[cc & 1];
        // The lane's place, unknown to the compiler to be the same in every chunk: the many LDS addresses made from it are cheap
        // to make again, and kept over the loop they would not fit the 128 registers that two blocks per compute unit leave.
        int tid = static_cast<int>(threadIdx.x);
        __asm__ volatile("" : "+v"(tid));
        const int here = tid & (kWave - 1);
        const int i16 = here & 15, qd = here >> 4;
        const int n = n0 + 4 * qd;   // the lane's result columns n .. n + 3, of token 16 it + lane % 16
        const int buf = kBufs == 2 ? cc & 1 : 0;
        T* const yc = yt + buf * kL * KD;
        T* const zc = zt + buf * kL * VD;
        const bool more = cc + 1 < chunks;
        const int next = REV ? c - 1 : c + 1;
        tile_barrier();   // the chunk's tiles and gate factors are complete
        // The compiler does not count the tile loads: its own wait for an ordinary load would take in those issued behind it.
        // So ordinary loads are waited for where no tile load is behind them: the next chunk's gates here, w's rows below.
        __asm__ volatile("" : "+v"(next_gate));
        Four<T> wx[DOT ? 4 : 1];   // the rows to dot the results with
        if constexpr (DOT) {
            const T* w = static_cast<const T*>(p.w.p) + b * p.w.b + (h / p.w.per) * p.w.h + static_cast<int64_t>(t0) * p.w.t + n;
#pragma unroll
            for (int it = 0; it < 4; ++it) wx[it].load(w + (16 * it + i16) * p.w.t, 16 * it + i16 < left ? vd - n : 0, p.w.wide);
        }
        if (kBufs == 2 && more) fill_yz(next, buf ^ 1, tid);
        // The next chunk's factors, by the last wave (it has one score tile, others two); its gates came a chunk ago.
        if (more && wave == kWaves - 1) gate_factors<REV>(gate_of(next, next_gate, here), p.m_o, p.m_s, gate_at[(cc + 1) & 1], here);
        next_gate = gate_load(REV ? c - 2 : min(c + 2, chunks - 1), here);

        if constexpr (OUT) {
            // The twelve score tiles, dealt to the waves.
            for (int e = wave; e < 12; e += kWaves) {
                const int pr = e >> 1, half = e & 1;
                int it = 0, jb = 0;
#pragma unroll
                for (int k = 0; k < 6; ++k) {
                    if (k == pr) {
                        it = Pairs<REV>::kIt[k];
                        jb = Pairs<REV>::kJb[k];
                    }
                }
                const int jt = 2 * jb + half;
                float s[4];
                if (REV ? jt < it : jt > it) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[r] = 0.0f;
                } else {
                    f32x4 a = {0, 0, 0, 0};   // token 16 jt + 4 quarter + r down, token 16 it + lane % 16 across
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
                        mma(row_frag<KD>(yc, 16 * jt + i16, kb, qd), row_frag<KD>(xt, 16 * it + i16, kb, qd), a);
                    if (jt == it) {
                        // Every row of y is part of a score here, and with it what is not finite in y.
                        const float odd = fmaf(a[0], 0.0f, fmaf(a[1], 0.0f, fmaf(a[2], 0.0f, a[3] * 0.0f)));
                        if (odd != odd) gates.odd = 1;
                        const float lhi = gates.lhi[16 * it + i16], llo = gates.llo[16 * it + i16];
                        const f32x4 jh = *reinterpret_cast<const f32x4*>(&gates.lhi[16 * jt + 4 * qd]);
                        const f32x4 jl = *reinterpret_cast<const f32x4*>(&gates.llo[16 * jt + 4 * qd]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int j = 4 * qd + r;
                            const float x = (lhi - jh[r]) + (llo - jl[r]);
                            const float w = __builtin_amdgcn_exp2f(REV ? -x : x);
                            s[r] = (REV ? j >= i16 : j <= i16) ? sdm_decayed(w * p.m_p, a[r]) : 0.0f;
                        }
                    } else {
                        const float ot = (REV ? gates.down : gates.up)[16 * it + i16] * (p.m_p * gates.tau[4 * it + jt]);
                        const f32x4 d = *reinterpret_cast<const f32x4*>(&(REV ? gates.up : gates.down)[16 * jt + 4 * qd]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[r] = sdm_decayed(ot * d[r], a[r]);
                    }
                }
                if constexpr (sizeof(T) == 2) {
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        *reinterpret_cast<u32x2*>(scores + ((pr * NP + k) * kWave + here) * kScoreWords + 2 * half) =
                            u32x2{__builtin_amdgcn_perm(__float_as_uint(s[1]), __float_as_uint(s[0]), 0x07060302u),
                                  __builtin_amdgcn_perm(__float_as_uint(s[3]), __float_as_uint(s[2]), 0x07060302u)};
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[r] -= __uint_as_float(__float_as_uint(s[r]) & 0xFFFF0000u);
                    }
                } else {
                    *reinterpret_cast<f32x4*>(scores + (pr * kWave + here) * kScoreWords + 4 * half) = f32x4{s[0], s[1], s[2], s[3]};
                }
            }
            // S^T x
            f32x4 O[4];   // tile it: columns n0 + 4 quarter + r down, token 16 it + lane % 16
#pragma unroll
            for (int it = 0; it < 4; ++it) O[it] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Parts<T, NP> sp;
                Frag<T> xf[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) xf[it] = row_frag<KD>(xt, 16 * it + i16, kb, qd);
                float s[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) { s[r] = S[2 * kb][r]; s[4 + r] = S[2 * kb + 1][r]; }
                cut(s, sp);
#pragma unroll
                for (int k = NP - 1; k >= 0; --k) {
#pragma unroll
                    for (int it = 0; it < 4; ++it) mma(sp.p[k], xf[it], O[it]);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) O[it] = decayed(gates.f[16 * it + i16], O[it]);
            lds_barrier();   // the scores are complete, and x's tile is free
            if constexpr (DOT) {
#pragma unroll
                for (int it = 0; it < 4; ++it) __asm__ volatile("" : "+v"(wx[it].w));
            }
            if (more) fill_x(next, tid);
            // The chunk's own tokens. A tile product multiplies z_j by the scores that are 0 as well (tokens before j, and those
            // that a reset cuts off), so what is not finite in the wave's columns of z is taken out of it, and put
            // where it belongs afterwards.
            Frag<T> zf[2];
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) zf[jb] = col_frag<VD, 4>(zc, jb, n0, i16, qd);
            const bool stray = __ballot(not_finite(zf[0], zf[1])) != 0;
            if (__builtin_expect(stray, 0)) {
#pragma unroll
                for (int jb = 0; jb < 2; ++jb) {
                    Frag<T> mark;
                    split_finite(zf[jb], zf[jb], mark);
                }
            }
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
#pragma unroll
                for (int s = NP - 1; s >= 0; --s) {
#pragma unroll
                    for (int pr = 0; pr < 6; ++pr) {
                        if (Pairs<REV>::kJb[pr] != jb) continue;
                        Frag<T> pf;
                        __builtin_memcpy(&pf, scores + ((pr * NP + s) * kWave + here) * kScoreWords, sizeof(pf));
                        mma(zf[jb], pf, O[Pairs<REV>::kIt[pr]]);
                    }
                }
            }
            if (__builtin_expect(stray, 0)) stray_values<T, VD, REV>(zc, gates, n0, i16, qd, O);
            // Results.
            if constexpr (DOT) {
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    float dot = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) dot = fmaf(wx[it].at(r), O[it][r], dot);
                    dot += lane_xor_f<16>(dot);
                    dot += lane_xor_f<32>(dot);
                    if (qd == 0) dots[wave * kL + 16 * it + i16] = dot;
                }
            }
            const int64_t o0 = b * p.o_b + h * p.o_h + static_cast<int64_t>(t0) * p.o_t;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int64_t at = o0 + (16 * it + i16) * p.o_t + n;
                if (16 * it + i16 >= left || n >= vd) continue;
                const f32x4 v = O[it];
                if (F32) {
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
        } else {
            decay += gates.sum;
        }

        // The state. Tokens that a later one's reset cuts off from it have a factor of 0; their rows of y are cleared, since 0
        // times what is not finite there would not be 0.
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(OUT ? gates.gone & gates.odd : gates.gone), 0)) {
            constexpr int kPieces = KD * static_cast<int>(sizeof(T)) / 16;
            for (int at = tid; at < kL * kPieces; at += kThreads) {
                const int row = at / kPieces;
                if (gates.u[row] == 0.0f) *reinterpret_cast<u32x4*>(piece<T, KD>(yc, row, at % kPieces)) = u32x4{0, 0, 0, 0};
            }
            lds_barrier();
        }
        const float all = gates.all;
#pragma unroll
        for (int d = 0; d < KT; ++d) S[d] = decayed(all, S[d]);
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            Parts<T, NP> zp;
            {
                const f32x4 ua = *reinterpret_cast<const f32x4*>(&gates.u[32 * jb + 4 * qd]);
                const f32x4 ub = *reinterpret_cast<const f32x4*>(&gates.u[32 * jb + 16 + 4 * qd]);
                float z[8];
                widen8(col_frag<VD, 4>(zc, jb, n0, i16, qd), z);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    z[r] = sdm_decayed(ua[r], z[r]);
                    z[4 + r] = sdm_decayed(ub[r], z[4 + r]);
                }
                cut(z, zp);
            }
#pragma unroll
            for (int d = 0; d < KT; d += 4) {
                Frag<T> yf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) yf[e] = col_frag<KD, 8>(yc, jb, 32 * ((d + e) >> 1) + 4 * (e & 1), i16, qd);
#pragma unroll
                for (int s = NP - 1; s >= 0; --s) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma(yf[e], zp.p[s], S[d + e]);
                }
            }
        }
        if (kBufs == 1) {
            lds_barrier();   // y's and z's tiles are free; the dots are complete
            if (more) fill_yz(next, 0, tid);
        }
        if (DOT && tid < min(kL, left)) {
            const int i = tid;
            float dot = dots[i];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) dot += dots[w * kL + i];
            p.dot[static_cast<int64_t>(bh) * p.T + t0 + i] = dot;
        }
    }

    if constexpr (OUT) {
        // Tokens past the row's length.
        const int t_dead = max(live, t_lo);
        for (int64_t e = threadIdx.x; e < static_cast<int64_t>(t_hi - t_dead) * vd; e += kThreads) {
            const int t = t_dead + static_cast<int>(e / vd), col = static_cast<int>(e % vd);
            const int64_t at = b * p.o_b + t * p.o_t + h * p.o_h + col;
            if (F32) static_cast<float*>(p.out)[at] = 0.0f;
            else static_cast<bf16_t*>(p.out)[at] = bf16_t{0};
        }
    }
    if constexpr (DOT) {
        for (int t = max(live, t_lo) + static_cast<int>(threadIdx.x); t < t_hi; t += kThreads)
            p.dot[static_cast<int64_t>(bh) * p.T + t] = 0.0f;
        // <S, R> at the segment's end (forwards only). R is made up like S, from the row's end.
        if (p.cross == nullptr) return;
        float x = 0.0f;
        if (p.r_segs != nullptr || p.r_start != nullptr) {
            const bool whole = p.r_segs != nullptr && p.chained;
            const float* r0 = whole ? p.r_segs + (static_cast<int64_t>(bh) * p.nseg + si) * one : p.r_start != nullptr ? p.r_start + bh * one : nullptr;
            f32x4 R[KT];
#pragma unroll
            for (int d = 0; d < KT; ++d) R[d] = f32x4{0, 0, 0, 0};
            if (r0 != nullptr) {
                const auto s = state_of(r0);
#pragma unroll
                for (int d = 0; d < KT; ++d) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[d][r] = state_read(s, d, r);
                }
            }
#pragma unroll 1
            for (int n = p.nseg - 1; !whole && n > si; --n) {
                const auto s = state_of(p.r_segs + (static_cast<int64_t>(bh) * p.nseg + n) * one);
                const float dec = p.r_decays[static_cast<int64_t>(bh) * p.nseg + n];
#pragma unroll
                for (int d = 0; d < KT; ++d) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[d][r] = decay_add(dec, R[d][r], state_read(s, d, r));
                }
            }
#pragma unroll
            for (int d = 0; d < KT; ++d) {
#pragma unroll
                for (int r = 0; r < 4; ++r) x = fmaf(S[d][r], R[d][r], x);
            }
        }
        x = group_sum<kWave>(x);
        __syncthreads();   // the last chunk's dots have been read
        if (lane == 0) dots[wave] = x;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWaves; ++w) x += dots[w];
            p.cross[static_cast<int64_t>(bh) * p.nseg + si] = x;
        }
    }
    if (!OUT && threadIdx.x == 0) p.decays[static_cast<int64_t>(bh) * p.nseg + si] = exp2_of(decay);
    float* so = OUT ? (p.last != nullptr && si == (REV ? 0 : p.nseg - 1) ? p.last + bh * one : nullptr)
                    : p.segs + (static_cast<int64_t>(bh) * p.nseg + si) * one;
    if (so != nullptr) {
        const auto s = state_of(so);
#pragma unroll
        for (int d = 0; d < KT; ++d) {
#pragma unroll
            for (int r = 0; r < 4; ++r) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[d][r]), s, state_at(d, r), 0, 0);
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
    constexpr int kU = 32;   // segments in flight
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
                s = decay_add(decay[bh * nseg + n], s, own[u]);
            }
        }
    }
}

struct GateGrad {
    const float *dq, *dk;     // [B H, T] the row dots q . dq and k . dk
    const float* cross;       // [B H, nseg]
    const float* g;
    int64_t g_b, g_t, g_h;
    const int32_t* lens;
    const float *state, *d_state;   // [B H, one] or NULL
    int64_t one;
    float* dg;
    int T, H, nseg, seg;
    int64_t waves;
};

// dg: one wave per (stream, head, segment), 256 tokens at a time from the segment's end, in float64. A token that
// resets, or has no state before it, has a gradient of 0, and with it the sums start afresh: nothing of a later sequence, be it large
// or not finite, is in an earlier one's. Where the sum from the end is not finite, that from the front,
//     dg_t = dg_{t0} - sum_{t0 <= s < t} (q_s . dq_s - k_s . dk_s),
// may be, since what makes q . dq infinite or NaN is a key or value behind t; dg_{t0} is <S, R> of the segment before,
// or <state, its gradient>.
__global__ __launch_bounds__(256) void glr_gate_grad_kernel(GateGrad p) {
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kWave;
    if (id >= p.waves) return;
    constexpr int kU = 4;
    const int lane = static_cast<int>(lane_id()), T = p.T;
    // Neighbouring waves take neighbouring heads, whose gates and results share cache lines.
    const int64_t h = id % p.H, bs = id / p.H, b = bs / p.nseg, bh = b * p.H + h;
    const int si = static_cast<int>(bs - b * p.nseg);
    int len = p.lens != nullptr ? p.lens[b] : T;
    len = len < 0 ? 0 : len > T ? T : len;
    const int t_lo = si * p.seg, t_hi = min(T, t_lo + p.seg);
    const float* gates = p.g + b * p.g_b + h * p.g_h;
    float* out = p.dg + b * T * p.H + h;
    const int nothing = p.state == nullptr ? 0 : -1;   // the token with no state before it, whatever its gate
    double carry = p.cross[bh * p.nseg + si];
    bool lost = false;
    for (int t1 = t_hi; t1 > t_lo; t1 -= kU * kWave) {   // lane l takes tokens t1 - 1 - l - 64 u
        float q[kU], k[kU], g[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = max(t1 - 1 - lane - u * kWave, t_lo);
            q[u] = p.dq[bh * T + t];
            k[u] = p.dk[bh * T + t];
            g[u] = t < len ? gates[t * p.g_t] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = t1 - 1 - lane - u * kWave;
            const double x = t >= t_lo ? static_cast<double>(q[u]) - static_cast<double>(k[u]) : 0.0;
            const uint64_t cuts = __ballot(t >= t_lo && (resets(g[u]) || t == nothing));
            double y;
            if (cuts == 0) {
                const double sum = scan_d(x);
                y = carry + sum;
                carry += uniform_d(sum, kWave - 1);
            } else {
                // A piece ends with the token that resets, the first one in time: the next starts behind it, from 0.
                y = 0.0;
                pieces(cuts << 1, x, lane, [&](int from, int to, double sum) {
                    if (lane >= from && lane < to) y = carry + sum;
                    carry = to < kWave || (cuts >> (kWave - 1)) != 0 ? 0.0 : carry + uniform_d(sum, kWave - 1);
                });
                if ((cuts >> lane) & 1) y = 0.0;
            }
            const float d = t < len ? static_cast<float>(y) : 0.0f;
            lost |= t >= t_lo && !(fabsf(d) < INFINITY);
            if (t >= t_lo) out[static_cast<int64_t>(t) * p.H] = d;
        }
    }
    if (__builtin_expect(__ballot(lost) == 0, 1)) return;
    double start;
    if (si > 0) {
        start = p.cross[bh * p.nseg + si - 1];
    } else if (p.d_state != nullptr) {
        float x = 0.0f;
        for (int64_t e = lane; e < p.one; e += kWave)
            x = fmaf(p.state != nullptr ? p.state[bh * p.one + e] : 0.0f, p.d_state[bh * p.one + e], x);
        start = group_sum<kWave>(x);
    } else {
        return;
    }
    __threadfence_block();   // what the lanes above stored is there for the others
    const int end = min(t_hi, len);
    for (int t0 = t_lo; t0 < end; t0 += kWave) {
        const int t = t0 + lane, at = min(t, end - 1);
        const double x = t < end ? static_cast<double>(p.dk[bh * T + at]) - static_cast<double>(p.dq[bh * T + at]) : 0.0;
        const uint64_t cuts = __ballot(t < end && (resets(gates[at * p.g_t]) || t == nothing));
        double y = 0.0;
        if (cuts & 1) start = 0.0;
        pieces(cuts, x, lane, [&](int from, int to, double sum) {   // a piece starts with the token that resets, from 0
            if (from > 0) start = 0.0;
            const double before = dpp_d<0x138, 0xF>(sum);   // wave_shr:1: the sum of the tokens before the lane's
            if (lane >= from && lane < to) y = start + (lane == from ? 0.0 : before);
            start += uniform_d(sum, kWave - 1);
        });
        const float d = static_cast<float>(y);
        float* o = out + static_cast<int64_t>(at) * p.H;
        if (t < end && fabsf(d) < INFINITY && !(fabsf(*o) < INFINITY)) *o = d;
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
// across the block in LDS in a fixed order. Bound by the state's bytes, read once and written once: 256 requests
// of 16 heads of 128 x 128 take 111 us, 4.9 TB/s (a copy of as much: 103).
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
    const float ga = token_factor(io.g[b * io.g_b + h * io.g_h]);
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
                    x[e] = fmaf(kd, v[e], sdm_decayed(ga, x[e]));
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

// Segments of the time axis: 256 blocks of (stream, head, segment), one per compute unit, if there are that many chunks. A
// second block per unit fills the first one's waits but doubles the states that the first kernel writes and the others read:
// it pays where segments stay long. Microseconds at 512 and at 256 blocks, forward / backward, heads of 128: 8 x 4096 tokens
// x 16 heads 230 / 722 and 258 / 803 (segments of 1024 and 2048 tokens); 1 x 16384 x 8 87 / 264 and 84 / 262 (256 and 512);
// 1 x 4096 x 16 63 / 191 and 60 / 174 (128 and 256); 16 x 256 x 16, whole rows at 256 blocks, 37 / 133 and 29 / 97. Down to
// single chunks: 4 x 1000 x 4 (width 100) with segments of 64, 128 and 256 tokens at least 45 / 125, 56 / 180 and 85 / 287.
constexpr int kGlrUnits = 256;
constexpr int kGlrLongSeg = 1024;
// Up to so many segments, each block adds up the segments before it by itself (half of them on average); past that a kernel
// chains the states in place. 8 x 4096 x 16, 4 segments: 230 by themselves, 248 chained; 2 x 2048 x 16 backward, 8
// segments: 230 and 174.
constexpr int kGlrOwnChain = 4;
struct SegPlan {
    int nseg, seg;
};
SegPlan seg_plan(int64_t bh, int T) {
    const int64_t chunks = (static_cast<int64_t>(T) + kL - 1) / kL;
    auto at = [&](int64_t blocks) {   // chunks per segment
        const int64_t want = (blocks + bh - 1) / bh, per = (chunks + want - 1) / want;
        return per < 1 ? 1 : per;
    };
    int64_t per = at(2 * kGlrUnits);
    if (per * kL < kGlrLongSeg) per = at(kGlrUnits);
    SegPlan s;
    s.seg = static_cast<int>(per * kL);
    s.nseg = static_cast<int>(chunks > 0 ? (chunks + per - 1) / per : 1);
    return s;
}

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
    const size_t tiles = out ? 2 * KD + VD : (sizeof(T) == 2 ? 2 : 1) * (KD + VD);
    return kL * tiles * sizeof(T) + (out ? 6 * kParts<T> * kWave * 8 * sizeof(T) : 0) + 2 * sizeof(Gates) +
           VD / 16 * kL * sizeof(float);
}

template <typename T, int KD, int VD, bool REV, bool OUT, bool DOT, bool FOLD>
hipError_t glr_go3(const GlrPass& p, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.H * (OUT ? p.nseg : p.nseg - 1));
    glr_kernel<T, KD, VD, REV, OUT, DOT, FOLD><<<grid, 4 * VD, glr_lds<T, KD, VD>(OUT), st>>>(p);
    return hipGetLastError();
}
template <typename T, bool REV, bool OUT, bool DOT, bool FOLD>
hipError_t glr_go2(const GlrPass& p, hipStream_t st) {
    const int kd = padded(p.y.width), vd = padded(p.z.width);
    if (kd == 64) return vd == 64 ? glr_go3<T, 64, 64, REV, OUT, DOT, FOLD>(p, st) : glr_go3<T, 64, 128, REV, OUT, DOT, FOLD>(p, st);
    return vd == 64 ? glr_go3<T, 128, 64, REV, OUT, DOT, FOLD>(p, st) : glr_go3<T, 128, 128, REV, OUT, DOT, FOLD>(p, st);
}
template <bool REV, bool OUT, bool DOT>
hipError_t glr_go(const GlrPass& p, int dtype, hipStream_t st) {
    // float32 results are not narrowed: one instance whatever out_f32.
    if (dtype != SDM_BF16) return glr_go2<float, REV, OUT, DOT, false>(p, st);
    if constexpr (DOT) {
        if (p.out_f32) return glr_go2<bf16_t, REV, OUT, DOT, true>(p, st);
    }
    return glr_go2<bf16_t, REV, OUT, DOT, false>(p, st);
}

// The segments' own states (y z^T), then chained when there are many.
template <bool REV>
hipError_t seg_states(GlrPass p, int dtype, int64_t one, int64_t bh, hipStream_t st) {
    hipError_t e = glr_go<REV, false, false>(p, dtype, st);
    if (e != hipSuccess || !p.chained) return e;
    const int64_t total = bh * one;
    glr_chain_kernel<REV><<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(p.segs, p.decays, p.start, p.nseg, one, total);
    return hipGetLastError();
}

template <typename T, bool REV, bool OUT, bool DOT, bool FOLD>
void list(const void** all, int& n) {
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 64, 64, REV, OUT, DOT, FOLD>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 64, 128, REV, OUT, DOT, FOLD>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 128, 64, REV, OUT, DOT, FOLD>);
    all[n++] = reinterpret_cast<const void*>(&glr_kernel<T, 128, 128, REV, OUT, DOT, FOLD>);
}
template <typename T>
void list_type(const void** all, int& n) {
    list<T, false, true, false, false>(all, n);   // o
    list<T, true, true, false, false>(all, n);    // dv
    list<T, false, true, true, false>(all, n);     // dq
    list<T, true, true, true, false>(all, n);      // dk
    if constexpr (sizeof(T) == 2) {
        list<T, false, true, true, true>(all, n);
        list<T, true, true, true, true>(all, n);
    }
    list<T, false, false, false, false>(all, n);
    list<T, true, false, false, false>(all, n);
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
    p.chained = sp.nseg > kGlrOwnChain;
    p.m_p = p.m_o = p.m_s = 1.0f;
    return p;
}

}  // namespace

int glr_lds_kernels(const void** fns, int cap) {
    const void* all[96];
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
    p.start = io->state;
    p.s_k = io->dv;
    p.s_v = 1;
    hipError_t e = hipSuccess;
    if (sp.nseg > 1) {
        p.segs = reinterpret_cast<float*>(ws + l.s);
        p.decays = reinterpret_cast<float*>(ws + l.sd);
        if ((e = seg_states<false>(p, io->dtype, one, bh, st)) != hipSuccess) return e;
    }
    p.last = io->last;
    p.m_p = p.m_o = io->scale;
    p.out = io->o;
    p.o_b = io->o_b;
    p.o_t = io->o_t;
    p.o_h = io->o_h;
    p.out_wide = reinterpret_cast<uintptr_t>(io->o) % (4 * es) == 0 && io->o_b % 4 == 0 && io->o_t % 4 == 0 && io->o_h % 4 == 0 && io->dv % 4 == 0;
    return glr_go<false, true, false>(p, io->dtype, st);
}

hipError_t glr_backward_launch(const sdm_glr_io* io, const sdm_glr_grad* g, hipStream_t st) {
    const int es = io->dtype == SDM_BF16 ? 2 : 4, per = io->H / io->Hk;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H, one = static_cast<int64_t>(io->dk) * io->dv;
    const SegPlan sp = seg_plan(bh, io->T);
    const GlrLayout l = glr_layout(io, true);
    char* ws = static_cast<char*>(io->workspace);
    const Rows q = rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, es), k = rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, es),
               v = rows_of(io->v, io->v_b, io->v_t, io->v_h, io->dv, 1, es), d = rows_of(g->d_o, g->do_b, g->do_t, g->do_h, io->dv, 1, es);
    hipError_t e = hipSuccess;
    // A pass forwards on the states, and one backwards on their gradients.
    GlrPass fwd = base_pass(io, sp), bwd = fwd;
    fwd.start = io->state;
    bwd.start = g->d_last;
    fwd.s_k = bwd.s_k = io->dv;
    fwd.s_v = bwd.s_v = 1;
    bwd.m_s = io->scale;
    if (sp.nseg > 1) {
        fwd.segs = reinterpret_cast<float*>(ws + l.s);
        fwd.decays = reinterpret_cast<float*>(ws + l.sd);
        bwd.segs = reinterpret_cast<float*>(ws + l.r);
        bwd.decays = reinterpret_cast<float*>(ws + l.rd);
        fwd.y = k;
        fwd.z = v;
        bwd.y = q;
        bwd.z = d;
        if ((e = seg_states<false>(fwd, io->dtype, one, bh, st)) != hipSuccess) return e;
        if ((e = seg_states<true>(bwd, io->dtype, one, bh, st)) != hipSuccess) return e;
    }
    const bool fold = per > 1;
    float* dqd = reinterpret_cast<float*>(ws + l.dqd);
    float* dkd = reinterpret_cast<float*>(ws + l.dkd);
    float* cross = reinterpret_cast<float*>(ws + l.cross);
    auto key_out = [&](GlrPass& p, void* out, size_t at) {   // [B, T, H or Hk, dk], on the transposed states
        p.out = fold ? static_cast<void*>(ws + at) : out;
        p.out_f32 = fold;
        p.o_h = io->dk;
        p.o_t = static_cast<int64_t>(io->H) * io->dk;
        p.o_b = p.o_t * io->T;
        p.out_wide = io->dk % 4 == 0;
        p.s_k = 1;
        p.s_v = io->dv;
    };
    {   // dq: keys and values exchanged
        GlrPass p = fwd;
        p.x = d;
        p.y = v;
        p.z = k;
        p.w = q;
        p.m_p = p.m_o = io->scale;
        key_out(p, g->dq, l.fq);
        p.dot = dqd;
        p.cross = cross;
        p.r_start = bwd.start;
        p.r_segs = bwd.segs;
        p.r_decays = bwd.decays;
        if ((e = glr_go<false, true, true>(p, io->dtype, st)) != hipSuccess) return e;
    }
    {   // dk
        GlrPass p = bwd;
        p.x = v;
        p.y = d;
        p.z = q;
        p.w = k;
        p.m_p = io->scale;
        key_out(p, g->dk, l.fk);
        p.dot = dkd;
        if ((e = glr_go<true, true, true>(p, io->dtype, st)) != hipSuccess) return e;
    }
    {   // dv
        GlrPass p = bwd;
        p.x = k;
        p.y = q;
        p.z = d;
        p.m_p = io->scale;
        p.last = g->d_state;
        p.out = g->dv;
        p.o_h = io->dv;
        p.o_t = static_cast<int64_t>(io->H) * io->dv;
        p.o_b = p.o_t * io->T;
        p.out_wide = io->dv % 4 == 0;
        if ((e = glr_go<true, true, false>(p, io->dtype, st)) != hipSuccess) return e;
    }
    if (io->T == 0) return hipSuccess;
    const int64_t waves = bh * sp.nseg;
    const GateGrad gg{dqd, dkd, cross, io->g, io->g_b, io->g_t, io->g_h, io->lens, io->state, g->d_state, one, g->dg, io->T, io->H,
                      sp.nseg, sp.seg, waves};
    glr_gate_grad_kernel<<<static_cast<unsigned>((waves * kWave + 255) / 256), 256, 0, st>>>(gg);
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
