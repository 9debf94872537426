// The gated delta rule with a dense state per head, forward, backward and by one token:
//     u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),    S_t = exp(g_t) S_{t-1} + k_t u_t^T,    o_t = scale S_t^T q_t.
//
// In chunks of L = 64 tokens, with G_i the sum of the chunk's gates up to i, S the state before it, D_ij = exp(G_i - G_j),
// r_i = u_i / beta_i what the state misses of v_i, and A_ij = D_ij (k_i . k_j) for j < i:
//     r = y - A (beta r),  y_i = v_i - exp(G_i) S^T k_i,    so    r = y - N (beta y),   N = (1 + A diag(beta))^-1 A;
//     o_i = scale (exp(G_i) S^T q_i + sum_{j <= i} D_ij (q_i . k_j) u_j),
//     S'  = exp(G_L) S + sum_j exp(G_L - G_j) k_j u_j^T.
// N is strictly lower triangular and has no division by beta; the gradient of u goes through its transpose.
#include <hip/hip_runtime.h>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"
#include "tiles.hpp"

namespace sdm {
namespace {

constexpr int kRow = 68;      // floats between the rows of a 64 x 64 matrix in LDS
constexpr int kFacBytes = 4 * kL * 4;

// Bytes of a chunk's score operands (Pairs) in all their parts.
template <typename T>
constexpr int kFragBytes = 6 * kParts<T> * kWave * 8 * static_cast<int>(sizeof(T));

// A chunk's factors, in its record behind the operands.
struct Factors {
    float f[kL];      // exp(G_i)
    float u[kL];      // exp(G_L - G_i)
    float beta[kL];   // 0 past the row's last token
    float one[kL];    // exp(g_i)
};
static_assert(sizeof(Factors) == kFacBytes, "a KiB");

// c += a b^T of two operands in parts: all products of 24 bits, the smallest first.
template <typename T, int NP>
__device__ __forceinline__ void mma_parts(const Parts<T, NP>& a, const Parts<T, NP>& b, f32x4& c) {
    if constexpr (NP == 3) {
        mma(a.p[2], b.p[0], c);
        mma(a.p[0], b.p[2], c);
        mma(a.p[1], b.p[1], c);
        mma(a.p[1], b.p[0], c);
        mma(a.p[0], b.p[1], c);
    }
    mma(a.p[0], b.p[0], c);
}

// Operand `pr` of a record's operands, as the lane holds it.
template <typename T, int NP>
__device__ __forceinline__ void frag_read(const char* at, int pr, int lane, Parts<T, NP>& o) {
#pragma unroll
    for (int s = 0; s < NP; ++s) __builtin_memcpy(&o.p[s], at + ((pr * NP + s) * kWave + lane) * (8 * static_cast<int>(sizeof(T))), sizeof(Frag<T>));
}
template <typename T, int NP>
__device__ __forceinline__ void frag_write(char* at, int pr, int lane, const Parts<T, NP>& o) {
#pragma unroll
    for (int s = 0; s < NP; ++s) __builtin_memcpy(at + ((pr * NP + s) * kWave + lane) * (8 * static_cast<int>(sizeof(T))), &o.p[s], sizeof(Frag<T>));
}

__device__ __forceinline__ int live_tokens(const int32_t* lens, int b, int T) {
    const int n = lens != nullptr ? lens[b] : T;
    return n < 0 ? 0 : n > T ? T : n;
}

// ------------------------------------------------------------------------------------------ chunk records
//
// What of a chunk does not depend on the state, for every chunk at once: N, the scores of its tokens, and its factors,
// as the operands that the kernels along the time axis take. Forward: N and D (q k^T). Backward: N, N^T and D (q k^T)
// transposed. A block of four waves per chunk. N's diagonal blocks of 16 come from substitution (a column of a
// block per lane, all four blocks at once), the rest by block columns, a wave each, through float32 products.
struct ChunkArgs {
    Rows q, k;
    const float *g, *beta;
    int64_t g_b, g_t, g_h, e_b, e_t, e_h;
    const int32_t* lens;
    int T, H, chunks;
    float scale;
    char* rec;
};

template <typename T, bool BACK>
constexpr int kRecBytes = (BACK ? 3 : 2) * kFragBytes<T> + kFacBytes;

template <typename T, int KD, bool BACK>
__global__ __launch_bounds__(256) void gdr_chunk_kernel(ChunkArgs p) {
    constexpr int KB = KD / 32, NP = kParts<T>;
    extern __shared__ __align__(16) char lds[];
    T* kt = reinterpret_cast<T*>(lds);
    T* qt = kt + kL * KD;
    float* A = reinterpret_cast<float*>(qt + kL * KD);
    float* N = A + kL * kRow;
    float* beta = N + kL * kRow;
    Gates& gates = *reinterpret_cast<Gates*>(beta + kL);

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int bh = blk / p.chunks, c = blk - bh * p.chunks, b = bh / p.H, h = bh - b * p.H;
    const int left = live_tokens(p.lens, b, p.T) - c * kL;
    if (left <= 0) return;
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(c) * kL;
    char* rec = p.rec + static_cast<int64_t>(blk) * kRecBytes<T, BACK>;

    Stage<T, KD, 256> sq, sk;
    sk.init(p.k);
    sq.init(p.q);
    sk.fill(p.k, static_cast<const T*>(p.k.p) + b * p.k.b + (h / p.k.per) * p.k.h + t0 * p.k.t, left, kt, wave, tid);
    sq.fill(p.q, static_cast<const T*>(p.q.p) + b * p.q.b + (h / p.q.per) * p.q.h + t0 * p.q.t, left, qt, wave, tid);
    if (wave == 3) {
        const int64_t t = t0 + min(lane, left - 1);
        const bool live = lane < left;
        const float g = live ? p.g[b * p.g_b + t * p.g_t + h * p.g_h] : 0.0f;
        const float e = live ? p.beta[b * p.e_b + t * p.e_t + h * p.e_h] : 0.0f;
        gate_factors<false>(g, 1.0f, 1.0f, gates, lane);
        beta[lane] = e;
        Factors* f = reinterpret_cast<Factors*>(rec + kRecBytes<T, BACK> - kFacBytes);
        f->f[lane] = gates.f[lane];
        f->u[lane] = gates.u[lane];
        f->beta[lane] = e;
        f->one[lane] = exp2_of(static_cast<double>(g < kGateMin ? kGateMin : g) * kLog2E);
    }
    tile_barrier();

    // Tiles of 16 x 16 tokens: twelve of the scores, dealt to the waves with the ten of A.
    char* const scores = rec + (BACK ? 2 : 1) * kFragBytes<T>;
    for (int e = wave; e < 22; e += 4) {
        int it = 0, jt = 0;
        const bool isA = e >= 12;
        if (isA) {
            const int n = e - 12;   // (it, jt), jt <= it, by rows
            it = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0;
            jt = n - it * (it + 1) / 2;
        } else {
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                if (k == e >> 1) {
                    it = Pairs<BACK>::kIt[k];
                    jt = 2 * Pairs<BACK>::kJb[k] + (e & 1);
                }
            }
        }
        const bool rev = BACK && !isA;
        T* const x = !isA && !BACK ? qt : kt;
        T* const y = !isA && BACK ? qt : kt;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // token 16 jt + 4 quarter + r down, token 16 it + lane % 16 across
        if (rev ? jt >= it : jt <= it) {
            f32x4 a = {0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) mma(row_frag<KD>(y, 16 * jt + i16, kb, qd), row_frag<KD>(x, 16 * it + i16, kb, qd), a);
            const float m = isA ? 1.0f : p.scale;
            if (jt == it) {
                const float lhi = gates.lhi[16 * it + i16], llo = gates.llo[16 * it + i16];
                const f32x4 jh = *reinterpret_cast<const f32x4*>(&gates.lhi[16 * jt + 4 * qd]);
                const f32x4 jl = *reinterpret_cast<const f32x4*>(&gates.llo[16 * jt + 4 * qd]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 4 * qd + r;
                    const float d = (lhi - jh[r]) + (llo - jl[r]);
                    const float w = __builtin_amdgcn_exp2f(rev ? -d : d);
                    s[r] = (rev ? j >= i16 : isA ? j < i16 : j <= i16) ? sdm_decayed(w * m, a[r]) : 0.0f;
                }
            } else {
                const float ot = (rev ? gates.down : gates.up)[16 * it + i16] * (m * gates.tau[4 * it + jt]);
                const f32x4 d = *reinterpret_cast<const f32x4*>(&(rev ? gates.up : gates.down)[16 * jt + 4 * qd]);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = sdm_decayed(ot * d[r], a[r]);
            }
        }
        if (isA) {
            *reinterpret_cast<f32x4*>(A + (16 * it + i16) * kRow + 16 * jt + 4 * qd) = f32x4{s[0], s[1], s[2], s[3]};
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                *reinterpret_cast<u32x2*>(scores + (((e >> 1) * NP + k) * kWave + lane) * 16 + 8 * (e & 1)) =
                    u32x2{__builtin_amdgcn_perm(__float_as_uint(s[1]), __float_as_uint(s[0]), 0x07060302u),
                          __builtin_amdgcn_perm(__float_as_uint(s[3]), __float_as_uint(s[2]), 0x07060302u)};
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] -= __uint_as_float(__float_as_uint(s[r]) & 0xFFFF0000u);
            }
        } else {
            *reinterpret_cast<f32x4*>(scores + ((e >> 1) * kWave + lane) * 32 + 16 * (e & 1)) = f32x4{s[0], s[1], s[2], s[3]};
        }
    }
    lds_barrier();

    if (wave == 0) {   // diagonal blocks: lane (quarter, i) has column i of block `quarter`
        const float* D = A + 16 * qd * kRow + 16 * qd;
        float xb[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = D[i * kRow + i16];
#pragma unroll
            for (int m = 0; m < i; ++m) x = fmaf(-D[i * kRow + m], xb[m], x);
            xb[i] = beta[16 * qd + i] * x;
            N[(16 * qd + i) * kRow + 16 * qd + i16] = x;
        }
    }
    lds_barrier();
    if (wave < 3) {   // block column `wave`, downwards: N_ij = (1 - N_ii beta) (A_ij - sum_{j <= m < i} A_im beta N_mj)
        f32x4 bn[4];   // beta N of the column's blocks, rows 4 quarter + r
        auto weigh = [&](int m, f32x4 x) { return x * *reinterpret_cast<const f32x4*>(&beta[16 * m + 4 * qd]); };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 x;
            if (i == wave) {
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = N[(16 * i + 4 * qd + r) * kRow + 16 * i + i16];
                bn[i] = weigh(i, x);
            }
            if (i <= wave) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = A[(16 * i + 4 * qd + r) * kRow + 16 * wave + i16];
#pragma unroll
            for (int m = 0; m < i; ++m) {
                if (m < wave) continue;
                const f32x4 a = *reinterpret_cast<const f32x4*>(A + (16 * i + i16) * kRow + 16 * m + 4 * qd);
#pragma unroll
                for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[e], bn[m][e], x, 0, 0, 0);
            }
            const f32x4 a = *reinterpret_cast<const f32x4*>(N + (16 * i + i16) * kRow + 16 * i + 4 * qd), bx = weigh(i, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[e], bx[e], x, 0, 0, 0);
            bn[i] = weigh(i, x);
#pragma unroll
            for (int r = 0; r < 4; ++r) N[(16 * i + 4 * qd + r) * kRow + 16 * wave + i16] = x[r];
        }
    }
    lds_barrier();

    for (int e = wave; e < (BACK ? 12 : 6); e += 4) {
        const bool tr = e >= 6;
        const int pr = tr ? e - 6 : e;
        int it = 0, jb = 0;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            if (k == pr) {
                it = tr ? Pairs<true>::kIt[k] : Pairs<false>::kIt[k];
                jb = tr ? Pairs<true>::kJb[k] : Pairs<false>::kJb[k];
            }
        }
        float x[8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int jt = 2 * jb + s;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (tr) x[4 * s + r] = jt >= it ? N[(16 * jt + 4 * qd + r) * kRow + 16 * it + i16] : 0.0f;
                else x[4 * s + r] = jt <= it ? N[(16 * it + i16) * kRow + 16 * jt + 4 * qd + r] : 0.0f;
            }
        }
        Parts<T, NP> o;
        cut(x, o);
        frag_write(rec + (tr ? kFragBytes<T> : 0), pr, lane, o);
    }
}

// ---------------------------------------------------------------------------------------- along the time axis
//
// A block owns 64 columns of one (stream, head)'s state, 16 for each of its four waves, in registers over all chunks
// as the accumulators of 16 x 16 matrix-product tiles; columns do not meet, so the waves only share the tiles in LDS.
struct MainArgs {
    Rows q, k, v;
    const int32_t* lens;
    int T, H, chunks, cols;   // cols: blocks of 64 columns
    int kd, vd;
    float scale;
    const char* rec;
    const float* start;       // [B H] states [kd, vd] (NULL: zero)
    float* last;              // [B H] (NULL: not kept)
    void* out;                // [B, T, H, vd] (OUT)
    int64_t o_b, o_t, o_h;
    int out_wide;
    float* states;            // the states before every chunk [B H, chunks] (!OUT), and r [B H, T, vd]
    float* miss;
};

// A wave's part of a state: rows 32 (d / 2) + 8 quarter + 4 (d % 2) + r of tile d, one column per lane, read and written
// through a buffer descriptor of the state's range; what lies past its widths is out of it (zero, and not written).
template <int KT>
struct StateAt {
    uint32_t at0;
    int vd, kd, col, qd;
    __device__ __forceinline__ StateAt(int col_, int qd_, int kd_, int vd_) : vd(vd_), kd(kd_), col(col_), qd(qd_) {
        at0 = 4u * static_cast<uint32_t>(col_ + 8 * qd_ * vd_);
    }
    __device__ __forceinline__ int at(int d, int r) const {
        const int k = 32 * (d >> 1) + 4 * (d & 1) + r;
        return static_cast<int>(col < vd && k + 8 * qd < kd ? at0 + 4u * static_cast<uint32_t>(k * vd) : 0xC0000000u);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t of(const float* s) const {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(s), 0, kd * vd * 4, 0x00027000);
    }
    __device__ __forceinline__ void read(const float* p, f32x4 (&S)[KT]) const {
        const auto s = of(p);
#pragma unroll
        for (int d = 0; d < KT; ++d) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[d][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(s, at(d, r), 0, 0));
        }
    }
    __device__ __forceinline__ void write(float* p, const f32x4 (&S)[KT]) const {
        const auto s = of(p);
#pragma unroll
        for (int d = 0; d < KT; ++d) {
#pragma unroll
            for (int r = 0; r < 4; ++r) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[d][r]), s, at(d, r), 0, 0);
        }
    }
};

// Copies KiB pieces of a record to LDS, dealt to four waves: the first n, then the factors.
__device__ __forceinline__ void record_fill(const char* rec, int n, int fac_off, char* to, int wave, int lane) {
    const u32x4 rsrc = buffer_of(rec, fac_off + kFacBytes);
    for (int i = wave; i <= n; i += 4) to_lds16(rsrc, to + i * 1024, static_cast<uint32_t>((i < n ? i * 1024 : fac_off) + lane * 16));
}

// 8 tokens' values at one column, as col_frag gives them.
template <typename T>
__device__ __forceinline__ float tile_at(T* tile, int row, int col) {
    constexpr int kElems = 16 / static_cast<int>(sizeof(T));
    return widen(*reinterpret_cast<const T*>(piece<T, 64>(tile, row, col / kElems) + (col % kElems) * static_cast<int>(sizeof(T))));
}

template <typename T>
__device__ __forceinline__ void store_four(void* out, int64_t at, f32x4 v, int left, int wide) {
    T* o = static_cast<T*>(out) + at;
    if (wide) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(o) = v;
        else *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < left) o[r] = narrow<T>(v[r]);
        }
    }
}

// OUT: the outputs (and the last state); else the states before every chunk and the rows r, for the backward pass.
template <typename T, int KD, bool OUT>
__global__ __launch_bounds__(256, 1) void gdr_kernel(MainArgs p) {
    constexpr int KB = KD / 32, KT = KD / 16, NP = kParts<T>;
    constexpr int kBufs = sizeof(T) == 2 ? 2 : 1;   // float32 tiles of two chunks do not fit
    constexpr int kTile = kL * KD * static_cast<int>(sizeof(T)), kTileV = kL * 64 * static_cast<int>(sizeof(T));
    constexpr int kN = kFragBytes<T> / 1024;
    constexpr int kBuf = (OUT ? 2 : 1) * kTile + kTileV + (OUT ? 2 : 1) * kFragBytes<T> + kFacBytes;
    extern __shared__ __align__(16) char lds[];

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int bh = blk / p.cols, cb = blk - bh * p.cols, b = bh / p.H, h = bh - b * p.H;
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int c0 = 64 * cb, n0 = 16 * wave, vw = min(64, p.vd - c0);   // the block's columns, the wave's first among them
    const int len = __builtin_amdgcn_readfirstlane(live_tokens(p.lens, b, p.T)), chunks = (len + kL - 1) / kL;

    Rows vr = p.v;
    vr.width = vw;
    const T* qb = OUT ? static_cast<const T*>(p.q.p) + b * p.q.b + (h / p.q.per) * p.q.h : nullptr;
    const T* kb_ = static_cast<const T*>(p.k.p) + b * p.k.b + (h / p.k.per) * p.k.h;
    const T* vb = static_cast<const T*>(p.v.p) + b * p.v.b + h * p.v.h + c0;
    const int64_t one = static_cast<int64_t>(p.kd) * p.vd;
    const StateAt<KT> place(c0 + n0 + i16, qd, p.kd, p.vd);

    f32x4 S[KT];
#pragma unroll
    for (int d = 0; d < KT; ++d) S[d] = f32x4{0, 0, 0, 0};
    if (p.start != nullptr) place.read(p.start + bh * one, S);

    Stage<T, KD, 256> sq, sk;
    Stage<T, 64, 256> sv;
    if (OUT) sq.init(p.q);
    sk.init(p.k);
    sv.init(vr);
    auto tiles = [&](int buf) { return lds + buf * kBuf; };
    auto fill = [&](int c, int buf) {
        const int64_t t0 = static_cast<int64_t>(c) * kL;
        const int left = len - c * kL;
        char* at = tiles(buf);
        sk.fill(p.k, kb_ + t0 * p.k.t, left, reinterpret_cast<T*>(at), wave, tid);
        sv.fill(vr, vb + t0 * p.v.t, left, reinterpret_cast<T*>(at + kTile), wave, tid);
        if (OUT) sq.fill(p.q, qb + t0 * p.q.t, left, reinterpret_cast<T*>(at + kTile + kTileV), wave, tid);
        record_fill(p.rec + (static_cast<int64_t>(bh) * p.chunks + c) * kRecBytes<T, !OUT>, (OUT ? 2 : 1) * kN,
                    kRecBytes<T, !OUT> - kFacBytes, at + (OUT ? 2 : 1) * kTile + kTileV, wave, lane);
    };
    if (chunks > 0) fill(0, 0);

    for (int c = 0; c < chunks; ++c) {
        const int buf = kBufs == 2 ? __builtin_amdgcn_readfirstlane(c & 1) : 0, t0 = c * kL, left = len - t0;
        char* const at = tiles(buf);
        T* const kt = reinterpret_cast<T*>(at);
        T* const vt = reinterpret_cast<T*>(at + kTile);
        T* const qt = reinterpret_cast<T*>(at + kTile + kTileV);
        const char* const nf = at + (OUT ? 2 : 1) * kTile + kTileV;
        const char* const pf = nf + kFragBytes<T>;
        const Factors& fac = *reinterpret_cast<const Factors*>(nf + (OUT ? 2 : 1) * kFragBytes<T>);
        tile_barrier();   // the chunk's tiles are complete, and the other buffer's are free
        if (kBufs == 2 && c + 1 < chunks) fill(c + 1, buf ^ 1);
        if (!OUT) place.write(p.states + (static_cast<int64_t>(bh) * p.chunks + c) * one, S);

        // S^T k and S^T q
        f32x4 Y[4], O[4];   // Y, tile it: tokens 16 it + 4 quarter + r down, column n0 + lane % 16; O: transposed
#pragma unroll
        for (int it = 0; it < 4; ++it) Y[it] = O[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            Parts<T, NP> sp;
            float s[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) { s[r] = S[2 * kb][r]; s[4 + r] = S[2 * kb + 1][r]; }
            cut(s, sp);
            Frag<T> kf[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) kf[it] = row_frag<KD>(kt, 16 * it + i16, kb, qd);
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) {
#pragma unroll
                for (int it = 0; it < 4; ++it) mma(kf[it], sp.p[n], Y[it]);
            }
            if constexpr (OUT) {
                Frag<T> qf[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) qf[it] = row_frag<KD>(qt, 16 * it + i16, kb, qd);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n) {
#pragma unroll
                    for (int it = 0; it < 4; ++it) mma(sp.p[n], qf[it], O[it]);
                }
            }
        }
        // y, then r = y - N (beta y)
        f32x4 X[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) X[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            float v[8], w[8];
            widen8(col_frag<64, 4>(vt, jb, n0, i16, qd), v);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 f = *reinterpret_cast<const f32x4*>(&fac.f[32 * jb + 16 * s + 4 * qd]);
                const f32x4 be = *reinterpret_cast<const f32x4*>(&fac.beta[32 * jb + 16 * s + 4 * qd]);
                f32x4& y = Y[2 * jb + s];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    y[r] = v[4 * s + r] - sdm_decayed(f[r], y[r]);
                    w[4 * s + r] = be[r] * y[r];
                }
            }
            Parts<T, NP> yp;
            cut(w, yp);
#pragma unroll
            for (int pr = 0; pr < 6; ++pr) {
                if (Pairs<false>::kJb[pr] != jb) continue;
                Parts<T, NP> np;
                frag_read(nf, pr, lane, np);
                mma_parts(np, yp, X[Pairs<false>::kIt[pr]]);
            }
        }
        float odd = 0.0f;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            Y[it] -= X[it];   // r
#pragma unroll
            for (int r = 0; r < 4; ++r) odd = fmaf(Y[it][r], 0.0f, odd);
        }
        if (__builtin_expect(__ballot(odd != odd) != 0, 0)) {
            // Something is not finite: what the products make of that reaches other tokens of the chunk too, so the wave's
            // columns go on token by token, by the definition.
            const int col = c0 + n0 + i16;
            for (int t = 0; t < min(left, kL); ++t) {
                const float a = fac.one[t];
                float pred = 0.0f, o = 0.0f, k[KB][8];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    widen8(row_frag<KD>(kt, t, kb, qd), k[kb]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float s = sdm_decayed(a, S[2 * kb + (e >> 2)][e & 3]);
                        S[2 * kb + (e >> 2)][e & 3] = s;
                        pred = fmaf(s, k[kb][e], pred);
                    }
                }
                pred += lane_xor_f<16>(pred);
                pred += lane_xor_f<32>(pred);
                const float r = tile_at(vt, t, n0 + i16) - pred, u = fac.beta[t] * r;
                float q[8];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    if (OUT) widen8(row_frag<KD>(qt, t, kb, qd), q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float s = 32 * kb + 8 * qd + e < p.kd ? fmaf(k[kb][e], u, S[2 * kb + (e >> 2)][e & 3]) : 0.0f;
                        S[2 * kb + (e >> 2)][e & 3] = s;
                        if (OUT) o = fmaf(s, q[e], o);
                    }
                }
                o += lane_xor_f<16>(o);
                o += lane_xor_f<32>(o);
                if (qd == 0 && col < p.vd) {
                    if (OUT) static_cast<T*>(p.out)[b * p.o_b + h * p.o_h + static_cast<int64_t>(t0 + t) * p.o_t + col] = narrow<T>(p.scale * o);
                    else p.miss[(static_cast<int64_t>(bh) * p.T + t0 + t) * p.vd + col] = r;
                }
            }
        } else {
            if constexpr (OUT) {
#pragma unroll
                for (int it = 0; it < 4; ++it) O[it] = decayed(fac.f[16 * it + i16] * p.scale, O[it]);
            }
            const float all = fac.f[kL - 1];
#pragma unroll
            for (int d = 0; d < KT; ++d) S[d] = decayed(all, S[d]);
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                float w[8], z[8];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const f32x4 be = *reinterpret_cast<const f32x4*>(&fac.beta[32 * jb + 16 * s + 4 * qd]);
                    const f32x4 f = *reinterpret_cast<const f32x4*>(&fac.u[32 * jb + 16 * s + 4 * qd]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        w[4 * s + r] = be[r] * Y[2 * jb + s][r];
                        z[4 * s + r] = sdm_decayed(f[r], w[4 * s + r]);
                    }
                }
                // The state takes the tokens' u
                Parts<T, NP> zp;
                cut(z, zp);
#pragma unroll
                for (int d = 0; d < KT; d += 4) {
                    Frag<T> kf[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) kf[e] = col_frag<KD, 8>(kt, jb, 32 * ((d + e) >> 1) + 4 * (e & 1), i16, qd);
#pragma unroll
                    for (int n = NP - 1; n >= 0; --n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) mma(kf[e], zp.p[n], S[d + e]);
                    }
                }
                if constexpr (OUT) {
                    Parts<T, NP> up;
                    cut(w, up);
#pragma unroll
                    for (int pr = 0; pr < 6; ++pr) {
                        if (Pairs<false>::kJb[pr] != jb) continue;
                        Parts<T, NP> pp;
                        frag_read(pf, pr, lane, pp);
                        mma_parts(up, pp, O[Pairs<false>::kIt[pr]]);
                    }
                }
            }
            if constexpr (OUT) {
                const int n = c0 + n0 + 4 * qd;   // the lane's result columns n .. n + 3, of token 16 it + lane % 16
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    if (16 * it + i16 >= left || n >= p.vd) continue;
                    store_four<T>(p.out, b * p.o_b + h * p.o_h + static_cast<int64_t>(t0 + 16 * it + i16) * p.o_t + n, O[it], p.vd - n, p.out_wide);
                }
            } else {
                float* miss = p.miss + (static_cast<int64_t>(bh) * p.T + t0) * p.vd + c0 + n0 + i16;
#pragma unroll
                for (int it = 0; it < 4; ++it) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * it + 4 * qd + r;
                        if (t < left && n0 + i16 < vw) miss[static_cast<int64_t>(t) * p.vd] = Y[it][r];
                    }
                }
            }
        }
        if (kBufs == 1) {
            lds_barrier();   // the tiles are free
            if (c + 1 < chunks) fill(c + 1, 0);
        }
    }
    if constexpr (OUT) {
        // Tokens past the row's length.
        for (int64_t e = tid; e < static_cast<int64_t>(p.T - len) * vw; e += 256) {
            const int t = len + static_cast<int>(e / vw), col = c0 + static_cast<int>(e % vw);
            static_cast<T*>(p.out)[b * p.o_b + t * p.o_t + h * p.o_h + col] = narrow<T>(0.0f);
        }
    }
    if (p.last != nullptr) place.write(p.last + bh * one, S);
}

// ------------------------------------------------------------------------------------------ one token
//
// A block owns up to 64 columns of one request's state, all their rows in its lanes' registers: read once, with both
// products (S^T k and S^T q) summed across the block in LDS in a fixed order, updated and written once;
// o = scale (exp(g) S^T q + (q . k) u).
struct GdrStep {
    sdm_gdr_step_io io;
    int cols, tiles;
};

template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&x)[V]) {
    if constexpr (V == 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = w[e];
    } else {
        x[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&x)[V]) {
    if constexpr (V == 4) *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
    else *p = x[0];
}

template <typename T, int V>
__global__ __launch_bounds__(256) void gdr_step_kernel(GdrStep a) {
    const sdm_gdr_step_io& io = a.io;
    __shared__ float qk[2][128];
    __shared__ float part[2][256 * V];
    __shared__ float us[64];
    const int tile = static_cast<int>(blockIdx.x % a.tiles);
    const int64_t bh = blockIdx.x / a.tiles;
    const int b = static_cast<int>(bh / io.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * io.H), hk = h / (io.H / io.Hk);
    const int n0 = tile * a.cols, nc = min(a.cols, io.dv - n0);
    const int64_t row = io.slots != nullptr ? io.slots[b] : b;
    T* o = static_cast<T*>(io.o) + b * io.o_b + h * io.o_h + n0;
    const int tid = static_cast<int>(threadIdx.x);
    if (row < 0 || row >= io.rows) {
        for (int n = tid; n < nc; n += 256) o[n] = narrow<T>(0.0f);
        return;
    }
    constexpr int kU = 32 / V;   // rows of a lane: 64 columns of 128 rows over 256 lanes
    const int per_row = (nc + V - 1) / V, groups = 256 / per_row;
    const int rg = tid / per_row, c = tid - rg * per_row;
    const bool on = rg < groups;
    const int64_t base = (row * io.H + h) * static_cast<int64_t>(io.dk) * io.dv + n0 + c * V;
    const float* from = io.state + base;
    float* to = io.new_state + base;
    float s[kU][V];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int d = rg + u * groups;
        load_row<V>(from + min(d, io.dk - 1) * io.dv, s[u]);   // rows past the last are not used
    }
    if (tid < 128) {
        qk[0][tid] = tid < io.dk ? widen((static_cast<const T*>(io.q) + b * io.q_b + hk * io.q_h)[tid]) : 0.0f;
    } else {
        qk[1][tid - 128] = tid - 128 < io.dk ? widen((static_cast<const T*>(io.k) + b * io.k_b + hk * io.k_h)[tid - 128]) : 0.0f;
    }
    const float ga = expf(io.g[b * io.g_b + h * io.g_h]);
    const float v = tid < nc ? widen((static_cast<const T*>(io.v) + b * io.v_b + h * io.v_h)[n0 + tid]) : 0.0f;
    const float beta = io.beta[b * io.e_b + h * io.e_h];
    __syncthreads();
    float sq[V], sk[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sq[e] = sk[e] = 0.0f;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int d = rg + u * groups, at = min(d, 127);
        const float qd = qk[0][at], kd = qk[1][at];   // 0 past the last row
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[u][e] = d < io.dk ? sdm_decayed(ga, s[u][e]) : 0.0f;
            sq[e] = fmaf(qd, s[u][e], sq[e]);
            sk[e] = fmaf(kd, s[u][e], sk[e]);
        }
    }
    if (on) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            part[0][(rg * per_row + c) * V + e] = sq[e];
            part[1][(rg * per_row + c) * V + e] = sk[e];
        }
    }
    const int lane = static_cast<int>(lane_id());
    const float dot = group_sum<kWave>(fmaf(qk[0][lane], qk[1][lane], qk[0][lane + 64] * qk[1][lane + 64]));
    __syncthreads();
    if (tid < nc) {
        float q = 0.0f, k = 0.0f;
        for (int r = 0; r < groups; ++r) {
            q += part[0][r * per_row * V + tid];
            k += part[1][r * per_row * V + tid];
        }
        const float u = beta * (v - k);
        us[tid] = u;
        o[tid] = narrow<T>(io.scale * fmaf(dot, u, q));
    }
    __syncthreads();
    if (!on) return;
    float x[V];
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = us[c * V + e];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int d = rg + u * groups;
        const float kd = qk[1][min(d, 127)];
#pragma unroll
        for (int e = 0; e < V; ++e) s[u][e] = fmaf(kd, x[e], s[u][e]);
        if (d < io.dk) store_row<V>(to + d * io.dv, s[u]);
    }
}

// --------------------------------------------------------------------------------------------- plans

template <typename T, int KD>
size_t chunk_lds() { return 2 * kL * KD * sizeof(T) + 2 * kL * kRow * 4 + sizeof(Gates) + kL * 4; }

template <typename T, int KD>
size_t main_lds(bool out) {
    return (sizeof(T) == 2 ? 2 : 1) * (kL * ((out ? 2 : 1) * KD + 64) * sizeof(T) + (out ? 2 : 1) * kFragBytes<T> + kFacBytes);
}

int chunks_of(int T) { return (T + kL - 1) / kL; }

struct GdrLayout {
    size_t rec, total;
};
GdrLayout gdr_layout(const sdm_gdr_io* io) {
    const size_t n = static_cast<size_t>(io->B) * io->H * chunks_of(io->T);
    GdrLayout l{};
    l.rec = 0;
    l.total = up256(n * (io->dtype == SDM_BF16 ? kRecBytes<bf16_t, false> : kRecBytes<float, false>));
    return l;
}

template <typename T, bool BACK>
hipError_t chunk_go(const sdm_gdr_io* io, char* rec, hipStream_t st) {
    const int per = io->H / io->Hk;
    ChunkArgs a{rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, sizeof(T)), rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, sizeof(T)),
                io->g, io->beta, io->g_b, io->g_t, io->g_h, io->e_b, io->e_t, io->e_h, io->lens, io->T, io->H, chunks_of(io->T), io->scale, rec};
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(io->B) * io->H * a.chunks);
    if (padded(io->dk) == 64) gdr_chunk_kernel<T, 64, BACK><<<grid, 256, chunk_lds<T, 64>(), st>>>(a);
    else gdr_chunk_kernel<T, 128, BACK><<<grid, 256, chunk_lds<T, 128>(), st>>>(a);
    return hipGetLastError();
}

template <typename T, bool OUT>
hipError_t main_go(const sdm_gdr_io* io, const MainArgs& a, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(io->B) * io->H * a.cols);
    if (padded(io->dk) == 64) gdr_kernel<T, 64, OUT><<<grid, 256, main_lds<T, 64>(OUT), st>>>(a);
    else gdr_kernel<T, 128, OUT><<<grid, 256, main_lds<T, 128>(OUT), st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const sdm_gdr_io* io, hipStream_t st) {
    const int per = io->H / io->Hk, es = sizeof(T);
    char* rec = static_cast<char*>(io->workspace) + gdr_layout(io).rec;
    if (io->T > 0) {
        const hipError_t e = chunk_go<T, false>(io, rec, st);
        if (e != hipSuccess) return e;
    }
    MainArgs a{};
    a.q = rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, es);
    a.k = rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, es);
    a.v = rows_of(io->v, io->v_b, io->v_t, io->v_h, io->dv, 1, es);
    a.lens = io->lens;
    a.T = io->T;
    a.H = io->H;
    a.chunks = chunks_of(io->T);
    a.cols = (io->dv + 63) / 64;
    a.kd = io->dk;
    a.vd = io->dv;
    a.scale = io->scale;
    a.rec = rec;
    a.start = io->state;
    a.last = io->last;
    a.out = io->o;
    a.o_b = io->o_b;
    a.o_t = io->o_t;
    a.o_h = io->o_h;
    a.out_wide = reinterpret_cast<uintptr_t>(io->o) % (4 * es) == 0 && io->o_b % 4 == 0 && io->o_t % 4 == 0 && io->o_h % 4 == 0 && io->dv % 4 == 0;
    return main_go<T, true>(io, a, st);
}

template <typename T>
void list(const void** all, int& n) {
    all[n++] = reinterpret_cast<const void*>(&gdr_chunk_kernel<T, 64, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_chunk_kernel<T, 128, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_kernel<T, 64, true>);
    all[n++] = reinterpret_cast<const void*>(&gdr_kernel<T, 128, true>);
}

}  // namespace

int gdr_lds_kernels(const void** fns, int cap) {
    const void* all[32];
    int n = 0;
    list<bf16_t>(all, n);
    list<float>(all, n);
    int k = 0;
    for (; k < n && k < cap; ++k) fns[k] = all[k];
    return k;
}

size_t gdr_workspace_bytes(const sdm_gdr_io* io, bool backward) {
    (void)backward;
    return io->B < 1 || io->T < 1 ? 0 : gdr_layout(io).total;
}

hipError_t gdr_forward_launch(const sdm_gdr_io* io, hipStream_t st) {
    return io->dtype == SDM_BF16 ? forward<bf16_t>(io, st) : forward<float>(io, st);
}

hipError_t gdr_step_launch(const sdm_gdr_step_io* io, hipStream_t st) {
    GdrStep a{*io, 64, 1};
    // Narrower column tiles until there are four blocks for each compute unit (or 16 columns a tile).
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    while (a.cols > 16 && bh * ((io->dv + a.cols - 1) / a.cols) < 1024) a.cols /= 2;
    a.tiles = (io->dv + a.cols - 1) / a.cols;
    const unsigned grid = static_cast<unsigned>(bh * a.tiles);
    const bool vec = io->dv % 4 == 0;
    if (io->dtype == SDM_BF16) {
        if (vec) gdr_step_kernel<bf16_t, 4><<<grid, 256, 0, st>>>(a);
        else gdr_step_kernel<bf16_t, 1><<<grid, 256, 0, st>>>(a);
    } else {
        if (vec) gdr_step_kernel<float, 4><<<grid, 256, 0, st>>>(a);
        else gdr_step_kernel<float, 1><<<grid, 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace sdm
