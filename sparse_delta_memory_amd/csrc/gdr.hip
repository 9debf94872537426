// The gated delta rule with a dense state per head, forward, backward and by one token:
//     u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),    S_t = exp(g_t) S_{t-1} + k_t u_t^T,    o_t = scale S_t^T q_t.
//
// In chunks of L = 64 tokens, with G_i the sum of the chunk's gates up to i, S the state before it, D_ij = exp(G_i - G_j),
// r_i = u_i / beta_i what the state misses of v_i, and A_ij = D_ij (k_i . k_j) for j < i:
//     r = y - A (beta r),  y_i = v_i - exp(G_i) S^T k_i,    so    r = y - N (beta y),   N = (1 + A diag(beta))^-1 A;
//     o_i = scale (exp(G_i) S^T q_i + sum_{j <= i} D_ij (q_i . k_j) u_j),
//     S'  = exp(G_L) S + sum_j exp(G_L - G_j) k_j u_j^T.
// N is strictly lower triangular and has no division by beta; the gradient of u goes through its transpose.
//
// Forward: a kernel over all chunks makes what does not depend on the state (N, the scores, the factors), another one goes along
// the chunks. Backward: the chunks' records; the states before every chunk and the rows r (forwards); the gradients of the
// states and of u (backwards); and a kernel over all chunks for the rest. States and their gradients go through memory, float32, a
// state per chunk. With few streams and heads the time axis is cut into segments (seg_plan).
//
// Layout. A wave owns 16 columns of the state in registers, as the accumulators of 16 x 16 matrix products (rows: the key
// dimension); cut into bfloat16 parts they are directly an operand of the products with k and q, and so are the results of
// those (y, r) of the products with N, the scores and k: nothing of the state or of r passes through LDS. Columns do not meet, so
// the waves share nothing but the chunk's tiles.
//
// Numbers. Products of bfloat16 inputs are exact; a float32 factor is cut into three bfloat16 parts, 24 bits, and a product of
// two such factors into the six products that count. float32 inputs go through the float32 matrix instructions. N's substitution
// is float32. Gates are summed in float64 per chunk; a gate of -infinity counts as -10000.
//
// What is not finite. A tile product takes a value that is not finite to other tokens of the chunk (0 times it is NaN). A wave
// whose r (backwards: du; in the last kernel: whose results) holds such a value goes over its columns of the chunk again token by
// token, by the definition, where it reaches what it is part of and nothing else; a factor of 0 leaves nothing of it. A key alone
// in its sequence (a reset at it and behind it) shows in no r, but the state's product takes the whole tile of keys: N's diagonal, 0
// otherwise, is NaN at a key that is not finite, and so is then some r of every column.
//
// What bounds it, 8 x 4096 tokens x 16 heads of 128 (bfloat16): forward 370 us, by the profile (whose kernels add up to a little more) 113 of
// them the records (53 KiB a chunk and head read and written) and 273 the way along 64 chunks: 4.2 us a chunk, where a wave's 216
// matrix instructions keep its SIMD's unit busy for 3456 of 8100 cycles; the steps of a chunk follow from each other, and with 16 columns
// a wave there is one computing wave per SIMD to fill them. Not kept: more waves for the outputs, with the state's parts handed over in LDS
// (430 us: loads of q in the operands' layout take 400 cycles each, and two barriers a chunk); reads from LDS a step ahead by hand
// (283 beside 283 for the kernel; past 256 registers 650); a chunk's results stored behind the next chunk's barrier (the same). Backward
// 1530 us: records 122, states 227, gradients 300, the rest 893, whose 304 KiB a chunk and head (192 of them float32 states, gradients, r and
// du) come and go at 2.9 TB/s: a block's loads and products follow each other, and its 157 KiB of LDS leave no room for a second block
// (all loads issued at once, ahead of the gates: the same time).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"
#include "tiles.hpp"

namespace sdm {
namespace {

constexpr int kRow = 68;      // floats between the rows of a 64 x 64 matrix in LDS
constexpr int kFacBytes = 4 * kL * 4;

// A triangle of 64 x 64 token pairs as operands of matrix products. In a record: its ten 16 x 16 tiles that are not 0, float32,
// a KiB each, the lane's four values together: row lane % 16 of tile row it, columns 4 (lane / 16) + r of tile column jt; lower
// triangles (jt <= it) by rows of tiles, upper ones by columns. In LDS:
// twelve halves of the six operands of Pairs, in parts.
constexpr int kTriBytes = 10 * 1024;
template <typename T>
constexpr int kFragBytes = 12 * kParts<T> * kWave * 4 * static_cast<int>(sizeof(T));
// A chunk's factors, in its record behind the operands.
struct Factors {
    float f[kL];      // exp(G_i)
    float u[kL];      // exp(G_L - G_i)
    float beta[kL];   // 0 past the row's last token
    float one[kL];    // exp(g_i)
};
static_assert(sizeof(Factors) == kFacBytes, "a KiB");

// The parts of 8 float32 values as in cut(): what a part leaves is x - hi as a product of two pairs, (hi, other) . (-1, 0) + x in one
// instruction (3.5 a value for the three parts, 5.5 with a mask and a subtraction; exact but for subnormal parts, which are dropped).
__device__ __forceinline__ void split(const float (&x)[8], Parts<bf16_t, 3>& o) {
    // Not constants to the compiler: as an instruction's own operand -1 would stand for a float32.
    uint32_t first = 0x0000BF80u, second = 0xBF800000u;
    __asm__("" : "+s"(first));
    __asm__("" : "+s"(second));
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int s = 0; s < 3; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = __builtin_amdgcn_perm(__float_as_uint(r[2 * e + 1]), __float_as_uint(r[2 * e]), 0x07060302u);
            o.p[s].w[e] = w;
            if (s < 2) {
                r[2 * e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, first), r[2 * e], false);
                r[2 * e + 1] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, second), r[2 * e + 1], false);
            }
        }
    }
}
__device__ __forceinline__ void split(const float (&x)[8], Parts<float, 1>& o) { cut(x, o); }

// c[n] += a[n] b^T of operands in parts, N products side by side: all of 24 bits, the smallest first.
template <typename T, int NP, int N, bool SWAP = false>
__device__ __forceinline__ void mma_parts(const Parts<T, NP> (&a)[N], const Parts<T, NP>& b, f32x4* const (&c)[N]) {
    constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
    for (int k = NP == 3 ? 0 : 5; k < 6; ++k) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (SWAP) mma(b.p[kB[k]], a[n].p[kA[k]], *c[n]);
            else mma(a[n].p[kA[k]], b.p[kB[k]], *c[n]);
        }
    }
}
template <typename T, int NP>
__device__ __forceinline__ void mma_parts(const Parts<T, NP>& a, const Parts<T, NP>& b, f32x4& c) {
    const Parts<T, NP> aa[1] = {a};
    f32x4* const cc[1] = {&c};
    mma_parts<T, NP, 1>(aa, b, cc);
}

// Operand `pr` of a record's operands, as the lane holds it.
template <int NP>
__device__ __forceinline__ void frag_read(const char* at, int pr, int lane, Parts<bf16_t, NP>& o) {
#pragma unroll
    for (int s = 0; s < NP; ++s) o.p[s].w = *reinterpret_cast<const u32x4*>(at + ((pr * NP + s) * kWave + lane) * 16);
}
template <int NP>
__device__ __forceinline__ void frag_read(const char* at, int pr, int lane, Parts<float, NP>& o) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(at + ((2 * pr + h) * kWave + lane) * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) o.p[0].v[4 * h + r] = x[r];
    }
}
// Half of an operand: tokens 16 jt + 4 quarter + r (half jt % 2) of row 16 it + lane % 16.
template <typename T>
__device__ __forceinline__ void half_write(char* at, int pr, int half, int lane, f32x4 s) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            *reinterpret_cast<u32x2*>(at + ((pr * 3 + k) * kWave + lane) * 16 + 8 * half) =
                u32x2{__builtin_amdgcn_perm(__float_as_uint(s[1]), __float_as_uint(s[0]), 0x07060302u),
                      __builtin_amdgcn_perm(__float_as_uint(s[3]), __float_as_uint(s[2]), 0x07060302u)};
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] -= __uint_as_float(__float_as_uint(s[r]) & 0xFFFF0000u);
        }
    } else {
        *reinterpret_cast<f32x4*>(at + ((2 * pr + half) * kWave + lane) * 16) = s;
    }
}

// x[it] += (the triangle's operand of token tile it) times y of the token pairs jb, for the pairs that there are (SWAP: transposed).
template <bool REV, bool SWAP, typename T, int NP>
__device__ __forceinline__ void mma_triangle(const char* at, int jb, int lane, const Parts<T, NP>& y, f32x4 (&x)[4]) {
    constexpr int kMany = REV ? 1 : 0;   // the jb that meets all four tiles
    if (jb == kMany) {
        Parts<T, NP> a[4];
        f32x4* c[4];
        int n = 0;
#pragma unroll
        for (int pr = 0; pr < 6; ++pr) {
            if (Pairs<REV>::kJb[pr] != jb) continue;
            frag_read(at, pr, lane, a[n]);
            c[n++] = &x[Pairs<REV>::kIt[pr]];
        }
        f32x4* const cc[4] = {c[0], c[1], c[2], c[3]};
        mma_parts<T, NP, 4, SWAP>(a, y, cc);
    } else {
        Parts<T, NP> a[2];
        f32x4* c[2];
        int n = 0;
#pragma unroll
        for (int pr = 0; pr < 6; ++pr) {
            if (Pairs<REV>::kJb[pr] != jb) continue;
            frag_read(at, pr, lane, a[n]);
            c[n++] = &x[Pairs<REV>::kIt[pr]];
        }
        f32x4* const cc[2] = {c[0], c[1]};
        mma_parts<T, NP, 2, SWAP>(a, y, cc);
    }
}

// The descriptor of a buffer that is the same for all lanes, in scalar registers (in vector registers every load is a loop).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_buffer(const void* p, int bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u)));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0, bytes, 0x00027000);
}

__device__ __forceinline__ int live_tokens(const int32_t* lens, int b, int T) {
    const int n = lens != nullptr ? lens[b] : T;
    return n < 0 ? 0 : n > T ? T : n;
}

// ------------------------------------------------------------------------------------------ chunk records
//
// What of a chunk does not depend on the state, for every chunk at once: N, the scores of its tokens, and its factors,
// in the layout that the kernels along the time axis take. Forward: N and D (q k^T). Backward: N, N^T and D (q k^T)
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

template <bool BACK>
constexpr int kRecBytes = (BACK ? 3 : 2) * kTriBytes + kFacBytes;

template <typename T, int KD>
constexpr int kChunkTiles = 2 * kL * KD * static_cast<int>(sizeof(T)) > kL * kRow * 4 ? 2 * kL * KD * static_cast<int>(sizeof(T)) : kL * kRow * 4;

template <typename T, int KD, bool BACK>
__global__ __launch_bounds__(256) void gdr_chunk_kernel(ChunkArgs p) {
    constexpr int KB = KD / 32;
    extern __shared__ __align__(16) char lds[];
    T* kt = reinterpret_cast<T*>(lds);
    T* qt = kt + kL * KD;
    float* N = reinterpret_cast<float*>(lds);   // over the tiles, once the products of them are done: three blocks fit a compute unit
    float* A = reinterpret_cast<float*>(lds + kChunkTiles<T, KD>);
    float* beta = A + kL * kRow;
    Gates& gates = *reinterpret_cast<Gates*>(beta + kL);

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    // Heads of the same tokens are neighbours: together they read and write whole rows.
    const int bc = blk / p.H, h = blk - bc * p.H, b = bc / p.chunks, c = bc - b * p.chunks, bh = b * p.H + h;
    const int left = live_tokens(p.lens, b, p.T) - c * kL;
    if (left <= 0) return;
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(c) * kL;
    char* rec = p.rec + (static_cast<int64_t>(bh) * p.chunks + c) * kRecBytes<BACK>;

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
        Factors* f = reinterpret_cast<Factors*>(rec + kRecBytes<BACK> - kFacBytes);
        f->f[lane] = gates.f[lane];
        f->u[lane] = gates.u[lane];
        f->beta[lane] = e;
        f->one[lane] = gate_factor(g);
    }
    tile_barrier();

    // Tiles of 16 x 16 tokens: ten of the scores, dealt to the waves with the ten of A.
    char* const scores = rec + (BACK ? 2 : 1) * kTriBytes;
    for (int e = wave; e < 20; e += 4) {
        const bool isA = e >= 10;
        const int n = isA ? e - 10 : e, hi = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0, lo = n - hi * (hi + 1) / 2;
        const int it = BACK && !isA ? lo : hi, jt = BACK && !isA ? hi : lo;
        const bool rev = BACK && !isA;
        T* const x = !isA && !BACK ? qt : kt;
        T* const y = !isA && BACK ? qt : kt;
        f32x4 a = {0, 0, 0, 0}, s;   // token 16 jt + 4 quarter + r down, token 16 it + lane % 16 across
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
                if (isA && j == i16) s[r] = 0.0f * a[r];   // NaN for a key that is not finite
            }
        } else {
            const float ot = (rev ? gates.down : gates.up)[16 * it + i16] * (m * gates.tau[4 * it + jt]);
            const f32x4 d = *reinterpret_cast<const f32x4*>(&(rev ? gates.up : gates.down)[16 * jt + 4 * qd]);
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = sdm_decayed(ot * d[r], a[r]);
        }
        if (isA) *reinterpret_cast<f32x4*>(A + (16 * it + i16) * kRow + 16 * jt + 4 * qd) = s;
        else *reinterpret_cast<f32x4*>(scores + n * 1024 + lane * 16) = s;
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

    for (int e = wave; e < (BACK ? 20 : 10); e += 4) {
        const int n = e >= 10 ? e - 10 : e, hi = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0, lo = n - hi * (hi + 1) / 2;
        f32x4 x;
        if (e < 10) {
            x = *reinterpret_cast<const f32x4*>(N + (16 * hi + i16) * kRow + 16 * lo + 4 * qd);
        } else {   // row 16 lo + lane % 16 of N^T
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = N[(16 * hi + 4 * qd + r) * kRow + 16 * lo + i16];
        }
        *reinterpret_cast<f32x4*>(rec + e * 1024 + lane * 16) = x;
    }
}

// What a segment of the time axis does to the state before it: takes it through its transition, leaves nothing of it (a gate
// resets), or nothing at all (past the row's length).
enum Kind { kMoves, kClears, kIdle };

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
    int rec_bytes;
    const float* start;       // [B H] states [kd, vd] (NULL: zero)
    float* last;              // [B H] (NULL: not kept)
    void* out;                // [B, T, H, vd] (OUT)
    int64_t o_b, o_t, o_h;
    int out_wide;
    float* states;            // the states before every chunk [B H, chunks] (states pass), and r [B H, T, vd]
    float* miss;
    // Segments of the time axis, `seg` chunks each. from: the states before every segment [B H, nseg] (NULL with one segment:
    // start). Segments pass: own and move take every segment's own state, from nothing, and its transition [kd, kd], of which
    // the first `made` are made; blocks past `cols` are the transition's.
    int nseg, seg, made;
    const float* from;
    float *own, *move;
    int32_t* kinds;           // [B H, nseg] (segments pass): what a segment does to a state before it (Kind)
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
        // Waited for here: left to the first use, in the loop over chunks, the wait would take in every chunk's tile loads.
#pragma unroll
        for (int d = 0; d < KT; ++d) __asm__ volatile("" : "+v"(S[d]));
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

// M triangles of a record (`tri`: the first) to LDS as operands, by four waves, and the factors behind them. The operands' halves
// that hold nothing are written once per buffer (record_zero).
template <typename T, int M, bool REV>
__device__ __forceinline__ void record_fill(const char* tri, const char* fac, char* to, int wave, int lane) {
    f32x4 x[(M * 10 + 3) / 4], f;
#pragma unroll
    for (int u = 0; u < (M * 10 + 3) / 4; ++u) {
        const int e = wave + 4 * u;
        if (e < M * 10) x[u] = *reinterpret_cast<const f32x4*>(tri + e * 1024 + lane * 16);
    }
    if (wave == 3) f = *reinterpret_cast<const f32x4*>(fac + lane * 16);
#pragma unroll
    for (int u = 0; u < (M * 10 + 3) / 4; ++u) {
        const int e = wave + 4 * u;
        if (e >= M * 10) continue;
        const int m = M > 1 && e >= 10 ? 1 : 0, n = e - 10 * m, hi = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0, lo = n - hi * (hi + 1) / 2;
        const int it = REV ? lo : hi, jt = REV ? hi : lo;
        // Pairs' place of (it, jt / 2)
        const int pr = REV ? (it < 2 ? 2 * it + (jt >> 1) : it + 2) : (it < 2 ? it : 2 * it - 2 + (jt >> 1));
        half_write<T>(to + m * kFragBytes<T>, pr, jt & 1, lane, x[u]);
    }
    if (wave == 3) *reinterpret_cast<f32x4*>(to + M * kFragBytes<T> + lane * 16) = f;
}
template <typename T, int M, bool REV>
__device__ __forceinline__ void record_zero(char* to, int wave, int lane) {
    // Forward the tiles (0, 1) and (2, 3), backwards (1, 0) and (3, 2).
    for (int e = wave; e < 2 * M; e += 4) {
        const int m = e >> 1, pr = REV ? (e & 1 ? 5 : 2) : (e & 1 ? 3 : 0);
        half_write<T>(to + m * kFragBytes<T>, pr, REV ? 0 : 1, lane, f32x4{0, 0, 0, 0});
    }
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

// Where the tiles of two chunks fit into LDS side by side, four more waves load the next chunk's while these compute (issuing
// its 77 KiB of loads by themselves kept the computing waves for 3000 of a chunk's 10000 cycles). float32 chunks of keys past 64
// columns do not fit twice and are loaded one by one (8 x 4096 x 16 heads, float32, 64 / 128 columns: forward 520 / 1240 us, backward
// 1505 / 3290).
template <typename T, int KD>
constexpr bool kTwo = sizeof(T) == 2 || KD == 64;
template <typename T, int KD>
constexpr int kMainThreads = kTwo<T, KD> ? 512 : 256;

// OUT: the outputs (and the last state). Else the states before every chunk and the rows r, for the backward pass; or (SEG)
// the segments' own states and transitions. The transition is the rule on the columns of the unit matrix, whose values are 0.
template <typename T, int KD, bool OUT, bool SEG>
__global__ __launch_bounds__((kMainThreads<T, KD>), (kMainThreads<T, KD> / 256)) void gdr_kernel(MainArgs p) {
    constexpr int KB = KD / 32, KT = KD / 16, NP = kParts<T>;
    constexpr bool kAhead = kTwo<T, KD>;
    constexpr int kTile = kL * KD * static_cast<int>(sizeof(T)), kTileV = kL * 64 * static_cast<int>(sizeof(T));
    constexpr int kBuf = (OUT ? 2 : 1) * kTile + kTileV + (OUT ? 2 : 1) * kFragBytes<T> + kFacBytes;
    extern __shared__ __align__(16) char lds[];

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int per = SEG ? p.cols + (p.kd + 63) / 64 : p.cols, nseg = SEG ? p.made : p.nseg;   // blocks of a segment, segments
    const int bs = blk / per, bh = bs / nseg, si = bs - bh * nseg, b = bh / p.H, h = bh - b * p.H;
    const bool unit = SEG && blk - bs * per >= p.cols;
    const int cb = blk - bs * per - (unit ? p.cols : 0), vd = unit ? p.kd : p.vd;
    const bool loads = threadIdx.x >= 256;   // the waves that load ahead
    const int tid = static_cast<int>(threadIdx.x) & 255, lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int c0 = 64 * cb, n0 = 16 * wave, vw = min(64, vd - c0);   // the block's columns, the wave's first among them
    const int len = __builtin_amdgcn_readfirstlane(live_tokens(p.lens, b, p.T));
    // The segment's chunks.
    const int first = si * p.seg, chunks = min((len + kL - 1) / kL, si + 1 == p.nseg ? p.chunks : first + p.seg);

    Rows vr = p.v;
    vr.width = vw;
    const T* qb = OUT ? static_cast<const T*>(p.q.p) + b * p.q.b + (h / p.q.per) * p.q.h : nullptr;
    const T* kb_ = static_cast<const T*>(p.k.p) + b * p.k.b + (h / p.k.per) * p.k.h;
    const T* vb = static_cast<const T*>(p.v.p) + b * p.v.b + h * p.v.h + c0;
    const int64_t one = static_cast<int64_t>(p.kd) * vd;
    const StateAt<KT> place(c0 + n0 + i16, qd, p.kd, vd);

    Stage<T, KD, 256> sq, sk;
    Stage<T, 64, 256> sv;
    auto tiles = [&](int buf) { return lds + buf * kBuf; };
    auto fill = [&](int c, int buf) {
        const int64_t t0 = static_cast<int64_t>(c) * kL;
        const int left = len - c * kL;
        char* at = tiles(buf);
        sk.fill(p.k, kb_ + t0 * p.k.t, left, reinterpret_cast<T*>(at), wave, tid);
        if (!unit) sv.fill(vr, vb + t0 * p.v.t, left, reinterpret_cast<T*>(at + kTile), wave, tid);
        if (OUT) sq.fill(p.q, qb + t0 * p.q.t, left, reinterpret_cast<T*>(at + kTile + kTileV), wave, tid);
        const char* rec = p.rec + (static_cast<int64_t>(bh) * p.chunks + c) * p.rec_bytes;
        record_fill<T, OUT ? 2 : 1, false>(rec, rec + p.rec_bytes - kFacBytes, at + (OUT ? 2 : 1) * kTile + kTileV, wave, lane);
    };
    if (!kAhead || loads) {
        if (OUT) sq.init(p.q, tid);
        sk.init(p.k, tid);
        sv.init(vr, tid);
        for (int n = 0; n < (kAhead ? 2 : 1); ++n) {
            record_zero<T, OUT ? 2 : 1, false>(tiles(n) + (OUT ? 2 : 1) * kTile + kTileV, wave, lane);
            if (unit) {   // no values
                for (int e = tid; e < kTileV / 16; e += 256) *reinterpret_cast<u32x4*>(tiles(n) + kTile + 16 * e) = u32x4{0, 0, 0, 0};
            }
        }
        if (chunks > first) fill(first, 0);
    }
    if (kAhead && loads) {
        for (int c = first; c < chunks; ++c) {
            tile_barrier();   // the chunk's tiles are complete, and the other buffer's are free
            if (c + 1 < chunks) fill(c + 1, __builtin_amdgcn_readfirstlane((c + 1 - first) & 1));
        }
        return;
    }
    f32x4 S[KT];
#pragma unroll
    for (int d = 0; d < KT; ++d) S[d] = f32x4{0, 0, 0, 0};
    if constexpr (SEG) {
        if (unit) {
#pragma unroll
            for (int d = 0; d < KT; ++d) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[d][r] = 32 * (d >> 1) + 8 * qd + 4 * (d & 1) + r == c0 + n0 + i16 ? 1.0f : 0.0f;
            }
        }
    } else if (p.from != nullptr) {
        place.read(p.from + (static_cast<int64_t>(bh) * p.nseg + si) * one, S);
    } else if (p.start != nullptr) {
        place.read(p.start + bh * one, S);
    }


    bool cut = false;   // a token of the lane's place resets
    for (int c = first; c < chunks; ++c) {
        const int buf = kAhead ? __builtin_amdgcn_readfirstlane((c - first) & 1) : 0, t0 = c * kL, left = len - t0;
        char* const at = tiles(buf);
        T* const kt = reinterpret_cast<T*>(at);
        T* const vt = reinterpret_cast<T*>(at + kTile);
        T* const qt = reinterpret_cast<T*>(at + kTile + kTileV);
        const char* const nf = at + (OUT ? 2 : 1) * kTile + kTileV;
        const char* const pf = nf + kFragBytes<T>;
        const Factors& fac = *reinterpret_cast<const Factors*>(nf + (OUT ? 2 : 1) * kFragBytes<T>);
        if (kAhead) lds_barrier();
        else tile_barrier();
        if (!OUT && !SEG) place.write(p.states + (static_cast<int64_t>(bh) * p.chunks + c) * one, S);
        if (SEG) cut |= fac.one[lane] == 0.0f;

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
            split(s, sp);
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
            split(w, yp);
            mma_triangle<false, false>(nf, jb, lane, yp, X);
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
                if (!SEG && qd == 0 && col < p.vd) {
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
                split(z, zp);
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
                    split(w, up);
                    mma_triangle<false, true>(pf, jb, lane, up, O);
                }
            }
            if constexpr (OUT) {
                const int n = c0 + n0 + 4 * qd;   // the lane's result columns n .. n + 3, of token 16 it + lane % 16
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    if (16 * it + i16 >= left || n >= p.vd) continue;
                    store_four<T>(p.out, b * p.o_b + h * p.o_h + static_cast<int64_t>(t0 + 16 * it + i16) * p.o_t + n, O[it], p.vd - n, p.out_wide);
                }
            } else if constexpr (!SEG) {
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
        if (!kAhead) {
            lds_barrier();   // the tiles are free
            if (c + 1 < chunks) fill(c + 1, 0);
        }
    }
    if constexpr (OUT) {
        // The segment's tokens past the row's length.
        const int from = max(len, first * kL), to = si + 1 == p.nseg ? p.T : min(p.T, (first + p.seg) * kL);
        for (int64_t e = tid; e < static_cast<int64_t>(to - from) * vw; e += 256) {
            const int t = from + static_cast<int>(e / vw), col = c0 + static_cast<int>(e % vw);
            static_cast<T*>(p.out)[b * p.o_b + t * p.o_t + h * p.o_h + col] = narrow<T>(0.0f);
        }
    }
    if constexpr (SEG) {
        place.write((unit ? p.move : p.own) + (static_cast<int64_t>(bh) * p.nseg + si) * one, S);
        const int kind = chunks <= first ? kIdle : __ballot(cut) != 0 ? kClears : kMoves;
        if (unit && cb == 0 && tid == 0) p.kinds[static_cast<int64_t>(bh) * p.nseg + si] = kind;
    } else if (p.last != nullptr && si + 1 == p.nseg) place.write(p.last + bh * one, S);
}

// The states before every segment (REV: the gradients behind every one) from the segments' own and their transitions,
//     S_{n+1} = M_n S_n + own_n    (REV: R_{n-1} = M_n^T R_n + own_n),
// one block per 16 columns of a (stream, head)'s state: each wave 16 rows, the columns in LDS between the steps, the next step's
// matrices in flight. Both factors in three bfloat16 parts, whatever the inputs. A segment with a reset leaves nothing of what was
// before, finite or not. One without does, also where its transition is 0 in float32: by the rule every token takes a column's
// infinity or NaN into the state again, as the product with it does. One past the row's length leaves every bit of the state.
struct ChainArgs {
    const float *move, *own;   // [B H, nseg]
    const int32_t* kinds;      // [B H, nseg]
    const float* start;        // [B H] (NULL: zero)
    float* to;                 // [B H, nseg]
    int nseg, kd, vd, cols;    // cols: blocks of 16 columns
};

template <int KD, bool REV>
__global__ __launch_bounds__(4 * KD) void gdr_chain_kernel(ChainArgs p) {
    constexpr int KB = KD / 32, kPad = KD + 4;
    __shared__ __align__(16) float cols[2][16 * kPad];   // [column][row]
    const int bh = static_cast<int>(blockIdx.x) / p.cols, cb = static_cast<int>(blockIdx.x) - bh * p.cols;
    const int lane = static_cast<int>(lane_id()), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int i16 = lane & 15, qd = lane >> 4, col = 16 * cb + i16, row = 16 * wave + i16, out = 16 * wave + 4 * qd;
    const int64_t one = static_cast<int64_t>(p.kd) * p.vd, sq = static_cast<int64_t>(p.kd) * p.kd;
    // Byte offsets of the lane's elements (row, 32 kb + 8 quarter + ..) of a transition, and of its part of a state; past any range
    // where there are none. Every step's loads go by them.
    uint32_t moff[KB], ooff[4];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int j = 32 * kb + 8 * qd;
        moff[kb] = row < p.kd && j < p.kd ? 4u * static_cast<uint32_t>(REV ? j * p.kd + row : row * p.kd + j) : 0xC0000000u;
        __asm__ volatile("" : "+v"(moff[kb]));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        ooff[r] = out + r < p.kd && col < p.vd ? 4u * static_cast<uint32_t>((out + r) * p.vd + col) : 0xC0000000u;
        __asm__ volatile("" : "+v"(ooff[r]));
    }
    const bool four = !REV && p.kd % 4 == 0;
    float m[KB][8];
    f32x4 own;
    int kind = kMoves;
    auto part = [&](const float* from, f32x4& x) {
        const auto b = uniform_buffer(from, static_cast<int>(one) * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, static_cast<int>(ooff[r]), 0, 0));
    };
    auto load = [&](int n) {
        const auto b = uniform_buffer(p.move + (static_cast<int64_t>(bh) * p.nseg + n) * sq, static_cast<int>(sq) * 4);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if (four) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(moff[kb] + 16u * h), 0, 0));
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[kb][4 * h + e] = w[e];
                }
            } else {
                const uint32_t step = REV ? 4u * static_cast<uint32_t>(p.kd) : 4u;
#pragma unroll
                for (int e = 0; e < 8; ++e) m[kb][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, static_cast<int>(moff[kb] + step * e), 0, 0));
            }
        }
        part(p.own + (static_cast<int64_t>(bh) * p.nseg + n) * one, own);
        kind = p.kinds[static_cast<int64_t>(bh) * p.nseg + n];
    };
    auto keep = [&](int n, f32x4 s, float* at) {
        float* to = p.to + (static_cast<int64_t>(bh) * p.nseg + n) * one;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (out + r < p.kd && col < p.vd) to[(out + r) * p.vd + col] = s[r];
        }
        *reinterpret_cast<f32x4*>(at + i16 * kPad + out) = s;
    };
    const int n0 = REV ? p.nseg - 1 : 0, n1 = REV ? 0 : p.nseg - 1, step = REV ? -1 : 1;
    f32x4 s = {0, 0, 0, 0};
    if (p.start != nullptr) {
        part(p.start + bh * one, s);
    }
    keep(n0, s, cols[0]);
    load(n0);
    int buf = 0;
    for (int n = n0; n != n1; n += step, buf ^= 1) {
        Parts<bf16_t, 3> mp[KB];
        const int now = kind;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (32 * kb + 8 * qd + e >= p.kd) m[kb][e] = 0.0f;   // the next row's
            }
            split(m[kb], mp[kb]);
        }
        f32x4 x = {0, 0, 0, 0}, part_[KB];
        const f32x4 add = own;
        if (n + step != n1) load(n + step);
        __syncthreads();   // the columns are complete
        if (now == kMoves) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const float* at = cols[buf] + i16 * kPad + 32 * kb + 8 * qd;
                const f32x4 a = *reinterpret_cast<const f32x4*>(at), b = *reinterpret_cast<const f32x4*>(at + 4);
                const float y[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                Parts<bf16_t, 3> yp;
                split(y, yp);
                part_[kb] = f32x4{0, 0, 0, 0};
                mma_parts(mp[kb], yp, part_[kb]);
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) x += part_[kb];
        }
        s = now == kIdle ? s : x + add;
        keep(n + step, s, cols[buf ^ 1]);
    }
}

// ------------------------------------------------------------------------------------------ backward
//
// With R the gradient of the state after a chunk and E_i the gradient of o_i times scale,
//     z_i = exp(G_L - G_i) R^T k_i + sum_{j >= i} D_ji (q_j . k_i) E_j,    du = z - N^T (beta z),    dv = beta du,
//     R before the chunk = exp(G_L) R + sum_i exp(G_i) (q_i E_i^T - k_i dv_i^T),
// the same shape of work as forward, back in time. The rest is local to a chunk, given S before it, R behind it, r and du:
//     dq_i = exp(G_i) S E_i + sum_{j <= i} D_ij (E_i . u_j) k_j,
//     dk_i = exp(G_L - G_i) R u_i + sum_{j >= i} D_ji (E_j . u_i) q_j
//            - exp(G_i) S dv_i - sum_{j < i} D_ij (dv_i . u_j) k_j - sum_{j > i} D_ji (dv_j . u_i) k_j,
//     dbeta_i = du_i . r_i,    dg_i = sum_{j >= i in the chunk} (q_j . dq_j - v_j . dv_j) + <S behind the chunk, R>,
// the last because a gate scales all that reaches its token or a later one from an earlier one; the sum starts afresh from
// 0 at every reset.
struct BackArgs {
    Rows q, k, d;             // d: the gradients of o
    const int32_t* lens;
    int T, H, chunks, cols;
    int kd, vd;
    float scale;
    const char* rec;
    const float* start;       // [B H] gradients of the last states (NULL: zero)
    float* first;             // [B H] gradients of the first states (NULL: not kept)
    float* grads;             // [B H, chunks] the gradients of the states behind every chunk
    float* du;                // [B H, T, vd]
    // Segments as in MainArgs. from: the gradients behind every segment; own: the segments pass's, from nothing (all but the first's).
    int nseg, seg;
    const float* from;
    float* own;
};

template <typename T, int KD, bool SEG>
__global__ __launch_bounds__((kMainThreads<T, KD>), (kMainThreads<T, KD> / 256)) void gdr_back_kernel(BackArgs p) {
    constexpr int KB = KD / 32, KT = KD / 16, NP = kParts<T>;
    constexpr bool kAhead = kTwo<T, KD>;
    constexpr int kTile = kL * KD * static_cast<int>(sizeof(T)), kTileV = kL * 64 * static_cast<int>(sizeof(T));
    constexpr int kBuf = 2 * kTile + kTileV + 2 * kFragBytes<T> + kFacBytes;
    extern __shared__ __align__(16) char lds[];

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int bs = blk / p.cols, cb = blk - bs * p.cols, nseg = SEG ? p.nseg - 1 : p.nseg;
    const int bh = bs / nseg, si = bs - bh * nseg + (SEG ? 1 : 0), b = bh / p.H, h = bh - b * p.H;
    const bool loads = threadIdx.x >= 256;   // the waves that load ahead
    const int tid = static_cast<int>(threadIdx.x) & 255, lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4;
    const int c0 = 64 * cb, n0 = 16 * wave, vw = min(64, p.vd - c0);
    const int len = __builtin_amdgcn_readfirstlane(live_tokens(p.lens, b, p.T));
    const int first = si * p.seg, chunks = min((len + kL - 1) / kL, si + 1 == p.nseg ? p.chunks : first + p.seg);

    Rows dr = p.d;
    dr.width = vw;
    const T* qb = static_cast<const T*>(p.q.p) + b * p.q.b + (h / p.q.per) * p.q.h;
    const T* kb_ = static_cast<const T*>(p.k.p) + b * p.k.b + (h / p.k.per) * p.k.h;
    const T* db = static_cast<const T*>(p.d.p) + b * p.d.b + h * p.d.h + c0;
    const int64_t one = static_cast<int64_t>(p.kd) * p.vd;
    const StateAt<KT> place(c0 + n0 + i16, qd, p.kd, p.vd);

    Stage<T, KD, 256> sq, sk;
    Stage<T, 64, 256> sd;
    auto fill = [&](int c, int buf) {
        const int64_t t0 = static_cast<int64_t>(c) * kL;
        const int left = len - c * kL;
        char* at = lds + buf * kBuf;
        sk.fill(p.k, kb_ + t0 * p.k.t, left, reinterpret_cast<T*>(at), wave, tid);
        sd.fill(dr, db + t0 * p.d.t, left, reinterpret_cast<T*>(at + kTile), wave, tid);
        sq.fill(p.q, qb + t0 * p.q.t, left, reinterpret_cast<T*>(at + kTile + kTileV), wave, tid);
        const char* rec = p.rec + (static_cast<int64_t>(bh) * p.chunks + c) * kRecBytes<true>;
        record_fill<T, 2, true>(rec + kTriBytes, rec + 3 * kTriBytes, at + 2 * kTile + kTileV, wave, lane);
    };
    if (!kAhead || loads) {
        sq.init(p.q, tid);
        sk.init(p.k, tid);
        sd.init(dr, tid);
        for (int n = 0; n < (kAhead ? 2 : 1); ++n) record_zero<T, 2, true>(lds + n * kBuf + 2 * kTile + kTileV, wave, lane);
        if (chunks > first) fill(chunks - 1, 0);
    }
    if (kAhead && loads) {
        for (int c = chunks - 1; c >= first; --c) {
            tile_barrier();
            if (c > first) fill(c - 1, __builtin_amdgcn_readfirstlane((chunks - c) & 1));
        }
        return;
    }
    f32x4 R[KT];
#pragma unroll
    for (int d = 0; d < KT; ++d) R[d] = f32x4{0, 0, 0, 0};
    if constexpr (!SEG) {
        if (p.from != nullptr) place.read(p.from + (static_cast<int64_t>(bh) * p.nseg + si) * one, R);
        else if (p.start != nullptr) place.read(p.start + bh * one, R);
    }


    for (int c = chunks - 1; c >= first; --c) {
        const int buf = kAhead ? __builtin_amdgcn_readfirstlane((chunks - 1 - c) & 1) : 0, t0 = c * kL, left = len - t0;
        char* const at = lds + buf * kBuf;
        T* const kt = reinterpret_cast<T*>(at);
        T* const dt = reinterpret_cast<T*>(at + kTile);
        T* const qt = reinterpret_cast<T*>(at + kTile + kTileV);
        const char* const nf = at + 2 * kTile + kTileV;
        const char* const pf = nf + kFragBytes<T>;
        const Factors& fac = *reinterpret_cast<const Factors*>(nf + 2 * kFragBytes<T>);
        if (kAhead) lds_barrier();
        else tile_barrier();
        if (!SEG) place.write(p.grads + (static_cast<int64_t>(bh) * p.chunks + c) * one, R);

        f32x4 Z[4];   // tile it: tokens 16 it + 4 quarter + r down, column n0 + lane % 16
#pragma unroll
        for (int it = 0; it < 4; ++it) Z[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            Parts<T, NP> rp;
            float s[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) { s[r] = R[2 * kb][r]; s[4 + r] = R[2 * kb + 1][r]; }
            split(s, rp);
            Frag<T> kf[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) kf[it] = row_frag<KD>(kt, 16 * it + i16, kb, qd);
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) {
#pragma unroll
                for (int it = 0; it < 4; ++it) mma(kf[it], rp.p[n], Z[it]);
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const f32x4 u = *reinterpret_cast<const f32x4*>(&fac.u[16 * it + 4 * qd]);
#pragma unroll
            for (int r = 0; r < 4; ++r) Z[it][r] = sdm_decayed(u[r], Z[it][r]);
        }
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            const Frag<T> df = col_frag<64, 4>(dt, jb, n0, i16, qd);
#pragma unroll
            for (int pr = 0; pr < 6; ++pr) {
                if (Pairs<true>::kJb[pr] != jb) continue;
                Parts<T, NP> pp;
                frag_read(pf, pr, lane, pp);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n) mma(pp.p[n], df, Z[Pairs<true>::kIt[pr]]);
            }
        }
        f32x4 X[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) X[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            float w[8];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 be = *reinterpret_cast<const f32x4*>(&fac.beta[32 * jb + 16 * s + 4 * qd]);
#pragma unroll
                for (int r = 0; r < 4; ++r) w[4 * s + r] = be[r] * Z[2 * jb + s][r];
            }
            Parts<T, NP> zp;
            split(w, zp);
            mma_triangle<true, false>(nf, jb, lane, zp, X);
        }
        float odd = 0.0f;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            Z[it] -= X[it];   // du
#pragma unroll
            for (int r = 0; r < 4; ++r) odd = fmaf(Z[it][r], 0.0f, odd);
        }
        if (__builtin_expect(__ballot(odd != odd) != 0, 0)) {   // token by token, as forward
            for (int t = min(left, kL) - 1; t >= 0; --t) {
                const float e = p.scale * tile_at(dt, t, n0 + i16), a = fac.one[t];
                float sum = 0.0f, k[KB][8], q[8];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    widen8(row_frag<KD>(kt, t, kb, qd), k[kb]);
                    widen8(row_frag<KD>(qt, t, kb, qd), q);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float s = 32 * kb + 8 * qd + n < p.kd ? fmaf(q[n], e, R[2 * kb + (n >> 2)][n & 3]) : 0.0f;
                        R[2 * kb + (n >> 2)][n & 3] = s;
                        sum = fmaf(s, k[kb][n], sum);
                    }
                }
                sum += lane_xor_f<16>(sum);
                sum += lane_xor_f<32>(sum);
                const float dv = fac.beta[t] * sum;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float s = 32 * kb + 8 * qd + n < p.kd ? fmaf(-k[kb][n], dv, R[2 * kb + (n >> 2)][n & 3]) : 0.0f;
                        R[2 * kb + (n >> 2)][n & 3] = sdm_decayed(a, s);
                    }
                }
                if (!SEG && qd == 0 && n0 + i16 < vw) p.du[(static_cast<int64_t>(bh) * p.T + t0 + t) * p.vd + c0 + n0 + i16] = sum;
            }
        } else {
            const float all = fac.f[kL - 1];
#pragma unroll
            for (int d = 0; d < KT; ++d) R[d] = decayed(all, R[d]);
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
                float e[8], w[8];
                widen8(col_frag<64, 4>(dt, jb, n0, i16, qd), e);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const f32x4 be = *reinterpret_cast<const f32x4*>(&fac.beta[32 * jb + 16 * s + 4 * qd]);
                    const f32x4 f = *reinterpret_cast<const f32x4*>(&fac.f[32 * jb + 16 * s + 4 * qd]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        e[4 * s + r] = sdm_decayed(f[r] * p.scale, e[4 * s + r]);
                        w[4 * s + r] = sdm_decayed(-f[r] * be[r], Z[2 * jb + s][r]);
                    }
                }
                Parts<T, NP> ep, wp;
                split(e, ep);
                split(w, wp);
#pragma unroll
                for (int d = 0; d < KT; d += 4) {
                    Frag<T> qf[4], kf[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        qf[m] = col_frag<KD, 8>(qt, jb, 32 * ((d + m) >> 1) + 4 * (m & 1), i16, qd);
                        kf[m] = col_frag<KD, 8>(kt, jb, 32 * ((d + m) >> 1) + 4 * (m & 1), i16, qd);
                    }
#pragma unroll
                    for (int n = NP - 1; n >= 0; --n) {
#pragma unroll
                        for (int m = 0; m < 4; ++m) mma(qf[m], ep.p[n], R[d + m]);
#pragma unroll
                        for (int m = 0; m < 4; ++m) mma(kf[m], wp.p[n], R[d + m]);
                    }
                }
            }
            float* const du = p.du + (static_cast<int64_t>(bh) * p.T + t0) * p.vd + c0 + n0 + i16;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * it + 4 * qd + r;
                    if (!SEG && t < left && n0 + i16 < vw) du[static_cast<int64_t>(t) * p.vd] = Z[it][r];
                }
            }
        }
        if (!kAhead) {
            lds_barrier();
            if (c > first) fill(c - 1, 0);
        }
    }
    if constexpr (SEG) place.write(p.own + (static_cast<int64_t>(bh) * p.nseg + si) * one, R);
    else if (p.first != nullptr && si == 0) place.write(p.first + bh * one, R);
}

// What is local to a chunk: a block per chunk, 16 key columns for each of its waves.
struct GradArgs {
    Rows q, k, v, d;
    const float *g, *beta;
    int64_t g_b, g_t, g_h, e_b, e_t, e_h;
    const int32_t* lens;
    int T, H, chunks, kd, vd;
    float scale;
    const float *states, *grads;   // [B H, chunks] before and behind every chunk
    const float *miss, *du;        // [B H, T, vd]
    int stateless;                 // no state before the first token
    void *dq, *dk;                 // [B, T, H or Hk, kd]: narrowed, or float32 per value head (FOLD)
    int key_wide;
    void* dv;                      // [B, T, H, vd]
    float *dg, *dbeta;             // [B, T, H]
};

// Tile of a 64-row operand in parts: part s at tile + s 64 VD.
template <typename T, int VD, int NP>
__device__ __forceinline__ void row_parts(T* tile, int row, int kb, int quarter, Parts<T, NP>& o) {
#pragma unroll
    for (int s = 0; s < NP; ++s) o.p[s] = row_frag<VD>(tile + s * kL * VD, row, kb, quarter);
}

// Four consecutive columns (a multiple of four) of a row.
template <int W>
__device__ __forceinline__ f32x4 tile_four(bf16_t* tile, int row, int col) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(piece<bf16_t, W>(tile, row, col >> 3) + 2 * (col & 7));
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
}
template <int W>
__device__ __forceinline__ f32x4 tile_four(float* tile, int row, int col) {
    return *reinterpret_cast<const f32x4*>(piece<float, W>(tile, row, col >> 2));
}

// Scores a[r] (token 16 jt + 4 quarter + r, for row 16 it + lane % 16) times m and the decay between the two; REV: of later
// tokens (jt >= it), else of earlier ones; STRICT: without the token itself.
template <bool REV, bool STRICT>
__device__ __forceinline__ void decay_scores(const Gates& gates, int it, int jt, int i16, int qd, float m, const f32x4& a, float (&s)[4]) {
    if (jt == it) {
        const float lhi = gates.lhi[16 * it + i16], llo = gates.llo[16 * it + i16];
        const f32x4 jh = *reinterpret_cast<const f32x4*>(&gates.lhi[16 * jt + 4 * qd]);
        const f32x4 jl = *reinterpret_cast<const f32x4*>(&gates.llo[16 * jt + 4 * qd]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 4 * qd + r;
            const float d = (lhi - jh[r]) + (llo - jl[r]);
            const float w = __builtin_amdgcn_exp2f(REV ? -d : d);
            s[r] = (REV ? (STRICT ? j > i16 : j >= i16) : STRICT ? j < i16 : j <= i16) ? sdm_decayed(w * m, a[r]) : 0.0f;
        }
    } else {
        const float ot = (REV ? gates.down : gates.up)[16 * it + i16] * (m * gates.tau[4 * it + jt]);
        const f32x4 d = *reinterpret_cast<const f32x4*>(&(REV ? gates.up : gates.down)[16 * jt + 4 * qd]);
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r] = sdm_decayed(ot * d[r], a[r]);
    }
}

template <typename T, int KD, int VD>
struct GradLds {   // bytes
    static constexpr int kD = kL * (KD > VD ? KD : VD) * static_cast<int>(sizeof(T));      // d_o's tile, then q's
    static constexpr int kK = kL * KD * static_cast<int>(sizeof(T));
    static constexpr int kU = kParts<T> * kL * VD * static_cast<int>(sizeof(T));           // u's parts; and dv's
    static constexpr int kS = 8 * kParts<T> * kWave * 8 * static_cast<int>(sizeof(T));     // score operands
    static constexpr int kWaves = KD / 16;
    static constexpr int kTotal = kD + kK + 2 * kU + kS + static_cast<int>(sizeof(Gates)) + (3 + kWaves) * kL * 4 + 64;
};

template <typename T, int KD, int VD, bool FOLD>
__global__ __launch_bounds__(4 * KD, KD == 128 ? 2 : 1) void gdr_grad_kernel(GradArgs p) {
    constexpr int VB = VD / 32, kThreads = 4 * KD, kWaves = KD / 16, NP = kParts<T>;
    using Lds = GradLds<T, KD, VD>;
    extern __shared__ __align__(16) char lds[];
    T* const dt = reinterpret_cast<T*>(lds);
    T* const qt = dt;
    T* const kt = reinterpret_cast<T*>(lds + Lds::kD);
    T* const ut = reinterpret_cast<T*>(lds + Lds::kD + Lds::kK);
    T* const wt = ut + NP * kL * VD;
    char* const scores = lds + Lds::kD + Lds::kK + 2 * Lds::kU;
    Gates& gates = *reinterpret_cast<Gates*>(scores + Lds::kS);
    float* const beta = reinterpret_cast<float*>(reinterpret_cast<char*>(&gates) + sizeof(Gates));
    float* const one_gate = beta + kL;
    float* const vdv = one_gate + kL;
    float* const dots = vdv + kL;           // [waves][64]
    float* const cross = dots + kWaves * kL;   // [waves]

    const int blk = xcd_block(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    // Heads of the same tokens are neighbours: together they read and write whole rows.
    const int bc = blk / p.H, h = blk - bc * p.H, b = bc / p.chunks, c = bc - b * p.chunks, bh = b * p.H + h;
    const int tid = static_cast<int>(threadIdx.x), lane = static_cast<int>(lane_id());
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, qd = lane >> 4, n0 = 16 * wave;
    const int t0 = c * kL, left = __builtin_amdgcn_readfirstlane(live_tokens(p.lens, b, p.T)) - t0, all = min(kL, p.T - t0);
    const int64_t row0 = (static_cast<int64_t>(b) * p.T + t0) * p.H + h;   // of [B, T, H]; a token's next one is p.H on
    using Out = typename std::conditional<FOLD, float, T>::type;
    // Key heads are added up later where they are shared; where not, H is Hk.
    Out* const dq = static_cast<Out*>(p.dq) + row0 * p.kd;
    Out* const dk = static_cast<Out*>(p.dk) + row0 * p.kd;
    T* const dv = static_cast<T*>(p.dv) + row0 * p.vd;
    if (left <= 0) {
        for (int e = tid; e < all * p.kd; e += kThreads) {
            const int64_t at = static_cast<int64_t>(e / p.kd) * p.H * p.kd + e % p.kd;
            dq[at] = narrow<Out>(0.0f);
            dk[at] = narrow<Out>(0.0f);
        }
        for (int e = tid; e < all * p.vd; e += kThreads) dv[static_cast<int64_t>(e / p.vd) * p.H * p.vd + e % p.vd] = narrow<T>(0.0f);
        if (tid < all) p.dg[row0 + static_cast<int64_t>(tid) * p.H] = p.dbeta[row0 + static_cast<int64_t>(tid) * p.H] = 0.0f;
        return;
    }

    Stage<T, KD, kThreads> sq, sk;
    Stage<T, VD, kThreads> sd;
    sq.init(p.q);
    sk.init(p.k);
    sd.init(p.d);
    const T* const db = static_cast<const T*>(p.d.p) + b * p.d.b + h * p.d.h + static_cast<int64_t>(t0) * p.d.t;
    sk.fill(p.k, static_cast<const T*>(p.k.p) + b * p.k.b + (h / p.k.per) * p.k.h + static_cast<int64_t>(t0) * p.k.t, left, kt, wave, tid);
    sd.fill(p.d, db, left, dt, wave, tid);
    if (wave == kWaves - 1) {
        const int64_t t = t0 + min(lane, left - 1);
        const bool live = lane < left;
        const float g = live ? p.g[b * p.g_b + t * p.g_t + h * p.g_h] : 0.0f;
        gate_factors<false>(g, 1.0f, 1.0f, gates, lane);
        one_gate[lane] = g;
        beta[lane] = live ? p.beta[b * p.e_b + t * p.e_t + h * p.e_h] : 0.0f;
    }
    lds_barrier();   // beta

    // u and dv in parts; dbeta, dv and v . dv of every token. A thread takes 8 columns of a token at a time.
    const int64_t vrow = (static_cast<int64_t>(bh) * p.T + t0) * p.vd;
    {
        constexpr int kUnits = VD / 8;
        static_assert(kThreads % kUnits == 0, "a token's columns are neighbouring lanes'");
        const T* const vb = static_cast<const T*>(p.v.p) + b * p.v.b + h * p.v.h + static_cast<int64_t>(t0) * p.v.t;
        const bool wide = p.vd % 8 == 0;
        for (int at = tid; at < kL * kUnits; at += kThreads) {
            const int t = at / kUnits, col = 8 * (at % kUnits);
            float r[8], d[8], v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = d[e] = v[e] = 0.0f;
            if (t < left && col < p.vd) {
                const float* rp = p.miss + vrow + t * p.vd + col;
                const float* dp = p.du + vrow + t * p.vd + col;
                const T* vp = vb + t * p.v.t + col;
                if (wide) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const f32x4 x = *reinterpret_cast<const f32x4*>(rp + 4 * s), y = *reinterpret_cast<const f32x4*>(dp + 4 * s);
#pragma unroll
                        for (int e = 0; e < 4; ++e) { r[4 * s + e] = x[e]; d[4 * s + e] = y[e]; }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (col + e < p.vd) { r[e] = rp[e]; d[e] = dp[e]; }
                    }
                }
                if (wide && p.v.wide) {
                    Frag<T> f;
                    __builtin_memcpy(&f, __builtin_assume_aligned(vp, 16), sizeof(f));
                    widen8(f, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = col + e < p.vd ? widen(vp[e]) : 0.0f;
                }
            }
            float db_ = 0.0f, vd_ = 0.0f, u[8], w[8];
            const float be = beta[t];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                db_ = fmaf(d[e], r[e], db_);
                u[e] = be * r[e];
                w[e] = be * d[e];
                vd_ = fmaf(v[e], w[e], vd_);
            }
            if (t < all && col < p.vd) {
                T* o = dv + static_cast<int64_t>(t) * p.H * p.vd + col;
                const f32x4 w0 = {w[0], w[1], w[2], w[3]}, w1 = {w[4], w[5], w[6], w[7]};
                store_four<T>(o, 0, w0, p.vd - col, wide);
                if (col + 4 < p.vd) store_four<T>(o, 4, w1, p.vd - col - 4, wide);
            }
            db_ = group_sum<kUnits>(db_);
            vd_ = group_sum<kUnits>(vd_);
            if (col == 0) {
                vdv[t] = vd_;
                if (t < all) p.dbeta[row0 + static_cast<int64_t>(t) * p.H] = db_;
            }
            Parts<T, NP> up, wp;
            split(u, up);
            split(w, wp);
#pragma unroll
            for (int s = 0; s < NP; ++s) {
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<u32x4*>(piece<T, VD>(ut + s * kL * VD, t, col >> 3)) = up.p[s].w;
                    *reinterpret_cast<u32x4*>(piece<T, VD>(wt + s * kL * VD, t, col >> 3)) = wp.p[s].w;
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        *reinterpret_cast<f32x4*>(piece<T, VD>(ut, t, (col >> 2) + n)) = f32x4{u[4 * n], u[4 * n + 1], u[4 * n + 2], u[4 * n + 3]};
                        *reinterpret_cast<f32x4*>(piece<T, VD>(wt, t, (col >> 2) + n)) = f32x4{w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]};
                    }
                }
            }
        }
    }
    // The wave's rows n0 + lane % 16 of the state and of its gradient: columns 32 kb + 8 quarter + ..
    float S[VB][8], R[VB][8];
    const int64_t one = static_cast<int64_t>(p.kd) * p.vd, at_state = (static_cast<int64_t>(bh) * p.chunks + c) * one;
    auto state_rows = [&](const float* from, float (&x)[VB][8]) {
        const auto s = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(from), 0, static_cast<int>(one) * 4, 0x00027000);
        const uint32_t at = 4u * static_cast<uint32_t>((n0 + i16) * p.vd + 8 * qd);
        const bool on = n0 + i16 < p.kd, four = p.vd % 4 == 0;
#pragma unroll
        for (int kb = 0; kb < VB; ++kb) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int col = 32 * kb + 8 * qd + 4 * n;
                if (four) {
                    const f32x4 w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                  s, static_cast<int>(on && col < p.vd ? at + 128u * kb + 16u * n : 0xC0000000u), 0, 0));
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[kb][4 * n + e] = w[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[kb][4 * n + e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                            s, static_cast<int>(on && col + e < p.vd ? at + 128u * kb + 16u * n + 4u * e : 0xC0000000u), 0, 0));
                }
            }
        }
    };
    state_rows(p.states + at_state, S);
    state_rows(p.grads + at_state, R);
    tile_barrier();

    // E_i . u_j for dq
    for (int e = wave; e < 12; e += kWaves) {
        const int pr = e >> 1;
        int it = 0, jb = 0;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            if (k == pr) { it = Pairs<false>::kIt[k]; jb = Pairs<false>::kJb[k]; }
        }
        const int jt = 2 * jb + (e & 1);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (jt <= it) {
            f32x4 a = {0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < VB; ++kb) {
                const Frag<T> df = row_frag<VD>(dt, 16 * it + i16, kb, qd);
                Parts<T, NP> up;
                row_parts<T, VD>(ut, 16 * jt + i16, kb, qd, up);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n) mma(up.p[n], df, a);
            }
            decay_scores<false, false>(gates, it, jt, i16, qd, p.scale, a, s);
        }
        half_write<T>(scores, pr, e & 1, lane, f32x4{s[0], s[1], s[2], s[3]});
    }
    // S E and S dv
    f32x4 Q[4], K[4];   // tile it: columns n0 + 4 quarter + r down, token 16 it + lane % 16
#pragma unroll
    for (int it = 0; it < 4; ++it) Q[it] = K[it] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < VB; ++kb) {
        Parts<T, NP> sp;
        split(S[kb], sp);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const Frag<T> df = row_frag<VD>(dt, 16 * it + i16, kb, qd);
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) mma(sp.p[n], df, Q[it]);
            Parts<T, NP> wp;
            row_parts<T, VD>(wt, 16 * it + i16, kb, qd, wp);
            mma_parts(sp, wp, K[it]);
        }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const float f = gates.f[16 * it + i16];
        Q[it] = decayed(f * p.scale, Q[it]);
        K[it] = decayed(-f, K[it]);
    }
    Frag<T> kf[2];
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) kf[jb] = col_frag<KD, 4>(kt, jb, n0, i16, qd);
    lds_barrier();   // the scores are complete
#pragma unroll
    for (int pr = 0; pr < 6; ++pr) {
        Parts<T, NP> pp;
        frag_read(scores, pr, lane, pp);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) mma(kf[Pairs<false>::kJb[pr]], pp.p[n], Q[Pairs<false>::kIt[pr]]);
    }
    lds_barrier();   // and read
    // E_j . u_i for dk
    for (int e = wave; e < 12; e += kWaves) {
        const int pr = e >> 1;
        int it = 0, jb = 0;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            if (k == pr) { it = Pairs<true>::kIt[k]; jb = Pairs<true>::kJb[k]; }
        }
        const int jt = 2 * jb + (e & 1);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (jt >= it) {
            f32x4 a = {0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < VB; ++kb) {
                const Frag<T> df = row_frag<VD>(dt, 16 * jt + i16, kb, qd);
                Parts<T, NP> up;
                row_parts<T, VD>(ut, 16 * it + i16, kb, qd, up);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n) mma(df, up.p[n], a);
            }
            decay_scores<true, false>(gates, it, jt, i16, qd, p.scale, a, s);
        }
        half_write<T>(scores, pr, e & 1, lane, f32x4{s[0], s[1], s[2], s[3]});
    }
    lds_barrier();   // complete, and d_o's tile is free
    sq.fill(p.q, static_cast<const T*>(p.q.p) + b * p.q.b + (h / p.q.per) * p.q.h + static_cast<int64_t>(t0) * p.q.t, left, qt, wave, tid);
    // R u; <S behind the chunk, R> = exp(G_L) <S, R> + sum_j exp(G_L - G_j) k_j . R u_j
    float x = 0.0f;
    {
        f32x4 A[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) A[it] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < VB; ++kb) {
            Parts<T, NP> rp;
            split(R[kb], rp);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                Parts<T, NP> up;
                row_parts<T, VD>(ut, 16 * it + i16, kb, qd, up);
                mma_parts(rp, up, A[it]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x = fmaf(S[kb][e], R[kb][e], x);
        }
        x = sdm_decayed(gates.all, x);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            A[it] = decayed(gates.u[16 * it + i16], A[it]);
            const f32x4 k = tile_four<KD>(kt, 16 * it + i16, n0 + 4 * qd);
#pragma unroll
            for (int r = 0; r < 4; ++r) x = fmaf(k[r], A[it][r], x);
            K[it] += A[it];
        }
    }
    tile_barrier();   // q's tile
    {
        Frag<T> qf[2];
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) qf[jb] = col_frag<KD, 4>(qt, jb, n0, i16, qd);
#pragma unroll
        for (int pr = 0; pr < 6; ++pr) {
            Parts<T, NP> pp;
            frag_read(scores, pr, lane, pp);
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) mma(qf[Pairs<true>::kJb[pr]], pp.p[n], K[Pairs<true>::kIt[pr]]);
        }
    }
    lds_barrier();   // the scores are read
    // - (dv_i . u_j) of earlier tokens j and of later ones the other way round
    for (int e = wave; e < 16; e += kWaves) {
        const int it = e >> 2, jt = e & 3;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s2[4];
        f32x4 a = {0, 0, 0, 0}, a2 = {0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < VB; ++kb) {
            Parts<T, NP> xp, yp;
            row_parts<T, VD>(jt <= it ? wt : ut, 16 * it + i16, kb, qd, xp);
            row_parts<T, VD>(jt <= it ? ut : wt, 16 * jt + i16, kb, qd, yp);
            mma_parts(yp, xp, a);
            if (jt == it) mma_parts(xp, yp, a2);
        }
        if (jt <= it) decay_scores<false, true>(gates, it, jt, i16, qd, -1.0f, a, s);
        else decay_scores<true, true>(gates, it, jt, i16, qd, -1.0f, a, s);
        if (jt == it) {
            decay_scores<true, true>(gates, it, jt, i16, qd, -1.0f, a2, s2);
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] += s2[r];   // one of the two is 0
        }
        half_write<T>(scores, e >> 1, e & 1, lane, f32x4{s[0], s[1], s[2], s[3]});
    }
    lds_barrier();
#pragma unroll
    for (int pr = 0; pr < 8; ++pr) {
        Parts<T, NP> pp;
        frag_read(scores, pr, lane, pp);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) mma(kf[pr & 1], pp.p[n], K[pr >> 1]);
    }
    // Results.
    float odd = 0.0f;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
#pragma unroll
        for (int r = 0; r < 4; ++r) odd = fmaf(Q[it][r], 0.0f, fmaf(K[it][r], 0.0f, odd));
    }
    if (__builtin_expect(__ballot(odd != odd) != 0, 0)) {
        // Something is not finite: the wave's columns token by token, forwards with the state, then backwards with its gradient.
        // u's and dv's tiles are not read any more; they take what dk is given forwards.
        float* const kept = reinterpret_cast<float*>(ut) + wave * (kL * 16);
        const int n = min(left, kL), col = n0 + i16;
        const float* const rp = p.miss + vrow;
        const float* const dp = p.du + vrow;
        constexpr int kElems = 16 / static_cast<int>(sizeof(T));
        auto key = [&](T* tile, int t) {   // column `col` of a token's row
            return widen(*reinterpret_cast<const T*>(piece<T, KD>(tile, t, col / kElems) + (col % kElems) * static_cast<int>(sizeof(T))));
        };
        for (int t = 0; t < n; ++t) {
            const float a = gate_factor(one_gate[t]), be = beta[t], k = key(kt, t);
            float sq_ = 0.0f, sk_ = 0.0f;
#pragma unroll
            for (int kb = 0; kb < VB; ++kb) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 32 * kb + 8 * qd + e;
                    if (j >= p.vd) continue;
                    const float s = sdm_decayed(a, S[kb][e]);
                    sk_ = fmaf(s, be * dp[t * p.vd + j], sk_);
                    S[kb][e] = fmaf(k, be * rp[t * p.vd + j], s);
                    sq_ = fmaf(S[kb][e], widen(db[t * p.d.t + j]), sq_);
                }
            }
            sq_ += lane_xor_f<16>(sq_);
            sq_ += lane_xor_f<32>(sq_);
            sk_ += lane_xor_f<16>(sk_);
            sk_ += lane_xor_f<32>(sk_);
            sq_ *= p.scale;
            if (qd == 0) {
                kept[t * 16 + i16] = sk_;
                if (col < p.kd) dq[static_cast<int64_t>(t) * p.H * p.kd + col] = narrow<Out>(sq_);
            }
            const float dot = group_sum<16>(col < p.kd ? key(qt, t) * sq_ : 0.0f);
            if (lane == 0) dots[wave * kL + t] = dot;
        }
        x = 0.0f;
#pragma unroll
        for (int kb = 0; kb < VB; ++kb) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (col < p.kd && 32 * kb + 8 * qd + e < p.vd) x = fmaf(S[kb][e], R[kb][e], x);
            }
        }
        for (int t = n - 1; t >= 0; --t) {
            const float a = gate_factor(one_gate[t]), be = beta[t], k = key(kt, t),
                        q = p.scale * key(qt, t);
            float sum = 0.0f;
#pragma unroll
            for (int kb = 0; kb < VB; ++kb) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 32 * kb + 8 * qd + e;
                    if (j >= p.vd) continue;
                    const float s = fmaf(q, widen(db[t * p.d.t + j]), R[kb][e]);
                    sum = fmaf(s, be * rp[t * p.vd + j], sum);
                    R[kb][e] = sdm_decayed(a, fmaf(-k, be * dp[t * p.vd + j], s));
                }
            }
            sum += lane_xor_f<16>(sum);
            sum += lane_xor_f<32>(sum);
            if (qd == 0 && col < p.kd) dk[static_cast<int64_t>(t) * p.H * p.kd + col] = narrow<Out>(sum - kept[t * 16 + i16]);
        }
        for (int e = lane; e < (all - n) * 16; e += kWave) {
            const int t = n + e / 16;
            if (n0 + e % 16 >= p.kd) continue;
            const int64_t at = static_cast<int64_t>(t) * p.H * p.kd + n0 + e % 16;
            dq[at] = narrow<Out>(0.0f);
            dk[at] = narrow<Out>(0.0f);
        }
    } else {
        const int n = n0 + 4 * qd;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int t = 16 * it + i16;
            const f32x4 q = tile_four<KD>(qt, t, n);
            float dot = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) dot = fmaf(q[r], Q[it][r], dot);
            dot += lane_xor_f<16>(dot);
            dot += lane_xor_f<32>(dot);
            if (qd == 0) dots[wave * kL + t] = dot;
            if (t >= all || n >= p.kd) continue;
            if (t >= left) Q[it] = K[it] = f32x4{0, 0, 0, 0};
            const int64_t at = static_cast<int64_t>(t) * p.H * p.kd + n;
            store_four<Out>(dq, at, Q[it], p.kd - n, p.key_wide);
            store_four<Out>(dk, at, K[it], p.kd - n, p.key_wide);
        }
    }
    x = group_sum<kWave>(x);
    if (lane == 0) cross[wave] = x;
    lds_barrier();
    if (wave == 0) {
        const int t = kL - 1 - lane;   // lanes go back in time
        double carry = 0.0, y = 0.0, d = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) carry += static_cast<double>(cross[w]);
        if (t < left) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) d += static_cast<double>(dots[w * kL + t]);
            d -= static_cast<double>(vdv[t]);
        }
        // A piece ends with the token that resets, the first one in time: the next starts behind it, from 0.
        const uint64_t cuts = __ballot(t < left && (resets(one_gate[t]) || (p.stateless && t0 + t == 0)));
        pieces(cuts << 1, d, lane, [&](int from, int to, double sum) {
            if (lane >= from && lane < to) y = carry + sum;
            carry = 0.0;
        });
        if ((cuts >> lane) & 1) y = 0.0;
        if (t < all) p.dg[row0 + static_cast<int64_t>(t) * p.H] = t < left ? static_cast<float>(y) : 0.0f;
    }
}

// The gradients of shared heads: the sum of `per` value heads' float32 rows, in head order (dq, then dk).
template <typename T>
__global__ __launch_bounds__(256) void gdr_fold_kernel(const float* fq, const float* fk, T* dq, T* dk, int64_t total, int d, int per) {
    const float* in = blockIdx.y ? fk : fq;
    T* out = blockIdx.y ? dk : dq;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = e / d, c = e - row * d;
        float s = 0.0f;
        for (int r = 0; r < per; ++r) s += in[(row * per + r) * d + c];
        out[e] = narrow<T>(s);
    }
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
    const float ga = token_factor(io.g[b * io.g_b + h * io.g_h]);
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
size_t chunk_lds() { return kChunkTiles<T, KD> + kL * kRow * 4 + sizeof(Gates) + kL * 4; }

template <typename T, int KD>
size_t main_lds(bool out) {
    return (kTwo<T, KD> ? 2 : 1) * (kL * ((out ? 2 : 1) * KD + 64) * sizeof(T) + (out ? 2 : 1) * kFragBytes<T> + kFacBytes);
}

int chunks_of(int T) { return (T + kL - 1) / kL; }

// Segments of the time axis. A block's way along it is most of the time where there are few blocks, so the axis is cut: a pass
// makes every segment's own state and transition (as many columns again as the state has rows), a kernel chains them, and the main
// pass runs on all segments at once. Rounds of blocks over the compute units times a segment's chunks, at 3.5 us a chunk, 3 without
// outputs, and 1.5 a step of the chain, say whether and how finely: 1 x 16384 tokens x 8 heads of 128, forward, 925 us whole and 230 in
// 16 segments; 8 x 4096 x 16 stays whole. The prices are those of bfloat16 forward at 128 columns; the backward pass, float32 (about twice
// as much) and narrower heads (half) are cut by them too. The same tokens and heads: backward 670, float32 595 and 1435, 64 columns 126 and 370.
constexpr int kUnits = 256;
struct SegPlan {
    int nseg, seg;
};
SegPlan seg_plan(const sdm_gdr_io* io) {
    const int64_t bh = static_cast<int64_t>(io->B) * io->H, chunks = chunks_of(io->T), cols = (io->dv + 63) / 64, kcols = (io->dk + 63) / 64;
    auto rounds = [](int64_t blocks) { return static_cast<double>((blocks + kUnits - 1) / kUnits); };
    SegPlan best{1, static_cast<int>(chunks > 0 ? chunks : 1)};
    double cost = rounds(bh * cols) * chunks * 3.5;
    for (int64_t per = (chunks + 1) / 2; per >= 2; per = per > 16 ? per * 3 / 4 : per - 1) {
        const int64_t n = (chunks + per - 1) / per;
        const double c = rounds(n * bh * (cols + kcols)) * per * 3.0 + 1.5 * n + 10.0 + rounds(n * bh * cols) * per * 3.5;
        if (c < cost) {
            cost = c;
            best = SegPlan{static_cast<int>(n), static_cast<int>(per)};
        }
    }
    return best;
}

// Byte offsets in the workspace.
struct GdrLayout {
    size_t rec, move, own, from, kinds, rown, rfrom, states, grads, miss, du, fq, fk, total;
};
GdrLayout gdr_layout(const sdm_gdr_io* io, bool backward) {
    const size_t bh = static_cast<size_t>(io->B) * io->H, n = bh * chunks_of(io->T), rows = bh * io->T;
    GdrLayout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    const SegPlan sp = seg_plan(io);
    if (sp.nseg > 1) {
        const size_t states = bh * sp.nseg * io->dk * io->dv * 4;
        l.move = take(bh * sp.nseg * io->dk * io->dk * 4);
        l.own = take(states);
        l.from = take(states);
        l.kinds = take(bh * sp.nseg * 4);
        if (backward) {
            l.rown = take(states);
            l.rfrom = take(states);
        }
    }
    if (backward) {
        l.rec = take(n * kRecBytes<true>);
        l.states = take(n * io->dk * io->dv * 4);
        l.grads = take(n * io->dk * io->dv * 4);
        l.miss = take(rows * io->dv * 4);
        l.du = take(rows * io->dv * 4);
        if (io->H > io->Hk) {
            l.fq = take(rows * io->dk * 4);
            l.fk = take(rows * io->dk * 4);
        }
    } else {
        l.rec = take(n * kRecBytes<false>);
    }
    l.total = at;
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

template <typename T, bool OUT, bool SEG>
hipError_t main_go(const sdm_gdr_io* io, const MainArgs& a, hipStream_t st) {
    const int64_t blocks = SEG ? static_cast<int64_t>(a.made) * (a.cols + (a.kd + 63) / 64) : static_cast<int64_t>(a.nseg) * a.cols;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(io->B) * io->H * blocks);
    if (padded(io->dk) == 64) gdr_kernel<T, 64, OUT, SEG><<<grid, kMainThreads<T, 64>, main_lds<T, 64>(OUT), st>>>(a);
    else gdr_kernel<T, 128, OUT, SEG><<<grid, kMainThreads<T, 128>, main_lds<T, 128>(OUT), st>>>(a);
    return hipGetLastError();
}

template <bool REV>
hipError_t chain_go(const sdm_gdr_io* io, const ChainArgs& a, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(io->B) * io->H * a.cols);
    if (padded(io->dk) == 64) gdr_chain_kernel<64, REV><<<grid, 256, 0, st>>>(a);
    else gdr_chain_kernel<128, REV><<<grid, 512, 0, st>>>(a);
    return hipGetLastError();
}

// The call without outputs, and the states before its segments (`made` of whose transitions are needed), if it has some.
template <typename T, bool BACK>
hipError_t begin(const sdm_gdr_io* io, const GdrLayout& l, MainArgs& a, hipStream_t st) {
    const int per = io->H / io->Hk, es = sizeof(T);
    char* ws = static_cast<char*>(io->workspace);
    const SegPlan sp = seg_plan(io);
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
    a.rec = ws + l.rec;
    a.rec_bytes = kRecBytes<BACK>;
    a.start = io->state;
    a.nseg = sp.nseg;
    a.seg = sp.seg;
    if (io->T == 0) return hipSuccess;
    hipError_t e = chunk_go<T, BACK>(io, ws + l.rec, st);
    if (e != hipSuccess || sp.nseg == 1) return e;
    a.made = BACK ? sp.nseg : sp.nseg - 1;   // what leaves the last one only the backward pass goes through
    a.own = reinterpret_cast<float*>(ws + l.own);
    a.move = reinterpret_cast<float*>(ws + l.move);
    a.kinds = reinterpret_cast<int32_t*>(ws + l.kinds);
    a.from = nullptr;
    if ((e = main_go<T, false, true>(io, a, st)) != hipSuccess) return e;
    float* from = reinterpret_cast<float*>(ws + l.from);
    a.from = from;
    return chain_go<false>(io, ChainArgs{a.move, a.own, a.kinds, a.start, from, sp.nseg, io->dk, io->dv, (io->dv + 15) / 16}, st);
}

template <typename T>
hipError_t forward(const sdm_gdr_io* io, hipStream_t st) {
    const int es = sizeof(T);
    MainArgs a{};
    const hipError_t e = begin<T, false>(io, gdr_layout(io, false), a, st);
    if (e != hipSuccess) return e;
    a.last = io->last;
    a.out = io->o;
    a.o_b = io->o_b;
    a.o_t = io->o_t;
    a.o_h = io->o_h;
    a.out_wide = reinterpret_cast<uintptr_t>(io->o) % (4 * es) == 0 && io->o_b % 4 == 0 && io->o_t % 4 == 0 && io->o_h % 4 == 0 && io->dv % 4 == 0;
    return main_go<T, true, false>(io, a, st);
}

template <typename T, int KD, bool FOLD>
hipError_t grad_go2(const GradArgs& a, unsigned grid, hipStream_t st) {
    if (padded(a.vd) == 64) gdr_grad_kernel<T, KD, 64, FOLD><<<grid, 4 * KD, GradLds<T, KD, 64>::kTotal, st>>>(a);
    else gdr_grad_kernel<T, KD, 128, FOLD><<<grid, 4 * KD, GradLds<T, KD, 128>::kTotal, st>>>(a);
    return hipGetLastError();
}
template <typename T, bool FOLD>
hipError_t grad_go(const GradArgs& a, unsigned grid, hipStream_t st) {
    return padded(a.kd) == 64 ? grad_go2<T, 64, FOLD>(a, grid, st) : grad_go2<T, 128, FOLD>(a, grid, st);
}

template <typename T>
hipError_t backward(const sdm_gdr_io* io, const sdm_gdr_grad* g, hipStream_t st) {
    const int per = io->H / io->Hk, es = sizeof(T);
    const GdrLayout l = gdr_layout(io, true);
    char* ws = static_cast<char*>(io->workspace);
    const Rows q = rows_of(io->q, io->q_b, io->q_t, io->q_h, io->dk, per, es), k = rows_of(io->k, io->k_b, io->k_t, io->k_h, io->dk, per, es),
               v = rows_of(io->v, io->v_b, io->v_t, io->v_h, io->dv, 1, es), d = rows_of(g->d_o, g->do_b, g->do_t, g->do_h, io->dv, 1, es);
    const int chunks = chunks_of(io->T), cols = (io->dv + 63) / 64;
    const int64_t bh = static_cast<int64_t>(io->B) * io->H;
    hipError_t e = hipSuccess;
    MainArgs m{};
    if ((e = begin<T, true>(io, l, m, st)) != hipSuccess) return e;
    m.states = reinterpret_cast<float*>(ws + l.states);
    m.miss = reinterpret_cast<float*>(ws + l.miss);
    if (io->T > 0 && (e = main_go<T, false, false>(io, m, st)) != hipSuccess) return e;
    BackArgs b{q, k, d, io->lens, io->T, io->H, chunks, cols, io->dk, io->dv, io->scale, ws + l.rec, g->d_last, g->d_state,
               reinterpret_cast<float*>(ws + l.grads), reinterpret_cast<float*>(ws + l.du), m.nseg, m.seg, nullptr, reinterpret_cast<float*>(ws + l.rown)};
    if (m.nseg > 1) {
        const unsigned grid = static_cast<unsigned>(bh * cols * (m.nseg - 1));
        if (padded(io->dk) == 64) gdr_back_kernel<T, 64, true><<<grid, kMainThreads<T, 64>, main_lds<T, 64>(true), st>>>(b);
        else gdr_back_kernel<T, 128, true><<<grid, kMainThreads<T, 128>, main_lds<T, 128>(true), st>>>(b);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        float* from = reinterpret_cast<float*>(ws + l.rfrom);
        if ((e = chain_go<true>(io, ChainArgs{m.move, b.own, m.kinds, g->d_last, from, m.nseg, io->dk, io->dv, (io->dv + 15) / 16}, st)) != hipSuccess) return e;
        b.from = from;
    }
    const unsigned grid = static_cast<unsigned>(bh * cols * m.nseg);
    if (padded(io->dk) == 64) gdr_back_kernel<T, 64, false><<<grid, kMainThreads<T, 64>, main_lds<T, 64>(true), st>>>(b);
    else gdr_back_kernel<T, 128, false><<<grid, kMainThreads<T, 128>, main_lds<T, 128>(true), st>>>(b);
    if ((e = hipGetLastError()) != hipSuccess || io->T == 0) return e;
    const bool fold = per > 1;
    GradArgs a{q, k, v, d, io->g, io->beta, io->g_b, io->g_t, io->g_h, io->e_b, io->e_t, io->e_h, io->lens, io->T, io->H, chunks, io->dk, io->dv,
               io->scale, m.states, b.grads, m.miss, b.du, io->state == nullptr, g->dq, g->dk, io->dk % 4 == 0, g->dv, g->dg, g->dbeta};
    if (!fold) return grad_go<T, false>(a, static_cast<unsigned>(bh * chunks), st);
    float *fq = reinterpret_cast<float*>(ws + l.fq), *fk = reinterpret_cast<float*>(ws + l.fk);
    a.dq = fq;
    a.dk = fk;
    if ((e = grad_go<T, true>(a, static_cast<unsigned>(bh * chunks), st)) != hipSuccess) return e;
    const int64_t total = static_cast<int64_t>(io->B) * io->T * io->Hk * io->dk, need = (total + 255) / 256;
    gdr_fold_kernel<T><<<dim3(static_cast<unsigned>(need < (1 << 20) ? need : 1 << 20), 2), 256, 0, st>>>(fq, fk, static_cast<T*>(g->dq),
                                                                                                          static_cast<T*>(g->dk), total, io->dk, per);
    return hipGetLastError();
}

template <typename T, int KD>
void list_grad(const void** all, int& n) {
    all[n++] = reinterpret_cast<const void*>(&gdr_grad_kernel<T, KD, 64, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_grad_kernel<T, KD, 64, true>);
    all[n++] = reinterpret_cast<const void*>(&gdr_grad_kernel<T, KD, 128, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_grad_kernel<T, KD, 128, true>);
}
template <typename T, int KD>
void list_width(const void** all, int& n) {
    all[n++] = reinterpret_cast<const void*>(&gdr_chunk_kernel<T, KD, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_chunk_kernel<T, KD, true>);
    all[n++] = reinterpret_cast<const void*>(&gdr_kernel<T, KD, true, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_kernel<T, KD, false, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_kernel<T, KD, false, true>);
    all[n++] = reinterpret_cast<const void*>(&gdr_back_kernel<T, KD, false>);
    all[n++] = reinterpret_cast<const void*>(&gdr_back_kernel<T, KD, true>);
    list_grad<T, KD>(all, n);
}
template <typename T>
void list(const void** all, int& n) {
    list_width<T, 64>(all, n);
    list_width<T, 128>(all, n);
}

}  // namespace

int gdr_lds_kernels(const void** fns, int cap) {
    const void* all[64];
    int n = 0;
    list<bf16_t>(all, n);
    list<float>(all, n);
    int k = 0;
    for (; k < n && k < cap; ++k) fns[k] = all[k];
    return k;
}

size_t gdr_workspace_bytes(const sdm_gdr_io* io, bool backward) {
    return io->B < 1 || io->T < 1 ? 0 : gdr_layout(io, backward).total;
}

hipError_t gdr_forward_launch(const sdm_gdr_io* io, hipStream_t st) {
    return io->dtype == SDM_BF16 ? forward<bf16_t>(io, st) : forward<float>(io, st);
}

hipError_t gdr_backward_launch(const sdm_gdr_io* io, const sdm_gdr_grad* g, hipStream_t st) {
    return io->dtype == SDM_BF16 ? backward<bf16_t>(io, g, st) : backward<float>(io, g, st);
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
