// RMS norm of every query and key head and the rotation by its token's position, in one pass over the
// heads, and the backward pass.
//
// For a head x of D columns, r = 1 / sqrt(mean(x^2) + eps), y = x r w, and the first `rot` columns of y
// turned pairwise by the token's angles (c, s): (y1, y2) -> (y1 c - y2 s, y2 c + y1 s), a pair being
// (i, i + rot/2) or, interleaved, (2i, 2i + 1). Backward, from the gradient d of the result: d is turned
// back by the transpose, dw = sum d x r, and with n = x r, dn = d w: dx = r (dn - n mean(dn n)).
//
// Everything is bound by the bytes of the heads (read once, written once). A team of lanes owns a head;
// a lane holds four PAIRS, both members, so the rotation needs no exchange between lanes and the angles
// of a pair are loaded once for both; only the sum of squares (and the backward's dot) crosses lanes.
// A team walks the heads of one token, four in flight, with the token's angles in registers: the angles
// are 8 bytes per pair in float32, twice a bfloat16 pair's bytes, and would otherwise be read for every
// head. Sums, norms and the rotation are float32; each result is rounded once. 32768 tokens of 16 + 4 heads
// of 128 (bfloat16): 71 us, 4.7 TB/s of the heads (a copy of as much: 67). Backward, 16381 tokens, half of each
// head turned: 63 us, 47 of them the walk (5.4 TB/s) and 4 the sum of the blocks' weight gradients.
#include <hip/hip_runtime.h>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"

namespace sdm {
namespace {

constexpr int kNrThreads = 256;
// Waves a launch should have before a team takes more than one head: two for each of the 1024 SIMDs.
// Above it, longer walks save loads of the angles; below it, more teams hide the latency.
constexpr int64_t kNrWaves = 2048;
constexpr int kNrAhead = 4;   // heads in flight per team

struct NrArgs {
    sdm_norm_rope_io io;
    int H;          // heads of a token, queries first
    int parts;      // teams a token's heads are dealt to
    int per;        // heads per team
};

// Four pairs of a head: columns of the first and second members.
struct Quad {
    int o1, o2;
    bool on, turn;
    bool one;   // scalar path only: the second member does not exist (the last column of an odd rest)
};

// Vector path: pairs 4l .. 4l+3 of the head, whose members lie in two runs of four columns (half
// layout; the columns after rot are split into two runs the same way) or in one run of eight.
template <bool INTER>
__device__ __forceinline__ Quad quad_of(int l, int D, int rot) {
    Quad q;
    const int p = 4 * l, h = rot >> 1;
    q.on = p < (D >> 1);
    q.turn = p < h;
    q.one = false;
    if (INTER) {
        q.o1 = 2 * p;
        q.o2 = 2 * p + 4;
    } else if (q.turn) {
        q.o1 = p;
        q.o2 = p + h;
    } else {
        q.o1 = rot + (p - h);
        q.o2 = q.o1 + ((D - rot) >> 1);
    }
    return q;
}

// x[0..3] the first members, x[4..7] the second ones.
template <bool INTER>
__device__ __forceinline__ void load_quad(const float* p, const Quad& q, float* x) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + q.o1), b = *reinterpret_cast<const f32x4*>(p + q.o2);
    if (INTER) {
        x[0] = a[0]; x[4] = a[1]; x[1] = a[2]; x[5] = a[3];
        x[2] = b[0]; x[6] = b[1]; x[3] = b[2]; x[7] = b[3];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
    }
}

template <bool INTER>
__device__ __forceinline__ void load_raw(const bf16_t* p, const Quad& q, u32x4& w) {
    if (INTER) {
        w = *reinterpret_cast<const u32x4*>(p + q.o1);
    } else {
        const u32x2 a = *reinterpret_cast<const u32x2*>(p + q.o1), b = *reinterpret_cast<const u32x2*>(p + q.o2);
        w = u32x4{a[0], a[1], b[0], b[1]};
    }
}

template <bool INTER>
__device__ __forceinline__ void unpack_raw(const u32x4& w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
        if (INTER) {
            x[i] = lo;
            x[4 + i] = hi;
        } else {
            x[2 * i] = lo;
            x[2 * i + 1] = hi;
        }
    }
}

template <bool INTER>
__device__ __forceinline__ void store_quad(float* p, const Quad& q, const float* x) {
    if (INTER) {
        *reinterpret_cast<f32x4*>(p + q.o1) = f32x4{x[0], x[4], x[1], x[5]};
        *reinterpret_cast<f32x4*>(p + q.o2) = f32x4{x[2], x[6], x[3], x[7]};
    } else {
        *reinterpret_cast<f32x4*>(p + q.o1) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4*>(p + q.o2) = f32x4{x[4], x[5], x[6], x[7]};
    }
}
template <bool INTER>
__device__ __forceinline__ void store_quad(bf16_t* p, const Quad& q, const float* x) {
    if (INTER) {
        *reinterpret_cast<u32x4*>(p + q.o1) =
            u32x4{pack_bf16(x[0], x[4]), pack_bf16(x[1], x[5]), pack_bf16(x[2], x[6]), pack_bf16(x[3], x[7])};
    } else {
        *reinterpret_cast<u32x2*>(p + q.o1) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        *reinterpret_cast<u32x2*>(p + q.o2) = u32x2{pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
}

// Norm weights of the lane's columns (ones where there are none), float32 or bfloat16.
template <bool INTER>
__device__ __forceinline__ void load_weights(const void* w, int bf, const Quad& q, float* x) {
    if (w == nullptr || !q.on) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 1.0f;
    } else if (bf) {
        u32x4 r;
        load_raw<INTER>(static_cast<const bf16_t*>(w), q, r);
        unpack_raw<INTER>(r, x);
    } else {
        load_quad<INTER>(static_cast<const float*>(w), q, x);
    }
}

__device__ __forceinline__ int64_t table_row(const sdm_norm_rope_io& io, int64_t t) {
    const int64_t p = io.pos_bytes == 8 ? static_cast<const int64_t*>(io.pos)[t] : static_cast<const int32_t*>(io.pos)[t];
    return p < 0 ? 0 : p >= io.table_rows ? io.table_rows - 1 : p;   // in bounds whatever the caller passed
}

// The four rows a team has in flight: raw words of bfloat16 rows, floats of float32 rows.
template <typename T>
struct Row;
template <>
struct Row<bf16_t> {
    u32x4 w;
    template <bool INTER>
    __device__ __forceinline__ void load(const bf16_t* p, const Quad& q) { load_raw<INTER>(p, q, w); }
    template <bool INTER>
    __device__ __forceinline__ void get(float* x) const { unpack_raw<INTER>(w, x); }
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
};
template <>
struct Row<float> {
    float v[8];
    template <bool INTER>
    __device__ __forceinline__ void load(const float* p, const Quad& q) { load_quad<INTER>(p, q, v); }
    template <bool INTER>
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
};

template <typename T, bool INTER, int TL>
__global__ __launch_bounds__(kNrThreads) void norm_rope_kernel(NrArgs a) {
    const sdm_norm_rope_io& io = a.io;
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kNrThreads + threadIdx.x) / TL;
    if (item >= io.N * a.parts) return;   // whole teams leave together
    const int64_t t = item / a.parts;
    const int part = static_cast<int>(item - t * a.parts);
    const Quad q = quad_of<INTER>(threadIdx.x % TL, io.D, io.rot);
    float c[4], s[4], wq[8], wk[8];
    if (q.on && q.turn) {
        const float* tab = io.table + table_row(io, t) * io.rot + 4 * (threadIdx.x % TL);
        const f32x4 cv = *reinterpret_cast<const f32x4*>(tab), sv = *reinterpret_cast<const f32x4*>(tab + (io.rot >> 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) { c[i] = cv[i]; s[i] = sv[i]; }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) { c[i] = 1.0f; s[i] = 0.0f; }
    }
    load_weights<INTER>(io.wq, io.w_dtype == SDM_BF16, q, wq);
    load_weights<INTER>(io.wk, io.w_dtype == SDM_BF16, q, wk);
    const float inv_d = 1.0f / static_cast<float>(io.D);
    const int h0 = part * a.per, h1 = min(a.H, h0 + a.per);
    for (int h = h0; h < h1; h += kNrAhead) {
        Row<T> rows[kNrAhead];
#pragma unroll
        for (int u = 0; u < kNrAhead; ++u) {
            rows[u].zero();
            if (h + u < h1 && q.on) {
                const int hh = h + u;
                const T* p = hh < io.Hq ? static_cast<const T*>(io.q) + t * io.q_row + hh * io.q_head
                                        : static_cast<const T*>(io.k) + t * io.k_row + (hh - io.Hq) * io.k_head;
                rows[u].template load<INTER>(p, q);
            }
        }
#pragma unroll
        for (int u = 0; u < kNrAhead; ++u) {
            if (h + u >= h1) break;
            const int hh = h + u;
            float x[8];
            rows[u].template get<INTER>(x);
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            ss = group_sum<TL>(ss);
            const float r = rsqrtf(fmaf(ss, inv_d, io.eps));
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y1 = x[i] * r * (hh < io.Hq ? wq[i] : wk[i]), y2 = x[4 + i] * r * (hh < io.Hq ? wq[4 + i] : wk[4 + i]);
                y[i] = fmaf(y1, c[i], -(y2 * s[i]));
                y[4 + i] = fmaf(y2, c[i], y1 * s[i]);
            }
            T* p = hh < io.Hq ? static_cast<T*>(io.q_out) + t * io.qo_row + hh * io.qo_head
                              : static_cast<T*>(io.k_out) + t * io.ko_row + (hh - io.Hq) * io.ko_head;
            if (q.on) store_quad<INTER>(p, q, y);
        }
    }
}

// One wave per head, pair by pair: any D, rot, stride and alignment.
constexpr int kNrPairs = 4;   // pairs per lane: D up to 512

__device__ __forceinline__ Quad pair_of(int p, int D, int rot, int inter) {
    Quad q;
    const int h = rot >> 1, rest = D - rot;
    q.turn = p < h;
    q.on = p < h + ((rest + 1) >> 1);
    if (q.turn) {
        q.o1 = inter ? 2 * p : p;
        q.o2 = inter ? 2 * p + 1 : p + h;
    } else {
        q.o1 = rot + 2 * (p - h);
        q.o2 = q.o1 + 1;
    }
    q.one = q.on && q.o2 >= D;
    return q;
}

__device__ __forceinline__ float weight_at(const void* w, int bf, int i) {
    return w == nullptr ? 1.0f : load_val(w, i, bf);
}

template <typename T>
__global__ __launch_bounds__(kNrThreads) void norm_rope_any_kernel(NrArgs a) {
    const sdm_norm_rope_io& io = a.io;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kNrThreads + threadIdx.x) / kWave;
    if (row >= io.N * a.H) return;
    const int64_t t = row / a.H;
    const int hh = static_cast<int>(row - t * a.H);
    const bool isq = hh < io.Hq;
    const T* p = isq ? static_cast<const T*>(io.q) + t * io.q_row + hh * io.q_head
                     : static_cast<const T*>(io.k) + t * io.k_row + (hh - io.Hq) * io.k_head;
    T* po = isq ? static_cast<T*>(io.q_out) + t * io.qo_row + hh * io.qo_head
                : static_cast<T*>(io.k_out) + t * io.ko_row + (hh - io.Hq) * io.ko_head;
    const void* w = isq ? io.wq : io.wk;
    const int bf = io.w_dtype == SDM_BF16;
    const float* tab = io.rot > 0 ? io.table + table_row(io, t) * io.rot : nullptr;
    float x1[kNrPairs], x2[kNrPairs], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < kNrPairs; ++j) {
        const Quad q = pair_of(lane_id() + j * kWave, io.D, io.rot, io.interleaved);
        x1[j] = q.on ? widen(p[q.o1]) : 0.0f;
        x2[j] = q.on && !q.one ? widen(p[q.o2]) : 0.0f;
        ss = fmaf(x1[j], x1[j], ss);
        ss = fmaf(x2[j], x2[j], ss);
    }
    const float r = rsqrtf(fmaf(group_sum<kWave>(ss), 1.0f / static_cast<float>(io.D), io.eps));
#pragma unroll
    for (int j = 0; j < kNrPairs; ++j) {
        const int pi = lane_id() + j * kWave;
        const Quad q = pair_of(pi, io.D, io.rot, io.interleaved);
        if (!q.on) continue;
        const float y1 = x1[j] * r * weight_at(w, bf, q.o1), y2 = q.one ? 0.0f : x2[j] * r * weight_at(w, bf, q.o2);
        const float c = q.turn ? tab[pi] : 1.0f, s = q.turn ? tab[(io.rot >> 1) + pi] : 0.0f;
        po[q.o1] = narrow<T>(fmaf(y1, c, -(y2 * s)));
        if (!q.one) po[q.o2] = narrow<T>(fmaf(y2, c, y1 * s));
    }
}

// ------------------------------------------------------------------------------------------ backward
//
// A team walks tokens grid-stride; it keeps the weight gradients of its columns in registers, the teams
// of a block add theirs in LDS in a fixed order, and a second kernel adds the blocks' rows in order: no
// atomics, so the sums are the same every run.
struct NrBack {
    NrArgs a;
    const void *dq, *dk;
    int64_t dq_row, dq_head, dk_row, dk_head;
    float* part;      // [blocks, 2, D]
    int64_t items;    // N * parts
};

template <typename T, bool INTER, int TL>
__global__ __launch_bounds__(kNrThreads) void norm_rope_back_kernel(NrBack b) {
    constexpr int kAhead = 2;   // two rows (head and gradient) per head in flight
    const sdm_norm_rope_io& io = b.a.io;
    extern __shared__ float sums[];   // [teams, 2, 8 TL]
    const int team = threadIdx.x / TL, teams = kNrThreads / TL, l = threadIdx.x % TL;
    const Quad q = quad_of<INTER>(l, io.D, io.rot);
    float wq[8], wk[8], gq[8], gk[8];
    load_weights<INTER>(io.wq, io.w_dtype == SDM_BF16, q, wq);
    load_weights<INTER>(io.wk, io.w_dtype == SDM_BF16, q, wk);
#pragma unroll
    for (int i = 0; i < 8; ++i) { gq[i] = 0.0f; gk[i] = 0.0f; }
    const float inv_d = 1.0f / static_cast<float>(io.D);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * teams + team; item < b.items;
         item += static_cast<int64_t>(gridDim.x) * teams) {
        const int64_t t = item / b.a.parts;
        const int part = static_cast<int>(item - t * b.a.parts);
        float c[4], s[4];
        if (q.on && q.turn) {
            const float* tab = io.table + table_row(io, t) * io.rot + 4 * l;
            const f32x4 cv = *reinterpret_cast<const f32x4*>(tab), sv = *reinterpret_cast<const f32x4*>(tab + (io.rot >> 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) { c[i] = cv[i]; s[i] = sv[i]; }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { c[i] = 1.0f; s[i] = 0.0f; }
        }
        const int h0 = part * b.a.per, h1 = min(b.a.H, h0 + b.a.per);
        for (int h = h0; h < h1; h += kAhead) {
            Row<T> xs[kAhead], ds[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                xs[u].zero();
                ds[u].zero();
                const int hh = h + u;
                if (hh < h1 && q.on) {
                    if (hh < io.Hq) {
                        xs[u].template load<INTER>(static_cast<const T*>(io.q) + t * io.q_row + hh * io.q_head, q);
                        ds[u].template load<INTER>(static_cast<const T*>(b.dq) + t * b.dq_row + hh * b.dq_head, q);
                    } else {
                        const int hk = hh - io.Hq;
                        xs[u].template load<INTER>(static_cast<const T*>(io.k) + t * io.k_row + hk * io.k_head, q);
                        ds[u].template load<INTER>(static_cast<const T*>(b.dk) + t * b.dk_row + hk * b.dk_head, q);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int hh = h + u;
                if (hh >= h1) break;
                const bool isq = hh < io.Hq;
                float x[8], e[8], d[8];
                xs[u].template get<INTER>(x);
                ds[u].template get<INTER>(e);
                float ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = fmaf(e[i], c[i], e[4 + i] * s[i]);
                    d[4 + i] = fmaf(e[4 + i], c[i], -(e[i] * s[i]));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(x[i], x[i], ss);
                    dot = fmaf(d[i] * (isq ? wq[i] : wk[i]), x[i], dot);
                }
                ss = group_sum<TL>(ss);
                dot = group_sum<TL>(dot);
                const float r = rsqrtf(fmaf(ss, inv_d, io.eps));
                const float m = dot * r * inv_d;   // mean of dn n
                float g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float n = x[i] * r, dw = d[i] * n;
                    gq[i] += isq ? dw : 0.0f;
                    gk[i] += isq ? 0.0f : dw;
                    g[i] = r * fmaf(-n, m, d[i] * (isq ? wq[i] : wk[i]));
                }
                T* p = isq ? static_cast<T*>(io.q_out) + t * io.qo_row + hh * io.qo_head
                           : static_cast<T*>(io.k_out) + t * io.ko_row + (hh - io.Hq) * io.ko_head;
                if (q.on) store_quad<INTER>(p, q, g);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sums[(team * 2) * 8 * TL + i * TL + l] = gq[i];
        sums[(team * 2 + 1) * 8 * TL + i * TL + l] = gk[i];
    }
    __syncthreads();
    // Column (i, l) of the quads: summed over the block's teams, stored at its column of the head.
    for (int e = threadIdx.x; e < 2 * 8 * TL; e += kNrThreads) {
        const int which = e / (8 * TL), i = e % (8 * TL) / TL, ll = e % TL;
        float v = 0.0f;
        for (int k = 0; k < teams; ++k) v += sums[(k * 2 + which) * 8 * TL + i * TL + ll];
        const Quad o = quad_of<INTER>(ll, io.D, io.rot);
        if (!o.on) continue;
        const int m = i & 3;
        const int col = INTER ? o.o1 + 2 * m + (i >> 2) : (i < 4 ? o.o1 : o.o2) + m;
        b.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * io.D + col] = v;
    }
}

template <typename T>
__global__ __launch_bounds__(kNrThreads) void norm_rope_back_any_kernel(NrBack b) {
    const sdm_norm_rope_io& io = b.a.io;
    extern __shared__ float sums[];   // [waves, 2, D]
    const int wave = threadIdx.x / kWave, waves = kNrThreads / kWave;
    const int bf = io.w_dtype == SDM_BF16;
    float g1[2][kNrPairs], g2[2][kNrPairs];
#pragma unroll
    for (int j = 0; j < kNrPairs; ++j) { g1[0][j] = g1[1][j] = g2[0][j] = g2[1][j] = 0.0f; }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * waves + wave; row < io.N * b.a.H;
         row += static_cast<int64_t>(gridDim.x) * waves) {
        const int64_t t = row / b.a.H;
        const int hh = static_cast<int>(row - t * b.a.H);
        const bool isq = hh < io.Hq;
        const int hk = hh - io.Hq;
        const T* p = isq ? static_cast<const T*>(io.q) + t * io.q_row + hh * io.q_head
                         : static_cast<const T*>(io.k) + t * io.k_row + hk * io.k_head;
        const T* pd = isq ? static_cast<const T*>(b.dq) + t * b.dq_row + hh * b.dq_head
                          : static_cast<const T*>(b.dk) + t * b.dk_row + hk * b.dk_head;
        T* po = isq ? static_cast<T*>(io.q_out) + t * io.qo_row + hh * io.qo_head
                    : static_cast<T*>(io.k_out) + t * io.ko_row + hk * io.ko_head;
        const void* w = isq ? io.wq : io.wk;
        const float* tab = io.rot > 0 ? io.table + table_row(io, t) * io.rot : nullptr;
        float x1[kNrPairs], x2[kNrPairs], d1[kNrPairs], d2[kNrPairs], ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kNrPairs; ++j) {
            const int pi = lane_id() + j * kWave;
            const Quad q = pair_of(pi, io.D, io.rot, io.interleaved);
            const bool two = q.on && !q.one;
            x1[j] = q.on ? widen(p[q.o1]) : 0.0f;
            x2[j] = two ? widen(p[q.o2]) : 0.0f;
            const float e1 = q.on ? widen(pd[q.o1]) : 0.0f, e2 = two ? widen(pd[q.o2]) : 0.0f;
            const float c = q.turn ? tab[pi] : 1.0f, s = q.turn ? tab[(io.rot >> 1) + pi] : 0.0f;
            d1[j] = fmaf(e1, c, e2 * s);
            d2[j] = fmaf(e2, c, -(e1 * s));
            ss = fmaf(x1[j], x1[j], ss);
            ss = fmaf(x2[j], x2[j], ss);
            dot = fmaf(d1[j] * (q.on ? weight_at(w, bf, q.o1) : 0.0f), x1[j], dot);
            dot = fmaf(d2[j] * (two ? weight_at(w, bf, q.o2) : 0.0f), x2[j], dot);
        }
        const float inv_d = 1.0f / static_cast<float>(io.D);
        const float r = rsqrtf(fmaf(group_sum<kWave>(ss), inv_d, io.eps));
        const float m = group_sum<kWave>(dot) * r * inv_d;
#pragma unroll
        for (int j = 0; j < kNrPairs; ++j) {
            const Quad q = pair_of(lane_id() + j * kWave, io.D, io.rot, io.interleaved);
            const float n1 = x1[j] * r, n2 = x2[j] * r;
            g1[0][j] += isq ? d1[j] * n1 : 0.0f;
            g2[0][j] += isq ? d2[j] * n2 : 0.0f;
            g1[1][j] += isq ? 0.0f : d1[j] * n1;
            g2[1][j] += isq ? 0.0f : d2[j] * n2;
            if (q.on) po[q.o1] = narrow<T>(r * fmaf(-n1, m, d1[j] * weight_at(w, bf, q.o1)));
            if (q.on && !q.one) po[q.o2] = narrow<T>(r * fmaf(-n2, m, d2[j] * weight_at(w, bf, q.o2)));
        }
    }
#pragma unroll
    for (int j = 0; j < kNrPairs; ++j) {
        const Quad q = pair_of(lane_id() + j * kWave, io.D, io.rot, io.interleaved);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (q.on) sums[(wave * 2 + which) * io.D + q.o1] = g1[which][j];
            if (q.on && !q.one) sums[(wave * 2 + which) * io.D + q.o2] = g2[which][j];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * io.D; e += kNrThreads) {
        float v = 0.0f;
        for (int k = 0; k < waves; ++k) v += sums[k * 2 * io.D + e];
        b.part[static_cast<int64_t>(blockIdx.x) * 2 * io.D + e] = v;
    }
}

// The blocks' rows added: 16 columns per block, 64 runs of rows side by side with 4 loads in flight each, then the 64
// partial sums in a fixed tree.
constexpr int kNrSumRuns = 64;
__global__ __launch_bounds__(16 * kNrSumRuns) void norm_rope_sum_kernel(const float* part, int rows, int D, float* dwq, float* dwk) {
    __shared__ float s[kNrSumRuns][17];
    const int c = threadIdx.x % 16, r0 = threadIdx.x / 16, col = blockIdx.x * 16 + c;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < 2 * D) {
        for (int r = r0; r < rows; r += 4 * kNrSumRuns) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = r + u * kNrSumRuns;
                const float x = part[static_cast<int64_t>(min(row, rows - 1)) * 2 * D + col];
                v[u] += row < rows ? x : 0.0f;
            }
        }
    }
    s[r0][c] = (v[0] + v[1]) + (v[2] + v[3]);
    for (int n = kNrSumRuns / 2; n > 0; n /= 2) {
        __syncthreads();
        if (r0 < n) s[r0][c] += s[r0 + n][c];
    }
    if (r0 == 0 && col < 2 * D) {
        float* o = col < D ? dwq : dwk;
        if (o != nullptr) o[col < D ? col : col - D] = s[0][c];
    }
}

// The call as the kernels take it: a tensor without heads has no weights either, whatever the pointer (every lane loads both
// tensors' weights before it walks the heads).
sdm_norm_rope_io nr_used(const sdm_norm_rope_io* io) {
    sdm_norm_rope_io u = *io;
    if (u.Hq == 0) u.wq = nullptr;
    if (u.Hk == 0) u.wk = nullptr;
    return u;
}

// Whether the vector path takes this call: pairs in whole runs of four on 16-byte addresses.
bool nr_vector(const sdm_norm_rope_io* io, const sdm_norm_rope_grad* g) {
    const int es = io->dtype == SDM_BF16 ? 2 : 4, unit = 16 / es;
    if (io->D % 8 != 0 || io->rot % 8 != 0) return false;
    auto ok = [&](const void* p, int64_t row, int64_t head) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % unit == 0 && head % unit == 0;
    };
    if (io->Hq > 0 && (!ok(io->q, io->q_row, io->q_head) || !ok(io->q_out, io->qo_row, io->qo_head))) return false;
    if (io->Hk > 0 && (!ok(io->k, io->k_row, io->k_head) || !ok(io->k_out, io->ko_row, io->ko_head))) return false;
    if (g != nullptr && io->Hq > 0 && !ok(g->dq, g->dq_row, g->dq_head)) return false;
    if (g != nullptr && io->Hk > 0 && !ok(g->dk, g->dk_row, g->dk_head)) return false;
    for (const void* p : {io->wq, io->wk, static_cast<const void*>(io->rot > 0 ? io->table : nullptr)}) {
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    }
    return true;
}

int team_lanes(int D) {
    int tl = 8;
    while (tl * 8 < D) tl *= 2;
    return tl;   // D <= 512: at most 64
}

// Heads per team: as many as leave kNrWaves waves, all of a token's at most.
void nr_split(NrArgs& a, int tl) {
    const int64_t waves_one = (a.io.N * a.H * tl + kWave - 1) / kWave;   // a head per team
    int per = static_cast<int>(waves_one / kNrWaves);
    per = per < 1 ? 1 : per > a.H ? a.H : per;
    a.parts = (a.H + per - 1) / per;
    a.per = (a.H + a.parts - 1) / a.parts;
}

// Blocks of the backward: 4 per compute unit keep the sum kernel's rows few.
constexpr int kNrBackBlocks = 1024;

template <typename T, bool INTER>
void nr_go(const NrArgs& a, int tl, hipStream_t st) {
    const int64_t teams = a.io.N * a.parts;
    const dim3 grid(static_cast<unsigned>((teams * tl + kNrThreads - 1) / kNrThreads));
    switch (tl) {
        case 8: norm_rope_kernel<T, INTER, 8><<<grid, kNrThreads, 0, st>>>(a); break;
        case 16: norm_rope_kernel<T, INTER, 16><<<grid, kNrThreads, 0, st>>>(a); break;
        case 32: norm_rope_kernel<T, INTER, 32><<<grid, kNrThreads, 0, st>>>(a); break;
        default: norm_rope_kernel<T, INTER, 64><<<grid, kNrThreads, 0, st>>>(a); break;
    }
}

template <typename T, bool INTER>
void nr_back_go(const NrBack& b, int tl, unsigned blocks, hipStream_t st) {
    const size_t lds = static_cast<size_t>(kNrThreads / tl) * 2 * 8 * tl * sizeof(float);
    switch (tl) {
        case 8: norm_rope_back_kernel<T, INTER, 8><<<blocks, kNrThreads, lds, st>>>(b); break;
        case 16: norm_rope_back_kernel<T, INTER, 16><<<blocks, kNrThreads, lds, st>>>(b); break;
        case 32: norm_rope_back_kernel<T, INTER, 32><<<blocks, kNrThreads, lds, st>>>(b); break;
        default: norm_rope_back_kernel<T, INTER, 64><<<blocks, kNrThreads, lds, st>>>(b); break;
    }
}

}  // namespace

hipError_t norm_rope_launch(const sdm_norm_rope_io* call, hipStream_t st) {
    const sdm_norm_rope_io used = nr_used(call), *io = &used;
    NrArgs a{*io, io->Hq + io->Hk, 1, 1};
    if (nr_vector(io, nullptr)) {
        const int tl = team_lanes(io->D);
        nr_split(a, tl);
        if (io->dtype == SDM_BF16) {
            io->interleaved ? nr_go<bf16_t, true>(a, tl, st) : nr_go<bf16_t, false>(a, tl, st);
        } else {
            io->interleaved ? nr_go<float, true>(a, tl, st) : nr_go<float, false>(a, tl, st);
        }
    } else {
        const int64_t rows = io->N * a.H;
        const dim3 grid(static_cast<unsigned>((rows * kWave + kNrThreads - 1) / kNrThreads));
        if (io->dtype == SDM_BF16) norm_rope_any_kernel<bf16_t><<<grid, kNrThreads, 0, st>>>(a);
        else norm_rope_any_kernel<float><<<grid, kNrThreads, 0, st>>>(a);
    }
    return hipGetLastError();
}

namespace {
// Blocks of a backward call: every team has work, at most kNrBackBlocks.
unsigned nr_back_blocks(int64_t items, int per_block) {
    const int64_t n = (items + per_block - 1) / per_block;
    return static_cast<unsigned>(n < kNrBackBlocks ? n : kNrBackBlocks);
}
}  // namespace

size_t norm_rope_back_workspace(int64_t N, int H, int D) {
    if (N < 1) return 0;
    const int64_t most = N * H < kNrBackBlocks ? N * H : kNrBackBlocks;
    return static_cast<size_t>(most) * 2 * D * sizeof(float);
}

hipError_t norm_rope_back_launch(const sdm_norm_rope_io* call, const sdm_norm_rope_grad* g, hipStream_t st) {
    const sdm_norm_rope_io used = nr_used(call), *io = &used;
    NrBack b;
    b.a = NrArgs{*io, io->Hq + io->Hk, 1, 1};
    b.dq = g->dq;
    b.dk = g->dk;
    b.dq_row = g->dq_row;
    b.dq_head = g->dq_head;
    b.dk_row = g->dk_row;
    b.dk_head = g->dk_head;
    b.part = static_cast<float*>(g->workspace);
    unsigned blocks = 0;
    if (io->N == 0) {
        // No token: the sum kernel below writes zeros.
    } else if (nr_vector(io, g)) {
        const int tl = team_lanes(io->D);
        nr_split(b.a, tl);
        b.items = io->N * b.a.parts;
        blocks = nr_back_blocks(b.items, kNrThreads / tl);
        if (io->dtype == SDM_BF16) {
            io->interleaved ? nr_back_go<bf16_t, true>(b, tl, blocks, st) : nr_back_go<bf16_t, false>(b, tl, blocks, st);
        } else {
            io->interleaved ? nr_back_go<float, true>(b, tl, blocks, st) : nr_back_go<float, false>(b, tl, blocks, st);
        }
    } else {
        b.items = io->N * b.a.H;
        blocks = nr_back_blocks(b.items, kNrThreads / kWave);
        const size_t lds = static_cast<size_t>(kNrThreads / kWave) * 2 * io->D * sizeof(float);
        if (io->dtype == SDM_BF16) norm_rope_back_any_kernel<bf16_t><<<blocks, kNrThreads, lds, st>>>(b);
        else norm_rope_back_any_kernel<float><<<blocks, kNrThreads, lds, st>>>(b);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (g->dwq == nullptr && g->dwk == nullptr)) return e;
    norm_rope_sum_kernel<<<(2 * io->D + 15) / 16, 16 * kNrSumRuns, 0, st>>>(b.part, static_cast<int>(blocks), io->D, g->dwq, g->dwk);
    return hipGetLastError();
}

}  // namespace sdm
