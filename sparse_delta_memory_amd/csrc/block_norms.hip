// The norms of a layer's block, each fused with what stands next to it, and their backward passes:
//   gate_norm:     y = x r(x) w silu(z) per head, r(x) = 1 / sqrt(mean(x^2) + eps), silu(z) = z / (1 + exp(-z));
//   residual_norm: h = x + a (y or y r(y) wy), n = h r(h) w per row, h as it is returned (rounded).
// Backward, with n = x r(x) the normed row and d the gradient of n w: dn = d w, dx = r (dn - n mean(dn n)), dw = sum d n;
// silu' = s (1 + z (1 - s)), s the sigmoid. The gradient of h is that of the residual and of its norm together; it is x's, and
// times a that of y (or of y's norm).
//
// The rows' bytes bound it, each read once and written once. A team of lanes owns a row: 8 to 64 lanes of a wave for rows of up to 512
// columns, a block of 256 or 512 threads for longer ones, 8 or 16 columns a lane. Teams walk rows with a stride, their columns' weights
// and weight gradients in registers. The next row's loads stand ahead of a row's work, but being conditional most of them are waited for
// there; what fills the wait is the other waves. The blocks' weight gradients are added in a fixed order by a second kernel (no
// atomics: the bits are the same every run).
//
// Of bfloat16 rows, 64 MiB a tensor, TB/s of these bytes at 64 / 512 / 1024 / 2048 / 4096 / 8192 columns: gate_norm 6.0, 5.5,
// 5.3, 5.4, 5.5, 5.5 and its backward 4.8, 4.7, 4.2, 4.4, 4.5, 4.4; residual_norm 6.0, 5.4, 5.4, 5.4, 4.8, 4.6. Its backward (4.6, 4.5,
// 3.9, 4.0, 3.5, 2.8) holds six arrays of weights and sums: past 2048 columns that is one wave per SIMD, past 4096 two with 46 to 201
// registers spilled (float32 there: 1.9), and rows of 513 to 1024 columns leave half of its waves without columns of their own.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"

namespace sdm {
namespace {

// Eight columns of a row as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<bf16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const bf16_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
    __device__ __forceinline__ void set(int e, bf16_t x) { w[e >> 1] |= static_cast<uint32_t>(x.bits) << (16 * (e & 1)); }
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ float at(int e) const { return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16); }
    static __device__ __forceinline__ void store(bf16_t* p, const float* x) {
        *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
};
template <>
struct Eight<float> {
    f32x4 w[2];
    __device__ __forceinline__ void load(const float* p) {
        w[0] = *reinterpret_cast<const f32x4*>(p);
        w[1] = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ __forceinline__ void set(int e, float x) { w[e >> 2][e & 3] = x; }
    __device__ __forceinline__ void zero() { w[0] = w[1] = f32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ float at(int e) const { return w[e >> 2][e & 3]; }
    static __device__ __forceinline__ void store(float* p, const float* x) {
        *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
};

// The columns of a team's lane l: 8 of each of its K units, consecutive (VEC: 16-byte accesses) or TW apart.
template <typename T, int TW, int K, bool VEC>
struct Cols {
    static constexpr int kRows = (TW > 256 ? TW : 256) / TW, kThreads = TW * kRows;
    int l, D;
    __device__ __forceinline__ int col(int k, int e) const { return VEC ? (k * TW + l) * 8 + e : (k * 8 + e) * TW + l; }
    // Whether the lane has columns in unit k. Waves past the row's end skip it (half of them at 1024 columns: 88 to 80 us of a gate's
    // backward pass of 32768 bfloat16 rows).
    __device__ __forceinline__ bool some(int k) const { return col(k, 0) < D; }
    __device__ __forceinline__ void load(const T* p, Eight<T> (&x)[K]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k].zero();
            if (VEC) {
                if (col(k, 0) < D) x[k].load(p + col(k, 0));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (col(k, e) < D) x[k].set(e, p[col(k, e)]);
                }
            }
        }
    }
    __device__ __forceinline__ void store(T* p, const float (&x)[K][8]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (VEC) {
                if (col(k, 0) < D) Eight<T>::store(p + col(k, 0), x[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (col(k, e) < D) p[col(k, e)] = narrow<T>(x[k][e]);
                }
            }
        }
    }
    // Weights, once per team (NULL: ones).
    __device__ __forceinline__ void weights(const void* w, int bf, float (&x)[K][8]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = w != nullptr && col(k, e) < D ? load_val(w, col(k, e), bf) : 1.0f;
        }
    }
};

// The sum over a team, in every lane of it, in a fixed order. red: a slot of [waves] of its own for each sum in flight.
template <int TW>
__device__ __forceinline__ float team_sum(float x, float* red) {
    if constexpr (TW <= kWave) {
        return group_sum<TW>(x);
    } else {
        x = group_sum<kWave>(x);
        if (lane_id() == 0) red[threadIdx.x / kWave] = x;
        __syncthreads();
        float s = red[0];
#pragma unroll
        for (int w = 1; w < TW / kWave; ++w) s += red[w];
        return s;
    }
}

// Two of them at once, given each wave's own sums (of the team's lanes, for teams of a wave or less).
template <int TW>
__device__ __forceinline__ float wave_sum(float x) { return group_sum<(TW < kWave ? TW : kWave)>(x); }
template <int TW>
__device__ __forceinline__ void team_sums(float& a, float& b, float* red_a, float* red_b) {
    if constexpr (TW > kWave) {
        if (lane_id() == 0) {
            red_a[threadIdx.x / kWave] = a;
            red_b[threadIdx.x / kWave] = b;
        }
        __syncthreads();
        a = red_a[0];
        b = red_b[0];
#pragma unroll
        for (int w = 1; w < TW / kWave; ++w) {
            a += red_a[w];
            b += red_b[w];
        }
    }
}

// 1 / (1 + exp(-z)), for z >= kFarGate. For float32 results the exponent's rounding, up to |z| / 2 units, is put back.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float z) {
    constexpr float kL2E = 1.44269504089f;
    const float t = -z * kL2E;
    float e = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(T) == 4) {
        const float lo = fmaf(-z, kL2E, -t) - z * 1.92596299e-8f;
        if (fabsf(t) < 126.0f) e = fmaf(e, lo * 0.69314718056f, e);   // past it e is as good as 0, or z is far out
    }
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// Gates so far out that exp(-z) reaches 2^126, whose reciprocal is subnormal (and comes out as 0), while z exp(z) is a normal number down
// to z = -91.9. There the sigmoid is exp(z), taken 2^64 times as large. Lanes look for such gates (by the largest of their bits) and
// go over their columns a second time if there are any: 1 to 2 % of the time of a norm whose rows have none.
constexpr float kFarGate = -87.3f;
__device__ __forceinline__ bool far_out(uint32_t bits) { return __builtin_expect(bits > __float_as_uint(kFarGate), 0); }   // or NaN
struct FarGate {
    float silu, slope;   // z exp(z), (1 + z) exp(z)
    __device__ __forceinline__ explicit FarGate(float z) {
        constexpr float kL2E = 1.44269504089f, kDown = 5.421010862427522e-20f;   // 2^-64
        const float c = fmaxf(z, -200.0f), t = c * kL2E, lo = fmaf(c, kL2E, -t) + c * 1.92596299e-8f;
        float e = __builtin_amdgcn_exp2f(t + 64.0f);
        e = fmaf(e, lo * 0.69314718056f, e);
        silu = z * e * kDown;
        slope = fmaf(z, e, e) * kDown;
    }
};

// A team's rows: every `step`-th from its own, as (token, head).
struct Walk {
    int64_t row, rows, t;
    int h, H, step, step_t, step_h;
    __device__ __forceinline__ Walk(int64_t first, int64_t rows_, int H_, int step_) : row(first), rows(rows_), H(H_), step(step_) {
        t = H > 1 ? first / H : first;
        h = H > 1 ? static_cast<int>(first - t * H) : 0;
        step_t = step / H;
        step_h = step - step_t * H;
    }
    __device__ __forceinline__ bool on() const { return row < rows; }
    __device__ __forceinline__ void next() {
        row += step;
        t += step_t;
        h += step_h;
        if (h >= H) {
            h -= H;
            ++t;
        }
    }
    __device__ __forceinline__ int64_t at(int64_t row_stride, int64_t head_stride) const { return t * row_stride + h * head_stride; }
};

template <typename T, int TW, int K, bool VEC>
__global__ __launch_bounds__(TW > 256 ? TW : 256) void gate_norm_kernel(sdm_gate_norm_io io) {
    using C = Cols<T, TW, K, VEC>;
    __shared__ float red[2][8];
    const C c{static_cast<int>(threadIdx.x) % TW, io.D};
    Walk w(static_cast<int64_t>(blockIdx.x) * C::kRows + threadIdx.x / TW, io.N * io.H, io.H, static_cast<int>(gridDim.x) * C::kRows);
    const T* x = static_cast<const T*>(io.x);
    const T* z = static_cast<const T*>(io.z);
    float wt[K][8];
    c.weights(io.w, io.w_dtype == SDM_BF16, wt);
    Eight<T> xr[K], zr[K];
    if (w.on()) {
        c.load(x + w.at(io.x_row, io.x_head), xr);
        c.load(z + w.at(io.z_row, io.z_head), zr);
    }
    const float inv = 1.0f / static_cast<float>(io.D);
    int turn = 0;
    while (w.on()) {
        Walk n = w;
        n.next();
        Eight<T> xn[K], zn[K];
        if (n.on()) {
            c.load(x + n.at(io.x_row, io.x_head), xn);
            c.load(z + n.at(io.z_row, io.z_head), zn);
        }
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(xr[k].at(e), xr[k].at(e), ss);
        }
        const float r = rsqrtf(fmaf(team_sum<TW>(ss, red[turn]), inv, io.eps));
        turn ^= 1;
        float y[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!c.some(k)) continue;
            uint32_t low = 0;   // the lowest gate's bits: negative floats order as their bits do
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = zr[k].at(e);
                low = max(low, __float_as_uint(g));
                y[k][e] = xr[k].at(e) * r * wt[k][e] * (g * sigmoid_of<T>(g));
            }
            if (far_out(low)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float g = zr[k].at(e);
                    if (g < kFarGate) y[k][e] = xr[k].at(e) * r * wt[k][e] * FarGate(g).silu;
                }
            }
        }
        c.store(static_cast<T*>(io.out) + w.at(io.o_row, io.o_head), y);
        w = n;
#pragma unroll
        for (int k = 0; k < K; ++k) { xr[k] = xn[k]; zr[k] = zn[k]; }
    }
}

// The teams' column sums of a block, added in order, to the block's row of the partial sums.
template <typename C, int TW, int K>
__device__ __forceinline__ void column_sums(const C& c, const float (&g)[K][8], float* sums, float* part) {
    if constexpr (C::kRows > 1) {
        const int team = static_cast<int>(threadIdx.x) / TW;
        __syncthreads();   // what was there before is read
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c.col(k, e) < c.D) sums[team * c.D + c.col(k, e)] = g[k][e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < c.D; i += C::kThreads) {
            float s = 0.0f;
            for (int t = 0; t < C::kRows; ++t) s += sums[t * c.D + i];
            part[i] = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c.col(k, e) < c.D) part[c.col(k, e)] = g[k][e];
            }
        }
    }
}

struct GateBack {
    sdm_gate_norm_io io;
    const void* d;
    int64_t d_row, d_head;
    void *dx, *dz;
    float* part;   // [blocks, D]
};

template <typename T, int TW, int K, bool VEC>
__global__ __launch_bounds__(TW > 256 ? TW : 256) void gate_norm_back_kernel(GateBack p) {
    using C = Cols<T, TW, K, VEC>;
    const sdm_gate_norm_io& io = p.io;
    __shared__ float red[4][8];
    extern __shared__ float sums[];
    const C c{static_cast<int>(threadIdx.x) % TW, io.D};
    Walk w(static_cast<int64_t>(blockIdx.x) * C::kRows + threadIdx.x / TW, io.N * io.H, io.H, static_cast<int>(gridDim.x) * C::kRows);
    const T* x = static_cast<const T*>(io.x);
    const T* z = static_cast<const T*>(io.z);
    const T* d = static_cast<const T*>(p.d);
    float wt[K][8], gw[K][8];
    c.weights(io.w, io.w_dtype == SDM_BF16, wt);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[k][e] = 0.0f;
    }
    Eight<T> xr[K], zr[K], dr[K];
    if (w.on()) {
        c.load(x + w.at(io.x_row, io.x_head), xr);
        c.load(z + w.at(io.z_row, io.z_head), zr);
        c.load(d + w.at(p.d_row, p.d_head), dr);
    }
    const float inv = 1.0f / static_cast<float>(io.D);
    int turn = 0;
    while (w.on()) {
        Walk n = w;
        n.next();
        Eight<T> xn[K], zn[K], dn_[K];
        if (n.on()) {
            c.load(x + n.at(io.x_row, io.x_head), xn);
            c.load(z + n.at(io.z_row, io.z_head), zn);
            c.load(d + n.at(p.d_row, p.d_head), dn_);
        }
        float ss = 0.0f, dot = 0.0f, dy[K][8], oz[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(xr[k].at(e), xr[k].at(e), ss);
        }
        ss = wave_sum<TW>(ss);   // its steps wait for each other: under the gates' work, not behind the branch
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[k][e] = oz[k][e] = 0.0f;
            if (!c.some(k)) continue;
            uint32_t low = 0;
            const float before = dot;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xe = xr[k].at(e), g = zr[k].at(e), de = dr[k].at(e), s = sigmoid_of<T>(g);
                low = max(low, __float_as_uint(g));
                dy[k][e] = de * (g * s);
                oz[k][e] = de * wt[k][e] * xe * (s * fmaf(g, 1.0f - s, 1.0f));
                dot = fmaf(dy[k][e] * wt[k][e], xe, dot);
            }
            if (far_out(low)) {
                dot = before;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xe = xr[k].at(e), g = zr[k].at(e), de = dr[k].at(e);
                    if (g < kFarGate) {
                        const FarGate far(g);
                        dy[k][e] = de * far.silu;
                        oz[k][e] = de * wt[k][e] * xe * far.slope;
                    }
                    dot = fmaf(dy[k][e] * wt[k][e], xe, dot);
                }
            }
        }
        dot = wave_sum<TW>(dot);
        team_sums<TW>(ss, dot, red[2 * turn], red[2 * turn + 1]);
        turn ^= 1;
        const float r = rsqrtf(fmaf(ss, inv, io.eps)), m = dot * r * inv;
        float ox[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ne = xr[k].at(e) * r;
                gw[k][e] = fmaf(dy[k][e], ne, gw[k][e]);
                ox[k][e] = r * fmaf(-ne, m, dy[k][e] * wt[k][e]);
                oz[k][e] *= r;
            }
        }
        const int64_t at = w.row * io.D;
        c.store(static_cast<T*>(p.dx) + at, ox);
        c.store(static_cast<T*>(p.dz) + at, oz);
        w = n;
#pragma unroll
        for (int k = 0; k < K; ++k) { xr[k] = xn[k]; zr[k] = zn[k]; dr[k] = dn_[k]; }
    }
    column_sums<C, TW, K>(c, gw, sums, p.part + static_cast<int64_t>(blockIdx.x) * io.D);
}

template <typename T, int TW, int K, bool VEC>
__global__ __launch_bounds__(TW > 256 ? TW : 256) void residual_norm_kernel(sdm_residual_norm_io io) {
    using C = Cols<T, TW, K, VEC>;
    __shared__ float red[4][8];
    const C c{static_cast<int>(threadIdx.x) % TW, io.D};
    const int64_t step = static_cast<int64_t>(gridDim.x) * C::kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * C::kRows + threadIdx.x / TW;
    const T* x = static_cast<const T*>(io.x);
    const T* y = static_cast<const T*>(io.y);
    const int bf = io.w_dtype == SDM_BF16;
    float wt[K][8], wy[K][8], wa[K][8];
    c.weights(io.w, bf, wt);
    c.weights(io.wy, bf, wy);
    c.weights(io.a, bf, wa);
    Eight<T> xr[K], yr[K];
    if (row < io.N) {
        c.load(x + row * io.x_row, xr);
        c.load(y + row * io.y_row, yr);
    }
    const float inv = 1.0f / static_cast<float>(io.D);
    int turn = 0;
    for (; row < io.N; row += step) {
        Eight<T> xn[K], yn[K];
        if (row + step < io.N) {
            c.load(x + (row + step) * io.x_row, xn);
            c.load(y + (row + step) * io.y_row, yn);
        }
        float h[K][8], ss = 0.0f;
        if (io.norm_y) {
            float sy = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sy = fmaf(yr[k].at(e), yr[k].at(e), sy);
            }
            const float r = rsqrtf(fmaf(team_sum<TW>(sy, red[2 * turn]), inv, io.eps));
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[k][e] = fmaf(wa[k][e], yr[k].at(e) * r * wy[k][e], xr[k].at(e));
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[k][e] = fmaf(wa[k][e], yr[k].at(e), xr[k].at(e));
            }
        }
        c.store(static_cast<T*>(io.h) + row * io.h_row, h);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[k][e] = widen(narrow<T>(h[k][e]));
                ss = fmaf(h[k][e], h[k][e], ss);
            }
        }
        const float r = rsqrtf(fmaf(team_sum<TW>(ss, red[2 * turn + 1]), inv, io.eps));
        turn ^= 1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[k][e] = h[k][e] * r * wt[k][e];
        }
        c.store(static_cast<T*>(io.n) + row * io.n_row, h);
#pragma unroll
        for (int k = 0; k < K; ++k) { xr[k] = xn[k]; yr[k] = yn[k]; }
    }
}

struct ResidualBack {
    sdm_residual_norm_io io;
    sdm_residual_norm_grad g;
    float* part;   // [blocks, 3, D]: dw, dwy, da
};

template <typename T, int TW, int K, bool VEC>
__global__ __launch_bounds__(TW > 256 ? TW : 256) void residual_norm_back_kernel(ResidualBack p) {
    using C = Cols<T, TW, K, VEC>;
    const sdm_residual_norm_io& io = p.io;
    __shared__ float red[8][8];
    extern __shared__ float sums[];
    const C c{static_cast<int>(threadIdx.x) % TW, io.D};
    const int64_t step = static_cast<int64_t>(gridDim.x) * C::kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * C::kRows + threadIdx.x / TW;
    const T* hp = static_cast<const T*>(io.h);
    const T* yp = static_cast<const T*>(io.y);
    const T* dhp = static_cast<const T*>(p.g.dh);
    const T* dnp = static_cast<const T*>(p.g.dn);
    const int bf = io.w_dtype == SDM_BF16;
    // y is only read where its norm or its scale's gradient needs it.
    const bool need_y = io.norm_y || p.g.da != nullptr;
    float wt[K][8], wy[K][8], wa[K][8], gw[K][8], gy[K][8], ga[K][8];
    c.weights(io.w, bf, wt);
    c.weights(io.wy, bf, wy);
    c.weights(io.a, bf, wa);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[k][e] = gy[k][e] = ga[k][e] = 0.0f;
    }
    Eight<T> hr[K], yr[K], er[K], nr[K];
    auto fetch = [&](int64_t at, Eight<T> (&h)[K], Eight<T> (&y)[K], Eight<T> (&e)[K], Eight<T> (&n)[K]) {
        c.load(hp + at * io.h_row, h);
        c.load(dnp + at * p.g.dn_row, n);
        if (dhp != nullptr) {
            c.load(dhp + at * p.g.dh_row, e);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) e[k].zero();
        }
        if (need_y) {
            c.load(yp + at * io.y_row, y);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) y[k].zero();
        }
    };
    if (row < io.N) fetch(row, hr, yr, er, nr);
    const float inv = 1.0f / static_cast<float>(io.D);
    int turn = 0;
    for (; row < io.N; row += step) {
        Eight<T> hn[K], yn[K], en[K], nn[K];
        if (row + step < io.N) fetch(row + step, hn, yn, en, nn);
        float* const slot = red[4 * turn];
        turn ^= 1;
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float he = hr[k].at(e);
                ss = fmaf(he, he, ss);
                dot = fmaf(nr[k].at(e) * wt[k][e], he, dot);
            }
        }
        const float r = rsqrtf(fmaf(team_sum<TW>(ss, slot), inv, io.eps));
        const float m = team_sum<TW>(dot, slot + 8) * r * inv;
        float o[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ne = hr[k].at(e) * r, de = nr[k].at(e);
                gw[k][e] = fmaf(de, ne, gw[k][e]);
                o[k][e] = fmaf(r, fmaf(-ne, m, de * wt[k][e]), er[k].at(e));
            }
        }
        const int64_t at = row * io.D;
        if (p.g.dx != nullptr) c.store(static_cast<T*>(p.g.dx) + at, o);
        if (io.norm_y) {
            float sy = 0.0f, dy = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float ye = yr[k].at(e);
                    sy = fmaf(ye, ye, sy);
                    dy = fmaf(o[k][e] * wa[k][e] * wy[k][e], ye, dy);
                }
            }
            const float ry = rsqrtf(fmaf(team_sum<TW>(sy, slot + 16), inv, io.eps));
            const float my = team_sum<TW>(dy, slot + 24) * ry * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float ne = yr[k].at(e) * ry, de = o[k][e] * wa[k][e];
                    ga[k][e] = fmaf(o[k][e], ne * wy[k][e], ga[k][e]);
                    gy[k][e] = fmaf(de, ne, gy[k][e]);
                    o[k][e] = ry * fmaf(-ne, my, de * wy[k][e]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ga[k][e] = fmaf(o[k][e], yr[k].at(e), ga[k][e]);
                    o[k][e] *= wa[k][e];
                }
            }
        }
        c.store(static_cast<T*>(p.g.dy) + at, o);
#pragma unroll
        for (int k = 0; k < K; ++k) { hr[k] = hn[k]; yr[k] = yn[k]; er[k] = en[k]; nr[k] = nn[k]; }
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 3 * io.D;
    if (p.g.dw != nullptr) column_sums<C, TW, K>(c, gw, sums, part);
    if (p.g.dwy != nullptr) column_sums<C, TW, K>(c, gy, sums, part + io.D);
    if (p.g.da != nullptr) column_sums<C, TW, K>(c, ga, sums, part + 2 * io.D);
}

// The blocks' rows added: 16 columns per block, 64 runs of rows side by side with 4 loads in flight each, then the 64
// partial sums in a fixed tree. out: the sums of each D columns (NULL: skipped).
constexpr int kRuns = 64;
struct SumArgs {
    const float* part;   // [rows, M, D]
    int rows, M, D;
    float* out[3];
};
__global__ __launch_bounds__(16 * kRuns) void block_norm_sum_kernel(SumArgs p) {
    __shared__ float s[kRuns][17];
    const int c = threadIdx.x % 16, r0 = threadIdx.x / 16, per = (p.D + 15) / 16, which = blockIdx.x / per, col = (blockIdx.x - which * per) * 16 + c;
    float* o = which == 0 ? p.out[0] : which == 1 ? p.out[1] : p.out[2];
    if (o == nullptr) return;   // the whole block
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < p.D) {
        const float* from = p.part + static_cast<int64_t>(which) * p.D + col;
        for (int r = r0; r < p.rows; r += 4 * kRuns) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = r + u * kRuns;
                const float x = from[static_cast<int64_t>(min(row, p.rows - 1)) * p.M * p.D];
                v[u] += row < p.rows ? x : 0.0f;
            }
        }
    }
    s[r0][c] = (v[0] + v[1]) + (v[2] + v[3]);
    for (int n = kRuns / 2; n > 0; n /= 2) {
        __syncthreads();
        if (r0 < n) s[r0][c] += s[r0 + n][c];
    }
    if (r0 == 0 && col < p.D) o[col] = s[0][c];
}

// --------------------------------------------------------------------------------------------- plans

// Teams by width: TW lanes, K units of 8 columns each.
template <typename F>
void by_width(int D, bool vec, F f) {
    // Rows that take no wide accesses go with the widest team of their class (lanes' columns are TW apart).
    if (D > 4096) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    else if (D > 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (D > 512) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    else if (D > 256 || !vec) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (D > 128) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    else if (D > 64) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
}

// Blocks: as many as the kernel's own registers let be resident at once, or as many as have rows; each walks its share. (A few more would
// run behind the others, alone: eight per compute unit for all, 2048 rows of 8192 float32 columns, took a residual 113 us, what fits
// takes 54.)
constexpr int64_t kUnits = 256;
unsigned grid_of(int64_t rows, int per_block, int64_t most) {
    const int64_t n = (rows + per_block - 1) / per_block;
    return static_cast<unsigned>(n < most ? n : most);
}

// Of a backward pass each block leaves a row of partial sums, at most 24 MiB of them: the workspace has a row for every block that
// the registers of such a pass may let be resident, for rows of one unit of columns a lane four per compute unit (a gate's, M 1) or
// three (a residual's, M 3), for longer ones two blocks of 256 threads (a gate's) or one. 5461 bfloat16 rows of 6144 columns, a
// gate's 108 us in 853 blocks, 87 in 256; a residual's 203 in 284 and 147 in 256.
int back_blocks(int64_t rows, int D, int M) {
    const int64_t most = kUnits * (D <= 2048 ? (M == 1 ? 4 : 3) : D <= 4096 && M == 1 ? 2 : 1);
    return static_cast<int>(rows < most ? rows : most);
}
template <auto Kernel>
int64_t resident(int threads) {
    static const int per_unit = [threads] {
        int n = 0;   // with the most LDS that its sums take: a block's teams hold 2048 columns
        const hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(Kernel), threads, 2048 * sizeof(float));
        return e == hipSuccess && n > 0 ? n : 1;
    }();
    return kUnits * per_unit;
}
template <auto Kernel, typename A>
void forward_go(const A& io, int64_t rows, int TW, int threads, hipStream_t st) {
    Kernel<<<grid_of(rows, threads / TW, resident<Kernel>(threads)), threads, 0, st>>>(io);
}
template <auto Kernel, typename A>
unsigned back_go(const A& args, int64_t rows, int most, int TW, int threads, hipStream_t st) {
    const int D = args.io.D, teams = threads / TW;
    const int64_t fit = resident<Kernel>(threads);
    const unsigned grid = grid_of(rows, teams, fit < most ? fit : most);
    Kernel<<<grid, threads, teams > 1 ? static_cast<size_t>(teams) * D * 4 : 0, st>>>(args);
    return grid;
}

bool wide(const void* p, int64_t a, int64_t b, int unit) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % unit == 0 && b % unit == 0; }

hipError_t sum_go(const float* part, int rows, int M, int D, float* a, float* b, float* c, hipStream_t st) {
    if (a == nullptr && b == nullptr && c == nullptr) return hipSuccess;
    const SumArgs s{part, rows, M, D, {a, b, c}};
    block_norm_sum_kernel<<<M * ((D + 15) / 16), 16 * kRuns, 0, st>>>(s);
    return hipGetLastError();
}

}  // namespace

hipError_t gate_norm_launch(const sdm_gate_norm_io* io, hipStream_t st) {
    const int unit = io->dtype == SDM_BF16 ? 8 : 4;
    const bool vec = io->D % 8 == 0 && wide(io->x, io->x_row, io->x_head, unit) && wide(io->z, io->z_row, io->z_head, unit) &&
                     wide(io->out, io->o_row, io->o_head, unit);
    by_width(io->D, vec, [&](auto tw, auto k) {
        constexpr int TW = tw, K = k, threads = TW > 256 ? TW : 256;
        const int64_t rows = io->N * io->H;
        if (io->dtype == SDM_BF16) {
            if (vec) forward_go<gate_norm_kernel<bf16_t, TW, K, true>>(*io, rows, TW, threads, st);
            else if constexpr (TW >= 64) forward_go<gate_norm_kernel<bf16_t, TW, K, false>>(*io, rows, TW, threads, st);
        } else {
            if (vec) forward_go<gate_norm_kernel<float, TW, K, true>>(*io, rows, TW, threads, st);
            else if constexpr (TW >= 64) forward_go<gate_norm_kernel<float, TW, K, false>>(*io, rows, TW, threads, st);
        }
    });
    return hipGetLastError();
}

size_t gate_norm_back_workspace(int64_t rows, int D) { return static_cast<size_t>(back_blocks(rows, D, 1)) * D * 4; }

hipError_t gate_norm_back_launch(const sdm_gate_norm_io* io, const sdm_gate_norm_grad* g, hipStream_t st) {
    const int unit = io->dtype == SDM_BF16 ? 8 : 4;
    const bool vec = io->D % 8 == 0 && wide(io->x, io->x_row, io->x_head, unit) && wide(io->z, io->z_row, io->z_head, unit) &&
                     wide(g->d, g->d_row, g->d_head, unit) && wide(g->dx, 0, 0, unit) && wide(g->dz, 0, 0, unit);
    const GateBack b{*io, g->d, g->d_row, g->d_head, g->dx, g->dz, static_cast<float*>(g->workspace)};
    unsigned grid = 0;
    if (io->N > 0) {
        by_width(io->D, vec, [&](auto tw, auto k) {
            constexpr int TW = tw, K = k, threads = TW > 256 ? TW : 256;
            const int64_t rows = io->N * io->H;
            const int most = back_blocks(rows, io->D, 1);
            if (io->dtype == SDM_BF16) {
                if (vec) grid = back_go<gate_norm_back_kernel<bf16_t, TW, K, true>>(b, rows, most, TW, threads, st);
                else if constexpr (TW >= 64) grid = back_go<gate_norm_back_kernel<bf16_t, TW, K, false>>(b, rows, most, TW, threads, st);
            } else {
                if (vec) grid = back_go<gate_norm_back_kernel<float, TW, K, true>>(b, rows, most, TW, threads, st);
                else if constexpr (TW >= 64) grid = back_go<gate_norm_back_kernel<float, TW, K, false>>(b, rows, most, TW, threads, st);
            }
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return sum_go(b.part, static_cast<int>(grid), 1, io->D, g->dw, nullptr, nullptr, st);
}

hipError_t residual_norm_launch(const sdm_residual_norm_io* io, hipStream_t st) {
    const int unit = io->dtype == SDM_BF16 ? 8 : 4;
    const bool vec = io->D % 8 == 0 && wide(io->x, io->x_row, 0, unit) && wide(io->y, io->y_row, 0, unit) && wide(io->h, io->h_row, 0, unit) &&
                     wide(io->n, io->n_row, 0, unit);
    by_width(io->D, vec, [&](auto tw, auto k) {
        constexpr int TW = tw, K = k, threads = TW > 256 ? TW : 256;
        const int64_t rows = io->N;
        if (io->dtype == SDM_BF16) {
            if (vec) forward_go<residual_norm_kernel<bf16_t, TW, K, true>>(*io, rows, TW, threads, st);
            else if constexpr (TW >= 64) forward_go<residual_norm_kernel<bf16_t, TW, K, false>>(*io, rows, TW, threads, st);
        } else {
            if (vec) forward_go<residual_norm_kernel<float, TW, K, true>>(*io, rows, TW, threads, st);
            else if constexpr (TW >= 64) forward_go<residual_norm_kernel<float, TW, K, false>>(*io, rows, TW, threads, st);
        }
    });
    return hipGetLastError();
}

size_t residual_norm_back_workspace(int64_t rows, int D) { return static_cast<size_t>(back_blocks(rows, D, 3)) * 3 * D * 4; }

hipError_t residual_norm_back_launch(const sdm_residual_norm_io* io, const sdm_residual_norm_grad* g, hipStream_t st) {
    const int unit = io->dtype == SDM_BF16 ? 8 : 4;
    const bool need_y = io->norm_y || g->da != nullptr;
    const bool vec = io->D % 8 == 0 && wide(io->h, io->h_row, 0, unit) && wide(g->dn, g->dn_row, 0, unit) && wide(g->dh, g->dh_row, 0, unit) &&
                     (!need_y || wide(io->y, io->y_row, 0, unit)) && wide(g->dx, 0, 0, unit) && wide(g->dy, 0, 0, unit);
    const ResidualBack b{*io, *g, static_cast<float*>(g->workspace)};
    unsigned grid = 0;
    if (io->N > 0) {
        by_width(io->D, vec, [&](auto tw, auto k) {
            constexpr int TW = tw, K = k, threads = TW > 256 ? TW : 256;
            const int most = back_blocks(io->N, io->D, 3);
            if (io->dtype == SDM_BF16) {
                if (vec) grid = back_go<residual_norm_back_kernel<bf16_t, TW, K, true>>(b, io->N, most, TW, threads, st);
                else if constexpr (TW >= 64) grid = back_go<residual_norm_back_kernel<bf16_t, TW, K, false>>(b, io->N, most, TW, threads, st);
            } else {
                if (vec) grid = back_go<residual_norm_back_kernel<float, TW, K, true>>(b, io->N, most, TW, threads, st);
                else if constexpr (TW >= 64) grid = back_go<residual_norm_back_kernel<float, TW, K, false>>(b, io->N, most, TW, threads, st);
            }
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return sum_go(b.part, static_cast<int>(grid), 3, io->D, g->dw, g->dwy, g->da, st);
}

}  // namespace sdm
