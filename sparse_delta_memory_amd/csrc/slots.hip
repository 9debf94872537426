// Slot selection: the slot ids and weights of a bank of n1 x n2 slots from two rows of scores per token,
// and the backward pass.
//
// A slot's score is a[i] + b[j], its id i n2 + j. The K best slots lie among the pairs of the K best a
// and the K best b, so the K best of each row are taken, and of the pairs (i-th best a, j-th best b)
// only those with (i + 1)(j + 1) <= K can be among the K best: all (i' <= i, j' <= j) are at least as
// good. Order, everywhere: the larger value first, of equal ones the lower place (column; for pairs the
// better a, then the better b). A NaN score counts as -infinity. The weights are the softmax of the K
// sums times `scale`; a sum of -infinity weighs 0, and so does every one when all are.
//
// One wave per token. The row sits in registers as integers of the same order (bfloat16 ones two to a
// word). The K-th best of the 64 lanes' own largest is a bound that at least K entries meet and few others
// do, so one sweep of ballots moves the few entries at or above it to LDS, and sorting networks over the 64
// lanes (compare-exchange across lanes, no LDS for most steps) order them; a bfloat16 entry and its place
// are one 32-bit word there. Reading the scores would take 105 us at 65536 tokens of 2 x 2048 bfloat16
// scores, K = 32; it takes 152, the issue of about 1400 vector instructions per token. (With 32-bit keys, 64-bit
// networks and the ordering inside the unrolled sweep, so that it did not fit the instruction cache: 283.) Rows
// of equal scores are ordered 64 entries at a time, the whole row swept again for each: both rows constant
// 2500 us, one row all -infinity 1360 (scores cut off at 0, half of them equal but not among the best, 141).
#include <hip/hip_runtime.h>

#include <climits>
#include <type_traits>

#include "mixer_device.hpp"
#include "sdm_launch.hpp"

namespace sdm {
namespace {

constexpr int kStThreads = 256;
constexpr int kStWaves = kStThreads / kWave;

// Entries up to which inserting them one by one is less than ordering and merging 64.
constexpr int kStInsert = 20;

struct StArgs {
    sdm_slot_topk_io io;
    int ka, kb;      // kept entries of each row: min(K, n)
    int pairs;       // pairs (i, j) with (i + 1)(j + 1) <= K
    int vec;         // rows take 16-byte loads
};

// Pairs (i, j) in the order of (i + 1)(j + 1), i in the high byte: the first pair_count(K) of them are
// those that can win for K.
constexpr int kStMaxPairs = 280;
struct PairTable {
    uint16_t at[kStMaxPairs];
    uint16_t count[65];
};
constexpr PairTable make_pairs() {
    PairTable t{};
    int n = 0;
    for (int p = 1; p <= 64; ++p) {
        for (int i = 1; i <= p; ++i) {
            if (p % i == 0) t.at[n++] = static_cast<uint16_t>(((i - 1) << 8) | (p / i - 1));
        }
        t.count[p] = static_cast<uint16_t>(n);
    }
    return t;
}
constexpr PairTable kPairsHost = make_pairs();
static_assert(kPairsHost.count[64] == kStMaxPairs, "pairs (i, j) with (i + 1)(j + 1) <= 64");
__constant__ PairTable kPairs = make_pairs();

// Float order as integer order: the magnitude's bits, negated under a minus sign, so that both zeros are
// 0. Of 16 bits for a bfloat16, of 32 for a float; beyond the infinities' lie the NaNs'.
template <typename T>
struct Order;
template <>
struct Order<bf16_t> {
    static constexpr int kInf = 0x7F80, kPad = -0x8000;   // kPad: below every value, places past a row's end
    static __device__ __forceinline__ int of(bf16_t x) {
        const int b = x.bits;
        return b & 0x8000 ? -(b & 0x7FFF) : b;
    }
    static __device__ __forceinline__ float value(int v) {
        return __uint_as_float(v < 0 ? (static_cast<uint32_t>(-v) | 0x8000u) << 16 : static_cast<uint32_t>(v) << 16);
    }
};
template <>
struct Order<float> {
    static constexpr int kInf = 0x7F800000, kPad = INT32_MIN;
    static __device__ __forceinline__ int of(float x) {
        const int b = __float_as_int(x);
        return b < 0 ? -(b & 0x7FFFFFFF) : b;
    }
    static __device__ __forceinline__ float value(int v) { return v < 0 ? -__int_as_float(-v) : __int_as_float(v); }
};
// The same of a float32 sum as unsigned key, a NaN as -infinity; 0 is below every key.
__device__ __forceinline__ uint32_t key_of(float f) {
    return static_cast<uint32_t>(Order<float>::of(f != f ? -INFINITY : f)) ^ 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) { return Order<float>::value(static_cast<int>(k ^ 0x80000000u)); }

// An entry: its key, and the complement of its place, so that the larger pair is the better entry.
struct Entry {
    uint32_t key, inv;
};
__device__ __forceinline__ bool above(const Entry& a, const Entry& b) {
    return ((static_cast<uint64_t>(a.key) << 32) | a.inv) > ((static_cast<uint64_t>(b.key) << 32) | b.inv);
}
__device__ __forceinline__ Entry pick(bool c, const Entry& a, const Entry& b) {
    return Entry{c ? a.key : b.key, c ? a.inv : b.inv};
}

// Compare-exchange with lane ^ M: the lanes of `up` keep the better entry.
template <int M>
__device__ __forceinline__ void exchange(Entry& e, bool up) {
    const Entry o{lane_xor<M>(e.key), lane_xor<M>(e.inv)};
    e = pick(above(e, o) == up, e, o);
}
template <int M>
__device__ __forceinline__ void exchange_key(uint32_t& k, bool up) {
    const uint32_t o = lane_xor<M>(k);
    k = up ? max(k, o) : min(k, o);
}

// One stage of the sorting network per merge length: best first when `up` holds for the whole length.
template <int M, typename E, typename F>
__device__ __forceinline__ void merge_steps(E& e, bool down, F step) {
    step(std::integral_constant<int, M>{}, e, down);
    if constexpr (M > 1) merge_steps<M / 2>(e, down, step);
}
template <int M, typename E, typename F>
__device__ __forceinline__ void sort_steps(E& e, F step) {
    if constexpr (M > 1) sort_steps<M / 2>(e, step);
    merge_steps<M>(e, M < 32 && (lane_id() & (2 * M)) != 0, step);
}
struct EntryStep {
    template <int M>
    __device__ __forceinline__ void operator()(std::integral_constant<int, M>, Entry& e, bool down) const {
        exchange<M>(e, ((lane_id() & M) == 0) != down);
    }
};
struct KeyStep {
    template <int M>
    __device__ __forceinline__ void operator()(std::integral_constant<int, M>, uint32_t& k, bool down) const {
        exchange_key<M>(k, ((lane_id() & M) == 0) != down);
    }
};
// The wave's 64 entries (or keys), best in lane 0.
__device__ __forceinline__ void sort64(Entry& e) { sort_steps<32>(e, EntryStep{}); }
__device__ __forceinline__ void sort64(uint32_t& k) { sort_steps<32>(k, KeyStep{}); }

// The best 64 of two sorted lists of 64, sorted: the better of lane l's entry and the other list's
// entry from the end is one of the 64 best, and those form one rising and falling run.
__device__ __forceinline__ void merge64(Entry& best, const Entry& other) {
    const int from = (63 - static_cast<int>(lane_id())) << 2;
    const Entry o{static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(other.key))),
                  static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(other.inv)))};
    best = pick(above(best, o), best, o);
    merge_steps<32>(best, false, EntryStep{});
}
__device__ __forceinline__ void merge64(uint32_t& best, uint32_t other) {
    best = max(best, static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute((63 - static_cast<int>(lane_id())) << 2, static_cast<int>(other))));
    merge_steps<32>(best, false, KeyStep{});
}

// Lane `from`'s entry of e into the sorted list: the entries below it move down by a lane, the last one out.
__device__ __forceinline__ void insert(Entry& best, const Entry& e, int from) {
    const Entry x{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(e.key), from)),
                  static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(e.inv), from))};
    const int pos = __popcll(__ballot(above(best, x)));   // lanes with a better one, the first ones
    if (pos >= kWave) return;
    const int lane = static_cast<int>(lane_id());
    const Entry up{static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(best.key), 0x138, 0xF, 0xF, false)),   // wave_shr:1
                   static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(best.inv), 0x138, 0xF, 0xF, false))};
    best = pick(lane > pos, up, best);
    best = pick(lane == pos, x, best);
}

__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(lane << 2, static_cast<int>(x)));
}

// The order values of a row's places: NV per lane, in runs of E (16 bytes' worth on the vector path, 1 on the
// element path). Places past the row's end hold kPad. bfloat16 vectors stay packed, two values to a word.
template <int E>
__device__ __forceinline__ uint32_t place(int v, uint32_t lane) {
    return static_cast<uint32_t>((v / E) * (kWave * E) + (v % E)) | (lane * E);
}
template <int E>
__device__ __forceinline__ uint32_t place(int v) { return place<E>(v, lane_id()); }
template <typename T, int E, int NV>
struct Values {
    int v[NV];
    __device__ __forceinline__ void load(const T* row, int n) {
        if constexpr (E == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t at = place<1>(i);
                v[i] = at < static_cast<uint32_t>(n) ? Order<T>::of(row[at]) : Order<T>::kPad;
            }
        } else {
            static_assert(sizeof(T) == 4 && E == 4 && NV % 4 == 0, "float vectors");
            u32x4 w[NV / 4];
#pragma unroll
            for (int c = 0; c < NV / 4; ++c) {
                const uint32_t at = place<4>(c * 4);
                w[c] = u32x4{0, 0, 0, 0};
                if (at < static_cast<uint32_t>(n)) w[c] = *reinterpret_cast<const u32x4*>(row + at);   // n is a multiple of 4
            }
#pragma unroll
            for (int c = 0; c < NV / 4; ++c) {
                const bool in = place<4>(c * 4) < static_cast<uint32_t>(n);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[c * 4 + e] = in ? Order<T>::of(__uint_as_float(w[c][e])) : Order<T>::kPad;
            }
        }
    }
    // The largest of the first and of the second half of the lane's values.
    __device__ __forceinline__ void largest(int& first, int& second) const {
        constexpr int kHalf = NV / 2;
        first = v[0];
        second = v[kHalf];
#pragma unroll
        for (int i = 1; i < kHalf; ++i) {
            first = max(first, v[i]);
            second = max(second, v[kHalf + i]);
        }
    }
    __device__ __forceinline__ int get(int i) const { return v[i]; }
    __device__ __forceinline__ void touch() {}
    // NaNs as -infinity.
    __device__ __forceinline__ void clean() {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (v[i] > Order<T>::kInf || (v[i] < -Order<T>::kInf && v[i] != Order<T>::kPad)) v[i] = -Order<T>::kInf;
        }
    }
};
template <int NV>
struct Values<bf16_t, 8, NV> {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 w[NV / 2];
    __device__ __forceinline__ void load(const bf16_t* row, int n) {
        u32x4 x[NV / 8];
#pragma unroll
        for (int c = 0; c < NV / 8; ++c) {
            const uint32_t at = place<8>(c * 8);
            x[c] = u32x4{0, 0, 0, 0};
            if (at < static_cast<uint32_t>(n)) x[c] = *reinterpret_cast<const u32x4*>(row + at);   // n is a multiple of 8
        }
#pragma unroll
        for (int c = 0; c < NV / 8; ++c) {
            const bool in = place<8>(c * 8) < static_cast<uint32_t>(n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t two = x[c][e];
                const s16x2 b = __builtin_bit_cast(s16x2, two), s = b >> 15;   // -1 under a minus sign
                const s16x2 y = ((b & static_cast<short>(0x7FFF)) ^ s) - s;
                w[c * 4 + e] = in ? y : s16x2{-0x8000, -0x8000};
            }
        }
    }
    __device__ __forceinline__ void largest(int& first, int& second) const {
        s16x2 a = w[0], b = w[NV / 4];
#pragma unroll
        for (int i = 1; i < NV / 4; ++i) {
            a = __builtin_elementwise_max(a, w[i]);
            b = __builtin_elementwise_max(b, w[NV / 4 + i]);
        }
        first = max(static_cast<int>(a[0]), static_cast<int>(a[1]));
        second = max(static_cast<int>(b[0]), static_cast<int>(b[1]));
    }
    __device__ __forceinline__ int get(int i) const { return w[i / 2][i % 2]; }
    // The words as if new: what is unpacked from them is not kept over a loop.
    __device__ __forceinline__ void touch() {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) __asm__ volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ void clean() {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = w[i][e];
                if (v > Order<bf16_t>::kInf || (v < -Order<bf16_t>::kInf && v != Order<bf16_t>::kPad))
                    w[i][e] = static_cast<short>(-Order<bf16_t>::kInf);
            }
        }
    }
};

// What the lists and networks hold of a row's entry: for bfloat16 one word (order value, place), compared as one
// unsigned number after Item<bf16_t>::sortable; for float32 two.
template <typename T>
struct Item;
template <>
struct Item<bf16_t> {
    typedef uint32_t type;
    typedef uint32_t sorted;
    static __device__ __forceinline__ type make(int v, uint32_t at) { return (static_cast<uint32_t>(v) << 16) | at; }
    static __device__ __forceinline__ sorted sortable(type w) { return w ^ 0x8000FFFFu; }
    static __device__ __forceinline__ sorted none() { return 0u; }
    static __device__ __forceinline__ float value(sorted s) { return Order<bf16_t>::value(static_cast<int16_t>((s ^ 0x80000000u) >> 16)); }
    static __device__ __forceinline__ uint32_t at(sorted s) { return ~s & 0xFFFFu; }
};
template <>
struct Item<float> {
    typedef u32x2 type;
    typedef Entry sorted;
    static __device__ __forceinline__ type make(int v, uint32_t at) { return u32x2{static_cast<uint32_t>(v), at}; }
    static __device__ __forceinline__ sorted sortable(type w) { return Entry{w[0] ^ 0x80000000u, ~w[1]}; }
    static __device__ __forceinline__ sorted none() { return Entry{0u, 0u}; }
    static __device__ __forceinline__ float value(const sorted& s) { return float_of(s.key); }
    static __device__ __forceinline__ uint32_t at(const sorted& s) { return ~s.inv; }
};

// The best `kept` entries of a row, best in lane 0. list: 64 items of LDS of this wave's own.
template <typename T, int E, int NV>
__device__ __forceinline__ typename Item<T>::sorted best_of_row(const void* base, int64_t from, int n, int kept, typename Item<T>::type* list) {
    using I = Item<T>;
    Values<T, E, NV> x;
    x.load(static_cast<const T*>(base) + from, n);
    if constexpr (NV == 1) {
        x.clean();
        typename I::sorted e = I::sortable(I::make(x.get(0), place<E>(0)));
        if (lane_id() >= static_cast<uint32_t>(n)) e = I::none();
        sort64(e);
        return e;
    } else {
        // At least `kept` entries are at or above the kept-th best of the lanes' largest, and not many more: of random
        // rows' 64 largest the 32nd leaves about 44 entries. For more than 32, of the 128 largest of the lanes' halves.
        auto bound_of = [&](int& top) {
            int first, second;
            x.largest(first, second);
            uint32_t m = static_cast<uint32_t>(max(first, second)) ^ 0x80000000u;
            if (kept > 32) {
                m = static_cast<uint32_t>(first) ^ 0x80000000u;
                uint32_t o = static_cast<uint32_t>(second) ^ 0x80000000u;
                sort64(m);
                sort64(o);
                merge64(m, o);
            } else {
                sort64(m);
            }
            top = static_cast<int>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(m), 0)) ^ 0x80000000u);
            return static_cast<int>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(m), kept - 1)) ^ 0x80000000u);
        };
        int top, bound = bound_of(top);
        // A NaN among the best, or too few entries above -infinity: with the NaNs as -infinity, once more. (Otherwise NaNs of either
        // sign are not at or above the bound.) The row's end stays below: it has at least `kept` entries.
        if (top > Order<T>::kInf || bound <= -Order<T>::kInf) {
            x.clean();
            bound = max(-Order<T>::kInf, bound_of(top));
        }
        // The entries at or above the bound in rounds of 64, in the order of the sweep: one round, but for rows of many
        // equal scores.
        typename I::sorted best = I::none();
        int count = 64;
        for (int round = 0; round < count; round += 64) {
            count = 0;
            // Comparisons, values and places are made in the round, not all kept for the next.
            __asm__ volatile("" : "+s"(bound));
            uint32_t lane = lane_id();
            __asm__ volatile("" : "+v"(lane));
            x.touch();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool in = x.get(i) >= bound;
                const uint64_t mask = __ballot(in);
                if (mask == 0) continue;
                const uint32_t at = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                                              __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), static_cast<uint32_t>(count - round)));
                if (in && at < 64u) list[at] = I::make(x.get(i), place<E>(i, lane));
                count += __popcll(mask);
            }
            __builtin_amdgcn_wave_barrier();
            typename I::sorted e = I::sortable(list[lane_id()]);
            __builtin_amdgcn_wave_barrier();
            if (round + static_cast<int>(lane_id()) >= count) e = I::none();
            sort64(e);
            if (round == 0) best = e;
            else merge64(best, e);
        }
        return best;
    }
}

__device__ __forceinline__ float wave_max_first(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); }

// Weights of the K sums, one per lane of each group of G lanes.
template <int G>
__device__ __forceinline__ float slot_weight(float v, float top, float scale, bool on) {
    const float e = on && v > -INFINITY ? expf((v - top) * scale) : 0.0f;
    const float s = group_sum<G>(e);
    return s > 0.0f ? e / s : (s != s ? s : 0.0f);
}

template <typename T, int E, int NV>
__global__ __launch_bounds__(kStThreads) void slot_topk_kernel(StArgs a) {
    const sdm_slot_topk_io& io = a.io;
    using I = Item<T>;
    __shared__ typename I::type lists[kStWaves][64];
    typename I::type* list = lists[threadIdx.x / kWave];
    const int lane = static_cast<int>(lane_id());
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kStWaves;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kStWaves + threadIdx.x / kWave; t < io.N; t += waves) {
        const auto ea = best_of_row<T, E, NV>(io.a, t * io.a_row, io.n1, a.ka, list);
        const auto eb = best_of_row<T, E, NV>(io.b, t * io.b_row, io.n2, a.kb, list);
        const float va = I::value(ea), vb = I::value(eb);
        // The pairs 64 at a time, those that (i + 1)(j + 1) lets come first first. Of the later ones only what beats the K-th
        // best so far matters: a few are inserted one by one (9 vector instructions each), many ordered and merged (220).
        auto pair_at = [&](int p) {
            const uint32_t ij = p < a.pairs ? kPairs.at[p] : 0xFFFFu;
            const int i = static_cast<int>(ij >> 8), j = static_cast<int>(ij & 255u);
            const float x = __uint_as_float(lane_value(__float_as_uint(va), i)) + __uint_as_float(lane_value(__float_as_uint(vb), j));
            return i < a.ka && j < a.kb ? Entry{key_of(x), ~ij} : Entry{0u, 0u};
        };
        Entry best = pair_at(lane);
        sort64(best);
        for (int p0 = kWave; p0 < a.pairs; p0 += kWave) {
            Entry e = pair_at(p0 + lane);
            const Entry low{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(best.key), io.K - 1)),
                            static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(best.inv), io.K - 1))};
            uint64_t in = __ballot(above(e, low));
            if (__popcll(in) > kStInsert) {
                sort64(e);
                merge64(best, e);
                continue;
            }
            for (; in != 0; in &= in - 1) insert(best, e, __builtin_ctzll(in));
        }
        const uint32_t ij = ~best.inv;
        const int i = static_cast<int>((ij >> 8) & 63u), j = static_cast<int>(ij & 63u);
        const int64_t ia = static_cast<uint32_t>(lane_value(I::at(ea), i)), jb = static_cast<uint32_t>(lane_value(I::at(eb), j));
        const float v = float_of(best.key);
        const float w = slot_weight<kWave>(v, wave_max_first(v), io.scale, lane < io.K);
        if (lane < io.K) {
            const int64_t off = io.chunk_rows > 0 ? (t / io.chunk_rows) % io.P * io.stream_offset : 0;
            const int64_t id = ia * io.n2 + jb + off;
            if (io.idx_bytes == 8) static_cast<int64_t*>(io.idx)[t * io.K + lane] = id;
            else static_cast<int32_t*>(io.idx)[t * io.K + lane] = static_cast<int32_t>(id);
            if (io.val_dtype == SDM_BF16) static_cast<bf16_t*>(io.val)[t * io.K + lane] = narrow<bf16_t>(w);
            else static_cast<float*>(io.val)[t * io.K + lane] = w;
        }
    }
}

// ------------------------------------------------------------------------------------------ backward
//
// With p the weights (recomputed from the K gathered sums in float32) and y the gradient of them,
// d_m = scale p_m (y_m - sum p y) is the gradient of sum m; a score's gradient is the sum of the d of
// the slots it is part of, the rest of the row 0. One wave per token: the row's gradient is collected
// in LDS, each score's entries added up in a fixed order by the lowest entry that has it,
// so nothing is atomic and the bits are the same every run; then the whole row is written in wide
// stores. 32768 tokens of 2 x 512 bfloat16 scores, K = 32: 27.6 us (80 MB, 2.9 TB/s; writing it alone
// would take 12 to 15). Comparing columns entry by entry through lane reads took 49.
struct StBack {
    sdm_slot_topk_io io;
    const float* dval;
    void *da, *db;
    int64_t da_row, db_row;
    int vec;
};

template <typename T, bool VEC>
__device__ __forceinline__ void write_row(T* out, int n, float* acc) {
    const int lane = static_cast<int>(lane_id());
    if constexpr (VEC && sizeof(T) == 2) {
        for (int c = lane * 8; c < n; c += kWave * 8) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(acc + c), y = *reinterpret_cast<const f32x4*>(acc + c + 4);
            *reinterpret_cast<u32x4*>(out + c) =
                u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        }
    } else if constexpr (VEC) {
        for (int c = lane * 4; c < n; c += kWave * 4) *reinterpret_cast<f32x4*>(out + c) = *reinterpret_cast<const f32x4*>(acc + c);
    } else {
        for (int c = lane; c < n; c += kWave) out[c] = narrow<T>(acc[c]);
    }
}

// acc (zero on entry and on return) gains the entries (col, d) of the wave's EN entry lanes (lane % EN; past K: col -1) and is
// written out. Each lane compares its entry's column with EN / (64 / EN) of the others', read from LDS two at a time, and with
// EN = 32 the two lanes of an entry add up their halves; the lowest entry of a column writes the sum. list: EN pairs.
template <typename T, bool VEC, int EN>
__device__ __forceinline__ void scatter_row(T* out, int n, int col, float d, float* acc, u32x2* list) {
    constexpr int kOwn = EN * EN / kWave;   // others per lane
    const int lane = static_cast<int>(lane_id()), part = lane / EN * kOwn;
    if (lane < EN) list[lane] = u32x2{static_cast<uint32_t>(col), __float_as_uint(d)};
    __builtin_amdgcn_wave_barrier();
    uint64_t firsts = 0;
    float sum = 0.0f;
#pragma unroll 8
    for (int m = 0; m < kOwn; m += 2) {
        const u32x4 two = *reinterpret_cast<const u32x4*>(list + part + m);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool same = static_cast<int>(two[2 * e]) == col;
            sum += same ? __uint_as_float(two[2 * e + 1]) : 0.0f;
            const uint64_t mask = __ballot(same);
            if constexpr (EN == kWave) {
                firsts |= mask & -mask;
            } else {   // the two parts' columns are two different ones
                const uint32_t lo = static_cast<uint32_t>(mask), hi = static_cast<uint32_t>(mask >> 32);
                firsts |= (lo & -lo) | (hi & -hi);
            }
        }
    }
    if constexpr (EN < kWave) sum += lane_xor_f<32>(sum);
    const bool first = lane < EN && col >= 0 && ((firsts >> lane) & 1);
    if (first) acc[col] = sum;
    __builtin_amdgcn_wave_barrier();
    write_row<T, VEC>(out, n, acc);
    __builtin_amdgcn_wave_barrier();
    if (first) acc[col] = 0.0f;
    __builtin_amdgcn_wave_barrier();
}

// EN: entry lanes, 32 (K up to 32: both halves of the wave hold the entries) or 64.
template <typename T, bool VEC, int EN>
__global__ __launch_bounds__(kStThreads) void slot_topk_back_kernel(StBack b) {
    const sdm_slot_topk_io& io = b.io;
    extern __shared__ __align__(16) float accs[];   // [waves, width]
    __shared__ __align__(16) u32x2 lists[kStWaves][EN];
    const int width = (max(io.n1, io.n2) + 7) & ~7;
    float* acc = accs + static_cast<size_t>(threadIdx.x / kWave) * width;
    u32x2* list = lists[threadIdx.x / kWave];
    const int lane = static_cast<int>(lane_id()), entry = lane & (EN - 1);
    for (int c = lane; c < width; c += kWave) acc[c] = 0.0f;
    __builtin_amdgcn_wave_barrier();
    const int64_t waves = static_cast<int64_t>(gridDim.x) * kStWaves;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kStWaves + threadIdx.x / kWave; t < io.N; t += waves) {
        const bool on = entry < io.K;
        int i = -1, j = -1;
        float v = -INFINITY, y = 0.0f;
        if (on) {
            int64_t id = io.idx_bytes == 8 ? static_cast<const int64_t*>(io.idx)[t * io.K + entry]
                                           : static_cast<const int32_t*>(io.idx)[t * io.K + entry];
            y = b.dval[t * io.K + entry];
            if (io.chunk_rows > 0) id -= (t / io.chunk_rows) % io.P * io.stream_offset;
            // In bounds whatever the caller passed.
            const int64_t last = static_cast<int64_t>(io.n1) * io.n2 - 1;
            id = id < 0 ? 0 : id > last ? last : id;
            const uint32_t local = static_cast<uint32_t>(id), n2 = static_cast<uint32_t>(io.n2);   // at most 2^24
            i = static_cast<int>(local / n2);
            j = static_cast<int>(local - static_cast<uint32_t>(i) * n2);
            const float x = widen(static_cast<const T*>(io.a)[t * io.a_row + i]) + widen(static_cast<const T*>(io.b)[t * io.b_row + j]);
            v = x != x ? -INFINITY : x;
        }
        float top = v;
        top = fmaxf(top, lane_xor_f<1>(top));
        top = fmaxf(top, lane_xor_f<2>(top));
        top = fmaxf(top, lane_xor_f<4>(top));
        top = fmaxf(top, lane_xor_f<8>(top));
        top = fmaxf(top, lane_xor_f<16>(top));
        if constexpr (EN == kWave) top = fmaxf(top, lane_xor_f<32>(top));
        const float p = slot_weight<EN>(v, top, io.scale, on);
        // A slot of weight 0 takes part in neither sum: its gradient is 0 whatever came in.
        const float py = p > 0.0f ? p * y : 0.0f;
        const float dot = group_sum<EN>(py);
        const float d = p > 0.0f ? p * (y - dot) * io.scale : p;
        if (b.da != nullptr) scatter_row<T, VEC, EN>(static_cast<T*>(b.da) + t * b.da_row, io.n1, i, d, acc, list);
        if (b.db != nullptr) scatter_row<T, VEC, EN>(static_cast<T*>(b.db) + t * b.db_row, io.n2, j, d, acc, list);
    }
}

bool rows16(const void* p, int64_t row, int n, int unit) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % unit == 0 && n % unit == 0;
}

// Rows per launch-resident wave: enough blocks to fill the device several times, then grid-stride.
constexpr int64_t kStBlocks = 1 << 16;

template <typename T, int E>
void st_go(const StArgs& a, hipStream_t st) {
    const int64_t need = (a.io.N + kStWaves - 1) / kStWaves;
    const unsigned grid = static_cast<unsigned>(need < kStBlocks ? need : kStBlocks);
    const int nv = ((a.io.n1 > a.io.n2 ? a.io.n1 : a.io.n2) + kWave - 1) / kWave;   // keys per lane of the longer row
    if constexpr (E == 1) {
        if (nv <= 1) { slot_topk_kernel<T, 1, 1><<<grid, kStThreads, 0, st>>>(a); return; }
        if (nv <= 2) { slot_topk_kernel<T, 1, 2><<<grid, kStThreads, 0, st>>>(a); return; }
    }
    if constexpr (E <= 4) {
        if (nv <= 4) { slot_topk_kernel<T, E, 4><<<grid, kStThreads, 0, st>>>(a); return; }
    }
    if (nv <= 8) slot_topk_kernel<T, E, 8><<<grid, kStThreads, 0, st>>>(a);
    else if (nv <= 16) slot_topk_kernel<T, E, 16><<<grid, kStThreads, 0, st>>>(a);
    else if (nv <= 32) slot_topk_kernel<T, E, 32><<<grid, kStThreads, 0, st>>>(a);
    else slot_topk_kernel<T, E, 64><<<grid, kStThreads, 0, st>>>(a);
}

}  // namespace

hipError_t slot_topk_launch(const sdm_slot_topk_io* io, hipStream_t st) {
    StArgs a;
    a.io = *io;
    a.ka = io->K < io->n1 ? io->K : io->n1;
    a.kb = io->K < io->n2 ? io->K : io->n2;
    a.pairs = kPairsHost.count[io->K];
    const bool bf = io->dtype == SDM_BF16;
    const int unit = bf ? 8 : 4;
    // 16-byte loads pay from rows of 64 lanes' worth of them; shorter rows leave lanes idle either way.
    const int longest = io->n1 > io->n2 ? io->n1 : io->n2;
    a.vec = longest > 2 * kWave && rows16(io->a, io->a_row, io->n1, unit) && rows16(io->b, io->b_row, io->n2, unit);
    if (bf) a.vec ? st_go<bf16_t, 8>(a, st) : st_go<bf16_t, 1>(a, st);
    else a.vec ? st_go<float, 4>(a, st) : st_go<float, 1>(a, st);
    return hipGetLastError();
}

int slot_lds_kernels(const void** fns, int cap) {
    const void* all[] = {reinterpret_cast<const void*>(&slot_topk_back_kernel<bf16_t, true, 32>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<bf16_t, false, 32>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<float, true, 32>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<float, false, 32>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<bf16_t, true, 64>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<bf16_t, false, 64>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<float, true, 64>),
                         reinterpret_cast<const void*>(&slot_topk_back_kernel<float, false, 64>)};
    int n = 0;
    for (const void* f : all) {
        if (n < cap) fns[n++] = f;
    }
    return n;
}

hipError_t slot_topk_back_launch(const sdm_slot_topk_io* io, const sdm_slot_topk_grad* g, hipStream_t st) {
    StBack b;
    b.io = *io;
    b.dval = g->dval;
    b.da = g->da;
    b.db = g->db;
    b.da_row = g->da_row;
    b.db_row = g->db_row;
    const bool bf = io->dtype == SDM_BF16;
    const int unit = bf ? 8 : 4;
    b.vec = (g->da == nullptr || rows16(g->da, g->da_row, io->n1, unit)) && (g->db == nullptr || rows16(g->db, g->db_row, io->n2, unit));
    const int width = ((io->n1 > io->n2 ? io->n1 : io->n2) + 7) & ~7;
    const size_t lds = static_cast<size_t>(kStWaves) * width * sizeof(float);
    const int64_t need = (io->N + kStWaves - 1) / kStWaves;
    const int64_t most = 4096;   // grid-stride past 16 blocks per compute unit: the LDS rows are zeroed once per wave
    const unsigned grid = static_cast<unsigned>(need < most ? need : most);
    auto go = [&](auto entries) {
        constexpr int EN = decltype(entries)::value;
        if (bf) {
            if (b.vec) slot_topk_back_kernel<bf16_t, true, EN><<<grid, kStThreads, lds, st>>>(b);
            else slot_topk_back_kernel<bf16_t, false, EN><<<grid, kStThreads, lds, st>>>(b);
        } else {
            if (b.vec) slot_topk_back_kernel<float, true, EN><<<grid, kStThreads, lds, st>>>(b);
            else slot_topk_back_kernel<float, false, EN><<<grid, kStThreads, lds, st>>>(b);
        }
    };
    if (io->K <= 32) go(std::integral_constant<int, 32>{});
    else go(std::integral_constant<int, 64>{});
    return hipGetLastError();
}

}  // namespace sdm
