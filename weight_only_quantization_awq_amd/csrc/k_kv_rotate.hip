// Queries and keys normalised for each head, rotated by their positions, and the keys and
// values quantised into the 4-bit cache, in one pass.
//
// For one row of one head x, in float32 but for the norm's inside:
//   u = fl32(1 / sqrt(mean x^2 + eps))        (64 bits inside, rounded once)
//   y = fl32(fl32(x u) w)                     (y = x where there is no weight)
//   channels (a, b) of a pair, angle's cosine c and sine s from the table:
//   a' = fl32(fl32(a c) - fl32(b s)),  b' = fl32(fl32(b c) + fl32(a s))
// Keys are turned by these very roundings, so what the cache holds does not depend on the order
// of a sum or on fused operations: the sum of squares is taken in 64 bits, where its order
// changes the rounded u about once in 2^28 rows.  Queries, which most callers round to 16 bits
// next, take fewer instructions: the squares' sum and u in float32 (u as the keys' where float32's range
// does not hold the squares) and the pair's sum in one fused operation, within 13 * 2^-24 of the sum of
// the two terms' sizes.  Values are formed in the definition's order, so that none leaves
// float32's range that does not leave it there (u (x1 (w1 c) - x2 (w2 s)) is no faster: 46.3 us both).
//
// Work split: units of 4 aligned positions and a head for keys and values as in k_kv.hip, and for
// queries a wave to a row and kQueryIter * 64 / (D/8) of its heads, whose loads are all in
// flight while the wave finds the row's sequence, position and angles.  Workgroups for keys,
// which compute more, are spread among those for queries, which move more (first all of
// them: 46.9 us and 45.2).
//
// Measured: 5 ragged bf16 chunks of up to 4099 rows, 64 query and 8 key heads of 128, with norms
// (188 MB in and out) 44.9 us, 4.2 TB/s; vector units are busy 71% of the cycles (95% with the
// queries' norms in 64 bits too, 49.5 us with a 64-bit root and division, 46.5 without).  One row: 4.5 us.
#include "kv_quant.h"

namespace awq {

namespace {

constexpr int kQueryIter = 4;   // heads of a lane
template <int D>
constexpr int kQueryHeads = kQueryIter * 64 / (D / 8);   // heads of a wave: 32, 16 or 8

// 1 / sqrt(x) in float32 for x > 0 (infinity too): the instruction's estimate (2^-23) and two
// Newton steps in 64 bits, each of which squares the error and half of it again, leave 2^-52 before the
// one rounding.  (A 64-bit root and division take 5 times as many instructions.)
__device__ __forceinline__ float inverse_root(double x) {
    double r = __builtin_amdgcn_rsq(x);
    const double h = 0.5 * x;
#pragma unroll
    for (int i = 0; i < 2; ++i) r = r * fma(-h * r, r, 1.5);
    return x > 1.0e300 ? 0.0f : static_cast<float>(r);
}

// What a lane needs to turn its 8 channels 8w .. 8w+7 of one row: the weights' and the
// angles' share of them.  Lanes whose channels are not rotated have turned = false.
template <int D>
struct Turner {
    static constexpr int LT = D / 8;
    float c[8], s[8], weight[8];   // s: with the sign of this channel's product
    bool norm, turned, neighbours, lost;
    int partner;                   // lane that holds the other channels of the pairs (halves)
    double eps;

    __device__ __forceinline__ void start(const KvTurn &t, const float *weights, int position, int w) {
        norm = weights != nullptr;
        neighbours = t.neighbours != 0;
        eps = t.eps;
        if (norm) load8(weights + 8 * w, weight);
        const int half = t.rot >> 1, lanes = half >> 3;   // lanes of half the rotated channels
        turned = w < 2 * lanes;
        lost = t.rot > 0 && position >= t.positions;
        partner = threadIdx.x & 63;
        const int at = position < 0 || lost ? 0 : position;
        if (turned) {
            const float *row = t.cos_sin + static_cast<int64_t>(at) * t.rot;
            if (neighbours) {
                const float4 a = *reinterpret_cast<const float4 *>(row + 4 * w), b = *reinterpret_cast<const float4 *>(row + half + 4 * w);
                c[0] = c[1] = a.x, c[2] = c[3] = a.y, c[4] = c[5] = a.z, c[6] = c[7] = a.w;
                s[0] = -b.x, s[1] = b.x, s[2] = -b.y, s[3] = b.y, s[4] = -b.z, s[5] = b.z, s[6] = -b.w, s[7] = b.w;
            } else {
                const bool second = w >= lanes;
                const int i = 8 * (second ? w - lanes : w);
                load8(row + i, c);
                load8(row + half + i, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = second ? s[e] : -s[e];
                partner += second ? -lanes : lanes;
            }
        }
    }

    // All lanes of the wave call.
    __device__ __forceinline__ void turn(float *x) const {
#pragma clang fp contract(off)
        if (norm) {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
#pragma unroll
            for (int m = 1; m < LT; m <<= 1) sum += __shfl_xor(sum, m);
            const float u = inverse_root(sum * (1.0 / D) + eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (x[i] * u) * weight[i];
        }
        float other[8];
        if (neighbours) {
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = x[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl(x[i], partner);
        }
        if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = x[i] * c[i], b = other[i] * s[i];
                x[i] = a + b;
            }
        }
        if (lost) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = NAN;
        }
    }
};

// Position of a wave's row, and whether the row belongs to a sequence.
__device__ __forceinline__ bool row_position(const KvCache &c, const KvBatch &s, int row, int lane, int &position) {
    int b;
    if (s.row_start)
        b = kv_wave_sequence<1, 0>(s, row, lane);
    else
        b = row / s.even;
    int r0, n;
    kv_rows(s, b, r0, n);
    position = kv_length(s, b, c.page_shift) - n + (row - r0);
    return row >= r0 && row < r0 + n;
}

// Turns queries (as the file's head says).
template <typename T, int D>
struct QueryTurner {
    static constexpr int LT = D / 8;
    typedef T vec8 __attribute__((ext_vector_type(8)));
    Turner<D> t;
    float theirs[8];   // weights of the pairs' other channels (halves)

    __device__ __forceinline__ void start(const KvTurn &turn, int position, int w) {
        t.start(turn, turn.q_weight, position, w);
        if (t.norm && !t.neighbours) load8(turn.q_weight + 8 * (w + t.partner - (threadIdx.x & 63)), theirs);
    }

    // All lanes of the wave call.  NORM, NEIGHBOURS: as `norm` and `neighbours` say.
    template <bool NORM, bool NEIGHBOURS>
    __device__ __forceinline__ void turn(vec8 in, float *x) const {
        float other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(in[i]);
        if constexpr (!NEIGHBOURS) {
            constexpr int kWords = sizeof(vec8) / 4;
            struct Words { uint32_t w[kWords]; } words = __builtin_bit_cast(Words, in);
#pragma unroll
            for (int i = 0; i < kWords; ++i) words.w[i] = __shfl(words.w[i], t.partner);
            const vec8 there = __builtin_bit_cast(vec8, words);
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = static_cast<float>(there[i]);
        }
        if constexpr (NORM) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int m = 1; m < LT; m <<= 1) sum += __shfl_xor(sum, m);
            const float mean = fmaf(sum, 1.0f / D, static_cast<float>(t.eps));
            float u = __builtin_amdgcn_rsqf(mean);
            if (__any(!(mean > 1.0e-30f && mean < 1.0e30f))) {   // (NaN, too)
                double wide = 0.0;
#pragma unroll
                for (int i = 0; i < 8; ++i) wide = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), wide);
#pragma unroll
                for (int m = 1; m < LT; m <<= 1) wide += __shfl_xor(wide, m);
                u = inverse_root(wide * (1.0 / D) + t.eps);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (x[i] * u) * t.weight[i];
            if constexpr (!NEIGHBOURS) {
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = (other[i] * u) * theirs[i];
            }
        }
        if (t.turned) {
            if constexpr (NEIGHBOURS) {
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = x[i ^ 1];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(other[i], t.s[i], x[i] * t.c[i]);
        }
    }
};

template <typename T, int D, int GROUP>
__global__ __launch_bounds__(kKvThreads) void kv_append_rotated_kernel(KvCache c, KvBatch s, KvTurn t, const T *Q,
                                                                       const T *__restrict__ K, const T *__restrict__ V,
                                                                       T *Qo, int64_t q_stride, int64_t k_stride,
                                                                       int64_t v_stride, int64_t o_stride, int q_heads,
                                                                       int units, int units_even, int key_groups, int apart) {
    constexpr int LT = D / 8, LU = 4 * LT, PER = kKvThreads / LU;
    __shared__ uint32_t bytes[PER][LU];
    // every `apart`th workgroup is one for keys and values, while there are any
    const int period = blockIdx.x / apart;
    const bool keys_here = period < key_groups && blockIdx.x == static_cast<unsigned>(period) * apart;
    if (keys_here) {
        Turner<D> turner;
        const int sub = threadIdx.x / LU, lane = threadIdx.x % LU, token = lane / LT, w = lane % LT;
        const int id = period * PER + sub, unit = id / c.heads, head = id - unit * c.heads;
        Finder<LU> f;
        f.row(c, s, unit, units, units_even, token);
        float k[8] = {}, v[8] = {};
        if (f.p.row >= 0) {
            load8(K + f.p.row * k_stride + head * D + 8 * w, k);
            load8(V + f.p.row * v_stride + head * D + 8 * w, v);
        }
        turner.start(t, t.k_weight, f.p.row >= 0 ? f.base + token : 0, w);
        f.page(c, s, head, token);
        turner.turn(k);
        store_unit<D, GROUP>(c, f.p, lane, token, w, k, v, bytes[sub]);
        return;
    }
    constexpr int kHeads = 64 / LT;   // of one step
    const int lane = threadIdx.x & 63, w = lane % LT;
    const int chunks = (q_heads + kQueryHeads<D> - 1) / kQueryHeads<D>;
    const int64_t id = static_cast<int64_t>(blockIdx.x - (period < key_groups ? period + 1 : key_groups)) * (kKvThreads / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t at = id / chunks;
    if (at >= s.T) return;
    const int row = static_cast<int>(at), head = static_cast<int>(id - at * chunks) * kQueryHeads<D> + lane / LT;
    typedef T vec8 __attribute__((ext_vector_type(8)));
    vec8 in[kQueryIter];
#pragma unroll
    for (int i = 0; i < kQueryIter; ++i) {
        in[i] = vec8{};
        if (head + i * kHeads < q_heads)
            in[i] = *reinterpret_cast<const vec8 *>(Q + row * q_stride + static_cast<int64_t>(head + i * kHeads) * D + 8 * w);
    }
    int position;
    if (!row_position(c, s, row, lane, position)) return;   // (one for the wave)
    QueryTurner<T, D> turner;
    turner.start(t, position, w);
    auto heads = [&](auto norm, auto neighbours) {
#pragma unroll
        for (int i = 0; i < kQueryIter; ++i) {
            float x[8];
            turner.template turn<decltype(norm)::value, decltype(neighbours)::value>(in[i], x);
            if (position < 0 || turner.t.lost) {   // (one for the wave)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = position < 0 ? 0.0f : NAN;
            }
            if (head + i * kHeads < q_heads) store8(Qo + row * o_stride + static_cast<int64_t>(head + i * kHeads) * D + 8 * w, x);
        }
    };
    if (turner.t.norm && turner.t.neighbours)
        heads(std::true_type{}, std::true_type{});
    else if (turner.t.norm)
        heads(std::true_type{}, std::false_type{});
    else if (turner.t.neighbours)
        heads(std::false_type{}, std::true_type{});
    else
        heads(std::false_type{}, std::false_type{});
}

template <typename T, int D, int GROUP>
hipError_t append_rotated(const KvCache &c, const KvBatch &s, const KvTurn &t, const void *Q, const void *K, const void *V, void *Qo,
                          int q_heads, int64_t qs, int64_t ks, int64_t vs, int64_t os, hipStream_t st) {
    int units, even;
    kv_unit_counts(s, units, even);
    const int64_t per = kKvThreads / (D / 2), keys = (static_cast<int64_t>(units) * c.heads + per - 1) / per;
    const int64_t waves = static_cast<int64_t>(s.T) * ((q_heads + kQueryHeads<D> - 1) / kQueryHeads<D>);
    const int64_t queries = (waves + kKvThreads / 64 - 1) / (kKvThreads / 64);
    auto launch = [&](int64_t groups, int64_t key_groups, int64_t apart) {
        hipLaunchKernelGGL((kv_append_rotated_kernel<T, D, GROUP>), dim3(static_cast<unsigned>(groups)), dim3(kKvThreads), 0, st, c, s, t,
                           static_cast<const T *>(Q), static_cast<const T *>(K), static_cast<const T *>(V), static_cast<T *>(Qo), qs, ks,
                           vs, os, q_heads, units, even, static_cast<int>(key_groups), static_cast<int>(apart));
    };
    if (t.keys_first) {
        launch(keys, keys, 1);
        launch(queries, 0, 1);
    } else {
        launch(keys + queries, keys, queries / keys + 1);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_rotated(const KvCache &c, const KvBatch &s, const KvTurn &t, const void *Q, const void *K,
                                    const void *V, void *Qo, int type, int q_heads, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, int64_t o_stride, hipStream_t st) {
    return kv_by_size(c, [&](auto d, auto g) {
        constexpr int D = decltype(d)::value, G = decltype(g)::value;
        if (type == 0) return append_rotated<float, D, G>(c, s, t, Q, K, V, Qo, q_heads, q_stride, k_stride, v_stride, o_stride, st);
        if (type == 1) return append_rotated<__bf16, D, G>(c, s, t, Q, K, V, Qo, q_heads, q_stride, k_stride, v_stride, o_stride, st);
        return append_rotated<_Float16, D, G>(c, s, t, Q, K, V, Qo, q_heads, q_stride, k_stride, v_stride, o_stride, st);
    });
}

}  // namespace awq
