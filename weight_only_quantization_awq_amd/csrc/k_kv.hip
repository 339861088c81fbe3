// Writing the 4-bit key/value cache and reading it back (layout: kv_internal.h).
//
// Quantiser, per group of one token and head, in float32:
//   lo   = fp16(min x), step = fp16(max(max x - lo, 0) * (1/15)), 1/15 in float32
//   code = clamp(rint((x - lo) / step), 0, 15)   (0 where step is 0)
// taken against the stored lo and step, with IEEE quotients, so the codes do
// not depend on the machine's approximations.  Reading: code*step is exact in
// float32 (4 + 11 significant bits), so code*step + lo rounds once there and
// once in the output type.
//
// A head's token that holds a NaN or a value beyond +-32768 in its key or its
// value row is stored as NaN key pairs and zero value pairs: it reads back as
// NaN (both), a query that attends to it gets NaN through its score, and a
// query that does not is untouched, since 0 * V stays 0.  The bound keeps
// code*step + lo inside fp16: lo + 15*step rounds to at most 65504.
//
// Work split: one unit per aligned block of 4 positions and head, 4 tokens x
// D/8 lanes of 8 channels (a wave at D = 128).  Keys leave as one word per lane.
// Values interleave 4 tokens by bytes, so a unit gathers its bytes in LDS and
// stores whole words where all 4 tokens are new, else single bytes (the other
// tokens of the block may be written by another call at the same time).
//
// Measured: appending 5 ragged bf16 chunks of up to 4099 rows, 8 heads of 128 (25 MB
// in and out), takes 12.8 us, two thirds of it the issue of 500 vector instructions a
// wave; reading 4 sequences of up to 16384 back takes 20.2 us for 94 MB, a large copy's
// rate; calls on few rows are a launch (4.0 and 3.0 us).
#include "kv_quant.h"

namespace awq {

namespace {

template <typename T, int D, int GROUP>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(KvCache c, KvBatch s, const T *__restrict__ K,
                                                               const T *__restrict__ V, int64_t k_stride,
                                                               int64_t v_stride, int units, int units_even) {
    constexpr int LT = D / 8;           // lanes of a token
    constexpr int LU = 4 * LT;          // lanes of a unit
    __shared__ uint32_t bytes[kKvThreads / LU][LU];   // value codes of each unit: 2*D bytes
    const int sub = threadIdx.x / LU, lane = threadIdx.x % LU, token = lane / LT, w = lane % LT;
    const int id = blockIdx.x * (kKvThreads / LU) + sub, unit = id / c.heads, head = id - unit * c.heads;
    Finder<LU> f;
    f.row(c, s, unit, units, units_even, token);
    float k[8] = {}, v[8] = {};
    if (f.p.row >= 0) {
        load8(K + f.p.row * k_stride + head * D + 8 * w, k);
        load8(V + f.p.row * v_stride + head * D + 8 * w, v);
    }
    f.page(c, s, head, token);
    store_unit<D, GROUP>(c, f.p, lane, token, w, k, v, bytes[sub]);
}

template <typename T, int D, int GROUP>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvCache c, KvBatch s, T *__restrict__ K,
                                                             T *__restrict__ V, int64_t k_stride, int64_t v_stride,
                                                             int units, int units_even) {
    constexpr int LT = D / 8, LU = 4 * LT, J = D / 32, NG = D / GROUP, GL = GROUP / 8;
    __shared__ uint32_t bytes[kKvThreads / LU][LU];
    const int sub = threadIdx.x / LU, lane = threadIdx.x % LU, token = lane / LT, w = lane % LT;
    const int id = blockIdx.x * (kKvThreads / LU) + sub, unit = id / c.heads, head = id - unit * c.heads;
    Finder<LU> f;
    f.row(c, s, unit, units, units_even, token);
    f.page(c, s, head, token);
    const Place p = f.p;
    const bool there = p.block != nullptr;
    const int P = 1 << c.page_shift, j = w >> 2, kb = w & 3;
    uint32_t kw = 0, kp = 0, vp = 0;
    const unsigned char *mine = reinterpret_cast<const unsigned char *>(bytes[sub]);
    if (there) {
        kw = *reinterpret_cast<const uint32_t *>(p.block + p.slot * (D / 2) + 4 * (kb * J + j));
        const uint32_t *pairs = reinterpret_cast<const uint32_t *>(p.block + P * D);
        kp = pairs[p.slot * NG + w / GL];
        vp = pairs[P * NG + p.slot * NG + w / GL];
        const unsigned char *vb = p.block + P * (D / 2) + (p.slot >> 2) * (2 * D);
        bytes[sub][lane] = reinterpret_cast<const uint32_t *>(vb)[lane];   // all 4 tokens' bytes, new or not
    }
    __syncthreads();
    if (p.row < 0) return;
    float k[8] = {}, v[8] = {};
    if (there) {
        const float ks = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(kp)));
        const float kl = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(kp >> 16)));
        const float vs = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(vp)));
        const float vl = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(vp >> 16)));
        const int m0 = 8 * (w & 1), b = w >> 2, shift = 2 * (w & 2);
        const bool lost = ks != ks;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] = fmaf(static_cast<float>((kw >> (4 * key_nibble(i))) & 15u), ks, kl);
            const uint32_t q = (static_cast<uint32_t>(mine[(m0 + i) * (4 * J) + 4 * b + token]) >> shift) & 15u;
            v[i] = lost ? ks : fmaf(static_cast<float>(q), vs, vl);
        }
    }
    store8(K + p.row * k_stride + head * D + 8 * w, k);
    store8(V + p.row * v_stride + head * D + 8 * w, v);
}

template <typename T, int D, int GROUP>
hipError_t append(const KvCache &c, const KvBatch &s, const void *K, const void *V, int64_t ks, int64_t vs,
                  hipStream_t st) {
    int units, even;
    kv_unit_counts(s, units, even);
    const int64_t per = kKvThreads / (D / 2), n = (static_cast<int64_t>(units) * c.heads + per - 1) / per;
    hipLaunchKernelGGL((kv_append_kernel<T, D, GROUP>), dim3(static_cast<unsigned>(n)), dim3(kKvThreads), 0, st, c, s,
                       static_cast<const T *>(K), static_cast<const T *>(V), ks, vs, units, even);
    return hipGetLastError();
}

template <typename T, int D, int GROUP>
hipError_t read(const KvCache &c, const KvBatch &s, void *K, void *V, int64_t ks, int64_t vs, hipStream_t st) {
    int units, even;
    kv_unit_counts(s, units, even);
    const int64_t per = kKvThreads / (D / 2), n = (static_cast<int64_t>(units) * c.heads + per - 1) / per;
    hipLaunchKernelGGL((kv_read_kernel<T, D, GROUP>), dim3(static_cast<unsigned>(n)), dim3(kKvThreads), 0, st, c, s,
                       static_cast<T *>(K), static_cast<T *>(V), ks, vs, units, even);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvCache &c, const KvBatch &s, const void *K, const void *V, int type,
                            int64_t k_stride, int64_t v_stride, hipStream_t st) {
    return kv_by_size(c, [&](auto d, auto g) {
        constexpr int D = decltype(d)::value, G = decltype(g)::value;
        if (type == 0) return append<float, D, G>(c, s, K, V, k_stride, v_stride, st);
        if (type == 1) return append<__bf16, D, G>(c, s, K, V, k_stride, v_stride, st);
        return append<_Float16, D, G>(c, s, K, V, k_stride, v_stride, st);
    });
}

hipError_t launch_kv_read(const KvCache &c, const KvBatch &s, void *K, void *V, int type, int64_t k_stride,
                          int64_t v_stride, hipStream_t st) {
    return kv_by_size(c, [&](auto d, auto g) {
        constexpr int D = decltype(d)::value, G = decltype(g)::value;
        if (type == 0) return read<float, D, G>(c, s, K, V, k_stride, v_stride, st);
        if (type == 1) return read<__bf16, D, G>(c, s, K, V, k_stride, v_stride, st);
        return read<_Float16, D, G>(c, s, K, V, k_stride, v_stride, st);
    });
}

}  // namespace awq
