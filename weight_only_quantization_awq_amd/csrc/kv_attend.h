// Attention over the 4-bit key/value cache: the kernels, instantiated per head
// dimension by k_kv_attend_{64,128,256}.hip.
//
//   S[t, i] = scale * sum_c k'[t, c] q[i, c],  k' = step*code + lo per group g
//           = scale * sum_g ( step[t,g] * sum_{c in g} code[t,c] q[i,c] + lo[t,g] * sum_{c in g} q[i,c] )
//   O[i]    = sum_t softmax(S[., i])_t v'[t]
//
// Both products run on 16x16x32 MFMAs, transposed (keys and values are the A
// operand, queries and scores the B operand), 32 tokens a step:
//  - S^T = codes·Q^T.  A code enters as the 16-bit float 16 + code, exact, made by a
//    shift and an and-or of the packed word; steps and lowest values are applied in
//    float32, where the base is taken out.
//  - A lane's result rows are tokens 4kb..4kb+3 of one query, which are the
//    tokens that its B operand of the second product takes: scores stay in
//    their lane.
//  - O^T = V'^T·P^T in fp16: codes become fp16 by and-or (1024 + code, 64 + code),
//    an exact packed subtraction, and one packed fma with (step, lo): v' is
//    rounded once, to 11 bits.  P = exp2(S - m) <= 2^15 is rounded to 11 bits, too.
//  - The softmax reference m of a query (shared by its 4 lanes) is put 2^7 below the
//    largest score (log2: 7 less) and moves only when one exceeds it by 2^15, so most
//    steps need no cross-lane maximum and no rescaling, and the largest P is 2^7 or more:
//    weights keep their 11 bits down to 2^-21 of the largest, and are off by 2^-32 of it
//    below.  (With m at the largest score itself those bounds were 2^-14 and 2^-25, and a key
//    that outweighs a long sequence 2^25 times made all of the others vanish.)  Sums l
//    and m stay in float32.
//
// Masked scores are set to -inf after the product, so whatever a masked key holds
// is dropped; value pairs of tokens that do not exist (behind the length, on a
// page outside the cache) or that no row's window reaches are zeroed, since 0 * NaN
// would not vanish.
#pragma once

#include "kv_internal.h"

namespace awq {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kHeadLog2 = 7.0f;    // the reference lies this far below the largest score (log2) when it is set,
constexpr float kMostLog2 = 15.0f;   // and scores may exceed it by this: P <= 2^15 fits fp16
constexpr float kFloorLog2 = 64.0f;  // the wide path's scores are formed relative to no less than -64

// ln sum exp S of a reference m (log2) and the sum l of exp2(S - m).  The head is taken out of
// both first, so that neither is larger than it has to be (with it, and three roundings,
// lse of 65 tokens was off by 4.2e-7 in the root mean square, which is 1.9e-7 now, as float32's).
__device__ __forceinline__ float kv_lse(float m, float l) {
    constexpr float kBelow = 1.0f / 128.0f;
    static_assert(kHeadLog2 == 7.0f, "");
    return l == 0.0f ? -INFINITY : fmaf(m + kHeadLog2, kLn2, __builtin_amdgcn_logf(l * kBelow) * kLn2);
}

// (x & mask) | bits in one instruction: VOP3 takes no literals, so the empty asm
// statements keep both constants in registers.  (The instruction itself is the
// compiler's: it has to see it to space it from MFMAs on the same registers.)
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    asm("" : "+s"(mask));
    asm("" : "+v"(bits));
    return (x & mask) | bits;
}

__device__ __forceinline__ float half_lo(uint32_t x) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(x)));
}
__device__ __forceinline__ float half_hi(uint32_t x) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(x >> 16)));
}

// Key codes enter as 16 + code, the lowest base whose steps of one are all exact.  It leaves a
// score by one of two ways, both with what float32 has left of sums that are (16 + code) / code
// times as large:
//  - in the lowest value's factor (a pair as the factors of (sum (base + code)*q, sum q) in a
//    score, scaled): no instruction, on the wide path, where one more for each score and group
//    takes 2.5 to 6%;
constexpr float kKeyBase = 16.0f;
__device__ __forceinline__ float2 key_factors(uint32_t pair, float scale) {
    const float step = half_lo(pair);
    return make_float2(step * scale, fmaf(-kKeyBase, step, half_hi(pair)) * scale);
}
//  - from the sum itself, with the middle of the codes, on the split path (a pair as the factors of
//    (sum (code - middle)*q, sum q), unscaled and exact; 0 to 1% of the time).  One token over 65
//    keys whose channels lie far apart, bf16: lse off by 1.5e-7 in the median of 100 inputs and by
//    1.5e-6 at most, by the first way 3.6e-7 and 1.8e-6, in float32 over the values 7e-8 and 3.2e-7.
constexpr float kKeyMiddle = 7.5f;
__device__ __forceinline__ float2 key_middle(uint32_t pair) {
    const float step = half_lo(pair);
    return make_float2(step, fmaf(kKeyMiddle, step, half_hi(pair)));
}

template <typename T>
struct KvType;
template <>
struct KvType<__bf16> {
    typedef bf16x8 vec8;
    // The codes of channels (2i, 2i+1) of a key word, + base.  (Base 128 would save the
    // shift of i = 0; its sums cancel 8 times as much.)
    static __device__ __forceinline__ uint32_t pair(uint32_t w, int i) {
        const uint32_t x = i == 0 ? w << 3 : w >> (4 * i - 3);
        return and_or(x, 0x00780078u, 0x41804180u);
    }
    static __device__ __forceinline__ floatx4 mfma(uint4 a, vec8 b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec8, a), b, c, 0, 0, 0);
    }
};
template <>
struct KvType<_Float16> {
    typedef half8 vec8;
    // Of the forms that take as long: 64 + code puts lse 3 to 4 times as far off (keys with
    // channels far apart, dim 128, 64 rows over 65 keys: 3.3e-5 in the root mean square and
    // 9.5e-6 with 16); a code's own bits as a subnormal need no base, but these MFMAs align
    // them as if they were 2^-14 (7.8e-5).
    static __device__ __forceinline__ uint32_t pair(uint32_t w, int i) {
        const uint32_t x = i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6);
        return and_or(x, 0x03C003C0u, 0x4C004C00u);
    }
    static __device__ __forceinline__ floatx4 mfma(uint4 a, vec8 b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec8, a), b, c, 0, 0, 0);
    }
};

typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// The bytes 0 and 2 of w hold two tokens' codes of two channels (low and high
// nibbles): those codes, exact, in fp16.
__device__ __forceinline__ void value_codes(uint32_t w, half2v &low, half2v &high) {
    low = __builtin_bit_cast(half2v, and_or(w, 0x000F000Fu, 0x64006400u)) -
          half2v{static_cast<_Float16>(1024), static_cast<_Float16>(1024)};
    high = __builtin_bit_cast(half2v, and_or(w, 0x00F000F0u, 0x54005400u)) -
           half2v{static_cast<_Float16>(64), static_cast<_Float16>(64)};
}

template <typename T>
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
    typedef T vec4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint2, vec4{static_cast<T>(a), static_cast<T>(b), static_cast<T>(c), static_cast<T>(d)});
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef T vec2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, vec2{static_cast<T>(a), static_cast<T>(b)});
}

template <int N>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t *w) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
}

// One step's codes, as a lane's operands, and pairs: lanes 0..31 hold the key
// pairs of tokens 0..31, lanes 32..63 the value pairs.
template <int D, int NG>
struct KvStep {
    uint32_t k[2][D / 32], v[2][D / 32], pair[NG];
    bool ok0, ok1;   // the two 16-token halves exist
};

// A wave's pairs in LDS, made for reading by result rows (4 tokens of a lane):
// keys as factors (key_middle), values as fp16 (step0, step2,
// step1, step3, lo0, lo2, lo1, lo3), the order of the value bytes.
template <int NG>
struct KvPairs {
    floatx4 k[2][NG][4][2];
    uint4 v[2][NG][4];
};

// Page of token `tok` (uniform in a wave), -1 where there is none.
__device__ __forceinline__ int kv_page(const KvAttend &a, const int32_t *table, int tok, int len) {
    if (tok >= len) return -1;
    const int id = table[tok >> a.c.page_shift];
    return id < 0 || id >= a.c.n_pages ? -1 : id;
}

template <int D, int NG>
__device__ __forceinline__ void kv_load(const KvAttend &a, int head, int tok, int page0, int page1, int lane,
                                        KvStep<D, NG> &s) {
    const int n = lane & 15, kb = lane >> 4, P = 1 << a.c.page_shift;
    s.ok0 = page0 >= 0;
    s.ok1 = page1 >= 0;
    const unsigned char *pairs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int page = h ? page1 : page0;
        const int slot = (tok + 16 * h) & (P - 1);
        // a half that does not exist reads page 0, which does, and is masked
        const unsigned char *b =
            a.c.pages + (page < 0 ? 0 : page) * a.c.page_stride + head * a.c.block;
        load_words<D / 32>(b + slot * (D / 2) + (n * (D / 2) + kb * (D / 8)), s.k[h]);
        load_words<D / 32>(b + P * (D / 2) + slot * (D / 2) + (kb * 16 + n) * (D / 8), s.v[h]);
        pairs[h] = b + P * D + slot * (4 * NG);
    }
    load_words<NG>((kb & 1 ? pairs[1] : pairs[0]) + (kb >> 1) * P * (4 * NG) + n * (4 * NG), s.pair);
}

// Whether a position is one of lowest .. len - 1 (0 <= lowest <= len).
__device__ __forceinline__ bool kv_seen(int p, int lowest, int len) {
    return static_cast<uint32_t>(p - lowest) < static_cast<uint32_t>(len - lowest);
}

// Orders a wave's LDS accesses for its own lanes: what one lane wrote, another reads, as other
// types (float and uint16_t, read as vectors), so nothing else keeps the compiler from moving
// either.  LDS itself runs a wave's accesses in turn: no instruction comes of this.
__device__ __forceinline__ void kv_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A step's pairs into LDS.  Value pairs of tokens that do not exist, or that no row
// sees, become zero (0 * NaN would not vanish).  One wave writes and reads them, in order.
template <typename T, int D, int NG>
__device__ __forceinline__ void kv_pairs(const KvAttend &a, const KvStep<D, NG> &s, int tok, int lowest, int len,
                                         int lane, KvPairs<NG> *lds) {
    const int n = lane & 15, h = (lane >> 4) & 1;
    kv_lds_order();   // the tile before has been read
    const bool there = (h ? s.ok1 : s.ok0) && kv_seen(tok + 16 * h + n, lowest, len);
    if (lane < 32) {
        float *k = reinterpret_cast<float *>(&lds->k[h][0][0][0]) + 2 * n;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float2 y = key_middle(s.pair[g]);
            k[32 * g] = y.x;
            k[32 * g + 1] = y.y;
        }
    } else {
        const int r = n & 3, at = 8 * (n >> 2) + (r >> 1) + 2 * (r & 1);   // tokens 0, 2, 1, 3
        uint16_t *v = reinterpret_cast<uint16_t *>(&lds->v[h][0][0]) + at;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t p = there ? s.pair[g] : 0u;
            v[32 * g] = static_cast<uint16_t>(p);
            v[32 * g + 4] = static_cast<uint16_t>(p >> 16);
        }
    }
    kv_lds_order();
}

// One wave's 16*NT columns: queries, running sums, output.
template <typename T, int D, int NG, int NT>
struct KvWave {
    static constexpr int J = D / 32;
    typename KvType<T>::vec8 q[NT][J];
    float qs[NT][NG];                 // sum of q over a group
    floatx4 o[NT][D / 16];            // channel 16i + 4kb + r of column lane & 15
    float m[NT], l[NT];               // reference (log2) and this lane's share of the sum
    int pos[NT], low[NT];             // last and first visible position (pos -1: no such column)

    __device__ __forceinline__ void start(const KvAttend &a, int head, int r0, int n, int len, int col0, int lane) {
        const int kb = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int c = col0 + 16 * t + (lane & 15), i = c / a.per;
            const bool real = i < n;
            const T *src = static_cast<const T *>(a.Q) + (r0 + (real ? i : 0)) * a.q_stride +
                           static_cast<int64_t>(head * a.per + (c - i * a.per)) * D + 8 * kb;
            pos[t] = real ? (a.causal ? len - n + i : len - 1) : -1;
            low[t] = a.window ? len - n + i - a.window + 1 : 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) qs[t][g] = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                typename KvType<T>::vec8 x = {};
                if (real) x = *reinterpret_cast<const typename KvType<T>::vec8 *>(src + 32 * j);
                q[t][j] = x;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += static_cast<float>(x[e]);
                qs[t][j * NG / J] += sum;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                qs[t][g] += __shfl_xor(qs[t][g], 16);
                qs[t][g] += __shfl_xor(qs[t][g], 32);
            }
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[t][d] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            m[t] = -INFINITY;
            l[t] = 0.0f;
        }
    }

    // Tokens tok .. tok+31.  edge: some of them may be hidden from some column.
    __device__ __forceinline__ void step(const KvAttend &a, const KvStep<D, NG> &s, int tok, int lowest, int len,
                                         bool edge, int lane, KvPairs<NG> *lds) {
        const int kb = lane >> 4;
        kv_pairs<T>(a, s, tok, lowest, len, lane, lds);
        floatx4 x[2][NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const floatx4 k0 = lds->k[h][g][kb][0], k1 = lds->k[h][g][kb][1];
                const float step[4] = {k0[0], k0[2], k1[0], k1[2]}, lo[4] = {k0[1], k0[3], k1[1], k1[3]};
                floatx4 acc[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = g * (J / NG); j < (g + 1) * (J / NG); ++j) {
                    const uint32_t w = s.k[h][j];
                    const uint4 f = make_uint4(KvType<T>::pair(w, 0), KvType<T>::pair(w, 1), KvType<T>::pair(w, 2),
                                               KvType<T>::pair(w, 3));
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t] = KvType<T>::mfma(f, q[t][j], acc[t]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x[h][t][r] = fmaf(step[r], fmaf(-(kKeyBase + kKeyMiddle), qs[t][g], acc[t][r]),
                                          g == 0 ? lo[r] * qs[t][g] : fmaf(lo[r], qs[t][g], x[h][t][r]));
            }
        }
        if (edge) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int p = tok + 16 * h + 4 * kb + r;
                    const bool there = h ? s.ok1 : s.ok0;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (!there || p > pos[t] || p < low[t]) x[h][t][r] = -INFINITY;
                }
        }
        half8 p[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float top = a.scale_log2 * fmaxf(fmaxf(fmaxf(x[0][t][0], x[0][t][1]), fmaxf(x[0][t][2], x[0][t][3])),
                                                   fmaxf(fmaxf(x[1][t][0], x[1][t][1]), fmaxf(x[1][t][2], x[1][t][3])));
            if (__any(top > m[t] + kMostLog2)) {
                float now = fmaxf(m[t], top - kHeadLog2);
                now = fmaxf(now, __shfl_xor(now, 16));
                now = fmaxf(now, __shfl_xor(now, 32));
                const float f = m[t] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[t] - now);
                m[t] = now;
                l[t] *= f;
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[t][d][r] *= f;
            }
            const float ref = m[t] == -INFINITY ? 0.0f : m[t];
            // operand order of the value bytes: tokens (0, 2), (1, 3) of each half
            constexpr int kOrder[4] = {0, 2, 1, 3};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = __builtin_amdgcn_exp2f(fmaf(x[h][t][kOrder[r]], a.scale_log2, -ref));
                    l[t] += e;
                    p[t][4 * h + r] = static_cast<_Float16>(e);
                }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            half2v vs[2][2], vl[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v = lds->v[h][g][kb];
                vs[h][0] = __builtin_bit_cast(half2v, v.x), vs[h][1] = __builtin_bit_cast(half2v, v.y);
                vl[h][0] = __builtin_bit_cast(half2v, v.z), vl[h][1] = __builtin_bit_cast(half2v, v.w);
            }
#pragma unroll
            for (int b = g * (J / NG); b < (g + 1) * (J / NG); ++b) {
                half2v lo[4], hi[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        half2v cl, ch;
                        value_codes(s.v[h][b] >> (8 * e), cl, ch);
                        lo[2 * h + e] = __builtin_elementwise_fma(cl, vs[h][e], vl[h][e]);
                        hi[2 * h + e] = __builtin_elementwise_fma(ch, vs[h][e], vl[h][e]);
                    }
                half8 fl, fh;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    fl[2 * e] = lo[e][0], fl[2 * e + 1] = lo[e][1];
                    fh[2 * e] = hi[e][0], fh[2 * e + 1] = hi[e][1];
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fl, p[t], o[t][2 * b], 0, 0, 0);
                    o[t][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fh, p[t], o[t][2 * b + 1], 0, 0, 0);
                }
            }
        }
    }

    // Tokens of tiles t0 .. t1-1 of one sequence and head.  The loads of the next tile,
    // and the page numbers of the one after, are in flight while a tile is computed
    // (loads two or three tiles ahead cost registers and with them waves: 64 sequences of
    // up to 8192 tokens 31 -> 39 and 50 us).  minpos / maxlow: the first last-visible and
    // the last first-visible position of the columns.
    __device__ __forceinline__ void run(const KvAttend &a, const int32_t *table, int head, int t0, int t1, int lowest,
                                        int len, int minpos, int maxlow, int lane, KvPairs<NG> *lds) {
        if (t0 >= t1) return;
        KvStep<D, NG> now, then;
        int tok = t0 * kKvTile, p0 = -1, p1 = -1;
        const int end = t1 * kKvTile;
        auto pages = [&](int t) {
            if (t < end) p0 = kv_page(a, table, t, len), p1 = kv_page(a, table, t + 16, len);
        };
        pages(tok);
        kv_load(a, head, tok, p0, p1, lane, now);
        pages(tok + kKvTile);
#pragma unroll 1
        while (true) {
            const int next = tok + kKvTile;
            if (next < end) {
                kv_load(a, head, next, p0, p1, lane, then);
                pages(next + kKvTile);
            }
            step(a, now, tok, lowest, len, hides(now, tok, minpos, maxlow), lane, lds);
            tok = next;
            if (tok >= end) return;
            now = then;
        }
    }
    static __device__ __forceinline__ bool hides(const KvStep<D, NG> &s, int tok, int minpos, int maxlow) {
        return tok + kKvTile - 1 > minpos || tok < maxlow || !s.ok0 || !s.ok1;   // (minpos < length)
    }

    // Output and lse of the columns col0 .. of a sequence's rows.
    __device__ __forceinline__ void finish(const KvAttend &a, int head, int r0, int n, int col0, int lane) {
        const int kb = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int c = col0 + 16 * t + (lane & 15), i = c / a.per, h = head * a.per + c - i * a.per;
            l[t] += __shfl_xor(l[t], 16);
            l[t] += __shfl_xor(l[t], 32);
            if (i >= n) continue;
            const float inv = l[t] == 0.0f ? 0.0f : 1.0f / l[t];
            T *dst = static_cast<T *>(a.O) + (r0 + i) * a.o_stride + static_cast<int64_t>(h) * D + 4 * kb;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                *reinterpret_cast<uint2 *>(dst + 16 * d) =
                    pack4<T>(o[t][d][0] * inv, o[t][d][1] * inv, o[t][d][2] * inv, o[t][d][3] * inv);
            if (a.lse && kb == 0)
                a.lse[static_cast<int64_t>(r0 + i) * a.q_heads + h] = kv_lse(m[t], l[t]);
        }
    }

    // Sums of the columns col0 .. < cols, for a join: ml[c] = (reference, sum), part[c] = output.
    __device__ __forceinline__ void keep(float *ml, float *part, int cols, int col0, int lane) {
        const int kb = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int c = col0 + 16 * t + (lane & 15);
            l[t] += __shfl_xor(l[t], 16);
            l[t] += __shfl_xor(l[t], 32);
            if (c >= cols) continue;
            if (kb == 0) *reinterpret_cast<float2 *>(ml + 2 * c) = make_float2(m[t], l[t]);
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                *reinterpret_cast<floatx4 *>(part + static_cast<int64_t>(c) * D + 16 * d + 4 * kb) = o[t][d];
        }
    }
};

// ---------------------------------------------------------------------------
// Split path: sequences with at most 16*NT columns per key head (decoding).
//
// The items (sequence, head) form one line, each kKvItemCost + its tiles long,
// which the workers (one wave each, as many as the GPU holds) share equally: ragged
// lengths and few long sequences load the GPU evenly, and nothing but the
// lengths on the device decides it.  A worker that holds a whole item writes
// its output; the pieces of an item that a boundary cuts go to the workspace
// and kv_merge_kernel joins them in order.  Boundaries within a.snap tiles of an
// item's ends move there.
//
// What bounds it is the wait for loads, one tile ahead and 3 waves a SIMD: waves spend 55 to 59%
// of their time in it, while vector units are active 44 to 59% of the cycles and the matrix
// cores 7 to 9% (24 x 2047 tokens, 32 heads, group 32, 252 MB: 64 us, 3.9 TB/s; 131072
// tokens, 8 heads, 143 MB: 42 us, 3.4 TB/s, and 6 for the join).  With fixed pieces of tokens
// instead of the line, ragged batches wait for their longest sequence.

// 64 sequences of the line, one to a lane.
struct KvLine {
    int chunk, base;          // sequences 64*chunk ..; where the first one's items begin
    int length, upto, total;  // of one head: this lane's sequence, up to its end, all 64

    __device__ __forceinline__ void load(const KvAttend &a, int c, int lane) {
        chunk = c;
        int r0, n, len;
        const int b = 64 * c + lane, t = b < a.s.B ? kv_item_tiles(a, b, r0, n, len) : 0;
        length = t > 0 ? t + kKvItemCost : 0;
        upto = length;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(upto, d);
            if (lane >= d) upto += up;
        }
        total = __builtin_amdgcn_readlane(upto, 63);
    }
};

struct KvItem {
    int b, head, r0, n, len, tiles, begin, end;   // begin, end: on the line
};

// The item at x (0 <= x < the line's length), at or behind the line's present chunk.
__device__ __forceinline__ KvItem kv_locate(const KvAttend &a, KvLine &line, int x, int lane) {
    const int H = a.c.heads;
    while (x >= line.base + H * line.total && 64 * (line.chunk + 1) < a.s.B) {
        line.base += H * line.total;
        line.load(a, line.chunk + 1, lane);
    }
    const int y = x - line.base;
    const int k = kv_clamp(__popcll(__ballot(H * line.upto <= y)), 0, 63);
    int length = __builtin_amdgcn_readlane(line.length, k);
    const int before = H * (__builtin_amdgcn_readlane(line.upto, k) - length);
    length = length > 0 ? length : 1;
    KvItem it;
    it.b = 64 * line.chunk + k;
    it.b = it.b < a.s.B ? it.b : a.s.B - 1;
    it.head = kv_clamp((y - before) / length, 0, H - 1);
    it.begin = line.base + before + it.head * length;
    it.end = it.begin + length;
    it.tiles = length - kKvItemCost;
    kv_rows(a.s, it.b, it.r0, it.n);
    it.len = kv_length(a.s, it.b, a.c.page_shift);
    return it;
}

template <typename T, int D, int NG, int NT>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(kv_split_waves(D, NT)))) void kv_split_kernel(
    KvAttend a) {
    const int lane = threadIdx.x;
    __shared__ KvPairs<NG> pairs;
    KvLine line;
    line.base = 0;
    int total = 0;
    for (int c = (a.s.B - 1) / 64; c >= 0; --c) {   // (ends with chunk 0 loaded)
        line.load(a, c, lane);
        total += line.total;
    }
    total *= a.c.heads;
    const int worker = blockIdx.x, workers = kv_workers(a, total);
    if (worker >= workers || total == 0) return;
    const int x0 = kv_share(worker, total, workers), x1 = kv_share(worker + 1, total, workers);

    KvWave<T, D, NG, NT> w;
    KvItem it = kv_locate(a, line, x0, lane);
    int t0 = x0 == it.begin ? 0 : kv_cut(a, it.begin, it.tiles, x0);
    while (true) {
        const int t1 = x1 >= it.end ? it.tiles : kv_cut(a, it.begin, it.tiles, x1);
        if (t0 < t1) {
            const int first = kv_first_token(a, it.len, it.n) / kKvTile;
            w.start(a, it.head, it.r0, it.n, it.len, 0, lane);
            const int minpos = a.causal ? it.len - it.n : it.len - 1;
            const int maxlow = a.window ? it.len - a.window : 0;
            w.run(a, a.s.table + static_cast<int64_t>(it.b) * a.s.max_pages, it.head, first + t0, first + t1,
                  kv_lowest(a, it.len, it.n), it.len, minpos, maxlow, lane, &pairs);
            const bool direct = t0 == 0 && t1 == it.tiles;
            if (direct) {
                w.finish(a, it.head, it.r0, it.n, 0, lane);
            } else {
                const int64_t at = kv_piece(a, worker, t0 == 0);
                w.keep(a.part_ml + 2 * at, a.part + at * D, it.n * a.per, 0, lane);
            }
            if (t0 == 0 && a.items && lane == 0) {
                // pieces: this worker's and those of the workers whose start cuts the item, the
                // last of them the last that starts before it.end - a.snap
                const int last = static_cast<int>((static_cast<int64_t>(it.end - a.snap) * workers + total - 1) / total) - 1;
                a.items[it.b * a.c.heads + it.head] = direct ? make_int2(0, 0) : make_int2(worker, last - worker + 1);
            }
        }
        if (it.end >= x1) return;
        it = kv_locate(a, line, it.end, lane);
        t0 = 0;
    }
}

// Joins the pieces of CH channels of one item's column: blockIdx = (item, column, channels).
// CH/4 threads hold the channels, and 1024/CH groups of them take every (1024/CH)th
// piece; the groups join in LDS.
template <typename T, int D, int CH>
__global__ __launch_bounds__(256) void kv_merge_kernel(KvAttend a) {
    constexpr int kLanes = CH / 4, kGroups = 256 / kLanes;
    const int item = blockIdx.x, col = blockIdx.y;
    int2 it = a.items[item];
    if (it.y <= 0 || it.x < 0 || it.x >= a.workers) return;
    it.y = it.y < a.workers - it.x ? it.y : a.workers - it.x;   // (inside, should tables change under the call)
    const int b = item / a.c.heads, head = item - b * a.c.heads;
    int r0, n;
    kv_rows(a.s, b, r0, n);
    if (n == 0 || static_cast<int64_t>(n) * a.per > a.split_cols || col >= n * a.per) return;
    const int x = threadIdx.x % kLanes, d = blockIdx.z * CH + 4 * x, group = threadIdx.x / kLanes;
    float top = -INFINITY, sum = 0.0f;
    floatx4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    auto join = [&](float m, float l, floatx4 z) {
        const float now = fmaxf(top, m);
        const float f0 = top == now ? 1.0f : __builtin_amdgcn_exp2f(top - now);
        const float f1 = m == now ? 1.0f : __builtin_amdgcn_exp2f(m - now);
        sum = sum * f0 + l * f1;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = y[r] * f0 + z[r] * f1;
        top = now;
    };
    constexpr int kAhead = 8;   // pieces in flight
    for (int k0 = group; k0 < it.y; k0 += kAhead * kGroups) {
        float2 ml[kAhead];
        floatx4 z[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i * kGroups;
            if (k >= it.y) break;
            const int64_t at = kv_piece(a, it.x + k, k == 0) + col;
            ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + at * 2);
            z[i] = *reinterpret_cast<const floatx4 *>(a.part + at * D + d);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k0 + i * kGroups >= it.y) break;
            join(ml[i].x, ml[i].y, z[i]);
        }
    }
    __shared__ floatx4 ys[kGroups][kLanes];
    __shared__ float2 mls[kGroups];
    for (int half = kGroups / 2; half > 0; half >>= 1) {
        if (group >= half && group < 2 * half) {
            ys[group][x] = y;
            if (x == 0) mls[group] = make_float2(top, sum);
        }
        __syncthreads();
        if (group < half) join(mls[group + half].x, mls[group + half].y, ys[group + half][x]);
    }
    if (group != 0) return;
    const int i = col / a.per, h = head * a.per + col - i * a.per;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *dst = static_cast<T *>(a.O) + (r0 + i) * a.o_stride + static_cast<int64_t>(h) * D + d;
    *reinterpret_cast<uint2 *>(dst) = pack4<T>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && d == 0)
        a.lse[static_cast<int64_t>(r0 + i) * a.q_heads + h] = kv_lse(top, sum);
}

// ---------------------------------------------------------------------------
// Wide path: sequences with more columns (prompts, chunks).
//
// A workgroup takes a unit, kv_wide_cols(D) columns of a sequence (rows x query
// heads of one key head, 32 a wave), over the tokens they see, in tiles of
// kv_wide_tile(D).  Where units are few, they form a line that one workgroup a CU
// shares equally, as on the split path (a unit costs kKvWideCost besides its
// tiles); else each has a workgroup of its own, the longest first.  Here the matrix
// cores and the vector work under them bound it, so a tile is unpacked once for all
// waves, into LDS, as 16-byte operands of 32x32x16 MFMAs in reading order (every LDS
// access is contiguous); the other half of the double buffer is filled between a
// tile's MFMAs, from loads issued a tile earlier, keys one tile ahead of values.
// The same two layouts serve this MFMA: result rows 8a + 4h + r of a lane are
// 4-token blocks, too.
//
// Measured: a causal prompt of 4096 rows, 32 query heads on 8 of 128, 172 to 190 us
// (0.72 to 0.80 PFLOP/s): the matrix cores are busy 35% of the cycles, the vector units 50%
// and LDS 43%; a wave waits for operands, loads and barriers 33% of its time and for its
// turn to issue 25%.  Two waves a SIMD beat one of 64 columns (187 and 269 us).  At dim 256 the
// output of 32 columns fills half the registers, so a SIMD has one wave: it issues
// (~740 instructions a tile, 32 of them MFMAs) 62% of its time and waits 29%, with no other
// to fill in (5 ragged chunks of up to 1031 rows over 6007 tokens: 300 us; MFMA 17%, VALU
// 36%, LDS 32%); two waves of 16 columns read every operand twice and took 337.

template <typename T>
struct KvWideType;
template <>
struct KvWideType<__bf16> {
    static __device__ __forceinline__ floatx16 mfma(uint4 a, bf16x8 b, floatx16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
    }
};
template <>
struct KvWideType<_Float16> {
    static __device__ __forceinline__ floatx16 mfma(uint4 a, half8 b, floatx16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), b, c, 0, 0, 0);
    }
};

constexpr int kv_wide_threads(int dim) { return 2 * kv_wide_cols(dim); }

// Unit u: a sequence's columns col0 .. (kv_wide_cols(D) of them at most), and the
// tiles t0 .. t1-1 that some of them see (one at least, so that every unit is visited).
struct KvUnit {
    int b, r0, n, len, col0, t0, t1;
};
template <int D>
__device__ __forceinline__ bool kv_unit(const KvAttend &a, int u, KvUnit &x) {
    constexpr int kCols = kv_wide_cols(D), TT = kv_wide_tile(D);
    int k;
    if (a.s.row_start) {
        x.b = kv_unit_sequence(a.s, u, a.per, kCols, 1);
        k = u - kv_unit_first(a.s, x.b, a.per, kCols, 1);
    } else {
        const int each = a.units / a.s.B;
        x.b = u / each;
        k = u - x.b * each;
    }
    kv_rows(a.s, x.b, x.r0, x.n);
    const int64_t cols = static_cast<int64_t>(x.n) * a.per;
    if (cols <= a.split_cols || k < 0 || static_cast<int64_t>(k) * kCols >= cols) return false;
    x.col0 = k * kCols;
    x.len = kv_length(a.s, x.b, a.c.page_shift);
    const int p0 = x.len - x.n, last = static_cast<int>(cols) - 1;
    const int end = x.col0 + kCols - 1 < last ? x.col0 + kCols - 1 : last;
    const int lo = a.window ? p0 + x.col0 / a.per - a.window + 1 : 0, hi = a.causal ? p0 + end / a.per + 1 : x.len;
    x.t0 = lo > 0 ? lo / TT : 0;
    x.t1 = hi > 0 ? (hi + TT - 1) / TT : 0;
    if (x.t1 <= x.t0) x.t1 = x.t0 + 1;
    return true;
}
// The tile at which a boundary `at` behind an item's begin cuts it (0 or tiles: not inside).
__device__ __forceinline__ int kv_wide_cut(int at, int tiles) {
    const int t = at - kKvWideCost;
    if (t <= kKvWideSnap) return 0;
    return tiles - t <= kKvWideSnap ? tiles : t;
}

// What a thread unpacks of one tile: KW key words of one token (and one of its
// pairs), VI pieces of 8 tokens x 2 channels of the values.
// Everything is loaded whether the token exists or not (from page 0 where it has
// none), so the loop that calls this has no branches for it.
template <int D, int NG, int THREADS>
struct KvWideLoad {
    static constexpr int J = D / 32, TT = kv_wide_tile(D), KW = TT * D / 8 / THREADS, VI = TT * D / 16 / THREADS;
    // What is done under each MFMA of the second product: the key words and pairs in the first
    // KW + 1 slots, then the 4 parts of each value piece, evenly spread; a piece's pairs are read
    // at the end of the slot before its first part.  -1: none in this slot.
    static constexpr int kSlots = TT / 32 * (D / 16), kFirst = KW + 1, kEach = (kSlots - kFirst - 3) / (4 * VI);
    static constexpr int part_at(int slot) {
        const int x = slot - kFirst;
        return x >= 0 && x % kEach == 0 && x / kEach < 4 * VI ? x / kEach : -1;
    }
    static constexpr int pairs_at(int slot) { return part_at(slot + 1) >= 0 && part_at(slot + 1) % 4 == 0 ? part_at(slot + 1) / 4 : -1; }
    static constexpr int kLoad = kFirst + kEach * (4 * VI - 1) + 1;   // the slot of the next loads, behind the last part
    uint32_t k[KW], kp, vp, v[VI][2];
    int k_id, v_id[VI];   // page numbers of the next tile, as the table holds them
    bool k_ok;
    uint32_t v_there;        // all ones where this lane's token exists and some row sees it
    uint4 pair[2];           // of the 8 tokens of a value piece being unpacked
    uint32_t lo[4], hi[4];
    int pair_from, pair_to, lost_to;

    // Where this lane's pairs come from and go, and the wave's mark of missing keys;
    // lanes and waves that have none write behind the others'.  (Opaque, or they
    // become branches in the loop.)
    __device__ __forceinline__ void init() {
        pair_from = ((threadIdx.x & 15) * NG + (chunk() < NG ? chunk() : 0)) * 4;
        pair_to = chunk() < NG ? chunk() * TT + token() : NG * TT;
        lost_to = chunk() == 0 ? key_block() : TT / 16;
        asm("" : "+v"(pair_from), "+v"(pair_to), "+v"(lost_to));
    }
    // The keys' 16-token block and the values' (u) are one for a wave, so pages,
    // their checks and addresses cost scalar instructions only.
    static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
    static __device__ __forceinline__ int key_block() { return wave() % (TT / 16); }
    static __device__ __forceinline__ int token() { return 16 * key_block() + (threadIdx.x & 15); }
    static __device__ __forceinline__ int chunk() { return ((threadIdx.x >> 4) & 3) + 4 * (wave() / (TT / 16)); }
    static __device__ __forceinline__ void piece(int i, int &m, int &b, int &h, int &u) {
        const int x = threadIdx.x + THREADS * i;
        m = x & 15, b = (x >> 4) % J, h = (x / (16 * J)) & 1, u = __builtin_amdgcn_readfirstlane(x / (32 * J));
    }
    // (A vector load: a scalar one in flight would make every
    // wait for an LDS operand a wait for all of them.)
    static __device__ __forceinline__ int id_of(const KvAttend &a, const int32_t *table, int tok, int len) {
        int at = (tok < len ? tok : len > 0 ? len - 1 : 0) >> a.c.page_shift;
        asm("" : "+v"(at));
        return table[at];
    }
    static __device__ __forceinline__ const unsigned char *block(const KvAttend &a, int head, int id, int tok, int len,
                                                                 bool &ok) {
        id = __builtin_amdgcn_readfirstlane(id);
        ok = (tok < len) & (id >= 0) & (id < a.c.n_pages);   // (no short circuit: no branches)
        return a.c.pages + (id & -static_cast<int>(ok)) * a.c.page_stride + head * a.c.block;
    }

    __device__ __forceinline__ void key_page(const KvAttend &a, const int32_t *table, int tok, int len) {
        k_id = id_of(a, table, tok + 16 * key_block(), len);
    }
    __device__ __forceinline__ void value_pages(const KvAttend &a, const int32_t *table, int tok, int len) {
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            int m, b, h, u;
            piece(i, m, b, h, u);
            v_id[i] = id_of(a, table, tok + 16 * u, len);
        }
    }

    // Keys, and both pairs of this lane's token.
    __device__ __forceinline__ void load_keys(const KvAttend &a, int head, int tok, int lowest, int len) {
        const int P = 1 << a.c.page_shift, at = tok + 16 * key_block(), slot = at & (P - 1), n = threadIdx.x & 15;
        const unsigned char *p = block(a, head, k_id, at, len, k_ok);
        load_words<KW>(p + slot * (D / 2) + static_cast<uint32_t>(n * (D / 2) + chunk() * (4 * KW)), k);
        const unsigned char *r = p + P * D + slot * (4 * NG);
        kp = *reinterpret_cast<const uint32_t *>(r + static_cast<uint32_t>(pair_from));
        vp = *reinterpret_cast<const uint32_t *>(r + P * (4 * NG) + static_cast<uint32_t>(pair_from));
        // a value that does not exist, or that no row sees, is worth zero (0 * NaN would not vanish)
        v_there = kv_seen(at + n, lowest, len) && k_ok ? ~0u : 0u;
    }
    __device__ __forceinline__ void load_values(const KvAttend &a, int head, int tok, int len) {
        const int P = 1 << a.c.page_shift;
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            int m, b, h, u;
            piece(i, m, b, h, u);
            bool ok;
            const int slot = (tok + 16 * u) & (P - 1);
            const unsigned char *q = block(a, head, v_id[i], tok + 16 * u, len, ok) + P * (D / 2) + slot * (D / 2);
            const uint32_t at = (h * 16 + m) * (D / 8) + 4 * b;
            v[i][0] = *reinterpret_cast<const uint32_t *>(q + at);
            v[i][1] = *reinterpret_cast<const uint32_t *>(q + 4 * D + at);
        }
    }

    // Key word i into ks[octet of channels][token].
    template <typename T>
    __device__ __forceinline__ void unpack_key(int i, uint4 *ks) const {
        const int w = chunk() * KW + i, octet = 4 * (w % J) + w / J;
        ks[octet * TT + token()] = make_uint4(KvType<T>::pair(k[i], 0), KvType<T>::pair(k[i], 1),
                                              KvType<T>::pair(k[i], 2), KvType<T>::pair(k[i], 3));
    }
    // Into pairs[group][token] (key factors), vpairs[group][token] and lost[16 tokens].
    template <typename T>
    __device__ __forceinline__ void unpack_pair(const KvAttend &a, float2 *pairs, uint32_t *vpairs, int *lost) const {
        pairs[pair_to] = key_factors(kp, a.scale_log2);
        vpairs[pair_to] = vp & v_there;
        lost[lost_to] = !k_ok;
    }
    // The pairs of value piece i, out of vpairs.
    __device__ __forceinline__ void read_pairs(int i, const uint32_t *vpairs) {
        int m, b, h, u;
        piece(i, m, b, h, u);
        const uint4 *p = reinterpret_cast<const uint4 *>(vpairs + b * NG / J * TT + 16 * u + 4 * h);
        pair[0] = p[0];
        pair[1] = p[2];
    }
    // Part 0..3 of value piece i: tokens (0, 2) or (1, 3) of one 4-token block; after
    // the last, into vs[16 tokens][h][b][channel of 32].
    __device__ __forceinline__ void unpack_value(int i, int part, uint4 *vs) {
        const int e = part >> 1, t = part & 1;
        const uint32_t q0 = t ? pair[e].y : pair[e].x, q2 = t ? pair[e].w : pair[e].z;
        const half2v s = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(q2, q0, 0x05040100u));
        const half2v l = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(q2, q0, 0x07060302u));
        half2v cl, ch;
        value_codes(v[i][e] >> (8 * t), cl, ch);
        lo[part] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(cl, s, l));
        hi[part] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(ch, s, l));
        if (part < 3) return;
        int m, b, h, u;
        piece(i, m, b, h, u);
        uint4 *dst = vs + ((u * 2 + h) * J + b) * 32 + m;
        dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        dst[16] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
};

template <typename T, int D, int NG>
__device__ __forceinline__ void kv_wide_piece(const KvAttend &a, const KvUnit &unit, int head, int t0, int t1, int piece,
                                              uint4 (&ks)[2][1024], uint4 (&vs)[2][1024],
                                              float2 (&pairs)[3][NG * kv_wide_tile(D) + 1],
                                              uint32_t (&vpairs)[2][NG * kv_wide_tile(D) + 4],
                                              int (&lost)[3][kv_wide_tile(D) / 16 + 1]) {
    constexpr int kCols = kv_wide_cols(D), kThreads = kv_wide_threads(D), J = D / 32, TT = kv_wide_tile(D), S = D / 16;
    constexpr int SUB = TT / 32;   // result tiles of 32 tokens x 32 columns a wave
    const int lane = threadIdx.x & 63, n32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r0 = unit.r0, n = unit.n, len = unit.len, p0 = len - n, lowest = kv_lowest(a, len, n);
    const int last_col = n * a.per - 1, col0 = unit.col0 + wave * 32;
    const int32_t *table = a.s.table + static_cast<int64_t>(unit.b) * a.s.max_pages;
    auto row_of = [&](int c) { return (c < last_col ? c : last_col) / a.per; };
    // where nothing is hidden from the wave's columns
    const int minpos = a.causal ? p0 + row_of(col0) : len - 1;
    const int maxlow = a.window ? p0 + row_of(col0 + 31) - a.window + 1 : 0;

    // this lane's column: its queries, their sums, its visible positions
    typedef typename KvType<T>::vec8 vec8;
    const int col = col0 + n32, row = col / a.per;
    const bool real = row < n;
    const int pos = real ? (a.causal ? p0 + row : len - 1) : -1, low = a.window ? p0 + row - a.window + 1 : 0;
    vec8 q[S];
    // Scores x are formed relative to ref: m, but no less than -kFloorLog2, and 0 before there is one.  Where m is
    // lower, limit sends every tile through the shift to m.  (x carries 2^-24 of its distance from ref: relative
    // to an m of -1000, later scores around 0 put lse off by 1e-5; now it is 2^-24 * (|S| + kFloorLog2) at most.)
    float qs[NG], m = -INFINITY, l = 0.0f, top = -INFINITY, ref = 0.0f, limit = -INFINITY;
    floatx16 o[J];
    {
        const T *src = static_cast<const T *>(a.Q) + (r0 + (real ? row : 0)) * a.q_stride +
                       static_cast<int64_t>(head * a.per + (col - row * a.per)) * D + 8 * h;
#pragma unroll
        for (int g = 0; g < NG; ++g) qs[g] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            vec8 x = {};
            if (real) x = *reinterpret_cast<const vec8 *>(src + 16 * s);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += static_cast<float>(x[e]);
            qs[s * NG / S] += sum;
            if (D > 128) asm("" : "+a"(x));   // (where the output fills the other registers)
            q[s] = x;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) qs[g] += __shfl_xor(qs[g], 32);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[j][r] = 0.0f;
    }

    // Both products are kSlots MFMAs a tile, each in a slot of its own: the operand
    // of some slots on is read from LDS, one MFMA issued, and a share of the tile's
    // vector work done under it.  (The slots are fenced: left to itself the
    // scheduler puts each read right before its MFMA and the vector work behind all.)
    constexpr int kSlots = SUB * S, kAhead = 4;
    static_assert(2 * SUB * J == kSlots && kSlots >= 2 * kAhead, "");
    // The next tile's scores: one group's sums of (base + code) * q (NG = 1), or the
    // scores themselves, into which the groups' sums are folded as they come.
    floatx16 next[SUB], part[2];
    uint4 f[kAhead];
    // operand i of the first product: with one group the result tiles alternate, else
    // the groups of one result tile follow each other
    auto key_operand = [&](int i, int &e, int &k) {
        if (NG == 1)
            e = i % SUB, k = i / SUB;
        else
            e = i / S, k = i % S;
    };
    auto read_key = [&](int t, int i) {
        int e, k;
        key_operand(i, e, k);
        return ks[t & 1][(2 * k + h) * TT + 32 * e + n32];
    };
    auto factors = [&](int t3, int g, int i) {   // of tokens 2i, 2i + 1 of a lane's 8 * SUB
        const float2 *kp = &pairs[t3][g * TT + 32 * (i / 8) + 4 * h + 8 * (i % 8 >> 1) + 2 * (i & 1)];
        return floatx4{kp[0].x, kp[0].y, kp[1].x, kp[1].y};
    };
    // One group's sums into the scores, in M parts under the next group's MFMAs; a
    // part's factors are read kFoldAhead slots earlier.
    constexpr int M = S / NG, kFold = NG == 1 ? 1 : 8 / M;   // operands of a group; factors of a part
    constexpr int kFoldAhead = M > 2 ? 2 : 1;   // slots (a part of M = 2 has 4 factors)
    floatx4 z[kFoldAhead][kFold];
    auto read_fold = [&](int t3, int i) {   // for operand i's slot: the group before
#pragma unroll
        for (int y = 0; y < kFold; ++y) z[i % kFoldAhead][y] = factors(t3, (i / M - 1) % NG, 8 * ((i / M - 1) / NG) + i % M * kFold + y);
    };
    auto fold = [&](int i) {
        const int e = (i / M - 1) / NG, g = (i / M - 1) % NG;
#pragma unroll
        for (int y = 0; y < kFold; ++y) {
            const floatx4 w = z[i % kFoldAhead][y];
            const floatx16 &sum = part[(i / M - 1) & 1];
            floatx16 &x = next[e];
            const int r = 2 * (i % M * kFold + y);
            x[r] = fmaf(w[0], sum[r], g == 0 ? w[1] * qs[g] : fmaf(w[1], qs[g], x[r]));
            x[r + 1] = fmaf(w[2], sum[r + 1], g == 0 ? w[3] * qs[g] : fmaf(w[3], qs[g], x[r + 1]));
        }
    };
    auto score_slot = [&](int t, int t3, int i) {
        int e, k;
        key_operand(i, e, k);
        const uint4 w = f[i % kAhead];
        if (i + kAhead < kSlots) f[i % kAhead] = read_key(t, i + kAhead);
        if constexpr (NG == 1) {
            next[e] = KvWideType<T>::mfma(w, q[k], k == 0 ? floatx16{} : next[e]);
        } else {
            floatx16 &y = part[(i / M) & 1];
            y = KvWideType<T>::mfma(w, q[k], k % M == 0 ? floatx16{} : y);
            if (i >= M) fold(i);
            if (i + kFoldAhead >= M) read_fold(t3, i + kFoldAhead);
        }
    };
    auto end_scores = [&](int t3) {   // the last group
        if constexpr (NG > 1) {
#pragma unroll
            for (int i = kSlots; i < kSlots + M; ++i) {
                fold(i);
                if (i + kFoldAhead < kSlots + M) read_fold(t3, i + kFoldAhead);
            }
        }
    };
    // The scores less the reference, two tokens at a time, and their maximum.
    floatx16 x[SUB];
    auto relative = [&](floatx4 y, int i) {
        const int e = i / 8, r = i % 8 * 2;
        if constexpr (NG == 1) {
            x[e][r] = fmaf(y[0], next[e][r], fmaf(y[1], qs[0], -ref));
            x[e][r + 1] = fmaf(y[2], next[e][r + 1], fmaf(y[3], qs[0], -ref));
        } else {
            x[e][r] = next[e][r] - ref;
            x[e][r + 1] = next[e][r + 1] - ref;
        }
        const float two = fmaxf(x[e][r], x[e][r + 1]);
        top = i == 0 ? two : fmaxf(top, two);
    };
    auto start_scores = [&](int t) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) f[i] = read_key(t, i);
    };

    KvWideLoad<D, NG, kThreads> in;
    in.init();
    int t3 = t0 % 3;   // t % 3
    if (t0 < t1) {
        // keys and pairs run one tile ahead of values: K(t0), K(t0 + 1), V(t0) into LDS,
        // K(t0 + 2), V(t0 + 1) on their way
        auto keys = [&](int t) {
#pragma unroll
            for (int i = 0; i < in.KW; ++i) in.template unpack_key<T>(i, ks[t & 1]);
            in.template unpack_pair<T>(a, pairs[t % 3], vpairs[t & 1], lost[t % 3]);
        };
        in.key_page(a, table, t0 * TT, len);
        in.value_pages(a, table, t0 * TT, len);
        in.load_keys(a, head, t0 * TT, lowest, len);
        in.load_values(a, head, t0 * TT, len);
        in.key_page(a, table, (t0 + 1) * TT, len);
        in.value_pages(a, table, (t0 + 1) * TT, len);
        keys(t0);
        in.load_keys(a, head, (t0 + 1) * TT, lowest, len);
        in.key_page(a, table, (t0 + 2) * TT, len);
        __syncthreads();   // the pairs of V(t0)
#pragma unroll
        for (int i = 0; i < 4 * in.VI; ++i) {
            if (i % 4 == 0) in.read_pairs(i / 4, vpairs[t0 & 1]);
            in.unpack_value(i / 4, i % 4, vs[t0 & 1]);
        }
        in.load_values(a, head, (t0 + 1) * TT, len);
        in.value_pages(a, table, (t0 + 2) * TT, len);
        keys(t0 + 1);
        in.load_keys(a, head, (t0 + 2) * TT, lowest, len);
        in.key_page(a, table, (t0 + 3) * TT, len);
        __syncthreads();
        start_scores(t0);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) score_slot(t0, t3, i);
        end_scores(t3);
#pragma unroll
        for (int i = 0; i < 8 * SUB; ++i) relative(NG == 1 ? factors(t3, 0, i) : floatx4{}, i);
    }
    for (int t = t0; t < t1; ++t) {
        const int tok = t * TT, buf = t & 1;
        const int n3 = t3 == 2 ? 0 : t3 + 1, w3 = t3 == 0 ? 2 : t3 - 1;   // (t + 1) % 3, (t + 2) % 3
        // K(t + 1) and V(t) are in LDS; K(t) and V(t - 1) have been read
        __syncthreads();
        bool gone[2 * SUB], some_gone = false;
#pragma unroll
        for (int e = 0; e < 2 * SUB; ++e) {
            gone[e] = __builtin_amdgcn_readfirstlane(lost[t3][e]) != 0;
            some_gone |= gone[e];
        }
        if (tok + TT - 1 > minpos || tok < maxlow || some_gone) {
#pragma unroll
            for (int e = 0; e < SUB; ++e)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int p = tok + 32 * e + 8 * (r >> 2) + 4 * h + (r & 3);
                    if (p > pos || p < low || gone[2 * e + (r >> 3)]) x[e][r] = -INFINITY;
                    top = e + r == 0 ? x[0][0] : fmaxf(top, x[e][r]);
                }
        }
        if (__any(top > limit)) {
            float now = fmaxf(m, top + ref - kHeadLog2);
            now = fmaxf(now, __shfl_xor(now, 32));
            const float g = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - now);
            m = now;
            const float back = (now == -INFINITY ? 0.0f : now) - ref;
            ref = now == -INFINITY ? 0.0f : fmaxf(now, -kFloorLog2);
            limit = now < -kFloorLog2 ? -INFINITY : kMostLog2;
            l *= g;
#pragma unroll
            for (int e = 0; e < SUB; ++e)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[e][r] -= back;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // (at D = 256 sums stay in accumulation registers; without this the
                // compiler copies all of them out before the branch, tile after tile)
                if constexpr (D == 256) asm("" : "+a"(o[j]));
#pragma unroll
                for (int r = 0; r < 16; ++r) o[j][r] *= g;
                if constexpr (D == 256) asm("" : "+a"(o[j]));
            }
        }
        // the first product of the next tile (of stale keys after the last one), under it P of this one
        half8 p[2 * SUB];
        constexpr int kOrder[4] = {0, 2, 1, 3};   // of the value bytes
        start_scores(t + 1);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            score_slot(t + 1, n3, i);
            constexpr int kEach = SUB * 16 / kSlots;
#pragma unroll
            for (int z = i * kEach; z < (i + 1) * kEach; ++z) {
                const int e = z / 16, r = z % 16;
                const float y = __builtin_amdgcn_exp2f(x[e][(r & ~3) + kOrder[r & 3]]);
                l += y;
                p[2 * e + (r >> 3)][r & 7] = static_cast<_Float16>(y);
            }
        }
        end_scores(n3);
        // the second product, under it the unpacking of K(t + 2) and V(t + 1), the loads
        // behind them, and what is left to do for the next tile's scores
        floatx4 y[2] = {};
        if (NG == 1) y[0] = factors(n3, 0, 0), y[1] = factors(n3, 0, 1);
        auto read_value = [&](int i) { return vs[buf][((i / J * 2 + h) * J + i % J) * 32 + n32]; };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) f[i] = read_value(i);
#pragma unroll
        for (int slot = 0; slot < kSlots; ++slot) {
            __builtin_amdgcn_sched_barrier(0);
            const uint4 w = f[slot % kAhead];
            if (slot + kAhead < kSlots) f[slot % kAhead] = read_value(slot + kAhead);
            o[slot % J] = KvWideType<_Float16>::mfma(w, p[slot / J], o[slot % J]);
            constexpr int kPairs = 8 * SUB;
#pragma unroll
            for (int z = slot * kPairs / kSlots; z < (slot + 1) * kPairs / kSlots; ++z) {   // (factors read two ahead)
                relative(y[z & 1], z);
                if (NG == 1 && z + 2 < kPairs) y[z & 1] = factors(n3, 0, z + 2);
            }
            if (slot < in.KW) in.template unpack_key<T>(slot, ks[buf]);
            if (slot == in.KW) {
                in.template unpack_pair<T>(a, pairs[w3], vpairs[buf], lost[w3]);
                in.load_keys(a, head, tok + 3 * TT, lowest, len);
            }
            if (in.part_at(slot) >= 0) in.unpack_value(in.part_at(slot) / 4, in.part_at(slot) % 4, vs[buf ^ 1]);
            if (in.pairs_at(slot) >= 0) in.read_pairs(in.pairs_at(slot), vpairs[buf ^ 1]);
            if (slot == in.kLoad) in.load_values(a, head, tok + 2 * TT, len);
            if (slot == kSlots - 1) {
                in.key_page(a, table, tok + 4 * TT, len);
                in.value_pages(a, table, tok + 3 * TT, len);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        t3 = n3;
    }
    l += __shfl_xor(l, 32);
    const int qh = head * a.per + col - row * a.per;
    if (piece >= 0) {   // kept for a join
        const int64_t at = static_cast<int64_t>(piece) * kCols + wave * 32 + n32;
        if (h == 0) *reinterpret_cast<float2 *>(a.wide_ml + 2 * at) = make_float2(m, l);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<floatx4 *>(a.wide_part + at * D + 32 * j + 8 * e + 4 * h) =
                    floatx4{o[j][4 * e], o[j][4 * e + 1], o[j][4 * e + 2], o[j][4 * e + 3]};
    } else if (real) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T *dst = static_cast<T *>(a.O) + (r0 + row) * a.o_stride + static_cast<int64_t>(qh) * D + 4 * h;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint2 *>(dst + 32 * j + 8 * e) = pack4<T>(
                    o[j][4 * e] * inv, o[j][4 * e + 1] * inv, o[j][4 * e + 2] * inv, o[j][4 * e + 3] * inv);
        if (a.lse && h == 0)
            a.lse[static_cast<int64_t>(r0 + row) * a.q_heads + qh] = kv_lse(m, l);
    }
}

template <typename T, int D, int NG>
__global__ __launch_bounds__(kv_wide_threads(D)) void kv_wide_kernel(KvAttend a) {
    constexpr int kThreads = kv_wide_threads(D), TT = kv_wide_tile(D);
    __shared__ uint4 ks[2][1024], vs[2][1024];
    __shared__ float2 pairs[3][NG * TT + 1];
    __shared__ __align__(16) uint32_t vpairs[2][NG * TT + 4];
    __shared__ int lost[3][TT / 16 + 1];
    __shared__ int before[kKvLineUnits + 1];   // line mode: tiles (and costs) of one head of the units before
    __shared__ uint16_t order[kKvLineUnits];   // the units, longest first
    __shared__ int jobs, span;                 // whole units to hand out instead of the line (0: none), and their time
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.c.heads;
    if (a.line) {
        for (int i = tid; i < a.units; i += kThreads) {
            KvUnit unit;
            before[i + 1] = kv_unit<D>(a, i, unit) ? unit.t1 - unit.t0 + kKvWideCost : 0;
        }
        if (tid == 0) before[0] = jobs = span = 0;
        __syncthreads();
        if (wave == 0) {   // prefix sums, 64 units at a time
            int sum = 0;
            for (int i = 0; i < a.units; i += 64) {
                int v = i + lane < a.units ? before[i + lane + 1] : 0;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int up = __shfl_up(v, d);
                    if (lane >= d) v += up;
                }
                if (i + lane < a.units) before[i + lane + 1] = sum + v;
                sum += __builtin_amdgcn_readlane(v, 63);
            }
        }
        __syncthreads();
        // Pieces cost time: their sums go through memory and a join.  Where whole units,
        // the longest first, take at most 6/5 of the line's share, they are handed out
        // instead: the first kKvCus to a CU each, the (kKvCus + i)th behind the
        // (kKvCus - 1 - i)th.  (6 ragged prompts of up to 6000 tokens, 94 tiles to a CU on
        // the line and 97 without: 278 us on the line, 263 us without; one of 2400 rows
        // over 4096, 59 tiles and 73: 176 us both ways.)
        auto length = [&](int i) { return before[i + 1] - before[i]; };
        for (int i = tid; i < a.units; i += kThreads) {
            const int mine = length(i);
            int rank = 0;
            for (int j = 0; j < a.units; ++j) rank += length(j) > mine || (length(j) == mine && j < i) ? 1 : 0;
            order[rank] = static_cast<uint16_t>(i);
            if (mine > 0) atomicAdd(&jobs, H);
        }
        __syncthreads();
        for (int i = tid; i < kKvCus; i += kThreads) {
            const int first = kKvCus - 1 - i, second = kKvCus + i;
            const int time = (first < jobs ? length(order[first / H]) : 0) + (second < jobs ? length(order[second / H]) : 0);
            atomicMax(&span, time);
        }
        __syncthreads();
        if (tid == 0 && 5 * static_cast<int64_t>(span) * a.wide_workers > 6 * static_cast<int64_t>(H) * before[a.units]) jobs = 0;
        __syncthreads();
    }

    // A piece at a time: unit u's tiles t0 .. t1-1 for one head.  (What the line needs is
    // worked out anew for each, so that no register holds it meanwhile.)
    for (int next_at = -1;;) {
        KvUnit unit;
        int head, t0, t1, piece = 0;
        bool whole = true, more = false;
        if (a.line) {
            const int all = __builtin_amdgcn_readfirstlane(before[a.units]), total = H * all;
            const int most = total / kKvWideMinShare > 1 ? total / kKvWideMinShare : 1;
            const int workers = a.wide_workers < most ? a.wide_workers : most;
            const int whole_jobs = __builtin_amdgcn_readfirstlane(jobs);
            if (static_cast<int>(blockIdx.x) >= (whole_jobs > 0 ? whole_jobs : workers) || total == 0) return;
            // Workgroups go round the 8 XCDs; neighbours on the line, which read the same
            // keys, get one XCD (and its L2).
            const int xcd = blockIdx.x & 7, rest = workers & 7;
            const int worker = xcd * (workers >> 3) + (xcd < rest ? xcd : rest) + (blockIdx.x >> 3);
            int x0 = static_cast<int>(static_cast<int64_t>(worker) * total / workers);
            int x1 = static_cast<int>((static_cast<int64_t>(worker) + 1) * total / workers);
            if (whole_jobs > 0) {   // this workgroup's unit, whole
                const int u = __builtin_amdgcn_readfirstlane(order[blockIdx.x / H]);
                x0 = (blockIdx.x % H) * all + __builtin_amdgcn_readfirstlane(before[u]);
                x1 = x0 + __builtin_amdgcn_readfirstlane(before[u + 1] - before[u]);
            }
            const int at = next_at < 0 ? x0 : next_at;
            head = kv_clamp(at / all, 0, H - 1);
            int lo = 0, hi = a.units;   // the last unit of the head that begins at or before it
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (head * all + __builtin_amdgcn_readfirstlane(before[mid]) <= at)
                    lo = mid;
                else
                    hi = mid;
            }
            const int item = head * all + __builtin_amdgcn_readfirstlane(before[lo]);
            const int length = __builtin_amdgcn_readfirstlane(before[lo + 1] - before[lo]), tiles = length - kKvWideCost;
            if (length <= 0 || !kv_unit<D>(a, lo, unit)) return;   // (not unless the tables change under the call)
            const int end = item + length;
            const int c0 = next_at < 0 ? kv_wide_cut(at - item, tiles) : 0;
            const int c1 = x1 >= end ? tiles : kv_wide_cut(x1 - item, tiles);
            whole = c0 == 0 && c1 == tiles;
            more = end < x1;
            next_at = end;
            if (c0 == 0 && c1 > 0 && a.wide_items && tid == 0) {   // (as in kv_split_kernel)
                const int last = static_cast<int>((static_cast<int64_t>(end - kKvWideSnap) * workers + total - 1) / total) - 1;
                a.wide_items[lo * H + head] = whole ? make_int2(0, 0) : make_int2(worker, last - worker + 1);
            }
            if (c0 >= c1) {   // all of it belongs to another workgroup
                if (!more) return;
                continue;
            }
            t0 = unit.t0 + c0;
            t1 = unit.t0 + c1;
            piece = 2 * worker + (c0 == 0 ? 1 : 0);
            __syncthreads();   // the piece before is done with LDS
        } else {
            head = blockIdx.x % H;
            if (!kv_unit<D>(a, a.units - 1 - blockIdx.x / H, unit)) return;   // (the longest first)
            t0 = unit.t0;
            t1 = unit.t1;
        }
        kv_wide_piece<T, D, NG>(a, unit, head, t0, t1, whole ? -1 : piece, ks, vs, pairs, vpairs, lost);
        if (!more) return;
    }
}

// Joins the pieces of one (unit, head), blockIdx.x: D/4 threads a column.
template <typename T, int D>
__global__ __launch_bounds__(256) void kv_wide_merge_kernel(KvAttend a) {
    constexpr int kLanes = D / 4, kPer = 256 / kLanes, kCols = kv_wide_cols(D);
    const int item = blockIdx.x, u = item / a.c.heads, head = item - u * a.c.heads;
    KvUnit unit;
    if (!kv_unit<D>(a, u, unit)) return;
    int2 it = a.wide_items[item];
    if (it.y <= 0 || it.x < 0 || it.x >= a.wide_workers) return;
    it.y = it.y < a.wide_workers - it.x ? it.y : a.wide_workers - it.x;   // (as in kv_merge_kernel)
    const int d = 4 * (threadIdx.x % kLanes);
    const int c = blockIdx.y * kPer + threadIdx.x / kLanes, col = unit.col0 + c, row = col / a.per;
    if (row >= unit.n) return;
    float top = -INFINITY, sum = 0.0f;
    floatx4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kAhead = 4;   // pieces in flight
    for (int k0 = 0; k0 < it.y; k0 += kAhead) {
        float2 ml[kAhead];
        floatx4 z[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k0 + i >= it.y) break;
            const int64_t at = (static_cast<int64_t>(it.x + k0 + i) * 2 + (k0 + i == 0 ? 1 : 0)) * kCols + c;
            ml[i] = *reinterpret_cast<const float2 *>(a.wide_ml + at * 2);
            z[i] = *reinterpret_cast<const floatx4 *>(a.wide_part + at * D + d);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k0 + i >= it.y) break;
            const float now = fmaxf(top, ml[i].x);
            const float f0 = top == now ? 1.0f : __builtin_amdgcn_exp2f(top - now);
            const float f1 = ml[i].x == now ? 1.0f : __builtin_amdgcn_exp2f(ml[i].x - now);
            sum = sum * f0 + ml[i].y * f1;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = y[r] * f0 + z[i][r] * f1;
            top = now;
        }
    }
    const int h = head * a.per + col - row * a.per;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *dst = static_cast<T *>(a.O) + (unit.r0 + row) * a.o_stride + static_cast<int64_t>(h) * D + d;
    *reinterpret_cast<uint2 *>(dst) = pack4<T>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && d == 0)
        a.lse[static_cast<int64_t>(unit.r0 + row) * a.q_heads + h] = kv_lse(top, sum);
}

// ---------------------------------------------------------------------------

template <typename T, int D, int NG>
hipError_t kv_attend_typed(const KvAttend &a, bool run_split, bool run_wide, bool merge, hipStream_t st) {
    if (run_split) {
        const dim3 grid(static_cast<unsigned>(a.workers)), threads(64);
        if (a.tiles_col == 1)
            hipLaunchKernelGGL((kv_split_kernel<T, D, NG, 1>), grid, threads, 0, st, a);
        else if (a.tiles_col == 2)
            hipLaunchKernelGGL((kv_split_kernel<T, D, NG, 2>), grid, threads, 0, st, a);
        else if constexpr (D < 256)   // (awq_kv.hip takes at most 2 column tiles at 256 channels)
            hipLaunchKernelGGL((kv_split_kernel<T, D, NG, 4>), grid, threads, 0, st, a);
        const int64_t columns = static_cast<int64_t>(a.s.B) * a.c.heads * a.split_cols;
        if (merge && columns <= kKvMergeFew)
            hipLaunchKernelGGL((kv_merge_kernel<T, D, 32>), dim3(a.s.B * a.c.heads, a.split_cols, D / 32), dim3(256), 0, st, a);
        else if (merge)
            hipLaunchKernelGGL((kv_merge_kernel<T, D, D>), dim3(a.s.B * a.c.heads, a.split_cols), dim3(256), 0, st, a);
    }
    if (run_wide) {
        hipLaunchKernelGGL((kv_wide_kernel<T, D, NG>), dim3(a.line && a.wide_workers > a.units * a.c.heads ? a.wide_workers : a.units * a.c.heads),
                           dim3(kv_wide_threads(D)), 0, st, a);
        if (a.wide_items)
            hipLaunchKernelGGL((kv_wide_merge_kernel<T, D>), dim3(a.units * a.c.heads, kv_wide_cols(D) / (1024 / D)),
                               dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

template <int D, int NG>
hipError_t kv_attend_group(const KvAttend &a, int type, bool run_split, bool run_wide, bool merge, hipStream_t st) {
    if (type == 1) return kv_attend_typed<__bf16, D, NG>(a, run_split, run_wide, merge, st);
    return kv_attend_typed<_Float16, D, NG>(a, run_split, run_wide, merge, st);
}

}  // namespace
}  // namespace awq
