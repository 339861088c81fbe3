// Device code that the kernels writing the 4-bit key/value cache share (k_kv.hip,
// k_kv_rotate.hip): vector loads and stores, where a unit's tokens go, the quantiser
// and the stores of a unit (definitions: k_kv.hip; layout: kv_internal.h).
#pragma once

#include "kv_internal.h"

namespace awq {
namespace {

constexpr int kKvThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *x);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float *x) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__bf16>(const __bf16 *p, float *x) {
    const bf16x8 v = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
}
template <>
__device__ __forceinline__ void load8<_Float16>(const _Float16 *p, float *x) {
    const half8 v = *reinterpret_cast<const half8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float *x);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float *x) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__bf16>(__bf16 *p, const float *x) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<__bf16>(x[i]);
    *reinterpret_cast<bf16x8 *>(p) = v;
}
template <>
__device__ __forceinline__ void store8<_Float16>(_Float16 *p, const float *x) {
    half8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<_Float16>(x[i]);
    *reinterpret_cast<half8 *>(p) = v;
}

// Where a unit's tokens go, or come from.
struct Place {
    int row;               // this lane's row of the call's tensors, -1: none
    unsigned char *block;  // the (page, head) block of the unit's 4 positions, NULL: there is none
    int slot;              // this lane's token within the page
};

// The place of a unit's token: row first, so that its loads can leave before the page's
// number is there.  `unit` is one for LU lanes (32 at least); all lanes of the wave call.
template <int LU>
struct Finder {
    int b, base;
    Place p{-1, nullptr, 0};

    __device__ __forceinline__ void row(const KvCache &c, const KvBatch &s, int unit, int units, int units_even, int token) {
        int k;
        b = 0;
        base = -1;
        if (s.row_start) {
            const int lane = threadIdx.x & 63, u0 = __builtin_amdgcn_readlane(unit, 0);
            b = kv_wave_sequence(s, u0, lane);
            if constexpr (LU < 64) {
                const int u1 = __builtin_amdgcn_readlane(unit, 32);
                const int b1 = u1 == u0 ? b : kv_wave_sequence(s, u1, lane);
                b = lane < 32 ? b : b1;
            }
            k = unit - kv_unit_first(s, b, 1, 4, 2);
        } else {
            if (unit >= units) return;
            b = unit / units_even;
            k = unit - b * units_even;
        }
        int r0, n;
        kv_rows(s, b, r0, n);
        const int first = kv_length(s, b, c.page_shift) - n;   // position of the first new row (may be negative)
        const int at = ((first >> 2) + k) * 4;                 // (arithmetic shift: floor)
        if (unit >= units || k < 0 || n == 0 || at >= first + n) return;   // (at + 3 >= first for every k >= 0)
        const int i = at + token - first;
        if (i >= 0 && i < n) p.row = r0 + i;
        base = at;
    }
    __device__ __forceinline__ void page(const KvCache &c, const KvBatch &s, int head, int token) {
        if (base < 0) return;
        // base < first + n <= the table's span, and 4 aligned positions share a page
        const int id = s.table[static_cast<int64_t>(b) * s.max_pages + (base >> c.page_shift)];
        if (id < 0 || id >= c.n_pages) return;
        p.block = c.pages + id * c.page_stride + head * c.block;
        p.slot = (base & ((1 << c.page_shift) - 1)) + token;
    }
};

// Nibble of channel i in a word of 8 codes: values' are in channel order, keys' are
// stored in the order 0,2,4,6,1,3,5,7.
__device__ __forceinline__ constexpr int key_nibble(int i) { return (i >> 1) + 4 * (i & 1); }

// Codes, as 8 nibbles of one word, and the group's pair (step, lowest) as fp16 bits.
// The lanes of a group are GL neighbours.  fits: the lane's 8 values are within
// +-kKvMaxAbs (their sum finds a NaN, which the minimum and maximum leave out).
//
// The quotients are IEEE's, from one reciprocal r = RN(1/step): q0 = RN(d*r) is off by
// less than 1.5 ulp, e = d - q0*step is exact, and q0 + e*r differs from d/step by
// less than 2^-23 ulp.  step has 11 bits, so d/step is no tie of 24-bit floats and is
// 2^-12 ulp or more from every one: both round alike.  (Where e underflows, the code
// is 0 either way.)  (With 16 divisions a lane the append of 25 MB took 16.5 us.)
// Four codes join as the float c0 + 16*c1 + 256*c2 + 4096*c3, exact below 2^24.
template <int GL, bool KEY>
__device__ __forceinline__ uint32_t quantise(const float *x, uint32_t &pair, bool &fits) {
    float lo = x[0], hi = x[0], sum = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]), sum += x[i];
    fits = (lo >= -kKvMaxAbs) & (hi <= kKvMaxAbs) & (sum == sum);
#pragma unroll
    for (int m = 1; m < GL; m <<= 1) lo = fminf(lo, __shfl_xor(lo, m)), hi = fmaxf(hi, __shfl_xor(hi, m));
    const _Float16 lo16 = static_cast<_Float16>(lo);
    lo = static_cast<float>(lo16);
    // (the product is rounded to float32 before fp16, which one instruction for both would leave out)
    float range = fmaxf(hi - lo, 0.0f) * (1.0f / 15.0f);
    asm("" : "+v"(range));
    const _Float16 step16 = static_cast<_Float16>(range);
    const float step = static_cast<float>(step16);
    pair = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, step16)) |
           (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, lo16)) << 16);
    const float r = step > 0.0f ? 1.0f / step : 0.0f;   // (a step of 0 makes codes of 0)
    float four[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = x[i] - lo, q0 = d * r, q1 = fmaf(fmaf(-q0, step, d), r, q0);
        const float q = rintf(__builtin_amdgcn_fmed3f(q1, 0.0f, 15.0f));   // (clamping to whole numbers first changes nothing)
        const int at = KEY ? key_nibble(i) : i;
        four[at >> 2] = fmaf(q, static_cast<float>(1 << (4 * (at & 3))), four[at >> 2]);
    }
    return static_cast<uint32_t>(four[0]) | (static_cast<uint32_t>(four[1]) << 16);
}

// Quantises a lane's 8 channels of a unit's keys and values and stores them: lane w of token
// `token`, `bytes` the unit's own part of LDS.  All threads of the workgroup call.
template <int D, int GROUP>
__device__ __forceinline__ void store_unit(const KvCache &c, const Place &p, int lane, int token, int w, const float *k,
                                           const float *v, uint32_t *bytes) {
    constexpr int LT = D / 8, J = D / 32, NG = D / GROUP, GL = GROUP / 8;
    const bool there = p.block != nullptr && p.row >= 0;
    bool k_fits, v_fits;
    uint32_t kp, vp, kw = quantise<GL, true>(k, kp, k_fits), vw = quantise<GL, false>(v, vp, v_fits);
    const unsigned long long any = __ballot(!(k_fits & v_fits));
    const int at = (threadIdx.x & 63) & ~(LT - 1);
    const bool bad = ((any >> at) & ((1ull << LT) - 1)) != 0;
    if (bad) kp = 0x7E007E00u, vp = 0, kw = 0, vw = 0;
    // lane w holds channels 8w..8w+7; the byte of channel 32b + m takes its high
    // nibble from 16 channels on, two lanes further
    const uint32_t up = __shfl_down(vw, 2);
    unsigned char *mine = reinterpret_cast<unsigned char *>(bytes);
    if ((w & 2) == 0) {
        const int m0 = 8 * (w & 1), b = w >> 2;
        const uint32_t even = (vw & 0x0F0F0F0Fu) | ((up & 0x0F0F0F0Fu) << 4);   // the bytes of channels m0, m0 + 2, ..
        const uint32_t odd = ((vw >> 4) & 0x0F0F0F0Fu) | (up & 0xF0F0F0F0u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mine[(m0 + i) * (4 * J) + 4 * b + token] = static_cast<unsigned char>((i & 1 ? odd : even) >> (8 * (i >> 1)));
    }
    const unsigned int here = __syncthreads_count(there);   // (also the barrier before the bytes are read)
    // all 4 tokens of this unit?  (one block of bytes: 4 aligned positions share a page)
    const bool whole_group = here == kKvThreads;
    if (there) {
        const int P = 1 << c.page_shift;
        const int j = w >> 2, kb = w & 3;
        *reinterpret_cast<uint32_t *>(p.block + p.slot * (D / 2) + 4 * (kb * J + j)) = kw;
        if (w % GL == 0) {
            uint32_t *pairs = reinterpret_cast<uint32_t *>(p.block + P * D);
            pairs[p.slot * NG + w / GL] = kp;
            pairs[P * NG + p.slot * NG + w / GL] = vp;
        }
        unsigned char *vb = p.block + P * (D / 2) + (p.slot >> 2) * (2 * D);
        if (whole_group) {
            reinterpret_cast<uint32_t *>(vb)[lane] = bytes[lane];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at4 = 4 * (w + LT * i) + token;
                vb[at4] = mine[at4];
            }
        }
    }
}

// Units of 4 aligned positions that T rows of B sequences can touch.
inline void kv_unit_counts(const KvBatch &s, int &units, int &units_even) {
    units_even = (s.even + 2) / 4 + 1;   // rows of one sequence, from the worst offset
    units = s.row_start ? s.T / 4 + 2 * s.B : s.B * units_even;
}

// f(D, GROUP), as integral constants, for the cache's sizes (checked by the caller)
template <typename F>
hipError_t kv_by_size(const KvCache &c, F f) {
#define AWQ_KV_SIZE(D, G) \
    if (c.dim == D && c.group == G) return f(std::integral_constant<int, D>{}, std::integral_constant<int, G>{});
    AWQ_KV_SIZE(64, 32)
    AWQ_KV_SIZE(64, 64)
    AWQ_KV_SIZE(128, 32)
    AWQ_KV_SIZE(128, 64)
    AWQ_KV_SIZE(128, 128)
    AWQ_KV_SIZE(256, 32)
    AWQ_KV_SIZE(256, 64)
    AWQ_KV_SIZE(256, 128)
#undef AWQ_KV_SIZE
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace awq
