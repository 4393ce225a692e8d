// Values of stored codes (Eq. 4), for the kernels that need them one by one: deq(c) =
// fl(fl(c * s) + z) in fp32 for b < 16 (product and sum rounded one after the other), the
// fp16 value itself for b = 16.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

__device__ __forceinline__ float2 h2_values(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// The 8 codes of width 2 << CLS in the 2 << CLS bytes of `w`, as values. A field at bit p joins
// the mantissa of m = 2^(23 - p), whose last place there is 1: the word m + c, and one fused
// multiply-add gives fl((m + c) s - m s) = fl(c s), m s being exact.
template <int CLS>
__device__ __forceinline__ void code_values(const uint4 &w, float s, float z, float (&x)[8])
{
    constexpr int BITS = 2 << CLS;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    if constexpr (CLS == 3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = h2_values(words[e]);
            x[2 * e] = v.x;
            x[2 * e + 1] = v.y;
        }
    } else {
        // P fields at bits 0, BITS, .. of a word shifted down by SH at a time
        constexpr int P = CLS == 2 ? 2 : 4, SH = P * BITS;
        constexpr uint32_t one = (1u << BITS) - 1u;
        float ms[P];
#pragma unroll
        for (int i = 0; i < P; ++i) ms[i] = s * __uint_as_float(0xCB000000u - ((uint32_t)(i * BITS) << 23));
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t v = words[e * BITS / 32] >> ((e * BITS & 31) / SH * SH);
            const int i = e % P;
            const uint32_t c0 = (v & (one << (i * BITS))) | (0x4B000000u - ((uint32_t)(i * BITS) << 23));
            const uint32_t c1 = (v & (one << (i * BITS + BITS))) | (0x4B000000u - ((uint32_t)(i * BITS + BITS) << 23));
            const float2 y = __fadd2_rn(__ffma2_rn(make_float2(__uint_as_float(c0), __uint_as_float(c1)), make_float2(s, s),
                                                   make_float2(ms[i], ms[i + 1])),
                                        make_float2(z, z));
            x[e] = y.x;
            x[e + 1] = y.y;
        }
    }
}

// The 2 << CLS bytes of 8 codes.
template <int CLS>
__device__ __forceinline__ uint4 load_codes(const uint8_t *p)
{
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (CLS == 0) w.x = __ldg(reinterpret_cast<const unsigned short *>(p));
    else if (CLS == 1) w.x = __ldg(reinterpret_cast<const uint32_t *>(p));
    else if (CLS == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w.x = v.x;
        w.y = v.y;
    } else w = __ldg(reinterpret_cast<const uint4 *>(p));
    return w;
}

} // namespace kvq
