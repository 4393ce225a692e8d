// Values of stored codes (Eq. 4), for the kernels that need them one by one: deq(c) =
// fl(fl(c * s) + z) in fp32 for b < 16 (product and sum rounded one after the other), the
// fp16 value itself for b = 16.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// N codes of width 2 << CLS from the low bits of `w` (N * bits bits, at most 64), as values.
template <int CLS, int N>
__device__ __forceinline__ void code_values(uint2 w, float s, float z, float (&x)[N])
{
    constexpr int BITS = 2 << CLS;
    static_assert(N * BITS <= 64, "one word pair");
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint32_t word = (e * BITS) < 32 ? w.x : w.y;
        const uint32_t f = (word >> ((e * BITS) & 31)) & ((1u << BITS) - 1u);
        if (CLS == 3) x[e] = __half2float(__ushort_as_half((unsigned short)f));
        else x[e] = __fadd_rn(__fmul_rn((float)f, s), z);
    }
}

} // namespace kvq
