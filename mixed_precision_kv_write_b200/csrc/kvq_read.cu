// Read-back of the newest cached tokens as plain K and V rows (no counterpart in the pages):
// the last n_s tokens of each sequence, dequantized (Eq. 4), in the row layout of kvq_write.
//
// read_kernel: D/8 adjacent lanes per (token, head), 8 channels of K and of V per lane: a lane
// loads b bytes of each part (2, 4, 8 or 16: its 8 codes) and stores 8 values. A CTA takes
// kPairs consecutive (token, head) pairs; one thread per pair first finds its sequence
// (binary search of cu_seqlens), its record offset and its scales. Bound: HBM (records and
// side entries in, rows out).
#include <cuda_bf16.h>

#include <type_traits>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 64;

struct ReadPair {
    float4 side;
    const uint8_t *base;      // contiguous: the record; paged: the pool
    const uint32_t *pt;       // paged: the stream's page table row
    uint32_t off;             // paged: record offset in the stream
    int32_t wc;               // width code; -1: not a cached token (row of zeros), -2: row left alone
};

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&x)[8])
{
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint4 o;
        uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *reinterpret_cast<uint4 *>(dst) = o;
    }
}

// the 8 values of chunk li of one record part
template <int D>
__device__ __forceinline__ void part_values(const RecLoc &L, int wc, int part, int li, float s, float z, float (&x)[8])
{
    const int b = 2 << wc;
    const uint8_t *p = L.at((uint32_t)(part * (b * D / 8) + b * li));
    if (wc == 0) {
        code_values<0, 8>(make_uint2(*reinterpret_cast<const uint16_t *>(p), 0u), s, z, x);
    } else if (wc == 1) {
        code_values<1, 8>(make_uint2(*reinterpret_cast<const uint32_t *>(p), 0u), s, z, x);
    } else if (wc == 2) {
        code_values<2, 8>(*reinterpret_cast<const uint2 *>(p), s, z, x);
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        float lo[4], hi[4];
        code_values<3, 4>(make_uint2(v.x, v.y), s, z, lo);
        code_values<3, 4>(make_uint2(v.z, v.w), s, z, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = lo[e];
            x[4 + e] = hi[e];
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads)
read_kernel(CacheView c, const int32_t *__restrict__ cu, int64_t n_rows, T *__restrict__ k_out, T *__restrict__ v_out)
{
    constexpr int VL = D / 8;
    __shared__ ReadPair pairs[kPairs];
    pdl_wait();
    pdl_trigger();
    const int64_t p0 = (int64_t)blockIdx.x * kPairs;
    const int n = (int)min((int64_t)kPairs, n_rows * c.H - p0);
    if (blockIdx.x == 0) {                       // cu_seqlens runs from 0 up to at most n_rows
        for (int s = threadIdx.x; s < c.B; s += kThreads)
            if (cu[s] < 0 || cu[s + 1] < cu[s] || cu[s + 1] > n_rows || (s == 0 && cu[0] != 0))
                set_status(c.status, KVQ_ERR_DEVICE_CHECK);
    }
    if (threadIdx.x < n) {
        const int64_t row = (p0 + threadIdx.x) / c.H;
        const int h = (int)((p0 + threadIdx.x) % c.H);
        int lo = 0, hi = c.B;                    // cu[lo] <= row < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= row) lo = mid;
            else hi = mid;
        }
        ReadPair pr;
        pr.side = make_float4(1.f, 0.f, 1.f, 0.f);
        pr.base = nullptr;
        pr.pt = nullptr;
        pr.off = 0;
        pr.wc = -2;
        const int64_t t0 = cu[lo], t1 = cu[lo + 1];
        if (row >= t0 && row < t1) {
            const int64_t j = c.len[lo * c.H + h] - (t1 - row);
            if (j >= 0) {
                const int64_t slot = slot_of(c, lo, h, j);
                const uint32_t mt = c.meta[slot];
                const RecLoc L = rec_loc(c, lo, h, mt & ~15u);
                pr.side = c.side[slot];
                pr.base = L.base;
                pr.pt = L.pt;
                pr.off = L.off;
                pr.wc = (int)(mt & 3u);
            } else {
                pr.wc = -1;
                set_status(c.status, KVQ_ERR_DEVICE_CHECK);
            }
        }
        pairs[threadIdx.x] = pr;
    }
    __syncthreads();
    for (int t = threadIdx.x; t < n * VL; t += kThreads) {
        const int pi = t / VL, li = t % VL;
        const int wc = pairs[pi].wc;
        if (wc == -2) continue;
        float kx[8] = {}, vx[8] = {};
        if (wc >= 0) {
            const float4 sd = pairs[pi].side;
            RecLoc L;
            L.base = const_cast<uint8_t *>(pairs[pi].base);
            L.pt = pairs[pi].pt;
            L.off = pairs[pi].off;
            L.shift = c.page_shift;
            if (k_out) part_values<D>(L, wc, 0, li, sd.x, sd.y, kx);
            if (v_out) part_values<D>(L, wc, 1, li, sd.z, sd.w, vx);
        }
        const int64_t at = (p0 + pi) * D + 8 * li;
        if (k_out) store8(k_out + at, kx);
        if (v_out) store8(v_out + at, vx);
    }
}

template <typename T>
cudaError_t launch_typed(const kvq_cache *cache, const int32_t *cu, int64_t n_rows, void *k_out, void *v_out,
                         cudaStream_t st)
{
    const CacheView &c = cache->view;
    const dim3 grid((unsigned)((n_rows * c.H + kPairs - 1) / kPairs));
    return c.D == 128 ? launch_pdl(read_kernel<128, T>, grid, dim3(kThreads), 0, st, c, cu, n_rows, (T *)k_out, (T *)v_out)
                      : launch_pdl(read_kernel<64, T>, grid, dim3(kThreads), 0, st, c, cu, n_rows, (T *)k_out, (T *)v_out);
}

} // namespace

cudaError_t launch_read(const kvq_cache *c, const int32_t *cu, int64_t n_rows, int dtype, void *k_out, void *v_out,
                        cudaStream_t st)
{
    if (n_rows == 0) return cudaSuccess;
    if (dtype == KVQ_F32) return launch_typed<float>(c, cu, n_rows, k_out, v_out, st);
    if (dtype == KVQ_BF16) return launch_typed<__nv_bfloat16>(c, cu, n_rows, k_out, v_out, st);
    return launch_typed<__half>(c, cu, n_rows, k_out, v_out, st);
}

} // namespace kvq
