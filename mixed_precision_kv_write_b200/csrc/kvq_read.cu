// Read-back of the newest cached tokens as plain K and V rows (no counterpart in the pages):
// the last n_s tokens of each sequence, dequantized (Eq. 4), in the row layout of kvq_write.
//
// read_kernel: D/8 adjacent lanes per (token, head), 8 channels of K and of V per lane: a lane
// loads b bytes of each part (2, 4, 8 or 16: its 8 codes) and stores 8 values. A CTA takes
// kPairs consecutive (token, head) pairs; one thread per pair first finds its sequence
// (binary search of cu_seqlens), its record offset and its scales, then the pairs are sorted
// by width, so that the lanes of a warp share one code path (69 -> 45 us unsorted to sorted at
// 284k pairs). Bound: HBM (records and side entries in, rows out); 284k pairs of head_dim 128 as
// fp16 take 43 us, 4.6 TB/s, the lookups in front of each CTA's loads being what is left.
#include <cuda_bf16.h>

#include <type_traits>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

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

// chunk li of both parts of one pair
template <int D, int CLS, typename T>
__device__ __forceinline__ void pair_values(const ReadPair &pr, uint32_t shift, int li, int64_t at, T *__restrict__ k_out,
                                            T *__restrict__ v_out)
{
    constexpr int BITS = 2 << CLS;
    RecLoc L;
    L.base = const_cast<uint8_t *>(pr.base);
    L.pt = pr.pt;
    L.off = pr.off;
    L.shift = shift;
    const uint4 kw = load_codes<CLS>(L.at(BITS * li)), vw = load_codes<CLS>(L.at(D * BITS / 8 + BITS * li));
    const float4 sd = pr.side;
    float x[8];
    if (k_out) {
        code_values<CLS>(kw, sd.x, sd.y, x);
        store8(k_out + at, x);
    }
    if (v_out) {
        code_values<CLS>(vw, sd.z, sd.w, x);
        store8(v_out + at, x);
    }
}

template <int D, typename T, int kPairs>
__global__ void __launch_bounds__(kThreads)
read_kernel(CacheView c, const int32_t *__restrict__ cu, int64_t n_rows, T *__restrict__ k_out, T *__restrict__ v_out)
{
    constexpr int VL = D / 8;
    __shared__ ReadPair pairs[kPairs];
    __shared__ uint8_t order[kPairs];
    __shared__ int cnt[5];                       // pairs by width: end of each width's run, [4] of the rows of zeros
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
    if (threadIdx.x < 32) {                      // sort by width; rows left alone are dropped
        const int lane = threadIdx.x;
        int base = 0;
#pragma unroll
        for (int w = 0; w < 5; ++w) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 32) {
                const bool in = i + lane < n && pairs[i + lane].wc == (w < 4 ? w : -1);
                const uint32_t m = __ballot_sync(0xffffffffu, in);
                if (in) order[base + __popc(m & ((1u << lane) - 1u))] = (uint8_t)(i + lane);
                base += __popc(m);
            }
            if (lane == 0) cnt[w] = base;
        }
    }
    __syncthreads();
    const int c0 = cnt[0], c1 = cnt[1], c2 = cnt[2], c3 = cnt[3], c4 = cnt[4];
    for (int t = threadIdx.x; t < c4 * VL; t += kThreads) {
        const int oi = t / VL, li = t % VL, pi = order[oi];
        const int64_t at = (p0 + pi) * D + 8 * li;
        const ReadPair &pr = pairs[pi];
        if (oi < c0) pair_values<D, 0>(pr, c.page_shift, li, at, k_out, v_out);
        else if (oi < c1) pair_values<D, 1>(pr, c.page_shift, li, at, k_out, v_out);
        else if (oi < c2) pair_values<D, 2>(pr, c.page_shift, li, at, k_out, v_out);
        else if (oi < c3) pair_values<D, 3>(pr, c.page_shift, li, at, k_out, v_out);
        else {
            const float zero[8] = {};
            if (k_out) store8(k_out + at, zero);
            if (v_out) store8(v_out + at, zero);
        }
    }
}

template <int D, typename T>
cudaError_t launch_typed(const kvq_cache *cache, const int32_t *cu, int64_t n_rows, void *k_out, void *v_out,
                         cudaStream_t st)
{
    const CacheView &c = cache->view;
    const int64_t n = n_rows * c.H;
    auto launch = [&](auto kernel, int pairs) {
        return launch_pdl(kernel, dim3((unsigned)((n + pairs - 1) / pairs)), dim3(kThreads), 0, st, c, cu, n_rows, (T *)k_out,
                          (T *)v_out);
    };
    // 128 pairs a CTA sort better and start fewer CTAs once 8 of them fill every SM (284k pairs:
    // 43.3 against 45.4 us), 64 spread a short call over more SMs (8k pairs: 6.6 against 9.8 us);
    // below 32 pairs an SM, one pass of the threads
    if (n >= (int64_t)128 * 8 * num_sms()) return launch(read_kernel<D, T, 128>, 128);
    if (n >= (int64_t)32 * num_sms()) return launch(read_kernel<D, T, 64>, 64);
    return launch(read_kernel<D, T, 16>, 16);
}

} // namespace

cudaError_t launch_read(const kvq_cache *c, const int32_t *cu, int64_t n_rows, int dtype, void *k_out, void *v_out,
                        cudaStream_t st)
{
    if (n_rows == 0) return cudaSuccess;
    auto go = [&](auto f128, auto f64) { return (c->D == 128 ? f128 : f64)(c, cu, n_rows, k_out, v_out, st); };
    if (dtype == KVQ_F32) return go(launch_typed<128, float>, launch_typed<64, float>);
    if (dtype == KVQ_BF16) return go(launch_typed<128, __nv_bfloat16>, launch_typed<64, __nv_bfloat16>);
    return go(launch_typed<128, __half>, launch_typed<64, __half>);
}

} // namespace kvq
