// Routed decode attention over chosen blocks (Eq. 2 with the full resolution replaced by a
// choice of blocks): one query per (sequence, query head) at t = len - 1. A skip query's
// output is 0, a local query attends over keys [max(0, t - w), t], a full query over the keys
// of the blocks listed for its KV head.
//
//   logit_j = q . deq(k_j) / sqrt(D),  p = softmax,  out = sum_j p_j deq(v_j)
//
// decode_blocks_kernel: one CTA per (sequence, query head), a key per warp at a time, D/32
// channels per lane, the running maximum and sum of the softmax in fp32 per warp; the warps'
// states are merged at the end.
#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads)
decode_blocks_kernel(CacheView c, const __half *__restrict__ q, const int32_t *__restrict__ ids, int k, int block,
                     const uint8_t *__restrict__ modes, int w, float *__restrict__ out)
{
    constexpr int N = D / 32;
    __shared__ float red[kWarps][D], rm[kWarps], rl[kWarps];
    pdl_wait();
    pdl_trigger();
    const int64_t hq = blockIdx.x;                             // (s * H + h) * G + g
    const int sh = (int)(hq / c.G), s = sh / c.H, h = sh % c.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = c.len[sh], mode = modes[hq];
    const int64_t slot0 = slot_of(c, s, h, 0);
    if (mode > 2 && threadIdx.x == 0) set_status(c.status, KVQ_ERR_MODE);
    float qv[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        qv[e] = __half2float(q[hq * D + lane * N + e]) * (kLog2e / sqrtf((float)D));
        o[e] = 0.f;
    }
    const int j_lo = mode == KVQ_MODE_LOCAL ? max(0, len - 1 - min(w, len)) : 0;
    const int n = mode == KVQ_MODE_FULL ? k * block : mode == KVQ_MODE_LOCAL ? len - j_lo : 0;
    for (int i = warp; i < n; i += kWarps) {
        int j = j_lo + i;
        if (mode == KVQ_MODE_FULL) {
            const int64_t at = (int64_t)sh * k + i / block;
            const int id = ids[at], before = i >= block ? ids[at - 1] : -1;
            if (id < 0) continue;
            if ((i >= block && before < 0) || id <= before || (int64_t)id * block >= len) {
                if (lane == 0) set_status(c.status, KVQ_ERR_DEVICE_CHECK);
                continue;
            }
            j = id * block + i % block;
            if (j >= len) continue;
        }
        const uint32_t mt = c.meta[slot0 + j];
        const float4 sd = c.side[slot0 + j];
        const int wc = (int)(mt & 3u), b = 2 << wc;
        const RecLoc L = rec_loc(c, s, h, mt & ~15u);
        float dot = 0.f, v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int bit = b * (lane * N + e);
            float x[2];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const uint32_t word = *reinterpret_cast<const uint32_t *>(L.at((uint32_t)(part * (b * D / 8) + 4 * (bit >> 5))));
                const uint32_t f = (word >> (bit & 31)) & ((1u << b) - 1u);
                x[part] = wc == 3 ? __half2float(__ushort_as_half((unsigned short)f))
                                  : __fadd_rn(__fmul_rn((float)f, part ? sd.z : sd.x), part ? sd.w : sd.y);
            }
            dot = fmaf(qv[e], x[0], dot);
            v[e] = x[1];
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        const float mn = fmaxf(m, dot), corr = exp2f(m - mn), p = exp2f(dot - mn);
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = o[e] * corr + p * v[e];
        m = mn;
    }
    if (lane == 0) {
        rm[warp] = m;
        rl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) red[warp][lane * N + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int x = 0; x < kWarps; ++x) M = fmaxf(M, rm[x]);
        for (int x = 0; x < kWarps; ++x) {
            if (rl[x] == 0.f) continue;
            const float f = exp2f(rm[x] - M);
            L += rl[x] * f;
            O += red[x][threadIdx.x] * f;
        }
        out[hq * D + threadIdx.x] = L > 0.f ? O / L : 0.f;
    }
}

} // namespace

int64_t decode_blocks_scratch(const kvq_cache *, int, int, int) { return 0; }

cudaError_t launch_decode_blocks(const __half *q, const kvq_cache *cache, const int32_t *ids, int k, int block,
                                 const uint8_t *modes, int w, float *, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const dim3 grid((unsigned)((int64_t)c.B * c.H * c.G));
    return c.D == 128 ? launch_pdl(decode_blocks_kernel<128>, grid, dim3(kThreads), 0, st, c, q, ids, k, block, modes, w, out)
                      : launch_pdl(decode_blocks_kernel<64>, grid, dim3(kThreads), 0, st, c, q, ids, k, block, modes, w, out);
}

} // namespace kvq
