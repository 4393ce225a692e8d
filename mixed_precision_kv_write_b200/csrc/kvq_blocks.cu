// Block-sparse decoding over the mixed-precision cache: per-block bounds of the keys and the
// choice of blocks. A block is `block` consecutive keys of one (sequence, KV head); the
// attention over chosen blocks is in kvq_blocks_attn.cu.
//
// Bounds. For block n and channel c: lo = min, hi = max over the block's keys j of
// deq(k_j)[c], rounded to fp16 (rounding is monotone, so it commutes with min and max).
// Score of a block for query q:  sum_c max(q_c lo_c, q_c hi_c)  >=  q . k_j for every key j
// of the block (up to the rounding of the bounds): an upper bound of the block's logits.
//
// Layout of the bounds: fp16 [B][H][nt][2][D][64], block n at [n / 64] and [n % 64], 0 = lo
// and 1 = hi. A channel's bounds of 64 blocks are one 128-byte line, so a query alone on its
// KV head reads, per channel, only the line that the sign of q_c asks for: half the bytes.
#include <algorithm>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kTile = KVQ_BLOCK_TILE;    // blocks per tile of the bounds layout

// ------------------------------------------------------------------ bounds
// A CTA takes groups of kGroup blocks of one (sequence, head): their 32-byte rows of the
// layout are whole sectors. Each block is cut into kSubs runs of keys, a run per warp at a
// time: D/4 lanes per key, 4 channels per lane. The runs' minima and maxima meet in shared
// memory as fp16.
constexpr int kBThreads = 256, kGroup = 16, kSubs = 4;

template <int D>
__global__ void __launch_bounds__(kBThreads)
bounds_kernel(CacheView c, int block, const int32_t *__restrict__ cu, __half *__restrict__ bounds, int nt, int per_sh)
{
    constexpr int LPK = D / 4, KPW = 32 / LPK;                 // lanes per key, keys per warp step
    constexpr int ROW = kSubs * 2 * D + 2;                     // one block's partials, padded
    __shared__ __half part[kGroup * ROW];
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x / per_sh, s = sh / c.H, h = sh % c.H;
    const int len = c.len[sh];
    int first = 0;                                             // first key that is new
    if (cu) {
        const int64_t n = (int64_t)cu[s + 1] - cu[s];
        if (n < 0 || n > len) {
            if (threadIdx.x == 0 && blockIdx.x % per_sh == 0) set_status(c.status, KVQ_ERR_DEVICE_CHECK);
            return;
        }
        if (n == 0) return;
        first = len - (int)n;
    }
    const int b_lo = first / block, b_hi = (len + block - 1) / block;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPK, gk = lane / LPK;
    const int run = block / kSubs;
    const int64_t slot0 = slot_of(c, s, h, 0);
    for (int g = b_lo / kGroup + blockIdx.x % per_sh; g * kGroup < b_hi; g += per_sh) {
        const int b0 = max(b_lo, g * kGroup), b1 = min(b_hi, (g + 1) * kGroup);
        for (int u = warp; u < (b1 - b0) * kSubs; u += kBThreads / 32) {
            const int b = b0 + u / kSubs, sub = u % kSubs;
            const int j0 = b * block + sub * run, n = min(run, len - j0);      // n <= 0: an empty run
            uint32_t mt = 0;
            float2 sd = make_float2(1.f, 0.f);
            if (lane < n) {
                mt = c.meta[slot0 + j0 + lane];
                sd = *reinterpret_cast<const float2 *>(&c.side[slot0 + j0 + lane]);
            }
            float lo[4], hi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] = INFINITY;
                hi[e] = -INFINITY;
            }
            for (int i0 = 0; i0 < n; i0 += KPW) {
                const int i = i0 + gk;
                const uint32_t m = __shfl_sync(0xffffffffu, mt, i & 31);
                const float sc = __shfl_sync(0xffffffffu, sd.x, i & 31), z = __shfl_sync(0xffffffffu, sd.y, i & 31);
                if (i >= n) continue;
                const int wc = (int)(m & 3u);
                const RecLoc L = rec_loc(c, s, h, m & ~15u);
                const uint8_t *p = L.at((uint32_t)(li << wc));                 // 4 channels: 1, 2, 4 or 8 bytes
                float x[4];
                if (wc == 0) code_values<0, 4>(make_uint2(*p, 0u), sc, z, x);
                else if (wc == 1) code_values<1, 4>(make_uint2(*reinterpret_cast<const uint16_t *>(p), 0u), sc, z, x);
                else if (wc == 2) code_values<2, 4>(make_uint2(*reinterpret_cast<const uint32_t *>(p), 0u), sc, z, x);
                else code_values<3, 4>(*reinterpret_cast<const uint2 *>(p), sc, z, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo[e] = fminf(lo[e], x[e]);
                    hi[e] = fmaxf(hi[e], x[e]);
                }
            }
#pragma unroll
            for (int d = LPK; d < 32; d <<= 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
                    hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
                }
            }
            if (gk == 0) {
                __half2 *dst = reinterpret_cast<__half2 *>(part + (b - g * kGroup) * ROW + sub * 2 * D + 4 * li);
                dst[0] = __floats2half2_rn(lo[0], lo[1]);
                dst[1] = __floats2half2_rn(lo[2], lo[3]);
                dst[D / 2] = __floats2half2_rn(hi[0], hi[1]);
                dst[D / 2 + 1] = __floats2half2_rn(hi[2], hi[3]);
            }
        }
        __syncthreads();
        for (int t = threadIdx.x; t < 2 * D * kGroup; t += kBThreads) {
            const int bi = t % kGroup, b = g * kGroup + bi, mc = t / kGroup;    // mc: [lo/hi][channel]
            if (b < b0 || b >= b1) continue;
            const __half *p = part + bi * ROW + mc;
            __half r = p[0];
#pragma unroll
            for (int q = 1; q < kSubs; ++q) r = mc < D ? __hmin(r, p[q * 2 * D]) : __hmax(r, p[q * 2 * D]);
            bounds[(((int64_t)sh * nt + b / kTile) * 2 * D + mc) * kTile + b % kTile] = r;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ scores
// Two blocks' scores can lie next to one another, and the choice between them has to be the
// same whatever order the channels are summed in: products of fp16 values are exact in
// fp64, and a sum of 128 of them there is off by at most 2^-46 of their largest sum, so the
// fp32 score is the correctly rounded one but for ties that close. fp16 -> fp64 takes one
// shift and one mask: the fp16 bits moved to the same field of a double (sign, exponent at
// bit 52 on) are the value times 2^-1008, subnormals included (fp64 arithmetic keeps them).
// q carries 2^1000, the score 2^8.
constexpr int kSThreads = 256, kSWarps = kSThreads / 32;
constexpr double kQUp = 1.0715086071862673e301;                // 2^1000

__device__ __forceinline__ double half_field(uint32_t top)     // the fp16 bits in bits 16..31 of `top`
{
    return __hiloint2double((int)((uint32_t)((int32_t)top >> 6) & 0x81FFFC00u), 0);
}

// One CTA per (sequence, KV head, tile of 64 blocks). Lane = (channel mod 4, group of 8
// blocks): a 16-byte load covers 8 blocks of a channel, a warp's load 4 channels.
template <int D, int NQ>
__global__ void __launch_bounds__(kSThreads)
score_kernel(CacheView c, const __half *__restrict__ q, const __half *__restrict__ bounds,
             const uint8_t *__restrict__ modes, int block, int nt, float *__restrict__ scores)
{
    __shared__ double qs[NQ][D];
    __shared__ double sum[kSWarps][NQ][kTile];
    __shared__ int act[64], n_act;
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x / nt, tile = blockIdx.x % nt, s = sh / c.H, h = sh % c.H;
    const int nb = (c.len[sh] + block - 1) / block;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane >> 3, b8 = lane & 7;
    const int64_t q0 = ((int64_t)s * c.H + h) * c.G;
    if (tid == 0) {
        int n = 0;
        for (int g = 0; g < c.G; ++g) {
            const int m = modes ? modes[q0 + g] : KVQ_MODE_FULL;
            if (m > 2) set_status(c.status, KVQ_ERR_MODE);
            if (m == KVQ_MODE_FULL) act[n++] = g;
        }
        n_act = n;
    }
    __syncthreads();
    float *dst = scores + ((int64_t)sh * nt + tile) * kTile;
    const int here = min(kTile, nb - tile * kTile);            // blocks of this tile
    float best = -INFINITY;
    if (here > 0) {
        const uint4 *lo = reinterpret_cast<const uint4 *>(bounds + ((int64_t)sh * nt + tile) * 2 * D * kTile);
        const uint4 *hi = lo + D * (kTile / 8);
        for (int a0 = 0; a0 < n_act; a0 += NQ) {
            const int n = min(NQ, n_act - a0);
            for (int t = tid; t < NQ * D; t += kSThreads)
                qs[t / D][t % D] = t / D < n ? (double)__half2float(q[(q0 + act[a0 + t / D]) * D + t % D]) * kQUp : 0.0;
            __syncthreads();
            double acc[NQ][8];
#pragma unroll
            for (int g = 0; g < NQ; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[g][e] = 0.0;
#pragma unroll 4
            for (int i = 0; i < D / (4 * kSWarps); ++i) {
                const int ch = (i * kSWarps + warp) * 4 + sub;
                uint4 l, u;
                if (NQ == 1) {
                    l = u = (qs[0][ch] < 0.0 ? lo : hi)[ch * (kTile / 8) + b8];
                } else {
                    l = lo[ch * (kTile / 8) + b8];
                    u = hi[ch * (kTile / 8) + b8];
                }
                const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int g = 0; g < NQ; ++g) {
                    const double qv = qs[g][ch];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = NQ == 1 ? uw[e] : (qv < 0.0 ? lw[e] : uw[e]);
                        acc[g][2 * e] = fma(qv, half_field(w << 16), acc[g][2 * e]);
                        acc[g][2 * e + 1] = fma(qv, half_field(w), acc[g][2 * e + 1]);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < NQ; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    double v = acc[g][e];
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    if (sub == 0) sum[warp][g][b8 * 8 + e] = v;
                }
            __syncthreads();
            if (tid < kTile) {
                for (int g = 0; g < n; ++g) {
                    double v = 0.0;
#pragma unroll
                    for (int w = 0; w < kSWarps; ++w) v += sum[w][g][tid];
                    best = fmaxf(best, (float)(v * 256.0));
                }
            }
            __syncthreads();
        }
    }
    if (tid < kTile) dst[tid] = tid < here ? best : -INFINITY;
}

// ------------------------------------------------------------------ choice
// One CTA per (sequence, KV head): the k blocks of the largest keys, ties to the lower
// index, written in ascending order. Keys are the scores mapped to unsigned integers of the
// same order; forced blocks get the largest key. The k-th largest key is found bit by bit
// (32 counts over the CTA), the output places by a prefix sum.
constexpr int kCThreads = 512, kPer = 8, kCChunk = kCThreads * kPer;

__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x) x = -INFINITY;                                 // NaN ranks lowest
    const uint32_t u = __float_as_uint(x + 0.0f);              // -0 and +0 are one value
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kCThreads)
choose_kernel(CacheView c, const float *__restrict__ scores, const uint8_t *__restrict__ modes, int block, int nt, int k,
              int first, int last, int32_t *__restrict__ ids)
{
    __shared__ int wsum[2][kCThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nb = (c.len[sh] + block - 1) / block;
    bool any = !modes;
    if (modes)
        for (int g = 0; g < c.G; ++g) any = any || modes[(int64_t)sh * c.G + g] == KVQ_MODE_FULL;
    int32_t *out = ids + (int64_t)sh * k;
    const int want = any ? min(k, nb) : 0;
    for (int i = want + tid; i < k; i += kCThreads) out[i] = -1;
    if (want == 0) return;
    const float *sc = scores + (int64_t)sh * nt * kTile;
    uint32_t key[kPer];
    auto load = [&](int base) {                                // keys of blocks base + tid * kPer ..; 0 past the end
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int b = base + tid * kPer + e;
            key[e] = 0;
            if (b < nb) key[e] = (b < first || b >= nb - last) ? 0xFFFFFFFFu : order_key(sc[b]);
        }
    };
    load(0);
    uint32_t T = 0;                                            // largest T with at least `want` keys >= T
    if (want < nb) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t t = T | (1u << bit);
            int n = 0;
            for (int base = 0; base < nb; base += kCChunk) {
                if (nb > kCChunk) load(base);
#pragma unroll
                for (int e = 0; e < kPer; ++e) n += key[e] >= t ? 1 : 0;
            }
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) wsum[bit & 1][warp] = n;
            __syncthreads();
            int all = 0;
#pragma unroll
            for (int w = 0; w < kCThreads / 32; ++w) all += wsum[bit & 1][w];
            if (all >= want) T = t;
        }
    }
    __syncthreads();
    // blocks above T, then those at T in index order until `want` are taken
    int above = 0;
    for (int base = 0; base < nb; base += kCChunk) {
        if (nb > kCChunk) load(base);
#pragma unroll
        for (int e = 0; e < kPer; ++e) above += key[e] > T ? 1 : 0;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0) wsum[0][warp] = above;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kCThreads / 32; ++w) all += wsum[0][w];
    const int ties = want - all;
    int gt0 = 0, eq0 = 0;                                      // taken so far: above T, at T
    __syncthreads();
    for (int base = 0; base < nb; base += kCChunk) {
        if (nb > kCChunk) load(base);
        int gt = 0, eq = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const bool in = base + tid * kPer + e < nb;
            gt += in && key[e] > T ? 1 : 0;
            eq += in && key[e] == T ? 1 : 0;
        }
        int gi = gt, ei = eq;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, gi, d), b = __shfl_up_sync(0xffffffffu, ei, d);
            if (lane >= d) {
                gi += a;
                ei += b;
            }
        }
        if (lane == 31) {
            wsum[0][warp] = gi;
            wsum[1][warp] = ei;
        }
        __syncthreads();
        int gp = gt0 + gi - gt, ep = eq0 + ei - eq, gall = 0, eall = 0;
        for (int w = 0; w < kCThreads / 32; ++w) {
            if (w < warp) {
                gp += wsum[0][w];
                ep += wsum[1][w];
            }
            gall += wsum[0][w];
            eall += wsum[1][w];
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int b = base + tid * kPer + e;
            if (b >= nb) break;
            if (key[e] > T) out[gp++ + min(ep, ties)] = b;
            else if (key[e] == T) {
                if (ep < ties) out[gp + ep] = b;
                ++ep;
            }
        }
        gt0 += gall;
        eq0 += eall;
        __syncthreads();
    }
}

} // namespace

cudaError_t launch_block_bounds(const kvq_cache *cache, int block, const int32_t *cu, __half *bounds, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const int nb = (cache->max_cap + block - 1) / block, nt = (nb + kTile - 1) / kTile;
    // CTAs per (sequence, head): one per group of blocks, at most about 8 per SM in all (they loop)
    const int64_t sh = (int64_t)c.B * c.H;
    const int64_t groups = (nb + kGroup - 1) / kGroup;
    const int per = (int)std::max<int64_t>(1, std::min<int64_t>(groups, (8 * num_sms() + sh - 1) / sh));
    const dim3 grid((unsigned)(sh * per));
    return c.D == 128 ? launch_pdl(bounds_kernel<128>, grid, dim3(kBThreads), 0, st, c, block, cu, bounds, nt, per)
                      : launch_pdl(bounds_kernel<64>, grid, dim3(kBThreads), 0, st, c, block, cu, bounds, nt, per);
}

namespace {
template <int D>
cudaError_t launch_scores(const kvq_cache *cache, const __half *q, const __half *bounds, const uint8_t *modes, int block,
                          int nt, float *scores, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const dim3 grid((unsigned)((int64_t)c.B * c.H * nt));
    if (c.G == 1) return launch_pdl(score_kernel<D, 1>, grid, dim3(kSThreads), 0, st, c, q, bounds, modes, block, nt, scores);
    if (c.G == 2) return launch_pdl(score_kernel<D, 2>, grid, dim3(kSThreads), 0, st, c, q, bounds, modes, block, nt, scores);
    return launch_pdl(score_kernel<D, 4>, grid, dim3(kSThreads), 0, st, c, q, bounds, modes, block, nt, scores);
}
} // namespace

cudaError_t launch_select_blocks(const __half *q, const kvq_cache *cache, const __half *bounds, int block,
                                 const uint8_t *modes, int k, int first, int last, float *scores, int32_t *ids,
                                 cudaStream_t st)
{
    const CacheView &c = cache->view;
    const int nb = (cache->max_cap + block - 1) / block, nt = (nb + kTile - 1) / kTile;
    cudaError_t e = c.D == 128 ? launch_scores<128>(cache, q, bounds, modes, block, nt, scores, st)
                               : launch_scores<64>(cache, q, bounds, modes, block, nt, scores, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(choose_kernel, dim3((unsigned)((int64_t)c.B * c.H)), dim3(kCThreads), 0, st, c,
                      (const float *)scores, modes, block, nt, k, first, last, ids);
}

} // namespace kvq
