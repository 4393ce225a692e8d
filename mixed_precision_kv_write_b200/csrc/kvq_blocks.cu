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
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kTile = KVQ_BLOCK_TILE;    // blocks per tile of the bounds layout

// ------------------------------------------------------------------ bounds
// A CTA takes groups of kGroup blocks of one (sequence, head): their 32-byte rows of the
// layout are whole sectors. A warp takes a run of up to 64 keys at a time, a whole block (half a
// one of 128) when the group has a block for every warp, else a quarter of one: it sorts the run's keys by width, asks for
// their records, then takes D/16 lanes per key, 16 channels per lane (two steps' loads in flight
// for the narrow widths: four cost more in code than they hide). A field at bit p joins the mantissa of m = 2^(23 - p), whose last place there is 1, and
// one fused multiply-add takes it to fl((m + c) s - m s) = fl(c s), m s being exact. The runs'
// minima and maxima meet in shared memory as fp16. 1.05 M keys of 128 channels take 60 us, 32
// instructions a key (8 channels a lane: 102; a key per warp at a time: 186), at 53 % issue-active
// and 34 % of DRAM's rate: the wait for the records behind the sort is what is left between them.
constexpr int kGroup = 16, kMaxSubs = 4, kMaxRun = 64, kRuns = 32;

template <int D, int W>
struct BoundsSmem {
    // per run of the group: lo and hi, padded
    __half part[kRuns][2 * D + 2];
    uint4 ent[W][kMaxRun];                               // a run's keys by width: offset, s, z
};

// lo and hi (a NaN stays one) over the n keys of `ent`, all of width 2 << CLS; gk, li: the lane's key of a step and
// its 16 channels. A last step's missing keys repeat the last one, which changes nothing.
template <int D, int CLS, bool PAGED>
__device__ __forceinline__ void bounds_class(__half2 (&lo)[8], __half2 (&hi)[8], const RecLoc &L, const uint4 *ent, int n, int gk,
                                             int li)
{
    constexpr int BITS = 2 << CLS, KPW = 512 / D, W = BITS / 2;      // W words of 16 codes
    constexpr int kFly = CLS >= 2 ? 1 : 2;
    for (int i0 = 0; i0 < n; i0 += kFly * KPW) {
        uint32_t w[kFly][W];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const uint32_t off = ent[min(i0 + f * KPW + gk, n - 1)].x + 2 * BITS * li;
            const uint8_t *p = PAGED ? L.at(off) : L.base + off;
            if (CLS == 0) {
                w[f][0] = __ldg(reinterpret_cast<const uint32_t *>(p));
            } else if (CLS == 1) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
                w[f][0] = v.x;
                w[f][1 % W] = v.y;
            } else {
#pragma unroll
                for (int x = 0; x < W / 4; ++x) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(PAGED && x ? L.at(off + 16 * x) : p + 16 * x));
                    w[f][4 * x % W] = v.x;
                    w[f][(4 * x + 1) % W] = v.y;
                    w[f][(4 * x + 2) % W] = v.z;
                    w[f][(4 * x + 3) % W] = v.w;
                }
            }
        }
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            if (f > 0 && i0 + f * KPW >= n) break;
            const uint4 en = ent[min(i0 + f * KPW + gk, n - 1)];
            const float sc = __uint_as_float(en.y), z = __uint_as_float(en.z);
            // P fields at bits 0, BITS, .. of a word shifted down by SH at a time
            constexpr int P = CLS == 2 ? 2 : 4, SH = P * BITS, N = CLS == 3 ? 1 : P;
            float ms[N];                                       // -m s by position
            if constexpr (CLS != 3) {
#pragma unroll
                for (int i = 0; i < P; ++i) ms[i] = sc * __uint_as_float(0xCB000000u - ((uint32_t)(i * BITS) << 23));
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                __half2 x;
                if constexpr (CLS == 3) {
                    x = *reinterpret_cast<const __half2 *>(&w[f][e / 2]);
                } else {
                    const uint32_t v = w[f][e * BITS / 32] >> ((e * BITS & 31) / SH * SH);
                    constexpr uint32_t one = (1u << BITS) - 1u;
                    const int i = e % P;
                    const uint32_t c0 = (v & (one << (i * BITS))) | (0x4B000000u - ((uint32_t)(i * BITS) << 23));
                    const uint32_t c1 = (v & (one << (i * BITS + BITS))) | (0x4B000000u - ((uint32_t)(i * BITS + BITS) << 23));
                    const float2 y = __fadd2_rn(__ffma2_rn(make_float2(__uint_as_float(c0), __uint_as_float(c1)), make_float2(sc, sc),
                                                           make_float2(ms[i % N], ms[(i + 1) % N])),
                                                make_float2(z, z));
                    x = __floats2half2_rn(y.x, y.y);
                }
                lo[e / 2] = __hmin2_nan(lo[e / 2], x);
                hi[e / 2] = __hmax2_nan(hi[e / 2], x);
            }
        }
    }
}

template <int D, bool PAGED, int W>
__global__ void __launch_bounds__(32 * W, 32 / W)
bounds_kernel(CacheView c, int block, const int32_t *__restrict__ cu, __half *__restrict__ bounds, int nt, int per_sh)
{
    constexpr int LPK = D / 16;                                // lanes per key
    constexpr int kBWarps = W, kBThreads = 32 * W;
    static_assert(kRuns >= kGroup * (128 / kMaxRun) && kRuns >= (W - 1) * kMaxSubs, "a row per run");
    extern __shared__ __align__(16) uint8_t raw[];
    BoundsSmem<D, W> &sm = *reinterpret_cast<BoundsSmem<D, W> *>(raw);
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x / per_sh, s = sh / c.H, h = sh % c.H;
    const int len = c.len[sh];
    int first = 0;                                             // first key that is new
    if (cu) {
        const int64_t n = (int64_t)cu[s + 1] - cu[s];
        if (n < 0 || n > len) {
            if (threadIdx.x == 0 && blockIdx.x % per_sh == 0) set_status(c.status, KVQ_ERR_DEVICE_CHECK);
            if (n < 0) return;
        }
        // without new tokens, the last block may have been cut by a roll-back (at its border it was whole)
        if (n == 0 && len % block == 0) return;
        first = max(0, len - (int)max(n, (int64_t)1));
    }
    const int b_lo = first / block, b_hi = (len + block - 1) / block;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPK, gk = lane / LPK;
    const int64_t slot0 = slot_of(c, s, h, 0);
    const RecLoc L = rec_loc(c, s, h, 0);
    uint4 *ent = sm.ent[warp];
    const uint32_t below = (1u << lane) - 1u;
    for (int g = b_lo / kGroup + blockIdx.x % per_sh; g * kGroup < b_hi; g += per_sh) {
        const int b0 = max(b_lo, g * kGroup), b1 = min(b_hi, (g + 1) * kGroup);
        const int subs = b1 - b0 < kBWarps ? kMaxSubs : block > kMaxRun ? block / kMaxRun : 1, run = block / subs;
        for (int u = warp; u < (b1 - b0) * subs; u += kBWarps) {
            const int b = b0 + u / subs, sub = u % subs;
            const int j0 = b * block + sub * run, n = min(run, len - j0);      // n <= 0: an empty run
            __half2 lo[8], hi[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo[e] = __half2half2(__ushort_as_half(0x7C00));                // +inf, -inf
                hi[e] = __half2half2(__ushort_as_half(0xFC00));
            }
            // the run's keys by width: counts, then places
            constexpr uint32_t kKey = 4u;                                      // (offsets are multiples of 16)
            uint32_t mt[kMaxRun / 32];
            float2 sd[kMaxRun / 32];
            int cnt[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kMaxRun / 32; ++i) {
                const int j = i * 32 + lane;
                mt[i] = 0u;
                if (j < n) {
                    mt[i] = c.meta[slot0 + j0 + j] | kKey;
                    sd[i] = *reinterpret_cast<const float2 *>(&c.side[slot0 + j0 + j]);
                }
            }
#pragma unroll
            for (int i = 0; i < kMaxRun / 32; ++i) {
                if (i * 32 >= n) continue;
                if (mt[i] & kKey) {
                    const uint32_t off = mt[i] & ~15u, bytes = (uint32_t)(D / 4) << (mt[i] & 3u);
                    for (uint32_t o = 0; o < bytes; o += 64) {
                        const uint8_t *p = PAGED ? L.at(off + o) : L.base + off + o;
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
                    }
                }
                const uint32_t v = __ballot_sync(0xffffffffu, mt[i] & kKey), w0 = __ballot_sync(0xffffffffu, mt[i] & 1u),
                               w1 = __ballot_sync(0xffffffffu, mt[i] & 2u);
                cnt[0] += __popc(v & ~w0 & ~w1);
                cnt[1] += __popc(w0 & ~w1);
                cnt[2] += __popc(w1 & ~w0);
                cnt[3] += __popc(w0 & w1);
            }
            int at[4] = {0, cnt[0], cnt[0] + cnt[1], cnt[0] + cnt[1] + cnt[2]};
#pragma unroll
            for (int i = 0; i < kMaxRun / 32; ++i) {
                if (i * 32 >= n) continue;
                const uint32_t v = __ballot_sync(0xffffffffu, mt[i] & kKey), w0 = __ballot_sync(0xffffffffu, mt[i] & 1u),
                               w1 = __ballot_sync(0xffffffffu, mt[i] & 2u);
                if (mt[i] & kKey) {
                    const uint32_t own = v & (mt[i] & 1u ? w0 : ~w0) & (mt[i] & 2u ? w1 : ~w1);
                    const int to = mt[i] & 2u ? (mt[i] & 1u ? at[3] : at[2]) : (mt[i] & 1u ? at[1] : at[0]);
                    ent[to + __popc(own & below)] = make_uint4(mt[i] & ~15u, __float_as_uint(sd[i].x), __float_as_uint(sd[i].y), 0u);
                }
                at[0] += __popc(v & ~w0 & ~w1);
                at[1] += __popc(w0 & ~w1);
                at[2] += __popc(w1 & ~w0);
                at[3] += __popc(w0 & w1);
            }
            __syncwarp();
            const uint4 *e0 = ent, *e1 = e0 + cnt[0], *e2 = e1 + cnt[1], *e3 = e2 + cnt[2];
            if (cnt[0]) bounds_class<D, 0, PAGED>(lo, hi, L, e0, cnt[0], gk, li);
            if (cnt[1]) bounds_class<D, 1, PAGED>(lo, hi, L, e1, cnt[1], gk, li);
            if (cnt[2]) bounds_class<D, 2, PAGED>(lo, hi, L, e2, cnt[2], gk, li);
            if (cnt[3]) bounds_class<D, 3, PAGED>(lo, hi, L, e3, cnt[3], gk, li);
            __syncwarp();
#pragma unroll
            for (int d = LPK; d < 32; d <<= 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    lo[e] = __hmin2_nan(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
                    hi[e] = __hmax2_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
                }
            }
            if (gk == 0) {
                __half2 *dst = reinterpret_cast<__half2 *>(&sm.part[(b - b0) * subs + sub][16 * li]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dst[e] = lo[e];
                    dst[D / 2 + e] = hi[e];
                }
            }
        }
        __syncthreads();
        if (b1 - b0 == kGroup && subs == 1) {
            // a thread per row: the group's 16 blocks are one 32-byte sector of it
            for (int mc = threadIdx.x; mc < 2 * D; mc += kBThreads) {
                uint32_t w[kGroup / 2];
#pragma unroll
                for (int i = 0; i < kGroup / 2; ++i) {
                    const __half2 v = __halves2half2(sm.part[2 * i][mc], sm.part[2 * i + 1][mc]);
                    // -0 and +0 are one value, stored as +0
                    const __half2 z = __hadd2(v, __half2half2(__ushort_as_half(0)));
                    w[i] = *reinterpret_cast<const uint32_t *>(&z);
                }
                uint4 *dst = reinterpret_cast<uint4 *>(bounds + (((int64_t)sh * nt + b0 / kTile) * 2 * D + mc) * kTile + b0 % kTile);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
            for (int t = threadIdx.x; t < 2 * D * (b1 - b0); t += kBThreads) {
                const int b = b0 + t / (2 * D), mc = t % (2 * D);               // mc: [lo/hi][channel]
                const __half *p = &sm.part[(b - b0) * subs][mc];
                __half r = p[0];
                for (int q = 1; q < subs; ++q) r = mc < D ? __hmin_nan(r, p[q * (2 * D + 2)]) : __hmax_nan(r, p[q * (2 * D + 2)]);
                bounds[(((int64_t)sh * nt + b / kTile) * 2 * D + mc) * kTile + b % kTile] = __hadd(r, __ushort_as_half(0));
            }
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
// q carries 2^1000, the score 2^8. Bounds that are not finite have no such form: a warp that has met
// one (the largest magnitude of its loads says so) takes its tile's sums again, by conversions. Bound by the latency of its one pass: 1024 heads x 128 blocks
// (33.5 MB of bounds) are scored and chosen in 14.5 us.
constexpr int kSThreads = 128, kSWarps = kSThreads / 32;
constexpr double kQUp = 1.0715086071862673e301;                // 2^1000

__device__ __forceinline__ double half_field(uint32_t top)     // the fp16 bits in bits 16..31 of `top`
{
    return __hiloint2double((int)((uint32_t)((int32_t)top >> 6) & 0x81FFFC00u), 0);
}

__device__ __forceinline__ double half_value(uint32_t top)     // the same for every value
{
    return (double)__half2float(__ushort_as_half((unsigned short)(top >> 16))) * (1.0 / (kQUp * 256.0));
}

// The scores of tiles [t0, t1) of 64 blocks of one (sequence, KV head), by a CTA. Two tiles at a
// time when there are two (half the warps each), else one. Lane = (channel mod 4, group of 8
// blocks): a 16-byte load covers 8 blocks of a channel, a warp's load 4 channels. Scores go to
// `dst`, and to `keep` (shared memory) when given.
template <int D, int NQ>
struct ScoreSmem {
    double qs[NQ][D];
    double sum[kSWarps][NQ][kTile];
    int act[64], n_act;
};

template <int D, int NQ>
__device__ __forceinline__ void score_tiles(const CacheView &c, const __half *__restrict__ q, const __half *__restrict__ bounds,
                                            const uint8_t *__restrict__ modes, int sh, int nb, int nt, int t0, int t1,
                                            float *__restrict__ dst, float *keep, ScoreSmem<D, NQ> &sm)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane >> 3, b8 = lane & 7;
    const int64_t q0 = (int64_t)sh * c.G;
    if (warp == 0) {                             // the group's full queries
        int n = 0;
        for (int g0 = 0; g0 < c.G; g0 += 32) {
            const int g = g0 + lane;
            int m = KVQ_MODE_SKIP;
            if (g < c.G) {
                m = modes ? modes[q0 + g] : KVQ_MODE_FULL;
                if (m > 2) set_status(c.status, KVQ_ERR_MODE);
            }
            const uint32_t in = __ballot_sync(0xffffffffu, m == KVQ_MODE_FULL);
            if (m == KVQ_MODE_FULL) sm.act[n + __popc(in & ((1u << lane) - 1u))] = g;
            n += __popc(in);
        }
        if (lane == 0) sm.n_act = n;
    }
    __syncthreads();
    const int n_act = sm.n_act;
    for (int t = t0; t < t1; t += 2) {
        const int pair = t + 1 < t1 ? 2 : 1, wpt = kSWarps / pair;     // warps per tile
        const int tile = t + warp / wpt, w0 = warp % wpt;
        const uint4 *lo = reinterpret_cast<const uint4 *>(bounds + ((int64_t)sh * nt + tile) * 2 * D * kTile);
        const uint4 *hi = lo + D * (kTile / 8);
        const bool some = nb > tile * kTile;                   // (otherwise nothing of the tile is read)
        float best = -INFINITY;
        for (int a0 = 0; a0 < n_act; a0 += NQ) {
            const int n = min(NQ, n_act - a0);
            if (t == t0 || n_act > NQ) {
                for (int x = tid; x < NQ * D; x += kSThreads)
                    sm.qs[x / D][x % D] = x / D < n ? (double)__half2float(q[(q0 + sm.act[a0 + x / D]) * D + x % D]) * kQUp : 0.0;
                __syncthreads();
            }
            double acc[NQ][8];
#pragma unroll
            for (int g = 0; g < NQ; ++g)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[g][e] = 0.0;
            __half2 top = __half2half2(__ushort_as_half(0));   // the largest magnitude met
            if (some) {
#pragma unroll(NQ == 1 ? 8 : NQ == 2 ? 4 : 2)
                for (int ch = w0 * 4 + sub; ch < D; ch += 4 * wpt) {
                    uint4 l, u;
                    if (NQ == 1) {
                        l = u = __ldg((sm.qs[0][ch] < 0.0 ? lo : hi) + ch * (kTile / 8) + b8);
                    } else {
                        l = __ldg(lo + ch * (kTile / 8) + b8);
                        u = __ldg(hi + ch * (kTile / 8) + b8);
                    }
                    const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2 *>(&uw[e])));
                        if (NQ > 1) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2 *>(&lw[e])));
                    }
#pragma unroll
                    for (int g = 0; g < NQ; ++g) {
                        const double qv = sm.qs[g][ch];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = NQ == 1 ? uw[e] : (qv < 0.0 ? lw[e] : uw[e]);
                            acc[g][2 * e] = fma(qv, half_field(w << 16), acc[g][2 * e]);
                            acc[g][2 * e + 1] = fma(qv, half_field(w), acc[g][2 * e + 1]);
                        }
                    }
                }
            }
            const bool odd = __hisnan(__hmul(__low2half(top), __ushort_as_half(0))) ||
                             __hisnan(__hmul(__high2half(top), __ushort_as_half(0)));
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
                for (int g = 0; g < NQ; ++g)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[g][e] = 0.0;
#pragma unroll 1
                for (int ch = w0 * 4 + sub; ch < D; ch += 4 * wpt) {
                    const uint4 l = __ldg(lo + ch * (kTile / 8) + b8), u = __ldg(hi + ch * (kTile / 8) + b8);
                    const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int g = 0; g < NQ; ++g) {
                        const double qv = sm.qs[g][ch];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = qv < 0.0 ? lw[e] : uw[e];
                            acc[g][2 * e] = fma(qv, half_value(w << 16), acc[g][2 * e]);
                            acc[g][2 * e + 1] = fma(qv, half_value(w), acc[g][2 * e + 1]);
                        }
                    }
                }
            }
            // over the 4 channels of the lanes that share blocks: halves change hands, so that lane
            // sub is left with blocks 2 sub, 2 sub + 1 of its 8
#pragma unroll
            for (int g = 0; g < NQ; ++g) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double give = sub & 2 ? acc[g][e] : acc[g][e + 4], have = sub & 2 ? acc[g][e + 4] : acc[g][e];
                    acc[g][e] = have + __shfl_xor_sync(0xffffffffu, give, 16);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const double give = sub & 1 ? acc[g][e] : acc[g][e + 2], have = sub & 1 ? acc[g][e + 2] : acc[g][e];
                    sm.sum[warp][g][b8 * 8 + 2 * sub + e] = have + __shfl_xor_sync(0xffffffffu, give, 8);
                }
            }
            __syncthreads();
            if (tid < pair * kTile) {
                for (int g = 0; g < n; ++g) {
                    double v = 0.0;
                    for (int w = 0; w < wpt; ++w) v += sm.sum[tid / kTile * wpt + w][g][tid % kTile];
                    best = fmaxf(best, (float)(v * 256.0));
                }
            }
            __syncthreads();
        }
        if (tid < pair * kTile) {
            const int b = t * kTile + tid;
            const float v = b < nb ? best : -INFINITY;
            dst[b] = v;
            if (keep) keep[b] = v;
        }
    }
}

// ------------------------------------------------------------------ choice
// The k blocks of the largest keys, ties to the lower index, written in ascending order. Keys
// are the scores mapped to unsigned integers of the same order; forced blocks get the largest
// key. The k-th largest key is found bit by bit, from the top, until a threshold leaves
// exactly k keys (or all 32 bits are known and ties are left); the output places come from a
// prefix sum over the blocks in order.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x) x = -INFINITY;                                 // NaN ranks lowest
    const uint32_t u = __float_as_uint(x + 0.0f);              // -0 and +0 are one value
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct Choice {
    int nb, k, first, last;
};

// Sum over WARPS warps (one: no barrier). `slot` alternates between calls.
template <int WARPS>
__device__ __forceinline__ int count_all(int n, int (*part)[32], int slot)
{
    n = __reduce_add_sync(0xffffffffu, n);
    if (WARPS == 1) return n;
    if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = n;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < WARPS ? part[slot][lane] : 0);
}

// By WARPS warps (warps 0 .. WARPS - 1 of the block; all threads of the block when more than
// one), PER keys a thread; more blocks than that are walked in chunks, scores read again.
template <int WARPS, int PER>
__device__ __forceinline__ void choose(const float *sc, const Choice &ch, int32_t *__restrict__ out, int (*part)[32])
{
    constexpr int T = 32 * WARPS, CH = T * PER;
    const int tid = threadIdx.x % T, warp = tid >> 5, lane = tid & 31;
    const int nb = ch.nb, want = min(ch.k, nb);
    for (int i = want + tid; i < ch.k; i += T) out[i] = -1;
    uint32_t key[PER];
    auto load = [&](int base) {                                // keys of blocks base + tid * PER ..; 0 past the end
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int b = base + tid * PER + e;
            key[e] = 0;
            if (b < nb) key[e] = (b < ch.first || b >= nb - ch.last) ? 0xFFFFFFFFu : order_key(sc[b]);
        }
    };
    load(0);
    // `thr`: the largest threshold known to leave at least `want` keys; `have`: how many it leaves
    uint32_t thr = 0;
    int have = nb, slot = 0;
    for (int bit = 31; bit >= 0 && have != want; --bit) {
        const uint32_t t = thr | (1u << bit);
        int n = 0;
        for (int base = 0; base < nb; base += CH) {
            if (nb > CH) load(base);
#pragma unroll
            for (int e = 0; e < PER; ++e) n += key[e] >= t ? 1 : 0;
        }
        n = count_all<WARPS>(n, part, slot ^= 1);
        if (n >= want) {
            thr = t;
            have = n;
        }
    }
    // every key above thr, and those at thr in index order until `want` are taken
    int above = 0;
    for (int base = 0; base < nb; base += CH) {
        if (nb > CH) load(base);
#pragma unroll
        for (int e = 0; e < PER; ++e) above += key[e] > thr ? 1 : 0;
    }
    above = count_all<WARPS>(above, part, slot ^= 1);
    const int ties = want - above;
    int gt0 = 0, eq0 = 0;                                      // before this chunk: above thr, at thr
    for (int base = 0; base < nb; base += CH) {
        if (nb > CH) load(base);
        int mine = 0;                                          // above thr | at thr << 16
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (base + tid * PER + e >= nb) break;
            mine += key[e] > thr ? 1 : key[e] == thr ? 0x10000 : 0;
        }
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        int before = upto - mine, all = __shfl_sync(0xffffffffu, upto, 31);
        if (WARPS > 1) {
            __syncthreads();
            if (lane == 31) part[0][warp] = upto;
            __syncthreads();
            const int v = lane < WARPS ? part[0][lane] : 0;
            before += __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
            all = __reduce_add_sync(0xffffffffu, v);
        }
        int gp = gt0 + (before & 0xFFFF), ep = eq0 + (before >> 16);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int b = base + tid * PER + e;
            if (b >= nb) break;
            if (key[e] > thr) out[gp++ + min(ep, ties)] = b;
            else if (key[e] == thr) {
                if (ep < ties) out[gp + ep] = b;
                ++ep;
            }
        }
        gt0 += all & 0xFFFF;
        eq0 += all >> 16;
    }
}

__device__ __forceinline__ void no_blocks(int32_t *out, int k)
{
    for (int i = threadIdx.x; i < k; i += blockDim.x) out[i] = -1;
}

// Scores of one (sequence, KV head, tile) per CTA.
template <int D, int NQ>
__global__ void __launch_bounds__(kSThreads)
score_kernel(CacheView c, const __half *__restrict__ q, const __half *__restrict__ bounds, const uint8_t *__restrict__ modes,
             int block, int nt, float *__restrict__ scores)
{
    __shared__ ScoreSmem<D, NQ> sm;
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x / nt, tile = blockIdx.x % nt;
    const int nb = (c.len[sh] + block - 1) / block;
    score_tiles<D, NQ>(c, q, bounds, modes, sh, nb, nt, tile, tile + 1, scores + (int64_t)sh * nt * kTile, nullptr, sm);
}

// The choice of one (sequence, KV head) per CTA, from scores in memory: long contexts, whose
// scores are read once per bit of the threshold.
constexpr int kCThreads = 1024, kCPer = 8;
__global__ void __launch_bounds__(kCThreads)
choose_kernel(CacheView c, const float *__restrict__ scores, const uint8_t *__restrict__ modes, int block, int nt, int k, int first,
              int last, int32_t *__restrict__ ids)
{
    __shared__ int part[2][32];
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x;
    bool any = !modes;
    if (modes)
        for (int g = 0; g < c.G; ++g) any = any || modes[(int64_t)sh * c.G + g] == KVQ_MODE_FULL;
    const Choice ch{(c.len[sh] + block - 1) / block, k, first, last};
    if (!any) no_blocks(ids + (int64_t)sh * k, k);
    else choose<kCThreads / 32, kCPer>(scores + (int64_t)sh * nt * kTile, ch, ids + (int64_t)sh * k, part);
}

// Both in one launch for up to kFuseTiles tiles: a cluster of CTAs per (sequence, KV head), each
// scoring a run of its tiles; the scores meet in the first one's shared memory, which chooses.
constexpr int kFuseTiles = 64, kMaxCluster = 8;
template <int D, int NQ>
__global__ void __launch_bounds__(kSThreads)
select_kernel(CacheView c, const __half *__restrict__ q, const __half *__restrict__ bounds, const uint8_t *__restrict__ modes,
              int block, int nt, int k, int first, int last, int n_cta, float *__restrict__ scores, int32_t *__restrict__ ids)
{
    namespace cg = cooperative_groups;
    __shared__ ScoreSmem<D, NQ> sm;
    __shared__ int part[2][32];
    extern __shared__ float keep[];              // nt tiles
    pdl_wait();
    pdl_trigger();
    const int sh = blockIdx.x / n_cta, rank = blockIdx.x % n_cta;
    const Choice ch{(c.len[sh] + block - 1) / block, k, first, last};
    const int per = (nt + n_cta - 1) / n_cta, t0 = min(nt, rank * per), t1 = min(nt, t0 + per);
    float *first_keep = keep;
    if (n_cta > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();                               // the first CTA has started: its shared memory may be written
        first_keep = cl.map_shared_rank(keep, 0);
    }
    score_tiles<D, NQ>(c, q, bounds, modes, sh, ch.nb, nt, t0, t1, scores + (int64_t)sh * nt * kTile, first_keep, sm);
    if (n_cta > 1) {
        cg::this_cluster().sync();
        if (rank > 0) return;
    } else {
        __syncthreads();
    }
    int32_t *out = ids + (int64_t)sh * k;
    if (sm.n_act == 0) no_blocks(out, k);
    else if (nt > 16) choose<kSWarps, kFuseTiles * kTile / kSThreads>(keep, ch, out, part);
    else if (nt > 4) choose<kSWarps, 16 * kTile / kSThreads>(keep, ch, out, part);
    else if (threadIdx.x < 32) {
        if (nt > 2) choose<1, 8>(keep, ch, out, part);
        else choose<1, 4>(keep, ch, out, part);
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
    auto launch = [&](auto kernel, size_t smem, int warps) {
        const cudaError_t e = ensure_smem_attr((const void *)kernel, smem);
        return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(32 * warps), smem, st, c, block, cu, bounds, nt, per);
    };
    // 4 warps a CTA when only new tokens' blocks are renewed (often one: a quarter of it per warp,
    // and twice as many CTAs in flight: 1024 heads 15.7 -> 13.3 us), 8 when all are
    if (c.D == 128) {
        if (cu) return c.ptab ? launch(bounds_kernel<128, true, 4>, sizeof(BoundsSmem<128, 4>), 4)
                              : launch(bounds_kernel<128, false, 4>, sizeof(BoundsSmem<128, 4>), 4);
        return c.ptab ? launch(bounds_kernel<128, true, 8>, sizeof(BoundsSmem<128, 8>), 8)
                      : launch(bounds_kernel<128, false, 8>, sizeof(BoundsSmem<128, 8>), 8);
    }
    if (cu) return c.ptab ? launch(bounds_kernel<64, true, 4>, sizeof(BoundsSmem<64, 4>), 4)
                          : launch(bounds_kernel<64, false, 4>, sizeof(BoundsSmem<64, 4>), 4);
    return c.ptab ? launch(bounds_kernel<64, true, 8>, sizeof(BoundsSmem<64, 8>), 8)
                  : launch(bounds_kernel<64, false, 8>, sizeof(BoundsSmem<64, 8>), 8);
}

namespace {
template <int D, int NQ>
cudaError_t launch_select(const __half *q, const kvq_cache *cache, const __half *bounds, int block, const uint8_t *modes, int k,
                          int first, int last, float *scores, int32_t *ids, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const int nb = (cache->max_cap + block - 1) / block, nt = (nb + kTile - 1) / kTile;
    const int64_t sh = (int64_t)c.B * c.H;
    if (nt <= kFuseTiles) {
        // a CTA per (sequence, KV head), more of them while there are fewer than two an SM
        const int64_t want = (2 * (int64_t)num_sms() + sh - 1) / sh;
        const int n_cta = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxCluster), nt));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sh * n_cta));
        cfg.blockDim = dim3(kSThreads);
        cfg.dynamicSmemBytes = (size_t)nt * kTile * sizeof(float);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)n_cta;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = n_cta > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, select_kernel<D, NQ>, c, q, bounds, modes, block, nt, k, first, last, n_cta, scores, ids);
    }
    const cudaError_t e = launch_pdl(score_kernel<D, NQ>, dim3((unsigned)(sh * nt)), dim3(kSThreads), 0, st, c, q, bounds, modes,
                                     block, nt, scores);
    if (e != cudaSuccess) return e;
    return launch_pdl(choose_kernel, dim3((unsigned)sh), dim3(kCThreads), 0, st, c, (const float *)scores, modes, block, nt, k,
                      first, last, ids);
}
} // namespace

cudaError_t launch_select_blocks(const __half *q, const kvq_cache *c, const __half *bounds, int block, const uint8_t *modes,
                                 int k, int first, int last, float *scores, int32_t *ids, cudaStream_t st)
{
    const int G = c->view.G;
    auto go = [&](auto f) { return f(q, c, bounds, block, modes, k, first, last, scores, ids, st); };
    if (c->D == 128) return G == 1 ? go(launch_select<128, 1>) : G == 2 ? go(launch_select<128, 2>) : go(launch_select<128, 4>);
    return G == 1 ? go(launch_select<64, 1>) : G == 2 ? go(launch_select<64, 2>) : go(launch_select<64, 4>);
}

} // namespace kvq
