// Routed decode attention over chosen blocks (Eq. 2 with the full resolution replaced by a
// choice of blocks): one query per (sequence, query head) at t = len - 1. A skip query's
// output is 0, a local query attends over keys [max(0, t - w), t], a full query over the keys
// of the blocks listed for its KV head.
//
//   logit_j = q . deq(k_j) / sqrt(D),  p = softmax,  out = sum_j p_j deq(v_j)
//
// With codes c, scale s, zero z (Eq. 4), the centred codes c' = c - 2^(b-1) (b < 16) and
// z' = z + 2^(b-1) s:
//   q . deq(k_j) = s_j (q . c_j) + z_j sum(q),   sum_j p_j deq(v_j) = sum_j (p_j s_j) c'_j + sum_j p_j z'_j
// Centring keeps the two sums of V, which run over many keys, from cancelling.
//
// One warp serves up to 8 query heads of a KV head at once with m16n8k16 matrix
// instructions (fp16 operands, fp32 sums), 16 keys at a time:
//   S^T [16 keys x 8 queries]      = C [16 x D] . Q^T [D x 8]            D/16 instructions
//   O^T [D channels x 8 queries]  += C'^T [D x 16] . W^T [16 x 8]        2 D/16 (up to 4 queries: D/16)
// The products are exact: q, the codes and native values are fp16 numbers. The weights
// w = p s are not, so each goes in as two fp16 numbers, w = hi + lo (22 bits), in units that
// keep them far from fp16's subnormals: a power of two above the largest s_V among the
// tile's keys of one width, times 2^-6 (p is at most 2^8, see below). Up to 4 queries leave
// columns 4..7 of the instruction to the second numbers. The queries are too few for the
// 128-row tiles of tcgen05 (G is 1 to 64, and the codes would have to be unpacked to shared
// memory first).
//
// The keys of a tile (up to 1024 of a CTA's share) are first sorted by width, so that 16 keys
// of one width unpack by one code path; the warps take the 16-key steps in turn. A 16-bit
// half of a word holds 16/b codes. For K the two halves are channels of one key (q is stored
// in the matching order, one order per width) and a mask alone makes an operand: a field in
// place IS the fp16 subnormal c 2^(pos - 24), and the sums of each position are scaled once
// per key. For V the halves are the same channels of two keys (one byte permutation), and
// the fields join the mantissa of 2^(10 - pos), whose last place there is 1, before
// 2^(10 - pos) + 2^(b-1) is subtracted.
//
// Online softmax: the running maximum of a query moves only when a logit exceeds it by
// more than 8 (log2 units), a warp-uniform branch. The warps of a CTA share a (sequence, KV
// head) and merge at the end; up to 8 CTAs that share one form a cluster and merge through
// distributed shared memory; more of them leave partial states in the caller's scratch, which
// a second launch merges.
//
// Latency: the records of a tile are asked for as soon as their offsets are known (bulk
// prefetches into L2, one per 16 consecutive keys), so the loads of the 16-key steps, which
// each warp issues one step at a time, find them there.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kQ = 8;                            // query heads per warp
constexpr int kSteps = 4;                        // 32-key steps of a warp's part of a tile
constexpr int kTileKeys = kWarps * kSteps * 32;  // keys sorted by width at a time
constexpr int kSlots = kTileKeys + 4 * 16;       // each width's keys are padded to 16
constexpr float kLazy = 8.f;                     // running-max slack, log2 units
constexpr float kMInit = -1e30f;                 // running max before the first key
constexpr int kMaxCluster = 8;                   // CTAs of a cluster
constexpr uint32_t kValid = 4u;                  // meta bit of a real key (bits 0..1: width code)

struct Tile {
    float4 side[kSlots];                         // (s_K cdot 2^24 (fp16: cdot), z_K cdot, s_V, z'_V), sorted
    uint32_t ent[kSlots];                        // record offset | kValid | width code, sorted
};

template <int D>
struct Smem {
    union {
        Tile tile;
        float o[kWarps][kQ][D + 4];              // the warps' states: o, then m and l
    };
    uint4 q[4][D / 32][32];                      // per width: a lane's query operands, 16 bytes at a time
    __half rows[kQ][D + 8];                      // the queries
    float qsum[kQ];
    float done[kQ][D + 4];                       // the CTA's state for the cluster: o, then m and l
    int cnt[kWarps][4];                          // keys of each width in each warp's part of the tile
    uint32_t some[4], smax[4];                   // per width: a real key's entry; the largest s_V's bits
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)     // an 8x8 matrix of 16-bit values
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// (a, b) minus the fp16 pair h, as an fp16 pair
__device__ __forceinline__ uint32_t rest_half(float a, float b, uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The field of BITS bits at SHIFT in both halves of p as fp16 subnormals: c 2^(SHIFT - 24) each.
template <int BITS, int SHIFT>
__device__ __forceinline__ uint32_t raw_field(uint32_t p)
{
    return p & ((((1u << BITS) - 1u) << SHIFT) * 0x10001u);
}

// The same field centred, c - 2^(BITS - 1): it joins the mantissa of 2^(10 - SHIFT), whose last
// place there is 1, then 2^(10 - SHIFT) + 2^(BITS - 1) is subtracted; every step is exact.
template <int BITS, int SHIFT>
__device__ __forceinline__ uint32_t mid_field(uint32_t p)
{
    constexpr uint32_t magic = (uint32_t)((25 - SHIFT) << 10) * 0x10001u;
    constexpr uint32_t off = (0x8000u | (uint32_t)((25 - SHIFT) << 10) | (1u << (BITS - 1 + SHIFT))) * 0x10001u;
    const uint32_t x = raw_field<BITS, SHIFT>(p) | magic, m = off;
    const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&m));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The 16/BITS centred codes in each half of p (LSB-first) as fp16 pairs: x[i] = (field i of
// the low half, field i of the high half) - 2^(BITS-1).
template <int BITS>
__device__ __forceinline__ void mid_fields(uint32_t p, uint32_t (&x)[16 / BITS])
{
    const uint32_t h = p >> 8;
    if constexpr (BITS == 8) {
        x[0] = mid_field<8, 0>(p);
        x[1] = mid_field<8, 0>(h);
    } else if constexpr (BITS == 4) {
        x[0] = mid_field<4, 0>(p);
        x[1] = mid_field<4, 4>(p);
        x[2] = mid_field<4, 0>(h);
        x[3] = mid_field<4, 4>(h);
    } else {
        x[0] = mid_field<2, 0>(p);
        x[1] = mid_field<2, 2>(p);
        x[2] = mid_field<2, 4>(p);
        x[3] = mid_field<2, 6>(p);
        x[4] = mid_field<2, 0>(h);
        x[5] = mid_field<2, 2>(h);
        x[6] = mid_field<2, 4>(h);
        x[7] = mid_field<2, 6>(h);
    }
}

// One word of K of two keys (rows g: x, g + 8: y) against its query operands: s[SHIFT / BITS]
// gains q . c 2^(SHIFT - 24) over the word's fields at SHIFT and SHIFT + 8 of both halves.
template <int BITS, int SHIFT>
__device__ __forceinline__ void k_fields(float (&s)[4][4], uint32_t x, uint32_t y, const uint32_t *q)
{
    if constexpr (SHIFT < 8) {
        constexpr int f = SHIFT / BITS;
        mma(s[f], raw_field<BITS, SHIFT>(x), raw_field<BITS, SHIFT>(y), raw_field<BITS, SHIFT>(x >> 8),
            raw_field<BITS, SHIFT>(y >> 8), q[f], q[f + 8 / BITS]);
        k_fields<BITS, SHIFT + BITS>(s, x, y, q);
    }
}

// Where a stream's bytes are: PAGED as RecLoc::at, else base + offset.
template <bool PAGED>
__device__ __forceinline__ const uint8_t *byte_at(const RecLoc &L, uint32_t off)
{
    return PAGED ? L.at(off) : L.base + off;
}

__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Bytes [o0, o1) of a stream (multiples of 16) into L2, page by page.
template <bool PAGED>
__device__ __forceinline__ void prefetch_records(const RecLoc &L, uint32_t o0, uint32_t o1)
{
    if constexpr (!PAGED) {
        prefetch_l2(L.base + o0, o1 - o0);
    } else {
        while (o0 < o1) {
            const uint32_t n = min(o1 - o0, (1u << L.shift) - (o0 & ((1u << L.shift) - 1u)));
            prefetch_l2(L.at(o0), n);
            o0 += n;
        }
    }
}

// BYTES bytes of a record at logical offset `off` of the stream (aligned to min(BYTES, 16), so a
// 16-byte piece lies in one page) into words; 2 bytes fill the low half of one word.
template <int BYTES, bool PAGED>
__device__ __forceinline__ void load_bytes(const RecLoc &L, uint32_t off, uint32_t (&w)[(BYTES + 3) / 4])
{
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(byte_at<PAGED>(L, off + 16u * i)));
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
    } else if constexpr (BYTES == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(byte_at<PAGED>(L, off)));
        w[0] = x.x;
        w[1] = x.y;
    } else if constexpr (BYTES == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(byte_at<PAGED>(L, off)));
    } else {
        w[0] = __ldg(reinterpret_cast<const unsigned short *>(byte_at<PAGED>(L, off)));
    }
}

// A warp's attention state. Lane (g, t) = (lane / 4, lane % 4): m, l, pz of queries 2t, 2t + 1
// (l and pz over the lane's own keys), o[mt] = channels g D/8 + 2 mt (entries 0, 1) and + 1
// (entries 2, 3) of those queries, in units of `unit`.
template <int D>
struct State {
    float o[D / 16][4];
    float m[2], l[2], pz[2];
    float unit;
};

// Slots base, base + 16 kWarps, .. below `end` of the sorted tile, 16 at a time, all of width
// 2 << CLS.
template <int D, int CLS, bool PAGED, int NQ>
__device__ __forceinline__ void run_class(State<D> &st, const Smem<D> &sm, const RecLoc &L, int base, int end, float fac, bool on0,
                                          bool on1)
{
    const Tile &tl = sm.tile;
    constexpr int BITS = 2 << CLS;
    constexpr int KW = D * BITS / 128;           // words of a lane's D/4 channels of K
    constexpr int VB = D * BITS / 64;            // bytes of a lane's D/8 channels of V
    constexpr int F = 16 / BITS;                 // fields per half word
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t q[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint4 x = sm.q[CLS][i][lane];
        q[4 * i] = x.x;
        q[4 * i + 1] = x.y;
        q[4 * i + 2] = x.z;
        q[4 * i + 3] = x.w;
    }
    const float qs0 = sm.qsum[2 * t], qs1 = sm.qsum[2 * t + 1];
    for (int c = base; c < end; c += 16 * kWarps) {
        const uint32_t e0 = tl.ent[c + g], e1 = tl.ent[c + 8 + g];
        const uint2 f0 = *reinterpret_cast<const uint2 *>(&tl.ent[c + 2 * t]);
        const uint2 f1 = *reinterpret_cast<const uint2 *>(&tl.ent[c + 8 + 2 * t]);
        uint32_t k0[KW], k1[KW];
        load_bytes<KW * 4, PAGED>(L, (e0 & ~15u) + 4 * KW * t, k0);
        load_bytes<KW * 4, PAGED>(L, (e1 & ~15u) + 4 * KW * t, k1);
        uint32_t v[4][(VB + 3) / 4];
        const uint32_t vo = D * BITS / 8 + VB * g;
        load_bytes<VB, PAGED>(L, (f0.x & ~15u) + vo, v[0]);
        load_bytes<VB, PAGED>(L, (f0.y & ~15u) + vo, v[1]);
        load_bytes<VB, PAGED>(L, (f1.x & ~15u) + vo, v[2]);
        load_bytes<VB, PAGED>(L, (f1.y & ~15u) + vo, v[3]);
        // S^T: a word gives 16/BITS operand pairs of its key; equal fields share a sum (for wide codes
        // two sums alternate), so no chain of dependent instructions is longer than 4
        float sf[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sf[i][0] = sf[i][1] = sf[i][2] = sf[i][3] = 0.f;
        if constexpr (CLS == 3) {
#pragma unroll
            for (int i = 0; i < KW; i += 2) mma(sf[i / 2 & 1], k0[i], k1[i], k0[i + 1], k1[i + 1], q[i], q[i + 1]);
        } else if constexpr (CLS == 2) {
#pragma unroll
            for (int i = 0; i < KW; ++i)
                mma(sf[i & 1], raw_field<8, 0>(k0[i]), raw_field<8, 0>(k1[i]), raw_field<8, 0>(k0[i] >> 8),
                    raw_field<8, 0>(k1[i] >> 8), q[2 * i], q[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < KW; ++i) k_fields<BITS, 0>(sf, k0[i], k1[i], q + i * F);
        }
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (CLS >= 2) s[i] = sf[0][i] + sf[1][i];
            else if (CLS == 1) s[i] = fmaf(sf[1][i], 0.0625f, sf[0][i]);
            else s[i] = fmaf(fmaf(fmaf(sf[3][i], 0.25f, sf[2][i]), 0.25f, sf[1][i]), 0.25f, sf[0][i]);
        }
        const float4 sd0 = tl.side[c + g], sd1 = tl.side[c + 8 + g];
        const bool v0 = e0 & kValid, v1 = e1 & kValid;
        float lg[4];
        lg[0] = v0 && on0 ? fmaf(sd0.x, s[0], sd0.y * qs0) : -INFINITY;
        lg[1] = v0 && on1 ? fmaf(sd0.x, s[1], sd0.y * qs1) : -INFINITY;
        lg[2] = v1 && on0 ? fmaf(sd1.x, s[2], sd1.y * qs0) : -INFINITY;
        lg[3] = v1 && on1 ? fmaf(sd1.x, s[3], sd1.y * qs1) : -INFINITY;
        float mx0 = fmaxf(lg[0], lg[2]), mx1 = fmaxf(lg[1], lg[3]);
        if (__any_sync(0xffffffffu, mx0 > st.m[0] + kLazy || mx1 > st.m[1] + kLazy)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
            }
            const float n0 = fmaxf(st.m[0], mx0), n1 = fmaxf(st.m[1], mx1);
            const float c0 = ex2(st.m[0] - n0), c1 = ex2(st.m[1] - n1);
            st.m[0] = n0;
            st.m[1] = n1;
            st.l[0] *= c0;
            st.l[1] *= c1;
            st.pz[0] *= c0;
            st.pz[1] *= c1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[i][0] *= c0;
                st.o[i][1] *= c1;
                st.o[i][2] *= c0;
                st.o[i][3] *= c1;
            }
        }
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(lg[i] - st.m[i & 1]);
        st.l[0] += p[0] + p[2];
        st.l[1] += p[1] + p[3];
        if (CLS != 3) {
            st.pz[0] = fmaf(p[0], sd0.w, fmaf(p[2], sd1.w, st.pz[0]));
            st.pz[1] = fmaf(p[1], sd0.w, fmaf(p[3], sd1.w, st.pz[1]));
        }
        const float w0 = CLS == 3 ? fac : sd0.z * fac, w1 = CLS == 3 ? fac : sd1.z * fac;
        p[0] *= w0;
        p[1] *= w0;
        p[2] *= w1;
        p[3] *= w1;
        uint32_t h0 = pack_half(p[0], p[1]), h1 = pack_half(p[2], p[3]);
        const uint32_t r0 = rest_half(p[0], p[1], h0), r1 = rest_half(p[2], p[3], h1);
        uint32_t bh0, bh1, bl0 = 0u, bl1 = 0u;
        if (NQ == 4) {                           // columns 4..7 carry the rests of queries 0..3
            bh0 = transpose8(t < 2 ? h0 : r0);
            bh1 = transpose8(t < 2 ? h1 : r1);
        } else {
            bh0 = transpose8(h0);
            bh1 = transpose8(h1);
            bl0 = transpose8(r0);
            bl1 = transpose8(r1);
        }
        // word i of the four keys, half by half: channels (32 i + 16 half)/BITS + field
#pragma unroll
        for (int i = 0; i < (VB + 3) / 4; ++i) {
#pragma unroll
            for (int half = 0; half < (VB >= 4 ? 2 : 1); ++half) {
                const uint32_t sel = half ? 0x7632 : 0x5410;
                const uint32_t pa = __byte_perm(v[0][i], v[1][i], sel), pb = __byte_perm(v[2][i], v[3][i], sel);
                if constexpr (F == 1) {
                    // one channel per half: rows g and g + 8 of the instruction are the word's two halves
                    if (half == 0) {
                        const uint32_t qa = __byte_perm(v[0][i], v[1][i], 0x7632), qb = __byte_perm(v[2][i], v[3][i], 0x7632);
                        mma(st.o[i], pa, qa, pb, qb, bh0, bh1);
                        if (NQ == 8) mma(st.o[i], pa, qa, pb, qb, bl0, bl1);
                    }
                } else {
                    uint32_t xa[F], xb[F];
                    mid_fields<BITS>(pa, xa);
                    mid_fields<BITS>(pb, xb);
#pragma unroll
                    for (int f = 0; f < F; f += 2) {
                        const int mt = ((2 * i + half) * F + f) / 2;
                        mma(st.o[mt], xa[f], xa[f + 1], xb[f], xb[f + 1], bh0, bh1);
                        if (NQ == 8) mma(st.o[mt], xa[f], xa[f + 1], xb[f], xb[f + 1], bl0, bl1);
                    }
                }
            }
        }
    }
}

struct Job {
    const int32_t *ids;
    const uint8_t *modes;
    int k, block_shift, w, n_split, n_sub, qs;   // qs: queries per partial in the scratch
    float *part;                                 // [unit][n_split][qs][D + 4]
};

template <int D, bool PAGED, int NQ>
__global__ void __launch_bounds__(kThreads, 2)
decode_blocks_kernel(CacheView c, const __half *__restrict__ q, Job job, float *__restrict__ out)
{
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    pdl_wait();
    pdl_trigger();
    const int split = blockIdx.x % job.n_split, unit = blockIdx.x / job.n_split;
    const int sub = unit % job.n_sub, sh = unit / job.n_sub, s = sh / c.H, h = sh % c.H;
    const int g0 = sub * NQ, nq = min(NQ, c.G - g0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3;
    const int64_t q0 = (int64_t)sh * c.G + g0;   // first query head of the unit
    const int len = c.len[sh];
    const int64_t slot0 = slot_of(c, s, h, 0);
    uint32_t full = 0, local = 0;
    for (int i = 0; i < nq; ++i) {
        const int m = job.modes[q0 + i];
        full |= (m == KVQ_MODE_FULL ? 1u : 0u) << i;
        local |= (m == KVQ_MODE_LOCAL ? 1u : 0u) << i;
        if (m > 2 && tid == 0 && split == 0) set_status(c.status, KVQ_ERR_MODE);
    }
    // the unit's entries: the listed blocks' keys (padded to 32), then the local window's; its
    // CTAs take equal shares, multiples of 32
    const int nb = (len + (1 << job.block_shift) - 1) >> job.block_shift;
    const int e_block = full ? ((min(job.k, nb) << job.block_shift) + 31) & ~31 : 0;
    if (full && sub == 0 && split == 0)          // no list of distinct blocks is longer than nb
        for (int x = nb + tid; x < job.k; x += kThreads)
            if (job.ids[(int64_t)sh * job.k + x] >= 0) set_status(c.status, KVQ_ERR_DEVICE_CHECK);
    const int wl = min(len, (int)min((int64_t)job.w + 1, (int64_t)len));
    const int e_all = e_block + (local ? wl : 0);
    const int share = ((e_all + job.n_split - 1) / job.n_split + 31) & ~31;

    // the queries, then their operands in each width's order and their sums over channels
    for (int x = tid; x < kQ * (D / 8); x += kThreads) {
        const int qi = x / (D / 8), ch = x % (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (qi < nq) v = __ldg(reinterpret_cast<const uint4 *>(q + (q0 + qi) * D) + ch);
        *reinterpret_cast<uint4 *>(&sm.rows[qi][8 * ch]) = v;
    }
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < 4 * (D / 32) * 32; x += kThreads) {
        const int cls = x / (D / 32 * 32), i = x / 32 % (D / 32), ln = x % 32;
        const int ch0 = (ln & 3) * (D / 4), fl = 3 - cls, f = 1 << fl;     // f = 16 / bits fields per half word
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = 4 * i + e;             // operand pair: word p / f, field p % f
            const __half *src = &sm.rows[(ln >> 2) & (NQ - 1)][ch0 + ((p >> fl) << (fl + 1)) + (p & (f - 1))];
            const __half2 v = __halves2half2(src[0], src[f]);
            r[e] = *reinterpret_cast<const uint32_t *>(&v);
        }
        sm.q[cls][i][ln] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    static_assert(kWarps == kQ, "a warp sums one query");
    {
        const int qi = warp;
        float a = 0.f;
#pragma unroll
        for (int ch = 0; ch < D; ch += 32) a += __half2float(sm.rows[qi & (NQ - 1)][ch + lane]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
        if (lane == 0) sm.qsum[qi] = a;
    }
    __syncthreads();

    State<D> st;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        st.m[i] = kMInit;
        st.l[i] = st.pz[i] = 0.f;
    }
    st.unit = 1.f;
    const float cdot = kLog2e / sqrtf((float)D);
    Tile &tl = sm.tile;
    const RecLoc L = rec_loc(c, s, h, 0);
    const int a0 = min(e_all, split * share), a1 = min(e_all, a0 + share);
    for (int a = a0; a < a1;) {
        // a tile: up to kTileKeys entries of one kind, the warps' parts multiples of 32
        const bool blocks = a < e_block;
        const int n = min(kTileKeys, (blocks ? min(a1, e_block) : a1) - a);
        const int per = ((n + kWarps - 1) / kWarps + 31) & ~31;
        const int p0 = warp * per, p1 = min(n, p0 + per);
        const uint32_t act = blocks ? full : local;
        uint32_t mt[kSteps], bal[kSteps][4];
        int64_t slot[kSteps];
        int cnt[4] = {0, 0, 0, 0};
        if (tid < 4) sm.smax[tid] = 0u;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            mt[i] = 0;
            slot[i] = slot0;
            const int e = a + p0 + i * 32 + lane;
            if (p0 + i * 32 >= p1) continue;
            int j = -1;
            if (e < a + p1) {
                if (blocks) {
                    const int x = e >> job.block_shift;
                    const int id = x < job.k ? job.ids[(int64_t)sh * job.k + x] : -1;
                    if (id >= 0) {
                        const int before = x > 0 ? job.ids[(int64_t)sh * job.k + x - 1] : -1;
                        if ((x > 0 && before < 0) || id <= before || id >= nb) {
                            set_status(c.status, KVQ_ERR_DEVICE_CHECK);
                        } else {
                            j = (id << job.block_shift) + (e & ((1 << job.block_shift) - 1));
                            if (j >= len) j = -1;
                        }
                    }
                } else {
                    j = len - wl + e - e_block;
                }
            }
            if (j >= 0) {
                slot[i] = slot0 + j;
                mt[i] = c.meta[slot[i]] | kValid;
            }
        }
        // 16 consecutive entries are consecutive keys, the valid ones in front: ask for their
        // side entries and records
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w) bal[i][w] = 0u;
            if (p0 + i * 32 >= p1) continue;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                bal[i][w] = __ballot_sync(0xffffffffu, (mt[i] & 7u) == (kValid | w));
                cnt[w] += __popc(bal[i][w]);
            }
            const uint32_t ok = bal[i][0] | bal[i][1] | bal[i][2] | bal[i][3];
            const int hb = lane & 16, keys = __popc((ok >> hb) & 0xFFFFu);
            const uint32_t last = __shfl_sync(0xffffffffu, mt[i], hb + max(keys - 1, 0));
            if (lane == hb && keys > 0) {
                prefetch_l2(&c.side[slot[i]], 16u * keys);
                prefetch_records<PAGED>(L, mt[i] & ~15u, (last & ~15u) + ((uint32_t)(D / 2) << (last & 3u)));
            }
        }
        if (lane < 4) sm.cnt[warp][lane] = lane == 0 ? cnt[0] : lane == 1 ? cnt[1] : lane == 2 ? cnt[2] : cnt[3];
        __syncthreads();
        // slots: width by width, each width's keys in the warps' order, padded to 16
        int all[4], at[4], first[5];
        first[0] = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            all[w] = 0;
            at[w] = 0;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const int m = sm.cnt[x][w];
                if (x < warp) at[w] += m;
                all[w] += m;
            }
            at[w] += first[w];
            first[w + 1] = first[w] + ((all[w] + 15) & ~15);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (p0 + i * 32 >= p1) continue;
            const int w = mt[i] & 3;
            const uint32_t b = w == 0 ? bal[i][0] : w == 1 ? bal[i][1] : w == 2 ? bal[i][2] : bal[i][3];
            const int to = w == 0 ? at[0] : w == 1 ? at[1] : w == 2 ? at[2] : at[3];
            float4 sd = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mt[i] & kValid) {
                sd = __ldg(&c.side[slot[i]]);
                const int pos = to + __popc(b & ((1u << lane) - 1u));
                const float mid = w == 3 ? 0.f : (float)(1 << ((2 << w) - 1));
                tl.ent[pos] = mt[i];
                tl.side[pos] = make_float4(sd.x * (w == 3 ? cdot : cdot * 16777216.f), sd.y * cdot, sd.z, fmaf(mid, sd.z, sd.w));
                sm.some[w] = mt[i];               // any one of them
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, w == x ? __float_as_uint(sd.z) : 0u);
                if (lane == 0 && bal[i][x]) atomicMax(&sm.smax[x], top);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) at[x] += __popc(bal[i][x]);
        }
        __syncthreads();
        // padding up to 16: a real record's offset, no kValid
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int to = first[w] + all[w] + lane;
            if (warp == w && all[w] > 0 && to < first[w + 1]) {
                tl.ent[to] = sm.some[w] & ~kValid;
                tl.side[to] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        __syncthreads();
        const bool on0 = (act >> (2 * t & (NQ - 1))) & 1u, on1 = (act >> ((2 * t & (NQ - 1)) + 1)) & 1u;
        // 16-key steps dealt to the warps in turn, so that they run one width's code at a time
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b0 = first[w] + ((warp - first[w] / 16) & (kWarps - 1)) * 16, b1 = first[w + 1];
            if (b0 >= b1) continue;
            // weights in units of S / 64, S a power of two above the largest scale (1 for fp16 values)
            float fac = 64.f, unit = 0.015625f;
            if (w != 3) {
                const int e = min(max((int)(sm.smax[w] >> 23) + 1, 87), 167);     // biased exponent of S
                unit = __uint_as_float((uint32_t)(e - 6) << 23);
                fac = __uint_as_float((uint32_t)(254 - e + 6) << 23);
            }
            if (unit != st.unit) {
                const float r = st.unit / unit;  // a power of two: exact
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    st.o[i][0] *= r;
                    st.o[i][1] *= r;
                    st.o[i][2] *= r;
                    st.o[i][3] *= r;
                }
                st.unit = unit;
            }
            if (w == 0) run_class<D, 0, PAGED, NQ>(st, sm, L, b0, b1, fac, on0, on1);
            else if (w == 1) run_class<D, 1, PAGED, NQ>(st, sm, L, b0, b1, fac, on0, on1);
            else if (w == 2) run_class<D, 2, PAGED, NQ>(st, sm, L, b0, b1, fac, on0, on1);
            else run_class<D, 3, PAGED, NQ>(st, sm, L, b0, b1, fac, on0, on1);
        }
        a += n;
        __syncthreads();                         // the tile's slots are read; the next one overwrites them
    }

    // this warp's sums over its lanes, then the warps' states through shared memory
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], d);
            st.pz[i] += __shfl_xor_sync(0xffffffffu, st.pz[i], d);
        }
    }
    if (NQ == 4) {                               // the rests join their queries
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[mt][i] += __shfl_down_sync(0xffffffffu, st.o[mt][i], 2);
    }
    if (2 * t < nq) {
        const int g = lane >> 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float *o = sm.o[warp][2 * t + i];
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                o[g * (D / 8) + 2 * mt] = fmaf(st.o[mt][i], st.unit, st.pz[i]);
                o[g * (D / 8) + 2 * mt + 1] = fmaf(st.o[mt][2 + i], st.unit, st.pz[i]);
            }
            if (g == 0) {
                o[D] = st.m[i];
                o[D + 1] = st.l[i];
            }
        }
    }
    __syncthreads();
    const bool cluster = job.n_split > 1 && job.n_split <= kMaxCluster;
    for (int x = tid; x < nq * D; x += kThreads) {
        const int qi = x / D, ch = x % D;
        float M = kMInit, l = 0.f, o = 0.f;
#pragma unroll
        for (int wp = 0; wp < kWarps; ++wp) M = fmaxf(M, sm.o[wp][qi][D]);
#pragma unroll
        for (int wp = 0; wp < kWarps; ++wp) {
            const float f = ex2(sm.o[wp][qi][D] - M);
            l = fmaf(sm.o[wp][qi][D + 1], f, l);
            o = fmaf(sm.o[wp][qi][ch], f, o);
        }
        if (job.n_split == 1) {
            out[(q0 + qi) * D + ch] = l > 0.f ? o / l : 0.f;
            continue;
        }
        float *p = cluster ? sm.done[qi] : job.part + (((int64_t)unit * job.n_split + split) * job.qs + qi) * (D + 4);
        p[ch] = o;
        if (ch == 0) {
            p[D] = M;
            p[D + 1] = l;
        }
    }
    if (!cluster) return;
    // the cluster's CTAs share the outputs; each reads every CTA's state
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int x = split * kThreads + tid; x < nq * D; x += job.n_split * kThreads) {
        const int qi = x / D, ch = x % D;
        float M = kMInit, l = 0.f, o = 0.f, m[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            m[r] = r < job.n_split ? cl.map_shared_rank(&sm.done[qi][D], r)[0] : kMInit;
            M = fmaxf(M, m[r]);
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            if (r >= job.n_split) break;
            const float f = ex2(m[r] - M);
            l = fmaf(cl.map_shared_rank(&sm.done[qi][D + 1], r)[0], f, l);
            o = fmaf(cl.map_shared_rank(&sm.done[qi][ch], r)[0], f, o);
        }
        out[(q0 + qi) * D + ch] = l > 0.f ? o / l : 0.f;
    }
    cl.sync();                                   // every CTA's state has been read
}

// Merges the n_split partial states of each (sequence, query head), a warp per output.
template <int D>
__global__ void __launch_bounds__(kThreads)
decode_blocks_combine_kernel(Job job, int64_t n_out, int G, int nq, float *__restrict__ out)
{
    constexpr int N = D / 32;
    pdl_wait();
    pdl_trigger();
    const int64_t hq = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (hq >= n_out) return;
    const int lane = threadIdx.x & 31, g = (int)(hq % G);
    const int64_t unit = hq / G * job.n_sub + g / nq;
    const float *p = job.part + (unit * job.n_split * job.qs + g % nq) * (D + 4);
    const int64_t step = (int64_t)job.qs * (D + 4);
    float M = kMInit;
    for (int i = lane; i < job.n_split; i += 32) M = fmaxf(M, p[i * step + D]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float l = 0.f, o[N] = {};
    for (int i = 0; i < job.n_split; ++i) {
        const float f = ex2(p[i * step + D] - M);
        l = fmaf(p[i * step + D + 1], f, l);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = fmaf(p[i * step + lane + 32 * e], f, o[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) out[hq * D + lane + 32 * e] = l > 0.f ? o[e] / l : 0.f;
}

int shift_of(int block)
{
    int s = 0;
    while ((1 << s) < block) ++s;
    return s;
}

// Query heads a warp serves: groups of up to 4 leave room for the weights' second halves in
// the same instructions.
int queries_per_warp(int G) { return G <= 4 ? 4 : kQ; }
int subgroups(int G) { return (G + queries_per_warp(G) - 1) / queries_per_warp(G); }

// CTAs per (sequence, KV head, subgroup): enough for a few warps on every SM, at least 64 keys
// a warp.
int splits(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int64_t units = (int64_t)c.B * c.H * (subgroups(c.G));
    const int64_t keys_b = std::min<int64_t>((int64_t)k * block, ((int64_t)cache->max_cap + block - 1) / block * block);
    const int64_t keys_w = std::min<int64_t>((int64_t)w + 1, cache->max_cap);
    const int64_t keys = c.G == 1 ? std::max(keys_b, keys_w) : keys_b + keys_w;
    const int64_t want = ((int64_t)num_sms() + units - 1) / units;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, (keys + 64 * kWarps - 1) / (64 * kWarps)));
}

template <int D, bool PAGED, int NQ>
cudaError_t launch_typed(const kvq_cache *cache, const __half *q, const Job &job, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const size_t smem = sizeof(Smem<D>);
    cudaError_t e = ensure_smem_attr((const void *)decode_blocks_kernel<D, PAGED, NQ>, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)c.B * c.H * job.n_sub;
    const dim3 grid((unsigned)(units * job.n_split));
    if (job.n_split > 1 && job.n_split <= kMaxCluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)job.n_split;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, decode_blocks_kernel<D, PAGED, NQ>, c, q, job, out);
    }
    e = launch_pdl(decode_blocks_kernel<D, PAGED, NQ>, grid, dim3(kThreads), smem, st, c, q, job, out);
    if (e != cudaSuccess || job.n_split == 1) return e;
    const int64_t n_out = (int64_t)c.B * c.H * c.G;
    return launch_pdl(decode_blocks_combine_kernel<D>, dim3((unsigned)((n_out + kWarps - 1) / kWarps)), dim3(kThreads), 0, st,
                      job, n_out, c.G, NQ, out);
}

template <int NQ>
cudaError_t launch_nq(const kvq_cache *cache, const __half *q, const Job &job, float *out, cudaStream_t st)
{
    if (cache->view.ptab)
        return cache->D == 128 ? launch_typed<128, true, NQ>(cache, q, job, out, st)
                               : launch_typed<64, true, NQ>(cache, q, job, out, st);
    return cache->D == 128 ? launch_typed<128, false, NQ>(cache, q, job, out, st)
                           : launch_typed<64, false, NQ>(cache, q, job, out, st);
}

} // namespace

int64_t decode_blocks_scratch(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int n = splits(cache, k, block, w);
    if (n <= kMaxCluster) return 0;
    return (int64_t)c.B * c.H * (subgroups(c.G)) * n * std::min(c.G, queries_per_warp(c.G)) * (c.D + 4) * (int64_t)sizeof(float);
}

cudaError_t launch_decode_blocks(const __half *q, const kvq_cache *cache, const int32_t *ids, int k, int block,
                                 const uint8_t *modes, int w, float *scratch, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    Job job;
    job.ids = ids;
    job.modes = modes;
    job.k = k;
    job.block_shift = shift_of(block);
    job.w = w;
    job.n_split = splits(cache, k, block, w);
    job.n_sub = subgroups(c.G);
    job.qs = std::min(c.G, queries_per_warp(c.G));
    job.part = scratch;
    if (queries_per_warp(c.G) == 4) return launch_nq<4>(cache, q, job, out, st);
    return launch_nq<8>(cache, q, job, out, st);
}

} // namespace kvq
