// Routed decode attention over chosen blocks (Eq. 2 with the full resolution replaced by a
// choice of blocks): one query per (sequence, query head) at t = len - 1. A skip query's
// output is 0, a local query attends over keys [max(0, t - w), t], a full query over the keys
// of the blocks listed for its KV head.
//
//   logit_j = q . deq(k_j) / sqrt(D),  p = softmax,  out = sum_j p_j deq(v_j)
//
// With codes c, scale s, zero z (Eq. 4), the centred codes c' = c - (2^b - 1)/2 (b < 16; exact in
// fp16) and z' = z + (2^b - 1)/2 s:
//   q . deq(k_j) = s_j (q . c'_j) + z'_j sum(q),   sum_j p_j deq(v_j) = sum_j (p_j s_j) c'_j + sum_j p_j z'_j
// Centring keeps the sums from cancelling: with K's codes as they are (a mask alone makes a field an
// fp16 subnormal, two instructions less a pair) the outputs were 9e-6 off, with centred ones 2e-7 to 6e-7.
//
// One warp serves up to 8 query heads of a KV head at once with m16n8k16 matrix
// instructions (fp16 operands, fp32 sums), 16 keys at a time:
//   S^T [16 keys x 8 queries]      = C' [16 x D] . Q^T [D x 8]           D/16 instructions
//   O^T [D channels x 8 queries]  += C'^T [D x 16] . W^T [16 x 8]        2 D/16 (up to 4 queries: D/16)
// The products are exact: q, the codes and native values are fp16 numbers. The weights
// w = p s are not, so each goes in as two fp16 numbers, w = hi + lo (22 bits), in a unit of the
// query's own: a power of two that puts the largest w the query has met (relative to its running
// maximum) at 2^11 to 2^15. A weight is then off by 2^-22 of itself or by 2^-36 of the largest one,
// whose key moved the sum by half of it or more (no centred code is 0), so keys of large V leave the
// weights of others alone unless they count. Native values have no scale that bounds them: their
// weights go in as two tf32 numbers, which have fp32's range, with the values as tf32 (exact), by
// m16n8k8 instructions, two for one of the others. Up to 4 queries leave
// columns 4..7 of the instruction to the second numbers. The queries are too few for the
// 128-row tiles of tcgen05 (G is 1 to 64, and the codes would have to be unpacked to shared
// memory first).
//
// The keys of a tile (up to 1024 of a CTA's share) are first sorted by width, so that 16 keys
// of one width unpack by one code path; the warps take the 16-key steps in turn. A 16-bit
// half of a word holds 16/b codes: for K the two halves are channels of one key (q is stored
// in the matching order, one order per width), for V the same channels of two keys (one byte
// permutation). A field at bit p joins the mantissa of 2^(10 - p), whose last place there is 1,
// by one mask-and-or, and one addition takes 2^(10 - p) + (2^b - 1)/2 off again. The fields are
// moved up one place first, so that this constant has its half.
//
// Online softmax: the running maximum of a query moves only when a logit exceeds it by
// more than 3 (log2 units), a warp-uniform branch. The warps of a CTA share a (sequence, KV
// head) and merge at the end; up to 16 CTAs that share one form a cluster and merge through
// distributed shared memory; more of them leave partial states in the caller's scratch, which
// a second launch merges.
//
// Bound by latency at 16 warps an SM (the state of 8 columns x D channels takes the registers):
// 656 k keys of 1024 heads take 66 us, 37 warp instructions a key, 2.0 TB/s of records. At 42 %
// issue-active and 23 % of DRAM's rate neither is a limit; the wait for a step's records is the top stall.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kQ = 8;                            // query heads per warp
constexpr int kTileKeys = 1024;                  // keys a CTA sorts by width at a time
constexpr int kSlots = kTileKeys + 4 * 16;       // each width's keys are padded to 16
constexpr float kPTop = 8.f;                     // 2^3: the running maximum's slack
constexpr float kWTop = 32768.f;                 // the largest weight in units of its query
constexpr int kMaxFac = 64;                      // the smallest unit is 2^-64
constexpr float kMInit = -1e30f;                 // running max before the first key
constexpr int kMaxCluster = 16;                  // CTAs of a cluster
constexpr uint32_t kValid = 4u;                  // meta bit of a real key (bits 0..1: width code)

struct Tile {
    uint2 ent[kSlots];                           // (record offset | kValid | width code, key), sorted
};

template <int D, int W>
struct Smem {
    union {
        Tile tile;
        float o[W][kQ][D + 4];                   // the warps' states: o, then m and l
    };
    uint4 q[4][D / 32][32];                      // per width: a lane's query operands, 16 bytes at a time
    __half rows[kQ][D + 8];                      // the queries
    float qsum[kQ];
    float done[kQ][D + 4];                       // the CTA's state for the cluster: o, then m and l
    int cnt[W][4];                               // keys of each width in each warp's part of the tile
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

__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ float to_tf32(float x)              // rounded to tf32's 11 bits
{
    uint32_t y;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
    return __uint_as_float(y);
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

// The fields of BITS bits at SHIFT in both halves of p, centred: c - (2^BITS - 1)/2. A field joins
// the mantissa of 2^(10 - SHIFT), then 2^(10 - SHIFT) + (2^BITS - 1)/2 is subtracted; every step is
// exact for SHIFT >= 1.
template <int BITS, int SHIFT>
__device__ __forceinline__ uint32_t mid_field(uint32_t p)
{
    constexpr uint32_t magic = (uint32_t)((25 - SHIFT) << 10) * 0x10001u;
    constexpr uint32_t off = (0x8000u | (uint32_t)((25 - SHIFT) << 10) | (((1u << BITS) - 1u) << (SHIFT - 1))) * 0x10001u;
    const uint32_t x = (p & ((((1u << BITS) - 1u) << SHIFT) * 0x10001u)) | magic, m = off;
    const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&m));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The 16/BITS centred codes in each half of p (LSB-first) as fp16 pairs: x[i] = (field i of
// the low half, field i of the high half).
template <int BITS>
__device__ __forceinline__ void mid_fields(uint32_t p, uint32_t (&x)[16 / BITS])
{
    const uint32_t l = p << 1, h = p >> 7;       // the lower and the upper 8 bits, one place up
    if constexpr (BITS == 8) {
        x[0] = mid_field<8, 1>(l);
        x[1] = mid_field<8, 1>(h);
    } else if constexpr (BITS == 4) {
        x[0] = mid_field<4, 1>(l);
        x[1] = mid_field<4, 5>(l);
        x[2] = mid_field<4, 1>(h);
        x[3] = mid_field<4, 5>(h);
    } else {
        x[0] = mid_field<2, 1>(l);
        x[1] = mid_field<2, 3>(l);
        x[2] = mid_field<2, 5>(l);
        x[3] = mid_field<2, 7>(l);
        x[4] = mid_field<2, 1>(h);
        x[5] = mid_field<2, 3>(h);
        x[6] = mid_field<2, 5>(h);
        x[7] = mid_field<2, 7>(h);
    }
}

// Where a stream's bytes are: PAGED as RecLoc::at, else base + offset.
template <bool PAGED>
__device__ __forceinline__ const uint8_t *byte_at(const RecLoc &L, uint32_t off)
{
    return PAGED ? L.at(off) : L.base + off;
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
// (entries 2, 3) of those queries, times fac (a power of two, 1 / unit).
template <int D>
struct State {
    float o[D / 16][4];
    float m[2], l[2], pz[2], fac[2];
};

// The running maxima take in the logits lg of the step's keys (entries 0, 1 of the key with scale
// sva, 2, 3 of the one with svb), the units their weights. A unit only grows relative to 2^m, so
// the sums shrink; the largest weight at hand comes to 2^11 to 2^12 units.
template <int D, int CLS>
__device__ __forceinline__ void raise(State<D> &st, const float (&lg)[4], float sva, float svb)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float n = fmaxf(lg[j], lg[2 + j]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
        n = fmaxf(st.m[j], n);
        const int have = (int)(__float_as_uint(st.fac[j]) >> 23) - 127;
        int f = min(kMaxFac, have + (int)fminf(n - st.m[j], 256.f));
        if (CLS != 3) {
            float w = fmaxf(ex2(lg[j] - n) * sva, ex2(lg[2 + j] - n) * svb);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, d));
            f = min(f, 12 + 126 - (int)(__float_as_uint(w) >> 23));            // w < 2^(exponent bits - 126)
        }
        const float c = ex2(st.m[j] - n), r = ex2(st.m[j] - n + (float)(f - have));
        st.m[j] = n;
        st.l[j] *= c;
        st.pz[j] *= c;
        st.fac[j] = __uint_as_float((uint32_t)(f + 127) << 23);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            st.o[i][j] *= r;
            st.o[i][2 + j] *= r;
        }
    }
}

// K's words and the side entries of a 16-key step's rows g and g + 8.
template <int D, int CLS, bool PAGED>
struct KRows {
    static constexpr int KW = D * (2 << CLS) / 128;      // words of a lane's D/4 channels of K
    uint32_t a[KW], b[KW];
    float4 sa, sb;
    bool va, vb;
    __device__ __forceinline__ void load(const Tile &tl, const RecLoc &L, const float4 *side, int c, int g, int t)
    {
        const uint2 e0 = tl.ent[c + g], e1 = tl.ent[c + 8 + g];
        load_bytes<KW * 4, PAGED>(L, (e0.x & ~15u) + 4 * KW * t, a);
        load_bytes<KW * 4, PAGED>(L, (e1.x & ~15u) + 4 * KW * t, b);
        if (CLS != 3) {
            sa = __ldg(side + e0.y);
            sb = __ldg(side + e1.y);
        }
        va = e0.x & kValid;
        vb = e1.x & kValid;
    }
};

// Slots base, base + 16 W, .. below `end` of the sorted tile, 16 at a time, all of width
// 2 << CLS. The next step's K and side entries are loaded while this one's weights are formed
// (not for native values, whose words take the registers), V while this one's logits are.
template <int D, int CLS, bool PAGED, int NQ, int W>
__device__ __forceinline__ void run_class(State<D> &st, const Smem<D, W> &sm, const RecLoc &L, const float4 *side, int base, int end,
                                          bool on0, bool on1)
{
    const Tile &tl = sm.tile;
    constexpr int BITS = 2 << CLS;
    constexpr int KW = KRows<D, CLS, PAGED>::KW;
    constexpr int VB = D * BITS / 64;            // bytes of a lane's D/8 channels of V
    constexpr int F = 16 / BITS;                 // fields per half word
    constexpr float mid = 0.5f * (float)((1 << BITS) - 1);
    const float cdot = kLog2e / sqrtf((float)D);
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
    const float qs0 = sm.qsum[2 * t] * cdot, qs1 = sm.qsum[2 * t + 1] * cdot;
    KRows<D, CLS, PAGED> kr;
    kr.load(tl, L, side, base, g, t);
    for (int c = base; c < end; c += 16 * W) {
        uint32_t v[4][(VB + 3) / 4];
        auto load_v = [&]() {
            const uint4 f0 = *reinterpret_cast<const uint4 *>(&tl.ent[c + 2 * t]);
            const uint4 f1 = *reinterpret_cast<const uint4 *>(&tl.ent[c + 8 + 2 * t]);
            const uint32_t vo = D * BITS / 8 + VB * g;
            load_bytes<VB, PAGED>(L, (f0.x & ~15u) + vo, v[0]);
            load_bytes<VB, PAGED>(L, (f0.z & ~15u) + vo, v[1]);
            load_bytes<VB, PAGED>(L, (f1.x & ~15u) + vo, v[2]);
            load_bytes<VB, PAGED>(L, (f1.z & ~15u) + vo, v[3]);
        };
        if (CLS != 3) load_v();
        // S^T: a word gives 16/BITS operand pairs of its key; two sums alternate, so that no chain of
        // dependent instructions is longer than D/32
        float sf[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) sf[i][0] = sf[i][1] = sf[i][2] = sf[i][3] = 0.f;
        if constexpr (CLS == 3) {
#pragma unroll
            for (int i = 0; i < KW; i += 2) mma(sf[i / 2 & 1], kr.a[i], kr.b[i], kr.a[i + 1], kr.b[i + 1], q[i], q[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                uint32_t xa[F], xb[F];
                mid_fields<BITS>(kr.a[i], xa);
                mid_fields<BITS>(kr.b[i], xb);
#pragma unroll
                for (int f = 0; f < F; f += 2)
                    mma(sf[(i * F + f) / 2 & 1], xa[f], xb[f], xa[f + 1], xb[f + 1], q[i * F + f], q[i * F + f + 1]);
            }
        }
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = sf[0][i] + sf[1][i];
        }
        // logits in log2 units: (s (q . c') + z' sum(q)) log2(e) / sqrt(D)
        const float ka = CLS == 3 ? cdot : kr.sa.x * cdot, kb = CLS == 3 ? cdot : kr.sb.x * cdot;
        const float za = CLS == 3 ? 0.f : fmaf(mid, kr.sa.x, kr.sa.y), zb = CLS == 3 ? 0.f : fmaf(mid, kr.sb.x, kr.sb.y);
        const float sva = CLS == 3 ? 1.f : kr.sa.z, svb = CLS == 3 ? 1.f : kr.sb.z;
        const float zva = CLS == 3 ? 0.f : fmaf(mid, kr.sa.z, kr.sa.w), zvb = CLS == 3 ? 0.f : fmaf(mid, kr.sb.z, kr.sb.w);
        float lg[4];
        lg[0] = kr.va && on0 ? fmaf(ka, s[0], za * qs0) : -INFINITY;
        lg[1] = kr.va && on1 ? fmaf(ka, s[1], za * qs1) : -INFINITY;
        lg[2] = kr.vb && on0 ? fmaf(kb, s[2], zb * qs0) : -INFINITY;
        lg[3] = kr.vb && on1 ? fmaf(kb, s[3], zb * qs1) : -INFINITY;
        if (c + 16 * W < end) kr.load(tl, L, side, c + 16 * W, g, t);
        if (CLS == 3) load_v();
        float p[4], w[4];
        auto weights = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = ex2(lg[i] - st.m[i & 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[i] * (CLS == 3 ? st.fac[i & 1] : (i < 2 ? sva : svb) * st.fac[i & 1]);
        };
        weights();
        bool over = fmaxf(p[0], p[2]) > kPTop || fmaxf(p[1], p[3]) > kPTop;
        if (CLS != 3) over = over || fmaxf(w[0], w[2]) > kWTop || fmaxf(w[1], w[3]) > kWTop;
        if (__any_sync(0xffffffffu, over)) {
            raise<D, CLS>(st, lg, sva, svb);
            weights();
        }
        st.l[0] += p[0] + p[2];
        st.l[1] += p[1] + p[3];
        if (CLS != 3) {
            st.pz[0] = fmaf(p[0], zva, fmaf(p[2], zvb, st.pz[0]));
            st.pz[1] = fmaf(p[1], zva, fmaf(p[3], zvb, st.pz[1]));
        }
        if constexpr (CLS == 3) {
            // the fp32 weights transposed as two 16-bit halves: x[i] is that of key 2t, 2t + 1, 8 + 2t,
            // 9 + 2t and the lane's query g
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const uint32_t w0 = __float_as_uint(w[i]), w1 = __float_as_uint(w[i + 1]);
                const uint32_t up = transpose8(__byte_perm(w0, w1, 0x7632)), low = transpose8(__byte_perm(w0, w1, 0x5410));
                x[i] = __uint_as_float(__byte_perm(low, up, 0x5410));
                x[i + 1] = __uint_as_float(__byte_perm(low, up, 0x7632));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float h = to_tf32(x[i]);
                y[i] = x[i] - h;
                x[i] = NQ == 4 && g >= 4 ? y[i] : h;                // columns 4..7 carry the rests of queries 0..3
            }
            // rows g and g + 8 of the instruction are a word's two channels
#pragma unroll
            for (int i = 0; i < VB / 4; ++i) {
                const float2 f0 = h2_values(v[0][i]), f1 = h2_values(v[1][i]);
                const float2 f2 = h2_values(v[2][i]), f3 = h2_values(v[3][i]);
                mma_tf32(st.o[i], f0.x, f0.y, f1.x, f1.y, x[0], x[1]);
                mma_tf32(st.o[i], f2.x, f2.y, f3.x, f3.y, x[2], x[3]);
                if (NQ == 8) {
                    mma_tf32(st.o[i], f0.x, f0.y, f1.x, f1.y, y[0], y[1]);
                    mma_tf32(st.o[i], f2.x, f2.y, f3.x, f3.y, y[2], y[3]);
                }
            }
            continue;
        }
        const uint32_t h0 = pack_half(w[0], w[1]), h1 = pack_half(w[2], w[3]);
        const uint32_t r0 = rest_half(w[0], w[1], h0), r1 = rest_half(w[2], w[3], h1);
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
                if constexpr (CLS != 3) {
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

template <int D, bool PAGED, int NQ, int W>
__global__ void __launch_bounds__(32 * W, 16 / W)
decode_blocks_kernel(CacheView c, const __half *__restrict__ q, Job job, float *__restrict__ out)
{
    constexpr int kThreads = 32 * W, kSteps = kTileKeys / kThreads;        // 32-key steps of a warp's part of a tile
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D, W> &sm = *reinterpret_cast<Smem<D, W> *>(raw);
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
    if (full && split == 0)                      // no list of distinct blocks is longer than nb
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
    // 16 bytes are four pairs (channel, channel + f), f = 16 / bits fields to a half word
    for (int x = tid; x < (D / 32) * 32; x += kThreads) {
        const int i = x / 32, ln = x % 32;
        const __half *row = &sm.rows[(ln >> 2) & (NQ - 1)][(ln & 3) * (D / 4)];
        const uint4 v = *reinterpret_cast<const uint4 *>(row + 8 * i);
        const uint2 va = *reinterpret_cast<const uint2 *>(row + (i >> 1) * 16 + (i & 1) * 4);
        const uint2 vb = *reinterpret_cast<const uint2 *>(row + (i >> 1) * 16 + (i & 1) * 4 + 8);
        sm.q[3][i][ln] = v;
        sm.q[2][i][ln] = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                                    __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        sm.q[1][i][ln] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        sm.q[0][i][ln] = make_uint4(__byte_perm(va.x, vb.x, 0x5410), __byte_perm(va.x, vb.x, 0x7632),
                                    __byte_perm(va.y, vb.y, 0x5410), __byte_perm(va.y, vb.y, 0x7632));
    }
    for (int qi = warp; qi < kQ; qi += W) {
        float a = 0.f;
#pragma unroll
        for (int ch = 0; ch < D; ch += 32) a += __half2float(sm.rows[qi & (NQ - 1)][ch + lane]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
        if (lane == 0) sm.qsum[qi] = a;
    }
    __syncthreads();

    Tile &tl = sm.tile;
    const RecLoc L = rec_loc(c, s, h, 0);
    const uint32_t *meta = c.meta + slot0;
    const float4 *side = c.side + slot0;
    const int bs = job.block_shift;
    const uint32_t below = (1u << lane) - 1u;
    const bool cluster = job.n_split > 1 && job.n_split <= kMaxCluster;
    const int a0 = min(e_all, split * share), a1 = min(e_all, a0 + share);
    // Where a unit has full and local queries, the blocks' keys are finished for the full ones before
    // the window's begin for the others: a value that is not finite gives NaN in a column of weight 0.
    const bool both = full && local;
    for (int part = 0; part < (both ? 2 : 1); ++part) {
        const int lo = part ? max(a0, e_block) : a0, hi = both && !part ? min(a1, e_block) : a1;
        const uint32_t mine = !both ? 0xFFu : part ? ~full : full;       // the queries finished in this part
        State<D> st;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.m[i] = kMInit;
            st.l[i] = st.pz[i] = 0.f;
            st.fac[i] = 1.f;
        }
        for (int a = lo; a < hi;) {
            // a tile: up to kTileKeys entries of one kind, the warps' parts multiples of 32
            const bool blocks = a < e_block;
            const int n = min(kTileKeys, (blocks ? min(hi, e_block) : hi) - a);
            const int per = ((n + W - 1) / W + 31) & ~31;
            const int p0 = warp * per, p1 = min(n, p0 + per);
            const uint32_t act = blocks ? full : local;
            // lane i < 17: the i-th block of the warp's part, or -1; an entry not above its predecessor
            // or past the length is dropped
            const int x0 = (a + p0) >> bs;
            int id = -1;
            if (blocks && p0 < p1) {
                const int x = x0 + lane;
                const bool in = x <= (a + p1 - 1) >> bs && x < job.k;
                id = in ? job.ids[(int64_t)sh * job.k + x] : -1;
                int before = __shfl_up_sync(0xffffffffu, id, 1);
                if (lane == 0 && x > 0) before = job.ids[(int64_t)sh * job.k + x - 1];
                if (id >= 0 && (id >= nb || (x > 0 && (before < 0 || id <= before)))) {
                    set_status(c.status, KVQ_ERR_DEVICE_CHECK);
                    id = -1;
                }
            }
            uint32_t mt[kSteps];
            int js[kSteps];
            int cnt[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                mt[i] = 0u;
                js[i] = 0;
                if (p0 + i * 32 >= p1) continue;
                const int e = a + p0 + i * 32 + lane;
                const int b = __shfl_sync(0xffffffffu, id, (e >> bs) - x0);
                js[i] = blocks ? (b << bs) + (e & ((1 << bs) - 1)) : len - wl + e - e_block;
                if (e < a + p1 && (!blocks || b >= 0) && js[i] < len) mt[i] = meta[js[i]] | kValid;
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if (p0 + i * 32 >= p1) continue;
                const uint32_t v = __ballot_sync(0xffffffffu, mt[i] & kValid), b0 = __ballot_sync(0xffffffffu, mt[i] & 1u),
                               b1 = __ballot_sync(0xffffffffu, mt[i] & 2u);
                cnt[0] += __popc(v & ~b0 & ~b1);
                cnt[1] += __popc(b0 & ~b1);
                cnt[2] += __popc(b1 & ~b0);
                cnt[3] += __popc(b0 & b1);
            }
            if (lane < 4) sm.cnt[warp][lane] = lane == 0 ? cnt[0] : lane == 1 ? cnt[1] : lane == 2 ? cnt[2] : cnt[3];
            __syncthreads();
            // slots: width by width, each width's keys in the warps' order, padded to 16. Lane
            // 4 x + w holds warp x's count of width w; sums over the warps, then over the widths
            int all[4], at[4], first[5];
            {
                const int my_cnt = lane < 4 * W ? sm.cnt[lane >> 2][lane & 3] : 0;
                int upto = my_cnt;
#pragma unroll
                for (int d = 4; d < 4 * W; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += y;
                }
                first[0] = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    all[w] = __shfl_sync(0xffffffffu, upto, 4 * (W - 1) + w);
                    at[w] = first[w] + __shfl_sync(0xffffffffu, upto - my_cnt, 4 * warp + w);
                    first[w + 1] = first[w] + ((all[w] + 15) & ~15);
                }
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if (p0 + i * 32 >= p1) continue;
                const uint32_t v = __ballot_sync(0xffffffffu, mt[i] & kValid), b0 = __ballot_sync(0xffffffffu, mt[i] & 1u),
                               b1 = __ballot_sync(0xffffffffu, mt[i] & 2u);
                if (mt[i] & kValid) {
                    const uint32_t own = v & (mt[i] & 1u ? b0 : ~b0) & (mt[i] & 2u ? b1 : ~b1);
                    const int to = mt[i] & 2u ? (mt[i] & 1u ? at[3] : at[2]) : (mt[i] & 1u ? at[1] : at[0]);
                    const int end = mt[i] & 2u ? (mt[i] & 1u ? first[3] + all[3] : first[2] + all[2])
                                               : (mt[i] & 1u ? first[1] + all[1] : all[0]);
                    int pos = to + __popc(own & below);
                    tl.ent[pos] = make_uint2(mt[i], (uint32_t)js[i]);
                    // the width's last key also fills its last 16, without kValid
                    if (++pos == end)
                        for (; pos & 15; ++pos) tl.ent[pos] = make_uint2(mt[i] & ~kValid, (uint32_t)js[i]);
                }
                at[0] += __popc(v & ~b0 & ~b1);
                at[1] += __popc(b0 & ~b1);
                at[2] += __popc(b1 & ~b0);
                at[3] += __popc(b0 & b1);
            }
            __syncthreads();
            const bool on0 = (act >> (2 * t & (NQ - 1))) & 1u, on1 = (act >> ((2 * t & (NQ - 1)) + 1)) & 1u;
            // 16-key steps dealt to the warps in turn, so that they run one width's code at a time
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int b0 = first[w] + ((warp - first[w] / 16) & (W - 1)) * 16, b1 = first[w + 1];
                if (b0 >= b1) continue;
                if (w == 0) run_class<D, 0, PAGED, NQ, W>(st, sm, L, side, b0, b1, on0, on1);
                else if (w == 1) run_class<D, 1, PAGED, NQ, W>(st, sm, L, side, b0, b1, on0, on1);
                else if (w == 2) run_class<D, 2, PAGED, NQ, W>(st, sm, L, side, b0, b1, on0, on1);
                else run_class<D, 3, PAGED, NQ, W>(st, sm, L, side, b0, b1, on0, on1);
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
        // columns 4..7 of up to 4 queries are the weights' second parts: left as states of their own
        if (2 * (t & (NQ / 2 - 1)) < nq) {
            const int g = lane >> 2;
            const bool rest = 2 * t >= NQ;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float *o = sm.o[warp][2 * t + i];
                const float add = rest ? 0.f : st.pz[i], unit = __uint_as_float((254u << 23) - __float_as_uint(st.fac[i]));
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt)
                    *reinterpret_cast<float2 *>(&o[g * (D / 8) + 2 * mt]) =
                        make_float2(fmaf(st.o[mt][i], unit, add), fmaf(st.o[mt][2 + i], unit, add));
                if (g == 0 && !rest) {
                    o[D] = st.m[i];
                    o[D + 1] = st.l[i];
                }
            }
        }
        __syncthreads();
        for (int x = tid; x < nq * D; x += kThreads) {
            const int qi = x / D, ch = x % D;
            if (!(mine >> qi & 1u)) continue;
            float M = kMInit, l = 0.f, o = 0.f;
#pragma unroll
            for (int wp = 0; wp < W; ++wp) M = fmaxf(M, sm.o[wp][qi][D]);
#pragma unroll
            for (int wp = 0; wp < W; ++wp) {
                const float f = ex2(sm.o[wp][qi][D] - M);
                l = fmaf(sm.o[wp][qi][D + 1], f, l);
                o = fmaf(sm.o[wp][qi][ch] + (NQ == 4 ? sm.o[wp][qi + 4][ch] : 0.f), f, o);
            }
            if (job.n_split == 1) {
                out[(q0 + qi) * D + ch] = l == 0.f ? 0.f : o / l;
                continue;
            }
            float *to = cluster ? sm.done[qi] : job.part + (((int64_t)unit * job.n_split + split) * job.qs + qi) * (D + 4);
            to[ch] = o;
            if (ch == 0) {
                to[D] = M;
                to[D + 1] = l;
            }
        }
        if (both) __syncthreads();                   // the states are read; the next part's tile overwrites them
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
        out[(q0 + qi) * D + ch] = l == 0.f ? 0.f : o / l;
    }
    cl.sync();                                   // every CTA's state has been read
}

// Merges the n_split partial states of each (sequence, query head), a warp per output.
constexpr int kCombineThreads = 128;
template <int D>
__global__ void __launch_bounds__(kCombineThreads)
decode_blocks_combine_kernel(Job job, int64_t n_out, int G, int nq, float *__restrict__ out)
{
    constexpr int N = D / 32;
    pdl_wait();
    pdl_trigger();
    const int64_t hq = (int64_t)blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5);
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
    for (int e = 0; e < N; ++e) out[hq * D + lane + 32 * e] = l == 0.f ? 0.f : o[e] / l;
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

// Warps per CTA and CTAs per (sequence, KV head, subgroup), a unit. An SM holds two CTAs of 8 warps
// or four of 4. Up to 2.5 units an SM: 8 warps, and as many CTAs a unit as one wave takes, with at
// least 64 keys a warp; above: a CTA of 4 warps a unit. Measured from cold caches, 1024 keys a full
// query, 513 a local one, us for 4 warps x 1 CTA, 8 x 1, 8 x 2 (first every query full, then 15 %
// skip, 45 % local; G = 1, D = 128):
//   144 units   38.9  28.7  24.6     37.2  26.6  23.9
//   256         43.0  32.8  43.0     41.0  30.7  38.9
//   320         47.1  51.2  58.9     43.0  33.0  41.0
//   384         49.1  54.8  61.5     43.9  43.2  49.2
//   512         53.3  59.4  77.9     49.2  49.6  61.5
//   640         83.3  77.4  94.8     51.2  55.3  72.0
//   1024        95.3 103.6 131.2     78.4  79.9 107.8
// (4 queries a head: 256 units 43.8 34.8 45.1 | 61.5 47.1 58.5, 512 units 55.3 61.4 82.2 | 75.8 84.9 99.9.)
struct Shape {
    int warps, n_split;
};
Shape shape_of(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int64_t units = (int64_t)c.B * c.H * subgroups(c.G), sms = num_sms();
    if (2 * units >= 5 * sms) return {4, 1};
    const int64_t keys_b = std::min<int64_t>((int64_t)k * block, ((int64_t)cache->max_cap + block - 1) / block * block);
    const int64_t keys_w = std::min<int64_t>((int64_t)w + 1, cache->max_cap);
    const int64_t keys = c.G == 1 ? std::max(keys_b, keys_w) : keys_b + keys_w;
    return {8, (int)std::max<int64_t>(1, std::min<int64_t>(2 * sms / units, (keys + 64 * 8 - 1) / (64 * 8)))};
}

template <int D, bool PAGED, int NQ, int W>
cudaError_t launch_typed(const kvq_cache *cache, const __half *q, const Job &job, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const size_t smem = sizeof(Smem<D, W>);
    cudaError_t e = ensure_smem_attr((const void *)decode_blocks_kernel<D, PAGED, NQ, W>, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)c.B * c.H * job.n_sub;
    const dim3 grid((unsigned)(units * job.n_split));
    if (job.n_split > 8 && job.n_split <= kMaxCluster) {
        e = ensure_cluster_attr((const void *)decode_blocks_kernel<D, PAGED, NQ, W>);
        if (e != cudaSuccess) return e;
    }
    if (job.n_split > 1 && job.n_split <= kMaxCluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(32 * W);
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
        return cudaLaunchKernelEx(&cfg, decode_blocks_kernel<D, PAGED, NQ, W>, c, q, job, out);
    }
    e = launch_pdl(decode_blocks_kernel<D, PAGED, NQ, W>, grid, dim3(32 * W), smem, st, c, q, job, out);
    if (e != cudaSuccess || job.n_split == 1) return e;
    const int64_t n_out = (int64_t)c.B * c.H * c.G;
    return launch_pdl(decode_blocks_combine_kernel<D>, dim3((unsigned)((n_out * 32 + kCombineThreads - 1) / kCombineThreads)),
                      dim3(kCombineThreads), 0, st,
                      job, n_out, c.G, NQ, out);
}

template <int NQ, int W>
cudaError_t launch_nq(const kvq_cache *cache, const __half *q, const Job &job, float *out, cudaStream_t st)
{
    if (cache->view.ptab)
        return cache->D == 128 ? launch_typed<128, true, NQ, W>(cache, q, job, out, st)
                               : launch_typed<64, true, NQ, W>(cache, q, job, out, st);
    return cache->D == 128 ? launch_typed<128, false, NQ, W>(cache, q, job, out, st)
                           : launch_typed<64, false, NQ, W>(cache, q, job, out, st);
}

} // namespace

int64_t decode_blocks_scratch(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int n = shape_of(cache, k, block, w).n_split;
    if (n <= kMaxCluster) return 0;
    return (int64_t)c.B * c.H * (subgroups(c.G)) * n * std::min(c.G, queries_per_warp(c.G)) * (c.D + 4) * (int64_t)sizeof(float);
}

cudaError_t launch_decode_blocks(const __half *q, const kvq_cache *cache, const int32_t *ids, int k, int block,
                                 const uint8_t *modes, int w, float *scratch, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const Shape shape = shape_of(cache, k, block, w);
    Job job;
    job.ids = ids;
    job.modes = modes;
    job.k = k;
    job.block_shift = shift_of(block);
    job.w = w;
    job.n_split = shape.n_split;
    job.n_sub = subgroups(c.G);
    job.qs = std::min(c.G, queries_per_warp(c.G));
    job.part = scratch;
    if (queries_per_warp(c.G) == 4)
        return shape.warps == 4 ? launch_nq<4, 4>(cache, q, job, out, st) : launch_nq<4, 8>(cache, q, job, out, st);
    return shape.warps == 4 ? launch_nq<8, 4>(cache, q, job, out, st) : launch_nq<8, 8>(cache, q, job, out, st);
}

} // namespace kvq
