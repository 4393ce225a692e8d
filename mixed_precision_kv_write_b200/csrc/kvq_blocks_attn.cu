// Routed decode attention over chosen blocks (Eq. 2 with the full resolution replaced by a
// choice of blocks): one query per (sequence, query head) at t = len - 1. A skip query's
// output is 0, a local query attends over keys [max(0, t - w), t], a full query over the keys
// of the blocks listed for its KV head.
//
//   logit_j = q . deq(k_j) / sqrt(D),  p = softmax,  out = sum_j p_j deq(v_j)
//
// With codes c, scale s, zero z (Eq. 4) and the centred codes c' = c - 2^(b-1) (b < 16; a small
// integer, exact in fp16), z' = z + 2^(b-1) s:
//   q . deq(k_j) = s_j (q . c'_j) + z'_j sum(q),   sum_j p_j deq(v_j) = sum_j (p_j s_j) c'_j + sum_j p_j z'_j
// Centring keeps the two terms from cancelling: for normal rows |q . c'| is a tenth of |q . c|.
//
// One warp serves up to 8 query heads of a KV head at once with m16n8k16 matrix
// instructions (fp16 operands, fp32 sums), 16 keys at a time:
//   S^T [16 keys x 8 queries]      = C' [16 x D] . Q^T [D x 8]            D/16 instructions
//   O^T [D channels x 8 queries]  += C'^T [D x 16] . W^T [16 x 8]         2 D/16 instructions
// The products are exact: q, the codes and native values are fp16 numbers. The weights
// w = p s are not, so each goes in as two fp16 numbers, w = hi + lo (22 bits), in units that
// keep them far from fp16's subnormals: a power of two above the largest s_V among the
// tile's keys of one width, times 2^-6 (p is at most 2^8, see below). The queries are too few
// for the 128-row tiles of tcgen05 (G is 1 to 64, and the codes would have to be unpacked to
// shared memory first); the loads, not the products, are what the time goes to.
//
// The keys of a tile (up to 256 of a warp's share) are first sorted by width, so that 16 keys
// of one width unpack by one code path: a 16-bit half of a word holds 16/b codes, one mask
// turns field i of both halves into the fp16 pair 1024 + 2^(b i) c, one fused multiply-add into
// c'. For K the two halves are channels of one key (q is stored in the matching order, one
// order per width); for V they are the same channels of two keys (one byte permutation).
//
// Online softmax: the running maximum of a query moves only when a logit exceeds it by
// more than 8 (log2 units), a warp-uniform branch. The warps of a CTA share a (sequence, KV
// head) and merge at the end; with more than one CTA per (sequence, KV head) the partial
// states go to the caller's scratch and a second launch merges them.
#include <algorithm>

#include "kvq_values.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kQ = 8;                            // query heads per warp
constexpr int kTileKeys = 256;                   // keys sorted by width at a time
constexpr int kSlots = kTileKeys + 4 * 16;       // each width's keys are padded to 16
constexpr float kLazy = 8.f;                     // running-max slack, log2 units
constexpr float kMInit = -1e30f;                 // running max before the first key
constexpr uint32_t kValid = 4u;                  // meta bit of a real key (bits 0..1: width code)

struct WarpTile {
    float4 side[kSlots];                         // (s_K cdot, z'_K cdot, s_V, z'_V), sorted
    uint32_t ent[kSlots];                        // record offset | kValid | width code, sorted
};

template <int D>
struct Smem {
    union {
        WarpTile tile[kWarps];
        float o[kWarps][kQ][D + 4];              // the warps' states: o, then m and l
    };
    uint4 q[4][D / 32][32];                      // per width: a lane's query operands, 16 bytes at a time
    float qsum[kQ];
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

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t hfma2u(uint32_t x, uint32_t m, uint32_t a)
{
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&m),
                              *reinterpret_cast<const __half2 *>(&a));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// fp16 bits of a power of two 2^e (-14 <= e <= 15), in both halves
__host__ __device__ constexpr uint32_t pow2h2(int e) { return (uint32_t)((15 + e) << 10) * 0x10001u; }
// fp16 bits of -(2^e + a), a a small power of two below 2^e (or 0), in both halves
__host__ __device__ constexpr uint32_t neg_sum_h2(int e, int a)
{
    return (0x8000u | (uint32_t)((15 + e) << 10) | (uint32_t)((a << 10) >> e)) * 0x10001u;
}

// The 16/BITS centred codes in each half of p (LSB-first) as fp16 pairs: x[i] = (field i of
// the low half, field i of the high half) - 2^(BITS-1); p itself for 16-bit values.
template <int BITS>
__device__ __forceinline__ void fields(uint32_t p, uint32_t (&x)[16 / BITS])
{
    if constexpr (BITS == 16) {
        x[0] = p;
    } else if constexpr (BITS == 8) {
        // bytes with 0x64 above them: 1024 + c; 1152 = 1024 + 128
        x[0] = hfma2u(__byte_perm(p, 0x64646464u, 0x4240), pow2h2(0), neg_sum_h2(10, 128));
        x[1] = hfma2u(__byte_perm(p, 0x64646464u, 0x4341), pow2h2(0), neg_sum_h2(10, 128));
    } else if constexpr (BITS == 4) {
        // fields at bits 0 and 4 (after one shift for the upper two): 1024 + 16^i c
        const uint32_t h = p >> 8;
        x[0] = hfma2u((p & 0x000F000Fu) | 0x64006400u, pow2h2(0), neg_sum_h2(10, 8));
        x[1] = hfma2u((p & 0x00F000F0u) | 0x64006400u, pow2h2(-4), neg_sum_h2(6, 8));
        x[2] = hfma2u((h & 0x000F000Fu) | 0x64006400u, pow2h2(0), neg_sum_h2(10, 8));
        x[3] = hfma2u((h & 0x00F000F0u) | 0x64006400u, pow2h2(-4), neg_sum_h2(6, 8));
    } else {
        // fields at bits 0 .. 8 (after one shift for the upper three): 1024 + 4^i c
        const uint32_t h = p >> 10;
        x[0] = hfma2u((p & 0x00030003u) | 0x64006400u, pow2h2(0), neg_sum_h2(10, 2));
        x[1] = hfma2u((p & 0x000C000Cu) | 0x64006400u, pow2h2(-2), neg_sum_h2(8, 2));
        x[2] = hfma2u((p & 0x00300030u) | 0x64006400u, pow2h2(-4), neg_sum_h2(6, 2));
        x[3] = hfma2u((p & 0x00C000C0u) | 0x64006400u, pow2h2(-6), neg_sum_h2(4, 2));
        x[4] = hfma2u((p & 0x03000300u) | 0x64006400u, pow2h2(-8), neg_sum_h2(2, 2));
        x[5] = hfma2u((h & 0x00030003u) | 0x64006400u, pow2h2(0), neg_sum_h2(10, 2));
        x[6] = hfma2u((h & 0x000C000Cu) | 0x64006400u, pow2h2(-2), neg_sum_h2(8, 2));
        x[7] = hfma2u((h & 0x00300030u) | 0x64006400u, pow2h2(-4), neg_sum_h2(6, 2));
    }
}

// BYTES bytes of a record at logical offset `off` of the stream (aligned to min(BYTES, 16), so a
// 16-byte piece lies in one page) into words; 2 bytes fill the low half of one word.
template <int BYTES>
__device__ __forceinline__ void load_bytes(const RecLoc &L, uint32_t off, uint32_t (&w)[(BYTES + 3) / 4])
{
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(L.at(off + 16u * i)));
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
    } else if constexpr (BYTES == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(L.at(off)));
        w[0] = x.x;
        w[1] = x.y;
    } else if constexpr (BYTES == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(L.at(off)));
    } else {
        w[0] = __ldg(reinterpret_cast<const unsigned short *>(L.at(off)));
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

// Keys [0, n) of the sorted tile from slot `base` on, all of width 2 << CLS, 16 at a time.
template <int D, int CLS>
__device__ __forceinline__ void run_class(State<D> &st, const Smem<D> &sm, const WarpTile &tl, const RecLoc &L, int base, int n,
                                          float fac, bool on0, bool on1)
{
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
    for (int c = base; c < base + n; c += 16) {
        const uint32_t e0 = tl.ent[c + g], e1 = tl.ent[c + 8 + g];
        const uint2 f0 = *reinterpret_cast<const uint2 *>(&tl.ent[c + 2 * t]);
        const uint2 f1 = *reinterpret_cast<const uint2 *>(&tl.ent[c + 8 + 2 * t]);
        uint32_t k0[KW], k1[KW];
        load_bytes<KW * 4>(L, (e0 & ~15u) + 4 * KW * t, k0);
        load_bytes<KW * 4>(L, (e1 & ~15u) + 4 * KW * t, k1);
        uint32_t v[4][(VB + 3) / 4];
        const uint32_t vo = D * BITS / 8 + VB * g;
        load_bytes<VB>(L, (f0.x & ~15u) + vo, v[0]);
        load_bytes<VB>(L, (f0.y & ~15u) + vo, v[1]);
        load_bytes<VB>(L, (f1.x & ~15u) + vo, v[2]);
        load_bytes<VB>(L, (f1.y & ~15u) + vo, v[3]);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        // a word gives F operand pairs of its key; two of them make one instruction's depth of 16
#pragma unroll
        for (int i = 0; i < KW; i += (F == 1 ? 2 : 1)) {
            uint32_t a[F == 1 ? 2 : F], b[F == 1 ? 2 : F];
            if constexpr (F == 1) {
                a[0] = k0[i];
                a[1] = k0[i + 1];
                b[0] = k1[i];
                b[1] = k1[i + 1];
            } else {
                fields<BITS>(k0[i], a);
                fields<BITS>(k1[i], b);
            }
#pragma unroll
            for (int f = 0; f < (F == 1 ? 2 : F); f += 2) mma(s, a[f], b[f], a[f + 1], b[f + 1], q[i * F + f], q[i * F + f + 1]);
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
        float p[4], hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(lg[i] - st.m[i & 1]);
        st.l[0] += p[0] + p[2];
        st.l[1] += p[1] + p[3];
        if (CLS != 3) {
            st.pz[0] = fmaf(p[0], sd0.w, fmaf(p[2], sd1.w, st.pz[0]));
            st.pz[1] = fmaf(p[1], sd0.w, fmaf(p[3], sd1.w, st.pz[1]));
        }
        const float w0 = CLS == 3 ? fac : sd0.z * fac, w1 = CLS == 3 ? fac : sd1.z * fac;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = p[i] * (i < 2 ? w0 : w1);
            hi[i] = __half2float(__float2half_rn(w));
            lo[i] = w - hi[i];
        }
        const uint32_t bh0 = transpose8(pack_half(hi[0], hi[1])), bh1 = transpose8(pack_half(hi[2], hi[3]));
        const uint32_t bl0 = transpose8(pack_half(lo[0], lo[1])), bl1 = transpose8(pack_half(lo[2], lo[3]));
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
                        mma(st.o[i], pa, qa, pb, qb, bl0, bl1);
                    }
                } else {
                    uint32_t xa[F], xb[F];
                    fields<BITS>(pa, xa);
                    fields<BITS>(pb, xb);
#pragma unroll
                    for (int f = 0; f < F; f += 2) {
                        const int mt = ((2 * i + half) * F + f) / 2;
                        mma(st.o[mt], xa[f], xa[f + 1], xb[f], xb[f + 1], bh0, bh1);
                        mma(st.o[mt], xa[f], xa[f + 1], xb[f], xb[f + 1], bl0, bl1);
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

template <int D>
__global__ void __launch_bounds__(kThreads, 4)
decode_blocks_kernel(CacheView c, const __half *__restrict__ q, Job job, float *__restrict__ out)
{
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    pdl_wait();
    pdl_trigger();
    const int split = blockIdx.x % job.n_split, unit = blockIdx.x / job.n_split;
    const int sub = unit % job.n_sub, sh = unit / job.n_sub, s = sh / c.H, h = sh % c.H;
    const int g0 = sub * kQ, nq = min(kQ, c.G - g0);
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
    // the unit's entries: the listed blocks' keys (padded to 32), then the local window's; the
    // warps of all its CTAs take equal shares
    const int nb = (len + (1 << job.block_shift) - 1) >> job.block_shift;
    const int e_block = full ? ((min(job.k, nb) << job.block_shift) + 31) & ~31 : 0;
    if (full && sub == 0 && split == 0)          // no list of distinct blocks is longer than nb
        for (int x = nb + tid; x < job.k; x += kThreads)
            if (job.ids[(int64_t)sh * job.k + x] >= 0) set_status(c.status, KVQ_ERR_DEVICE_CHECK);
    const int wl = min(len, (int)min((int64_t)job.w + 1, (int64_t)len));
    const int e_all = e_block + (local ? wl : 0);
    const int share = ((e_all + job.n_split * kWarps - 1) / (job.n_split * kWarps) + 31) & ~31;

    // query operands in each width's order, and the sums over channels
    for (int x = tid; x < 4 * (D / 32) * 32; x += kThreads) {
        const int cls = x / (D / 32 * 32), i = x / 32 % (D / 32), ln = x % 32;
        const int qi = ln >> 2, ch0 = (ln & 3) * (D / 4), bits = 2 << cls, f = 16 / bits;
        uint32_t r[4] = {0u, 0u, 0u, 0u};
        if (qi < nq) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = 4 * i + e;         // operand pair: word p / f, field p % f
                const __half *src = q + (q0 + qi) * D + ch0 + p / f * (2 * f) + p % f;
                const __half2 v = __halves2half2(src[0], src[f]);
                r[e] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        sm.q[cls][i][ln] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    for (int qi = warp; qi < kQ; qi += kWarps) {
        float a = 0.f;
        if (qi < nq)
            for (int ch = lane; ch < D; ch += 32) a += __half2float(q[(q0 + qi) * D + ch]);
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
    WarpTile &tl = sm.tile[warp];
    const RecLoc L = rec_loc(c, s, h, 0);
    const int a0 = min(e_all, (split * kWarps + warp) * share), a1 = min(e_all, a0 + share);
    int a = a0;
    while (a < a1) {
        // a tile: up to kTileKeys entries of one kind
        const bool blocks = a < e_block;
        const int n = min(kTileKeys, (blocks ? min(a1, e_block) : a1) - a);
        const uint32_t act = blocks ? full : local;
        uint32_t mt[kTileKeys / 32];
        float4 sd[kTileKeys / 32];
        int cnt[4] = {0, 0, 0, 0};
        float smax[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kTileKeys / 32; ++i) {
            mt[i] = 0;
            const int e = i * 32 + lane;
            int j = -1;
            if (e < n) {
                if (blocks) {
                    const int x = (a + e) >> job.block_shift;
                    const int id = x < job.k ? job.ids[(int64_t)sh * job.k + x] : -1;
                    if (id >= 0) {
                        const int before = x > 0 ? job.ids[(int64_t)sh * job.k + x - 1] : -1;
                        if ((x > 0 && before < 0) || id <= before || id >= nb) {
                            set_status(c.status, KVQ_ERR_DEVICE_CHECK);
                        } else {
                            j = (id << job.block_shift) + ((a + e) & ((1 << job.block_shift) - 1));
                            if (j >= len) j = -1;
                        }
                    }
                } else {
                    j = len - wl + (a - e_block) + e;
                }
            }
            if (j >= 0) {
                mt[i] = c.meta[slot0 + j] | kValid;
                sd[i] = c.side[slot0 + j];
            }
        }
#pragma unroll
        for (int i = 0; i < kTileKeys / 32; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const bool in = (mt[i] & 7u) == (kValid | w);
                cnt[w] += __popc(__ballot_sync(0xffffffffu, in));
                if (in) smax[w] = fmaxf(smax[w], sd[i].z);
            }
        }
        int first[5];
        first[0] = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) first[w + 1] = first[w] + ((cnt[w] + 15) & ~15);
        int at[4] = {first[0], first[1], first[2], first[3]};
        uint32_t some[4] = {0u, 0u, 0u, 0u};     // an offset of a real record of each width
#pragma unroll
        for (int i = 0; i < kTileKeys / 32; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const bool in = (mt[i] & 7u) == (kValid | w);
                const uint32_t b = __ballot_sync(0xffffffffu, in);
                if (in) {
                    const int pos = at[w] + __popc(b & ((1u << lane) - 1u));
                    const float mid = w == 3 ? 0.f : (float)(1 << ((2 << w) - 1));
                    tl.ent[pos] = mt[i];
                    tl.side[pos] = make_float4(sd[i].x * cdot, fmaf(mid, sd[i].x, sd[i].y) * cdot, sd[i].z,
                                               fmaf(mid, sd[i].z, sd[i].w));
                    some[w] = mt[i];
                }
                at[w] += __popc(b);
            }
        }
        // padding up to 16: a real record's offset, no kValid
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (cnt[w] == 0) continue;
            const uint32_t any = __reduce_max_sync(0xffffffffu, some[w]);
            if (at[w] + lane < first[w + 1]) {
                tl.ent[at[w] + lane] = any & ~kValid;
                tl.side[at[w] + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        __syncwarp();
        const bool on0 = (act >> (2 * t)) & 1u, on1 = (act >> (2 * t + 1)) & 1u;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (cnt[w] == 0) continue;
            // weights in units of S / 64, S a power of two above the largest scale (1 for fp16 values)
            float fac = 64.f, unit = 0.015625f;
            if (w != 3) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(smax[w]));
                const int e = min(max((int)(top >> 23) + 1, 87), 167);     // biased exponent of S
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
            const int len16 = first[w + 1] - first[w];
            if (w == 0) run_class<D, 0>(st, sm, tl, L, first[w], len16, fac, on0, on1);
            else if (w == 1) run_class<D, 1>(st, sm, tl, L, first[w], len16, fac, on0, on1);
            else if (w == 2) run_class<D, 2>(st, sm, tl, L, first[w], len16, fac, on0, on1);
            else run_class<D, 3>(st, sm, tl, L, first[w], len16, fac, on0, on1);
        }
        __syncwarp();                            // the tile's slots are read; the next one overwrites them
        a += n;
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
    __syncthreads();
    {
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
        } else {
            float *p = job.part + (((int64_t)unit * job.n_split + split) * job.qs + qi) * (D + 4);
            p[ch] = o;
            if (ch == 0) {
                p[D] = M;
                p[D + 1] = l;
            }
        }
    }
}

// Merges the n_split partial states of each (sequence, query head), a warp per output.
template <int D>
__global__ void __launch_bounds__(kThreads)
decode_blocks_combine_kernel(Job job, int64_t n_out, int G, float *__restrict__ out)
{
    constexpr int N = D / 32;
    pdl_wait();
    pdl_trigger();
    const int64_t hq = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (hq >= n_out) return;
    const int lane = threadIdx.x & 31, g = (int)(hq % G);
    const int64_t unit = hq / G * job.n_sub + g / kQ;
    const float *p = job.part + (unit * job.n_split * job.qs + g % kQ) * (D + 4);
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

// CTAs per (sequence, KV head, subgroup): enough for a few warps on every SM, at least 64 keys
// a warp.
int splits(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int64_t units = (int64_t)c.B * c.H * ((c.G + kQ - 1) / kQ);
    const int64_t keys_b = std::min<int64_t>((int64_t)k * block, ((int64_t)cache->max_cap + block - 1) / block * block);
    const int64_t keys_w = std::min<int64_t>((int64_t)w + 1, cache->max_cap);
    const int64_t keys = c.G == 1 ? std::max(keys_b, keys_w) : keys_b + keys_w;
    const int64_t want = (12 * (int64_t)num_sms() + units * kWarps - 1) / (units * kWarps);
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, (keys + 64 * kWarps - 1) / (64 * kWarps)));
}

template <int D>
cudaError_t launch_typed(const kvq_cache *cache, const __half *q, const Job &job, float *out, cudaStream_t st)
{
    const CacheView &c = cache->view;
    const size_t smem = sizeof(Smem<D>);
    cudaError_t e = ensure_smem_attr((const void *)decode_blocks_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)c.B * c.H * job.n_sub;
    e = launch_pdl(decode_blocks_kernel<D>, dim3((unsigned)(units * job.n_split)), dim3(kThreads), smem, st, c, q, job, out);
    if (e != cudaSuccess || job.n_split == 1) return e;
    const int64_t n_out = (int64_t)c.B * c.H * c.G;
    return launch_pdl(decode_blocks_combine_kernel<D>, dim3((unsigned)((n_out + kWarps - 1) / kWarps)), dim3(kThreads), 0, st,
                      job, n_out, c.G, out);
}

} // namespace

int64_t decode_blocks_scratch(const kvq_cache *cache, int k, int block, int w)
{
    const CacheView &c = cache->view;
    const int n = splits(cache, k, block, w);
    if (n == 1) return 0;
    return (int64_t)c.B * c.H * ((c.G + kQ - 1) / kQ) * n * std::min(c.G, kQ) * (c.D + 4) * (int64_t)sizeof(float);
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
    job.n_sub = (c.G + kQ - 1) / kQ;
    job.qs = std::min(c.G, kQ);
    job.part = scratch;
    return c.D == 128 ? launch_typed<128>(cache, q, job, out, st) : launch_typed<64>(cache, q, job, out, st);
}

} // namespace kvq
