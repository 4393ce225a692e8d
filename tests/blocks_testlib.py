"""Plain 64-bit forms of the rotating write, the read-back and block-sparse decoding, for the
GPU tests, and the rounding bounds that their tolerances count."""
from __future__ import annotations

import math

import torch

from mixed_precision_kv_write_b200 import kvq

U32, U16, UB16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8      # half a step of fp32, fp16, bf16
TILE = kvq.BLOCK_TILE


def cu_of(counts, device="cuda"):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


def rows(n, heads, D, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn((n, heads, D), generator=g, device=device).half()


def widths(n, heads, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    pick = torch.randint(0, 4, (n, heads), generator=g, device=device)
    return torch.tensor([2, 4, 8, 16], dtype=torch.uint8, device=device)[pick]


def stored(x, bits):
    """(codes fp64, scale, zero) of Eq. 4 for fp16 rows: scale and zero in fp32 as the cache holds them."""
    x32, b = x.float(), bits.float()[..., None]
    lo, hi = x32.amin(-1, keepdim=True), x32.amax(-1, keepdim=True)
    s, z = (hi - lo) / (torch.exp2(b) - 1), lo + 0.0
    code = torch.where(s == 0, 0.0, ((x32 - z) / s).round())
    native = b == 16
    return (torch.where(native, x32, code).double(), torch.where(native, 1.0, s)[..., 0],
            torch.where(native, 0.0, z)[..., 0])


def values64(x, bits):
    c, s, z = stored(x, bits)
    return c * s.double()[..., None] + z.double()[..., None]


def values32(x, bits):
    """The same with the product and the sum rounded to fp32 one after the other."""
    c, s, z = stored(x, bits)
    return c.float() * s[..., None] + z[..., None]


def rope_table(n, rot, device="cuda", base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), -1).float().to(device)


def rotate(x, pos, table, interleaved, wide=False):
    """Rows x [n, heads, D] rotated to positions pos [n]: in fp32 with every operation rounded on its
    own and the result in fp16, or (wide) in fp64 without rounding."""
    rot = table.shape[1]
    t = table[pos.long()].to(torch.float64 if wide else torch.float32)
    c, s = t[:, None, :rot // 2], t[:, None, rot // 2:]
    y = x.to(t.dtype).clone()
    ia = torch.arange(0, rot, 2, device=x.device) if interleaved else torch.arange(rot // 2, device=x.device)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia], y[..., ib]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    y[..., ia], y[..., ib] = ac - bs, bc + as_
    return y if wide else y.half()


class Filled:
    """A cache holding given lengths, with its rows at hand."""

    def __init__(self, lens, H, D, G=1, page=0, seed=0, capacity=None, widths_of=None):
        self.lens, self.H, self.D, self.G = list(lens), H, D, G
        n = sum(lens)
        self.k, self.v = rows(n, H, D, seed), rows(n, H, D, seed + 1)
        self.bits = widths(n, H, seed + 2) if widths_of is None else torch.full((n, H), widths_of, dtype=torch.uint8,
                                                                             device="cuda")
        self.cu = cu_of(lens)
        cap = [max(1, L) for L in lens] if capacity is None else capacity
        pages = sum(H * (c * 4 * D // page + 2) for c in cap) if page else 0
        self.cache = kvq.KVQCache(len(lens), H, D, cap, query_group=G, page_bytes=page, pool_pages=pages)
        if n:
            kvq.kvq_write(self.k, self.v, self.bits, self.cu, self.cache)
        self.start = [int(x) for x in self.cu.tolist()]

    def seq(self, s, what="k"):
        """fp64 values [L, H, D] of sequence s."""
        r = slice(self.start[s], self.start[s] + self.lens[s])
        return values64(getattr(self, what)[r], self.bits[r])


def bounds64(f: Filled, block, nt):
    """{(s, h): (lo, hi)} as [nb, D] fp64, before rounding."""
    out = {}
    for s, L in enumerate(f.lens):
        x = f.seq(s)
        for h in range(f.H):
            parts = [x[a:a + block, h] for a in range(0, L, block)]
            out[s, h] = (torch.stack([p.amin(0) for p in parts]) if parts else x.new_zeros((0, f.D)),
                         torch.stack([p.amax(0) for p in parts]) if parts else x.new_zeros((0, f.D)))
    return out


def flat_bounds(b):
    """[B, H, nt, 2, D, 64] as [B, H, 2, D, nt * 64]."""
    return b.permute(0, 1, 3, 4, 2, 5).flatten(-2)


def scores64(q, bounds, modes, lens, block, G):
    """fp64 scores [B, H, nt * 64] with -inf where the call gives -inf."""
    fb = flat_bounds(bounds).double()
    B, H = fb.shape[:2]
    out = torch.full((B, H, fb.shape[-1]), -math.inf, dtype=torch.float64, device=q.device)
    for s in range(B):
        nb = -(-lens[s] // block)
        for h in range(H):
            for g in range(G):
                if modes is None or int(modes[s, h * G + g]) == 2:
                    qv = q[s, h * G + g].double()[:, None]
                    sc = torch.maximum(qv * fb[s, h, 0], qv * fb[s, h, 1]).sum(0)
                    out[s, h, :nb] = torch.maximum(out[s, h, :nb], sc[:nb])
    return out


def choose(scores, lens, block, k, first, last):
    """ids [B, H, k] from fp32 scores: by key descending, index ascending; -1 without a full query."""
    B, H, _ = scores.shape
    ids = torch.full((B, H, k), -1, dtype=torch.int32)
    sc = scores.cpu()
    for s in range(B):
        nb = -(-lens[s] // block)
        for h in range(H):
            row = sc[s, h, :nb].tolist()
            if nb == 0 or all(x == -math.inf for x in row):
                continue
            key = [(-math.inf if (b < first or b >= nb - last) else -row[b], b) for b in range(nb)]
            take = sorted(b for _, b in sorted(key)[:k])
            ids[s, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
    return ids


def attention64(f: Filled, q, ids, block, modes, w):
    """fp64 outputs [B, HQ, D] and, per output, the error that fp32 arithmetic may leave.

    Logits: a D-term fp32 dot product and the few operations around it are off by at most
    (D + 16) U32 times the sum of the terms' magnitudes |q_c| (c s + |z|); a weight by twice that and
    the exponential's 2^-21; the output sums n terms: (n + 16) U32 of sum p |v|, |v| <= c s + |z|."""
    B, HQ, D = q.shape
    out = torch.zeros((B, HQ, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for s, L in enumerate(f.lens):
        r = slice(f.start[s], f.start[s] + L)
        kc, ks, kz = stored(f.k[r], f.bits[r])
        vc, vs, vz = stored(f.v[r], f.bits[r])
        ks, kz, vs, vz = (t.double()[..., None] for t in (ks, kz, vs, vz))
        for hq in range(HQ):
            h, m = hq // f.G, int(modes[s, hq])
            if m == 0 or L == 0:
                continue
            if m == 1:
                j = torch.arange(max(0, L - 1 - w), L, device=q.device)
            else:
                b = ids[s, h]
                j = (b[b >= 0].long()[:, None] * block + torch.arange(block, device=q.device)).flatten()
                j = j[j < L]
            if j.numel() == 0:
                continue
            qv = q[s, hq].double()
            a = ((kc[j, h] * ks[j, h] + kz[j, h]) @ qv) / math.sqrt(D)
            mag = ((kc[j, h].abs() * ks[j, h] + kz[j, h].abs()) @ qv.abs()) / math.sqrt(D)
            p = torch.softmax(a, 0)
            out[s, hq] = p @ (vc[j, h] * vs[j, h] + vz[j, h])
            off = 2 * (D + 16) * U32 * float(mag.max()) + 2.0 ** -21
            tol[s, hq] = (off + (j.numel() + 16) * U32) * 2 * (p @ (vc[j, h].abs() * vs[j, h] + vz[j, h].abs()))
    return out, tol


def assert_attention(got, ref, tol, what=""):
    """Every output within its bound, and all together within sqrt-like growth of the same
    roundings: independent errors of n and D terms of 2^-24 stay below 2e-5 of the result."""
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{what}: {float((err - tol).max()):.3e} past the bound"
    norm = float(ref.norm())
    assert float((got.double() - ref).norm()) <= 2e-5 * norm, f"{what}: rel L2 {float((got.double() - ref).norm()) / norm:.3e}"
