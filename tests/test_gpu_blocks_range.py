"""Attention over chosen blocks with values of very different magnitudes, against 64 bits: a key's
error may count only as far as its weight does."""
import math

import pytest
import torch

from blocks_testlib import U32, Filled, cu_of, rows, stored, widths
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu


def _own(k, v, bits, G, page=0):
    """A one-sequence cache of these rows."""
    n, H, D = k.shape
    f = Filled([0], H, D, G=G, page=page, capacity=[n])
    f.lens, f.start, f.k, f.v, f.bits = [n], [0, n], k, v, bits
    kvq.kvq_write(k, v, bits, cu_of([n]), f.cache)
    return f


def _centred(x, bits):
    """Centred codes, scales and zeros as the attention uses them: c' s + z' is the value."""
    c, s, z = stored(x, bits)
    mid = torch.where(bits == 16, 0.0, (torch.exp2(bits.double()) - 1) / 2)
    s, z = s.double(), z.double()
    return c - mid[..., None], s[..., None], (z + mid * s)[..., None]


def _one_channel_attention64(f, q, keys):
    """fp64 outputs of one head's queries q [G, D], of which only channel 0 is not 0, over `keys`, and
    the error fp32 arithmetic may leave.

    A logit has two terms, of magnitude q s |c'| and q |z'|, and 7 roundings on the way to the
    exponent, the last one of its distance to the maximum: 8 U32 of the magnitudes of both, times
    ln 2 in log2 units. The exponential adds 2^-21, the split of the weight 2^-22, the sums of n terms
    2 (n + 16) U32. The same error of the weights' sum comes on top, relative."""
    D, n = q.shape[1], len(keys)
    kc, ks, kz = (t[keys, 0] for t in _centred(f.k, f.bits))
    vc, vs, vz = (t[keys, 0] for t in _centred(f.v, f.bits))
    qd = q.double()
    a = qd @ (kc * ks + kz).T / math.sqrt(D)
    mag = qd.abs()[:, :1] * (kc.abs() * ks + kz.abs())[:, :1].T / math.sqrt(D) / math.log(2)
    top = torch.gather(mag, 1, a.argmax(1, keepdim=True))
    p = torch.softmax(a, 1)
    mv = vc.abs() * vs + vz.abs()
    e = math.log(2) * 8 * U32 * (mag + top) + 2.0 ** -21 + 2.0 ** -22 + 2 * (n + 16) * U32
    return p @ (vc * vs + vz), (p * e) @ mv + (p * e).sum(1, keepdim=True) * (p @ mv)


@pytest.mark.parametrize("order", ["large first", "small first", "mixed"])
@pytest.mark.parametrize("b,G,D", [(2, 1, 64), (4, 4, 128), (8, 2, 64), (16, 1, 128), (16, 4, 64), (2, 8, 128), (16, 8, 128),
                                   (8, 5, 64), (0, 4, 128)])
def test_weights_beside_much_larger_values(b, G, D, order):
    """Rows of V about 2^14 and rows about 2^-14; one half of the queries puts its weight on the
    first, the other half on the second, the others' weight going from a lot to nothing."""
    n = 160
    g = torch.Generator(device="cuda").manual_seed(7)
    at = torch.arange(n, device="cuda")
    large = {"large first": at < n // 2, "small first": at >= n // 2, "mixed": at * 7 % 5 < 2}[order]
    v = torch.randint(-1023, 1024, (n, 1, D), generator=g, device="cuda").double()
    v = (v * torch.where(large, 16.0, 2.0 ** -24)[:, None, None]).half()
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    k[large, 0, 0] = 1.0
    bits = widths(n, 1, 3) if b == 0 else torch.full((n, 1), b, dtype=torch.uint8, device="cuda")
    f = _own(k, v, bits, G)
    modes = torch.full((1, G), 2, dtype=torch.uint8, device="cuda")
    ids = torch.arange(n // 16, dtype=torch.int32, device="cuda").reshape(1, 1, -1).contiguous()
    for far in (0.0, 12.0, 20.0, 30.0, 60.0, 200.0):
        q = torch.zeros((1, G, D), dtype=torch.float16, device="cuda")
        q[0, 0::2, 0], q[0, 1::2, 0] = -far * math.sqrt(D), far * math.sqrt(D)
        got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, modes, 0)
        f.cache.check()
        ref, tol = _one_channel_attention64(f, q[0], list(range(n)))
        err = (got[0].double() - ref).abs()
        assert bool((err <= tol).all()), f"far {far}: {float((err / tol).max()):.3g} times the bound"


def test_weights_after_rows_without_values():
    """Constant rows of V (scale 0) hold the weight, rows of a tiny scale the rest, then large rows."""
    D, n = 64, 96
    v = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    v[32:64] = rows(32, 1, D, 1) * 2.0 ** -12
    v[64:] = rows(32, 1, D, 2) * 2.0 ** 12
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    k[32:64, 0, 0], k[64:, 0, 0] = -1.0, -2.0
    for b in (2, 4, 8, 16):
        f = _own(k, v, torch.full((n, 1), b, dtype=torch.uint8, device="cuda"), 1)
        for blocks in ([0, 1, 2, 3], [2, 3], [0, 1], [0, 1, 2, 3, 4, 5], [0, 4, 5]):
            ids = torch.tensor([[blocks]], dtype=torch.int32, device="cuda")
            keys = [j for x in blocks for j in range(16 * x, 16 * x + 16)]
            for far in (0.0, 8.0, 25.0):
                q = torch.zeros((1, 1, D), dtype=torch.float16, device="cuda")
                q[..., 0] = far * math.sqrt(D)
                got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, torch.full((1, 1), 2, dtype=torch.uint8, device="cuda"),
                                                    0)
                f.cache.check()
                ref, tol = _one_channel_attention64(f, q[0], keys)
                assert bool(((got[0].double() - ref).abs() <= tol).all()), (b, blocks, far)
