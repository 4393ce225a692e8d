"""Attention over chosen blocks with values that are not finite: they reach the queries that attend
over them, and no others."""
import math

import pytest
import torch

from blocks_testlib import Filled, assert_attention, attention64, cu_of, flat_bounds, rows
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _filled(lens, H, D, G, page, seed, at, poison, b, part):
    """A cache whose token `at` of every sequence and head holds one value `poison` in K or V, at width b."""
    f = Filled([0] * len(lens), H, D, G=G, page=page, seed=seed, capacity=lens)
    g = Filled(lens, H, D, seed=seed)                          # (its rows)
    f.lens, f.k, f.v, f.bits, f.cu, f.start = g.lens, g.k, g.v, g.bits, g.cu, g.start
    for s in f.start[:-1]:
        getattr(f, part)[s + at, :, 5] = poison
        f.bits[s + at] = b
    kvq.kvq_write(f.k, f.v, f.bits, f.cu, f.cache)
    f.cache.check()
    return f


SHAPES = [
    # lens, H, G, D, block, k, w, page: one CTA a unit, a cluster, scratch and second launch, small CTAs
    ([300, 211], 2, 2, 64, 16, 8, 40, 0),
    ([300], 1, 5, 128, 32, 4, 40, 4096),
    ([3000], 1, 8, 64, 16, 120, 900, 0),
    ([20000], 1, 4, 128, 128, 150, 6000, 0),
    ([300, 150] * 75, 4, 3, 64, 16, 8, 40, 0),
]


@pytest.mark.parametrize("b,poison,part", [(16, INF, "v"), (16, NAN, "v"), (4, INF, "v"), (2, -INF, "v"), (8, NAN, "k"),
                                           (16, NAN, "k")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("where", ["chosen block", "window", "neither"])
def test_values_that_are_not_finite_stay_with_their_queries(shape, b, poison, part, where):
    lens, H, G, D, block, k, w, page = SHAPES[shape]
    B, short = len(lens), min(lens)
    at = {"chosen block": 2 * block + 3, "window": short - 1, "neither": 5}[where]
    if where == "window":
        lens = [short] * B                                     # (its last block is in every window)
    f = _filled(lens, H, D, G, page, shape, at, poison, b, part)
    ids = torch.full((B, H, k), -1, dtype=torch.int32)
    for s, L in enumerate(lens):
        listed = [x for x in range(1, -(-L // block) - 1) if where != "window" or (x + 1) * block <= at][:k]
        ids[s, :, :len(listed)] = torch.tensor(listed, dtype=torch.int32)
        assert at < L - 1 - w or where == "window"
    ids = ids.cuda()
    modes = torch.tensor([[(2, 1, 0, 2, 1, 1, 0, 2)[g % 8] for g in range(H * G)]] * B, dtype=torch.uint8, device="cuda")
    q = rows(B, H * G, D, 40 + shape)
    got = kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w)
    f.cache.check()
    hit = modes == {"chosen block": 2, "window": 1, "neither": 3}[where]
    # what the cache holds: a quantized row takes its minimum and maximum over numbers and a NaN in it gets
    # code 0, its minimum (finite); an infinite one gives it an infinite scale, and every value is NaN
    own = slice(f.start[0] + at, f.start[0] + at + 1)
    held = kvq.kvq_read(f.cache, f.cu, f.start[-1], torch.float32)[part == "v"]
    if b < 16 and math.isnan(poison):
        hit = torch.zeros_like(hit)
        assert bool(held.isfinite().all())
        for x in f.start[:-1]:
            getattr(f, part)[x + at, :, 5] = held[x + at, :, 5].half()
    else:
        assert not bool(held[own, :, 5].isfinite().any())
    # a value that is not finite in a quantized row leaves no channel of it; in a native V row, its own
    ch = got if part == "k" or b < 16 else got[..., 5:6]
    assert not bool(ch[hit].isfinite().any())
    assert bool((got[modes == 0] == 0).all())
    rest = ~hit & (modes != 0)
    assert bool(got[rest].isfinite().all())
    f.k, f.v = f.k.nan_to_num(0, 0, 0), f.v.nan_to_num(0, 0, 0)
    ref, tol = attention64(f, q, ids, block, modes, w)
    assert_attention(got[rest], ref[rest], tol[rest], f"{where} {b} {poison}")


@pytest.mark.parametrize("G", [1, 3, 8])
def test_a_query_that_is_not_a_number(G):
    f = Filled([300, 40], 2, 64, G=G, seed=1)
    q = rows(2, 2 * G, 64, 2)
    ids = torch.tensor([[[0, 1]] * 2] * 2, dtype=torch.int32, device="cuda")
    modes = torch.full((2, 2 * G), 2, dtype=torch.uint8, device="cuda")
    modes[1, 0] = 1
    ref, tol = attention64(f, q, ids, 16, modes, 7)
    q[0, G - 1, 3] = NAN
    q[1, 0, 9] = INF                                           # inf and -inf logits, and their difference
    got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, modes, 7)
    f.cache.check()
    bad = torch.zeros((2, 2 * G), dtype=torch.bool, device="cuda")
    bad[0, G - 1] = bad[1, 0] = True
    assert bool(got[bad].isnan().all())
    assert_attention(got[~bad], ref[~bad], tol[~bad])


def test_no_keys_is_still_zero():
    f = Filled([5], 1, 64, G=2)
    ids = torch.full((1, 1, 3), -1, dtype=torch.int32, device="cuda")
    got = kvq.routed_attn_decode_blocks(rows(1, 2, 64, 1), f.cache, ids, 16, torch.tensor([[2, 0]], dtype=torch.uint8,
                                                                                         device="cuda"), 0)
    assert bool((got == 0).all())


# ------------------------------------------------------------------ bounds and choice
@pytest.mark.parametrize("block,new", [(16, None), (64, None), (128, None), (16, 1), (64, 70), (128, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_bounds_of_keys_that_are_not_finite(block, new, D):
    """Infinite keys bound their channel, a NaN makes both bounds NaN; the other blocks are as ever."""
    lens, H = [700, 129], 2
    f = Filled([0, 0], H, D, seed=1, capacity=lens)
    g = Filled(lens, H, D, seed=1)
    k, bits = g.k, g.bits
    for i, (at, b, x) in enumerate([(3, 16, INF), (40, 16, -INF), (41, 16, INF), (200, 4, INF), (333, 16, NAN), (690, 16, -INF),
                                    (699, 2, -INF), (699 + 100, 16, NAN), (699 + 129, 16, INF)]):
        k[at, i % H, 7 * i], bits[at] = x, b
    kvq.kvq_write(k, g.v, bits, g.cu, f.cache)
    bounds = kvq.block_bounds(f.cache, block)
    if new is not None:
        fresh, cu = bounds, torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
        bounds = kvq.block_bounds(f.cache, block, cu, out=fresh.clone())
    f.cache.check()
    held, _ = kvq.kvq_read(f.cache, g.cu, g.start[-1], torch.float32)
    fb = flat_bounds(bounds)
    for s, L in enumerate(lens):
        x = held[g.start[s]:g.start[s] + L].half()
        for n in range(-(-L // block)):
            part = x[n * block:(n + 1) * block]
            assert torch.equal(fb[s, :, 0, :, n].isnan(), part.isnan().any(0))
            for i, pick in enumerate(("amin", "amax")):
                assert torch.equal(fb[s, :, i, :, n].nan_to_num(9.0, INF, -INF),
                                   getattr(part, pick)(0).nan_to_num(9.0, INF, -INF))


@pytest.mark.parametrize("L,G,D,block", [(700, 1, 64, 16), (700, 2, 128, 16), (9000, 4, 64, 32), (9000, 1, 128, 64),
                                         (70000, 3, 64, 16)])
def test_choice_with_bounds_that_are_not_finite(L, G, D, block):
    """Scores in 64 bits with IEEE rules; a sum that is not a number counts as -inf."""
    B, H, k = 2, 2, 9
    cache = kvq.KVQCache(B, H, D, L, query_group=G)
    x = torch.zeros((B * L, H, D), dtype=torch.float16, device="cuda")
    kvq.kvq_write(x, x, torch.full((B * L, H), 2, dtype=torch.uint8, device="cuda"), cu_of([L] * B), cache)
    nt, nb = kvq.block_tiles(cache, block), -(-L // block)
    g = torch.Generator(device="cuda").manual_seed(5)
    mid = torch.randn((B, H, nt, 1, D, 64), generator=g, device="cuda")
    b = torch.cat((mid - 2, mid + 2), 3).half()
    u = torch.rand(b.shape, generator=g, device="cuda")
    lo, hi = b[:, :, :, 0], b[:, :, :, 1]
    lo[u[:, :, :, 0] < 0.3 / D] = -INF
    hi[u[:, :, :, 1] < 0.3 / D] = INF
    both = u[:, :, :, 0] > 1 - 0.1 / D                         # a NaN key's channel
    lo[both], hi[both] = NAN, NAN
    same = u[:, :, :, 1] > 1 - 0.1 / D                         # every key of the block the same infinity
    lo[same], hi[same] = -INF, -INF
    q = rows(B, H * G, D, 3)
    q[q == 0] = 1.0
    ids, scores = kvq.select_blocks(q, cache, b, block, k, first=0, last=0)
    cache.check()
    fb, qd = flat_bounds(b).double(), q.double().view(B, H, G, D, 1)
    ref = torch.where(qd < 0, qd * fb[:, :, None, 0], qd * fb[:, :, None, 1]).sum(3).nan_to_num(-INF, INF, -INF).amax(2)
    ref[..., nb:] = -INF
    got = scores.double()
    odd = ~ref.isfinite()
    assert torch.equal(got[odd], ref[odd]) and bool((ref[..., :nb] == INF).any()) and bool((ref[..., :nb] == -INF).any())
    mag = float(q.double().abs().sum(-1).max()) * 8
    assert bool(((got - ref)[~odd].abs() <= 2.0 ** -24 * ref[~odd].abs() + D * 2.0 ** -52 * mag).all())
    for s in range(B):                                         # by score, ties to the lower index
        for h in range(H):
            row = scores[s, h, :nb].tolist()
            want = sorted(sorted(range(nb), key=lambda n: (-row[n], n))[:k])
            assert ids[s, h].tolist() == want
