"""Attention over chosen blocks with values that are not finite: they reach the queries that attend
over them, and no others."""
import math

import pytest
import torch

from blocks_testlib import Filled, assert_attention, attention64, rows
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
