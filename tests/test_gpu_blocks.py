"""Block-sparse decoding: the blocks' bounds, the choice of blocks and the routed attention over
them, against plain 64-bit forms, and the chain of them as a decode loop runs it."""
import math

import pytest
import torch

from blocks_testlib import (TILE, U16, U32, Filled, assert_attention, attention64, bounds64, choose, cu_of, flat_bounds,
                            rope_table, rotate, rows, scores64, values32, widths)
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bounds
@pytest.mark.parametrize("lens,H,D,block,page", [
    ([1], 1, 64, 16, 0),
    ([16, 0, 17, 15], 2, 128, 16, 0),
    ([333, 64, 129, 1], 3, 64, 32, 4096),
    ([5000, 65], 2, 128, 64, 4096),
    ([1500, 128, 127], 2, 128, 128, 0),
    ([4200], 1, 64, 64, 0),
])
def test_bounds(lens, H, D, block, page):
    f = Filled(lens, H, D, page=page, seed=5)
    nt = kvq.block_tiles(f.cache, block)
    out = torch.full((len(lens), H, nt, 2, D, TILE), 3.0, dtype=torch.float16, device="cuda")
    assert kvq.block_bounds(f.cache, block, out=out) is out
    f.cache.check()
    fb = flat_bounds(out)
    for (s, h), (lo, hi) in bounds64(f, block, nt).items():
        nb = lo.shape[0]
        r = slice(f.start[s], f.start[s] + lens[s])
        x = values32(f.k[r, h:h + 1], f.bits[r, h:h + 1])[:, 0]
        for i, (want, pick) in enumerate(((lo, "amin"), (hi, "amax"))):
            got = fb[s, h, i, :, :nb].T
            exact = [getattr(x[a:a + block], pick)(0).half() for a in range(0, lens[s], block)]
            assert not exact or torch.equal(got, torch.stack(exact))
            # fp32 product and sum (terms up to 4 max|x|), then half a step of fp16
            tol = 12 * U32 * float(f.k.abs().max()) + U16 * want.abs() + 2.0 ** -25
            assert bool(((got.double() - want).abs() <= tol).all())
        assert bool((fb[s, h, :, :, nb:] == 3.0).all())       # entries past the last block stay


@pytest.mark.parametrize("block", [16, 64])
def test_bounds_kept_up_through_writes_and_roll_backs(block):
    B, H, D = 3, 2, 128
    cache = kvq.KVQCache(B, H, D, [400, 200, 90])
    bounds = kvq.block_bounds(cache, block)
    assert bool((bounds == 0).all())
    have = [0, 0, 0]
    for i, (back, new) in enumerate([(None, [200, 65, 0]), (None, [1, 1, 1]), ([190, 64, -1], [3, 1, 80]),
                                     (None, [0, 0, 0]), ([0, 10, 81], [1, 100, 2]), ([-1, 5, 3], [300, 1, 1])]):
        if back is not None:
            have = [min(h, b) if b >= 0 else h for h, b in zip(have, back)]
            cache.truncate(torch.tensor(back, dtype=torch.int32, device="cuda"))
        n = sum(new)
        if n:
            kvq.kvq_write(rows(n, H, D, i), rows(n, H, D, i + 50), widths(n, H, i), cu_of(new), cache)
        have = [h + m for h, m in zip(have, new)]
        kvq.block_bounds(cache, block, cu_of(new), out=bounds)
        cache.check()
        fresh = flat_bounds(kvq.block_bounds(cache, block))
        for s in range(B):
            nb = -(-have[s] // block)
            assert torch.equal(flat_bounds(bounds)[s, ..., :nb], fresh[s, ..., :nb]), (i, s)


def test_bounds_refusals():
    f = Filled([20], 1, 64)
    for block in (0, 8, 48, 256):
        with pytest.raises((kvq.KVQError, ValueError)):
            kvq.block_bounds(f.cache, block)
    with pytest.raises(ValueError):
        kvq.block_bounds(f.cache, 16, cu_of([1]))
    with pytest.raises(ValueError):
        kvq.block_bounds(f.cache, 16, out=torch.zeros((1, 1, 1, 2, 64, 32), dtype=torch.float16, device="cuda"))
    out = kvq.block_bounds(f.cache, 16)
    kvq.block_bounds(f.cache, 16, cu_of([21]), out=out)        # more new tokens than the sequence holds
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK


# ------------------------------------------------------------------ choice
def _random_bounds(B, H, nt, D, seed, grid=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mid = 0.5 * torch.randn((B, H, nt, 1, D, TILE), generator=g, device="cuda")
    rad = (2.3 + 0.4 * torch.randn((B, H, nt, 1, D, TILE), generator=g, device="cuda")).abs()
    b = torch.cat((mid - rad, mid + rad), 3)
    return (b if grid is None else (b * grid).round() / grid).half()


@pytest.mark.parametrize("lens,H,G,D,block,k,first,last", [
    ([1], 1, 1, 64, 16, 1, 0, 0),
    ([777, 0, 64, 65], 2, 1, 128, 16, 5, 1, 1),
    ([5000, 3, 4096], 1, 2, 64, 32, 17, 0, 1),
    ([9000, 2500], 2, 4, 128, 64, 64, 1, 2),
    ([3000], 3, 3, 64, 128, 2, 1, 1),
    ([2000, 800], 1, 9, 128, 16, 40, 2, 0),
    ([70000], 1, 1, 64, 16, 100, 1, 1),                        # more blocks than one pass of the CTA holds
    ([140000, 9], 1, 2, 64, 16, 4096, 3, 5),
    ([300, 0, 17, 1030] * 25, 3, 1, 128, 16, 9, 1, 1),         # a CTA per (sequence, head)
    ([5000, 4000] * 50, 3, 2, 64, 64, 20, 0, 1),
])
def test_choice(lens, H, G, D, block, k, first, last):
    cache = kvq.KVQCache(len(lens), H, D, [max(1, L) for L in lens], query_group=G)
    n, B = sum(lens), len(lens)
    x = torch.zeros((n, H, D), dtype=torch.float16, device="cuda")
    kvq.kvq_write(x, x, torch.full((n, H), 2, dtype=torch.uint8, device="cuda"), cu_of(lens), cache)
    nt = kvq.block_tiles(cache, block)
    bounds = _random_bounds(B, H, nt, D, 3)
    q = rows(B, H * G, D, 4)
    g = torch.Generator().manual_seed(k)
    for modes in (None, torch.randint(0, 3, (B, H * G), generator=g).to(torch.uint8).cuda(),
                  torch.ones((B, H * G), dtype=torch.uint8, device="cuda")):
        ids, scores = kvq.select_blocks(q, cache, bounds, block, k, modes, first=first, last=last)
        cache.check()
        ref = scores64(q, bounds, modes, lens, block, G)
        assert torch.equal(scores.isfinite(), ref.isfinite())
        # a sum in fp64 (D terms, each 2^-53 of the largest partial sum), rounded to fp32 once
        fin = ref.isfinite()
        mag = float(q.double().abs().sum(-1).max() * bounds.double().abs().max())
        assert bool(((scores.double() - ref)[fin].abs() <= U32 * ref[fin].abs() + D * 2.0 ** -52 * mag).all())
        assert torch.equal(ids.cpu(), choose(scores, lens, block, k, first, last))


def test_choice_in_a_very_long_context():
    # one head of 600000 keys, 37500 blocks: several passes of the choosing CTA
    L, block, k = 600000, 16, 300
    cache = kvq.KVQCache(1, 1, 64, L)
    x = torch.zeros((L, 1, 64), dtype=torch.float16, device="cuda")
    kvq.kvq_write(x, x, torch.full((L, 1), 2, dtype=torch.uint8, device="cuda"), cu_of([L]), cache)
    bounds = _random_bounds(1, 1, kvq.block_tiles(cache, block), 64, 3, grid=1)
    q = rows(1, 1, 64, 5).round()                              # many ties
    ids, scores = kvq.select_blocks(q, cache, bounds, block, k)
    cache.check()
    assert torch.equal(ids.cpu(), choose(scores, [L], block, k, 1, 1))
    out = kvq.routed_attn_decode_blocks(q, cache, ids, block, torch.full((1, 1), 2, dtype=torch.uint8, device="cuda"), 0)
    cache.check()
    assert bool((out == 0).all())                              # every value is 0


def test_ties_go_to_the_lowest_index_and_order_of_sums_does_not_matter():
    # values on a coarse grid: many equal scores; and channels permuted give the same scores
    lens, H, D, block = [64 * 128], 2, 128, 64
    f = Filled(lens, H, D, widths_of=2)
    q = (rows(1, H, D, 1) * 2).round() / 2
    b = _random_bounds(1, H, 2, D, 9, grid=2)
    b[:, :, 1] = b[:, :, 0]                                    # every block of tile 1 equals one of tile 0
    ids, scores = kvq.select_blocks(q, f.cache, b, block, 20, first=0, last=0)
    assert torch.equal(ids.cpu(), choose(scores, lens, block, 20, 0, 0))
    assert torch.equal(scores[..., :64], scores[..., 64:])
    perm = torch.randperm(D, generator=torch.Generator().manual_seed(1)).cuda()
    ids2, s2 = kvq.select_blocks(q[..., perm].contiguous(), f.cache, b[..., perm, :].contiguous(), block, 20, first=0, last=0)
    assert torch.equal(s2, scores) and torch.equal(ids2, ids)
    same = torch.zeros_like(b)                                 # every score 0 (some -0): the lowest blocks
    ids, _ = kvq.select_blocks(-q, f.cache, same, block, 7, first=0, last=0)
    assert ids.cpu().tolist() == [[list(range(7))] * H]


def test_scores_at_the_ends_of_fp16():
    lens, D, block = [64 * 3], 64, 64
    f = Filled(lens, 1, D, widths_of=2)
    b = torch.zeros((1, 1, 1, 2, D, TILE), dtype=torch.float16, device="cuda")
    q = torch.zeros((1, 1, D), dtype=torch.float16, device="cuda")
    q[0, 0, 0], q[0, 0, 1], q[0, 0, 2] = 65504.0, 2.0 ** -24, -65504.0
    b[..., 0, 0], b[..., 2, 0] = 65504.0, -65504.0             # the largest product twice
    b[..., 1, 1] = 2.0 ** -24                                  # a subnormal product alone
    b[0, 0, 0, 0, 2, 2], b[0, 0, 0, 1, 2, 2] = -2.0 ** -24, 2.0 ** -24
    _, scores = kvq.select_blocks(q, f.cache, b, block, 1, first=0, last=0)
    assert scores[0, 0, :3].tolist() == [2 * 65504.0 ** 2, 2.0 ** -48, 65504.0 * 2.0 ** -24]


def test_choice_refusals():
    f = Filled([100], 2, 64, G=2)
    b, q = kvq.block_bounds(f.cache, 16), rows(1, 4, 64, 1)
    for change in (dict(k=0), dict(k=4097), dict(k=2, first=2, last=1), dict(first=-1), dict(block=48), dict(q=q[:, :2]),
                   dict(q=q.float()), dict(bounds=b[..., :32]), dict(modes=torch.zeros((1, 2), dtype=torch.uint8, device="cuda")),
                   dict(ids=torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda"))):
        args = dict(q=q, cache=f.cache, bounds=b, block=16, k=4) | change
        with pytest.raises((kvq.KVQError, ValueError, TypeError)):
            kvq.select_blocks(**args)
    m = torch.tensor([[2, 3, 2, 2]], dtype=torch.uint8, device="cuda")
    kvq.select_blocks(q, f.cache, b, 16, 4, m)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_MODE


# ------------------------------------------------------------------ attention
def _random_ids(lens, H, block, k, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.full((len(lens), H, k), -1, dtype=torch.int32)
    for s, L in enumerate(lens):
        nb = -(-L // block)
        for h in range(H):
            n = int(torch.randint(0, min(k, nb) + 1, (1,), generator=g))
            ids[s, h, :n] = torch.randperm(nb, generator=g)[:n].sort().values.to(torch.int32)
    return ids.cuda()


ATTN = [
    # lens, H, G, D, block, k, w, page
    ([1], 1, 1, 64, 16, 1, 0, 0),
    ([777, 0, 64, 65], 2, 1, 128, 16, 5, 100, 0),
    ([3000, 3, 2049], 3, 2, 64, 32, 17, 33, 4096),
    ([9000, 2500], 2, 4, 128, 64, 64, 512, 65536),
    ([3000, 1], 3, 3, 64, 128, 9, 5000, 0),
    ([2000, 800, 1999], 1, 9, 128, 16, 90, 0, 4096),
    ([1300], 2, 16, 64, 64, 21, 64, 0),
    ([20000], 1, 1, 128, 128, 157, 20000, 0),
    ([500] * 40, 4, 1, 128, 64, 3, 20, 0),
    ([5000], 2, 20, 128, 32, 130, 257, 4096),
    # as many (sequence, head)s as start small CTAs, one of them short of a tile, several tiles, or empty
    ([300, 1, 0, 77] * 20, 8, 1, 128, 64, 5, 33, 0),
    ([1500, 1100] * 74, 4, 1, 64, 64, 24, 1200, 4096),
    ([90] * 100, 6, 5, 64, 16, 4, 20, 0),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case):
    lens, H, G, D, block, k, w, page = ATTN[case]
    B = len(lens)
    f = Filled(lens, H, D, G=G, page=page, seed=case)
    q = rows(B, H * G, D, 40 + case)
    ids = _random_ids(lens, H, block, k, case)
    for modes in (torch.full((B, H * G), 2, dtype=torch.uint8, device="cuda"),
                  torch.randint(0, 3, (B, H * G), generator=torch.Generator().manual_seed(case)).to(torch.uint8).cuda(),
                  torch.ones((B, H * G), dtype=torch.uint8, device="cuda")):
        got = kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w)
        f.cache.check()
        ref, tol = attention64(f, q, ids, block, modes, w)
        assert_attention(got, ref, tol, f"case {case} modes {modes.flatten()[:3].tolist()}")
        empty = ref.abs().amax(-1) == 0
        assert bool((got[empty] == 0).all())
        again = kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w)
        assert torch.equal(again, got)                         # repeatable bit for bit


@pytest.mark.parametrize("b", [2, 4, 8, 16])
def test_attention_one_width_at_a_time(b):
    f = Filled([260, 1000], 2, 128, seed=b, widths_of=b)
    q = rows(2, 2, 128, 3)
    ids = torch.arange(16, dtype=torch.int32, device="cuda").expand(2, 2, 16).contiguous()
    ids[0, :, 5:] = -1
    modes = torch.full((2, 2), 2, dtype=torch.uint8, device="cuda")
    got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 64, modes, 0)
    f.cache.check()
    assert_attention(got, *attention64(f, q, ids, 64, modes, 0), f"b={b}")


@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (4, 128), (8, 128)])
def test_attention_keeps_single_precision(G, D):
    """Normal rows, all widths: independent roundings of 2^-24 in the logits (about log2(e) |q||k| /
    sqrt(D), a few units) and 2^-22 of the weights' exponentials leave a few 1e-7 of the result."""
    f = Filled([6000] * 3, 2, D, G=G, seed=12)
    q = rows(3, 2 * G, D, 5)
    ids = _random_ids(f.lens, 2, 64, 60, 2)
    ids[:, :, 0] = ids[:, :, 0].clamp(min=0)
    modes = torch.full((3, 2 * G), 2, dtype=torch.uint8, device="cuda")
    got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 64, modes, 0).double()
    ref, _ = attention64(f, q, ids, 64, modes, 0)
    assert float((got - ref).norm()) <= 1e-6 * float(ref.norm())


def test_attention_all_blocks_equals_routed_decode():
    for D, G, page in ((128, 1, 0), (64, 4, 4096)):
        f = Filled([1000, 17, 333], 2, D, G=G, page=page, seed=2)
        q = rows(3, 2 * G, D, 1)
        modes = torch.randint(0, 3, (3, 2 * G), generator=torch.Generator().manual_seed(1)).to(torch.uint8).cuda()
        ids = torch.full((3, 2, 32), -1, dtype=torch.int32, device="cuda")
        for s, L in enumerate(f.lens):
            nb = -(-L // 32)
            ids[s, :, :nb] = torch.arange(nb, dtype=torch.int32, device="cuda")
        a = kvq.routed_attn_decode_blocks(q, f.cache, ids, 32, modes, 50)
        b = kvq.routed_attn_decode(q, f.cache, modes, 50)
        f.cache.check()
        _, tol = attention64(f, q, ids, 32, modes, 50)
        assert bool(((a - b).double().abs() <= 2 * tol).all())


def test_large_and_small_magnitudes():
    # values near fp16's ends in V, logits far apart, tiny V beside large V
    D, n = 128, 256
    k, v = rows(n, 1, D, 1), rows(n, 1, D, 2)
    v[:64] *= 3.0e4 / 6
    v[64:128] *= 1.0e-4
    v[128:192] = 0.125
    k[200] *= 8
    bits = widths(n, 1, 3)
    f = Filled([n], 1, D)
    f.cache = kvq.KVQCache(1, 1, D, n)
    f.k, f.v, f.bits = k, v, bits
    kvq.kvq_write(k, v, bits, cu_of([n]), f.cache)
    modes = torch.full((1, 1), 2, dtype=torch.uint8, device="cuda")
    for scale in (1.0, 30.0, 0.0):
        q = rows(1, 1, D, 5) * scale
        for picked in ([0, 1, 2, 3], [1], [2], [3], [1, 3]):
            ids = torch.tensor([[picked + [-1] * (4 - len(picked))]], dtype=torch.int32, device="cuda")
            got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 64, modes, 0)
            assert_attention(got, *attention64(f, q, ids, 64, modes, 0), f"scale {scale} {picked}")


def test_bad_entries_are_passed_over_and_reported():
    f = Filled([200, 100], 1, 64, seed=4)
    q = rows(2, 1, 64, 2)
    modes = torch.full((2, 1), 2, dtype=torch.uint8, device="cuda")
    want_ids = torch.tensor([[[1, 5, -1, -1, -1, -1]], [[0, 6, -1, -1, -1, -1]]], dtype=torch.int32, device="cuda")
    ref, tol = attention64(f, q, want_ids, 16, modes, 0)
    for bad in ([[1, 5, 5, -1, -1, -1], [0, 6, -1, -1, -1, -1]],            # the same block twice
                [[1, 5, 3, -1, -1, -1], [0, 6, -1, -1, -1, -1]],            # not ascending
                [[1, 5, -1, 7, -1, -1], [0, 6, -1, -1, -1, -1]],            # a block behind the padding
                [[1, 5, 13, -1, -1, -1], [0, 6, 7, 2 ** 31 - 1, -1, -1]],   # past the length
                [[1, 5, 2 ** 28, -1, -1, -1], [0, 6, -1, -1, -2 ** 31, -1]]):
        ids = torch.tensor(bad, dtype=torch.int64).to(torch.int32)[:, None].contiguous().cuda()
        got = kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, modes, 0)
        code = 0
        try:
            f.cache.check()
        except kvq.KVQError as e:
            code = e.code
        assert code == kvq.KVQ_ERR_DEVICE_CHECK, bad
        assert_attention(got, ref, tol, str(bad))


def test_attention_refusals():
    f = Filled([100], 2, 64, G=2)
    q, m = rows(1, 4, 64, 1), torch.full((1, 4), 2, dtype=torch.uint8, device="cuda")
    ids = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")
    for change in (dict(block=24), dict(w=-1), dict(ids=ids[:, :1]), dict(ids=ids.long()), dict(ids=ids[0]), dict(modes=m[:, :2]),
                   dict(q=q[:, :2]), dict(ids=torch.zeros((1, 2, 0), dtype=torch.int32, device="cuda")),
                   dict(out=torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda"))):
        args = dict(q=q, cache=f.cache, ids=ids, block=16, modes=m, w=4) | change
        with pytest.raises((kvq.KVQError, ValueError, TypeError)):
            kvq.routed_attn_decode_blocks(**args)
    lib = kvq.load_library()
    assert lib.routed_attn_decode_blocks_scratch(f.cache.handle, 0, 16, 4) == -1
    assert lib.routed_attn_decode_blocks_scratch(f.cache.handle, 1, 17, 4) == -1
    kvq.routed_attn_decode_blocks(q, f.cache, torch.full((1, 2, 1), -1, dtype=torch.int32, device="cuda"), 16,
                                  torch.full((1, 4), 9, dtype=torch.uint8, device="cuda"), 4)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_MODE


# ------------------------------------------------------------------ the chain
def _step(cache, table, x, bits, one, bounds, modes, block, k, w, pos=None):
    q = kvq.kvq_write_rope(x["q"], x["k"], x["v"], bits, one, cache, table, positions=pos)
    kvq.block_bounds(cache, block, one, out=bounds)
    ids, _ = kvq.select_blocks(q, cache, bounds, block, k, modes)
    return q, ids, kvq.routed_attn_decode_blocks(q, cache, ids, block, modes, w)


@pytest.mark.parametrize("D,G,page,captured", [(128, 1, 0, False), (64, 4, 4096, False), (128, 4, 8192, True)])
def test_decode_loop(D, G, page, captured):
    """A prompt, then decode steps: append with rotation, renew the bounds, choose, attend; each
    step against the plain forms over all rows so far, eager or captured once and replayed."""
    B, H, block, k, w, steps = 3, 2, 32, 6, 40, 4
    pre = [500, 31, 260]
    cap = [L + steps for L in pre]
    f = Filled([0] * B, H, D, G=G, page=page, capacity=cap)
    cache, table = f.cache, rope_table(max(cap), D)
    kp, vp, bp = rows(sum(pre), H, D, 1), rows(sum(pre), H, D, 2), widths(sum(pre), H, 3)
    kvq.kvq_write_rope(None, kp, vp, bp, cu_of(pre), cache, table)
    bounds = kvq.block_bounds(cache, block)
    pos = torch.cat([torch.arange(L, device="cuda") for L in pre])
    kr = rotate(kp, pos, table, False)
    hist = [[kr[a:a + L], vp[a:a + L], bp[a:a + L]] for a, L in zip(cu_of(pre).tolist(), pre)]
    x = {"q": rows(B, H * G, D, 0), "k": rows(B, H, D, 0), "v": rows(B, H, D, 0)}
    bits, modes, one = widths(B, H, 0), torch.zeros((B, H * G), dtype=torch.uint8, device="cuda"), cu_of([1] * B)
    back = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    if captured:
        roll = torch.tensor(pre, dtype=torch.int32, device="cuda")
        _step(cache, table, x, bits, one, bounds, modes, block, k, w, roll)      # warm-up, rolled back by the first replay
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _step(cache, table, x, bits, one, bounds, modes, block, k, w, back)
    for t in range(steps):
        for n in x:
            x[n].copy_(rows(B, x[n].shape[1], D, 100 * t + ord(n)))
        bits.copy_(widths(B, H, 10 + t))
        modes.copy_(torch.randint(0, 3, (B, H * G), generator=torch.Generator().manual_seed(t)).to(torch.uint8))
        modes[:, 0] = 2
        if captured:
            back.fill_(-1) if t else back.copy_(roll)
            graph.replay()
        else:
            outs = _step(cache, table, x, bits, one, bounds, modes, block, k, w)
        q, ids, out = outs
        cache.check()
        at = torch.tensor([L + t for L in pre], device="cuda")
        assert torch.equal(q, rotate(x["q"], at, table, False))
        krt = rotate(x["k"], at, table, False)
        for s in range(B):
            hist[s] = [torch.cat((a, b[s:s + 1])) for a, b in zip(hist[s], (krt, x["v"], bits))]
        f.lens = [L + t + 1 for L in pre]
        f.start = cu_of(f.lens).tolist()
        f.k, f.v, f.bits = (torch.cat([hh[i] for hh in hist]) for i in range(3))
        fresh = kvq.block_bounds(cache, block)
        want = choose(scores64(q, fresh, modes, f.lens, block, G).float(), f.lens, block, k, 1, 1)
        assert torch.equal(ids.cpu(), want)
        assert_attention(out, *attention64(f, q, ids, block, modes, w), f"step {t}")


def test_two_streams_share_a_cache_for_reading():
    f = Filled([2000, 900], 2, 128, G=2, seed=8)
    q = [rows(2, 4, 128, i) for i in range(2)]
    modes = torch.full((2, 4), 2, dtype=torch.uint8, device="cuda")
    bounds = kvq.block_bounds(f.cache, 16)
    want = []
    for i in range(2):
        ids, _ = kvq.select_blocks(q[i], f.cache, bounds, 16, 50, modes)
        want.append((ids, kvq.routed_attn_decode_blocks(q[i], f.cache, ids, 16, modes, 0)))
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            ids, _ = kvq.select_blocks(q[i], f.cache, bounds, 16, 50, modes, stream=st[i])
            got[i] = (ids, kvq.routed_attn_decode_blocks(q[i], f.cache, ids, 16, modes, 0, stream=st[i]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bounds_hold_every_logit():
    f = Filled([1000], 2, 128, seed=1)
    bounds = kvq.block_bounds(f.cache, 64)
    q = rows(1, 2, 128, 2)
    _, scores = kvq.select_blocks(q, f.cache, bounds, 64, 4)
    for h in range(2):
        a = f.seq(0)[:, h] @ q[0, h].double()
        top = torch.stack([a[i:i + 64].max() for i in range(0, 1000, 64)])
        slack = U16 * float((q[0, h].double().abs().sum() * f.k.double().abs().max()))
        assert bool((scores[0, h, :16].double() >= top - slack).all())
        assert math.isinf(float(scores[0, h, 16]))
