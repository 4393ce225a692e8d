"""The rotating write (kvq_write_rope): q rotated bit for bit as the fp32 formula with every
operation rounded on its own, within rounding of the formula in 64 bits, and the cache equal
to kvq_write of the rotated rows, for both launch forms (short appends; scan + quantize)."""
import pytest
import torch

from blocks_testlib import U16, U32, cu_of, rope_table, rotate, rows, widths
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu


def _same_cache(a, b, H, lens):
    for s, L in enumerate(lens):
        for h in range(H):
            if L:
                for x, y in zip(a.export(s, h, 0, L), b.export(s, h, 0, L)):
                    assert torch.equal(x, y), (s, h)


def _inputs(counts, H, G, D, fused, seed):
    n = sum(counts)
    if fused:
        x = rows(n, H * (G + 2), D, seed)
        return x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):]
    return rows(n, H * G, D, seed), rows(n, H, D, seed + 1), rows(n, H, D, seed + 2)


def _positions(start, counts):
    return torch.tensor([p + i for p, c in zip(start, counts) for i in range(c)], device="cuda")


CASES = [
    # counts per call, H, G, D, rot, interleaved, fused, page
    ([[5, 0, 3], [1, 1, 1], [0, 2, 0]], 2, 1, 128, 128, False, False, 0),
    ([[1, 1, 1, 1]] * 3, 3, 4, 64, 64, False, True, 0),
    ([[1, 1]] * 2, 5, 2, 128, 96, False, True, 4096),
    ([[300, 17, 1, 0]], 4, 2, 128, 32, True, True, 0),
    ([[700, 3]], 3, 3, 64, 48, False, False, 4096),
    ([[1200, 0, 2500], [1, 1, 1], [64, 1, 999]], 2, 1, 128, 128, False, True, 8192),
    ([[33], [2], [1]], 1, 8, 64, 16, True, False, 0),
    ([[40, 9], [1, 1]], 70, 1, 64, 64, True, True, 0),          # more heads than the append keeps on chip
    ([[20000]], 2, 1, 64, 64, False, False, 0),                 # scan chunks past the direct sums
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rotates_and_appends(case):
    calls, H, G, D, rot, inter, fused, page = CASES[case]
    B = len(calls[0])
    lens = [sum(c[s] for c in calls) for s in range(B)]
    cap = [max(1, L) for L in lens]
    pool = sum(H * (c * 4 * D // page + 2) for c in cap) if page else 0
    mk = lambda: kvq.KVQCache(B, H, D, cap, query_group=G, page_bytes=page, pool_pages=pool)  # noqa: E731
    cache, plain = mk(), mk()
    table = rope_table(max(lens), rot)
    start = [0] * B
    for i, counts in enumerate(calls):
        q, k, v = _inputs(counts, H, G, D, fused, 100 * case + 10 * i)
        bits = widths(sum(counts), H, 7 * case + i)
        pos = _positions(start, counts)
        got = kvq.kvq_write_rope(q, k, v, bits, cu_of(counts), cache, table, interleaved=inter)
        assert torch.equal(got.view(torch.int16), rotate(q, pos, table, inter).view(torch.int16))
        wide = rotate(q, pos, table, inter, wide=True)
        # two products and a sum in fp32, then half a step of fp16 (2^-25 where it is subnormal)
        tol = 4 * U32 * q.double().abs().amax(-1, keepdim=True) * 2 + U16 * wide.abs() + 2.0 ** -25
        assert bool(((got.double() - wide).abs() <= tol).all())
        kvq.kvq_write(rotate(k, pos, table, inter).contiguous(), v.contiguous(), bits, cu_of(counts), plain)
        start = [p + c for p, c in zip(start, counts)]
    cache.check()
    plain.check()
    assert cache.lengths().tolist() == lens
    _same_cache(cache, plain, H, lens)


@pytest.mark.parametrize("inter", [False, True])
def test_every_rounding_of_the_rotation(inter):
    """Many values, so that a product left unrounded would show (about one row value in 10^5)."""
    H, D, n = 16, 128, 4096
    cache = kvq.KVQCache(1, H, D, n)
    table = rope_table(n, D)
    q, k, v = _inputs([n], H, 1, D, False, 77)
    pos = torch.arange(n, device="cuda")
    got = kvq.kvq_write_rope(q, k, v, torch.full((n, H), 16, dtype=torch.uint8, device="cuda"), cu_of([n]), cache, table,
                             interleaved=inter)
    assert torch.equal(got, rotate(q, pos, table, inter))
    kd, vd = kvq.kvq_read(cache, cu_of([n]), n)
    assert torch.equal(kd, rotate(k, pos, table, inter)) and torch.equal(vd, v)


@pytest.mark.parametrize("n_new", [1, 50])
def test_positions_roll_back_first(n_new):
    B, H, D = 3, 2, 128
    cache, plain = (kvq.KVQCache(B, H, D, 200) for _ in range(2))
    table = rope_table(200, D)
    counts = [100, 60, 1]
    q, k, v = _inputs(counts, H, 1, D, False, 1)
    bits = widths(sum(counts), H, 2)
    for c in (cache, plain):
        kvq.kvq_write_rope(None, k, v, bits, cu_of(counts), c, table)
    back = torch.tensor([80, -1, 0], dtype=torch.int32, device="cuda")
    start, new = [80, 60, 0], [n_new] * B
    q2, k2, v2 = _inputs(new, H, 1, D, True, 5)
    b2 = widths(sum(new), H, 6)
    pos = _positions(start, new)
    for _ in range(2):                       # decoded again after a roll-back: the same cache and queries
        back2 = torch.tensor(start, dtype=torch.int32, device="cuda")
        got = kvq.kvq_write_rope(q2, k2, v2, b2, cu_of(new), cache, table, positions=back)
        back = back2
        assert torch.equal(got, rotate(q2, pos, table, False))
    plain.truncate(torch.tensor(start, dtype=torch.int32, device="cuda"))
    kvq.kvq_write(rotate(k2, pos, table, False), v2.contiguous(), b2, cu_of(new), plain)
    cache.check()
    lens = [p + n for p, n in zip(start, new)]
    assert cache.lengths().tolist() == lens
    _same_cache(cache, plain, H, lens)


@pytest.mark.parametrize("n_new", [1, 40])
def test_refused_sequences_keep_rows_and_cache(n_new):
    # sequence 0 would pass the table's last position, sequence 1 has a bad width, 2 its capacity
    B, H, G, D = 4, 2, 2, 64
    cache = kvq.KVQCache(B, H, D, [200, 200, 30 + n_new - 1, 200], query_group=G)
    table = rope_table(100 + n_new - 1, D)
    counts = [100, 10, 30, 20]
    q, k, v = _inputs(counts, H, G, D, False, 3)
    kvq.kvq_write_rope(q, k, v, widths(sum(counts), H, 4), cu_of(counts), cache, rope_table(200, D))
    cache.check()
    new = [n_new] * B
    q, k, v = _inputs(new, H, G, D, False, 9)
    bits = widths(B * n_new, H, 5)
    bits[2 * n_new - 1, 1] = 3
    out = torch.full((B * n_new, H * G, D), 7.0, dtype=torch.float16, device="cuda")
    kvq.kvq_write_rope(q, k, v, bits, cu_of(new), cache, table, q_out=out)
    with pytest.raises(kvq.KVQError) as e:
        cache.check()
    assert e.value.code in (kvq.KVQ_ERR_BITS, kvq.KVQ_ERR_CAPACITY)
    assert cache.lengths().tolist() == [100, 10, 30, 20 + n_new]
    assert bool((out[:3 * n_new] == 7.0).all())
    assert torch.equal(out[3 * n_new:], rotate(q[3 * n_new:], _positions([20], [n_new]), table, False))


@pytest.mark.parametrize("n_new", [1, 40])
def test_queries_in_place_and_rows_past_the_last_sequence(n_new):
    B, H, D = 2, 3, 128
    cache = kvq.KVQCache(B, H, D, 100)
    table = rope_table(100, 64)
    n = B * n_new
    q, k, v = _inputs([n + (2 if n_new > 1 else 0)], H, 1, D, False, 11)
    want = rotate(q[:n], _positions([0, 0], [n_new] * B), table, True)
    tail = q[n:].clone()
    same = kvq.kvq_write_rope(q, k, v, widths(q.shape[0], H, 1), cu_of([n_new] * B), cache, table, interleaved=True, q_out=q)
    cache.check()
    assert same is q and torch.equal(q[:n], want) and torch.equal(q[n:], tail)


def test_short_write_replays_in_a_graph_and_a_long_one_is_refused():
    B, H, G, D = 4, 2, 2, 128
    cache, plain = (kvq.KVQCache(B, H, D, 64, query_group=G) for _ in range(2))
    table = rope_table(64, D)
    one = cu_of([1] * B)
    q, k, v = _inputs([B], H, G, D, False, 1)
    bits = widths(B, H, 1)
    pos = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    kvq.kvq_write_rope(q, k, v, bits, one, cache, table)         # warm-up
    kvq.kvq_write_rope(None, k, v, bits, one, plain, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kvq.kvq_write_rope(q, k, v, bits, one, cache, table, positions=pos)
    for step in range(1, 6):
        for t, seed in ((q, 1), (k, 2), (v, 3)):
            t.copy_(rows(t.shape[0], t.shape[1], D, 50 * step + seed))
        bits.copy_(widths(B, H, 90 + step))
        if step == 3:
            bits[1, 0] = 5                                       # refused in this replay only
        graph.replay()
        start = [step if s != 1 or step <= 3 else step - 1 for s in range(B)]
        ok = [s for s in range(B) if step != 3 or s != 1]
        want = rotate(q, torch.tensor(start, device="cuda"), table, False)
        assert torch.equal(out[ok], want[ok])
        if step == 3:
            with pytest.raises(kvq.KVQError):
                cache.check()
        cu = cu_of([1 if s in ok else 0 for s in range(B)])
        pp = torch.tensor(start, device="cuda")
        kvq.kvq_write(rotate(k, pp, table, False)[ok].contiguous(), v[ok].contiguous(), bits[ok].contiguous(), cu, plain)
    cache.check()
    lens = cache.lengths().tolist()
    assert lens == [6, 5, 6, 6] == plain.lengths().tolist()
    _same_cache(cache, plain, H, lens)
    x = rows(9, H, D, 5)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g2 = torch.cuda.CUDAGraph()
        cu9, b9 = cu_of([9, 0, 0, 0]), widths(9, H, 1)
        torch.cuda.synchronize()
        g2.capture_begin()
        try:
            with pytest.raises(kvq.KVQError) as e:
                kvq.kvq_write_rope(None, x, x, b9, cu9, cache, table)
        finally:
            g2.capture_end()
    assert e.value.code == kvq.KVQ_ERR_ARG
    assert cache.lengths().tolist() == lens


def test_another_stream():
    B, H, D = 2, 2, 64
    cache, plain = (kvq.KVQCache(B, H, D, 300) for _ in range(2))
    table = rope_table(300, D)
    q, k, v = _inputs([250, 3], H, 1, D, True, 2)
    bits = widths(253, H, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = kvq.kvq_write_rope(q, k, v, bits, cu_of([250, 3]), cache, table, stream=side)
    side.synchronize()
    want = kvq.kvq_write_rope(q, k, v, bits, cu_of([250, 3]), plain, table)
    assert torch.equal(out, want)
    _same_cache(cache, plain, H, [250, 3])


def test_refusals():
    cache = kvq.KVQCache(1, 2, 64, 10)
    x, b, cu, t = rows(1, 2, 64, 1), widths(1, 2, 1), cu_of([1]), rope_table(10, 64)
    bad = [
        dict(cos_sin=rope_table(10, 64)[:, :40].contiguous()), dict(cos_sin=rope_table(10, 128)),
        dict(cos_sin=t.half()), dict(cos_sin=t.cpu()), dict(bits=b.int()), dict(k=rows(1, 3, 64, 1)),
        dict(v=rows(2, 2, 64, 1)), dict(q=x.transpose(1, 2)), dict(k=x.float()), dict(q=rows(1, 4, 64, 1)[:, ::2]),
        dict(cu_seqlens=cu.long()), dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
        dict(q=None, q_out=x), dict(cos_sin=t[0]),
    ]
    for change in bad:
        args = dict(q=x, k=x, v=x, bits=b, cu_seqlens=cu, cache=cache, cos_sin=t) | change
        with pytest.raises((kvq.KVQError, TypeError, ValueError)):
            kvq.kvq_write_rope(**args)
    # row strides that are not multiples of 8 elements, and rows that are not 16-byte aligned
    flat = torch.zeros(4 * 140, dtype=torch.float16, device="cuda")
    odd = flat[:280].view(2, 140)[:, :128].view(2, 2, 64)
    with pytest.raises(kvq.KVQError):
        kvq.kvq_write_rope(None, odd, odd, widths(2, 2, 1), cu_of([2]), cache, t)
    off = flat[4:4 + 128].view(1, 2, 64)
    with pytest.raises(kvq.KVQError):
        kvq.kvq_write_rope(None, off, off, b, cu, cache, t)
    cache.check()
    assert cache.lengths().tolist() == [0]
