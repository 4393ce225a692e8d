"""Calls of the rotating write and of block-sparse decoding at the edges of what their contracts
allow: sequences without new tokens, roll-backs, empty and refused writes."""
import pytest
import torch

from blocks_testlib import Filled, cu_of, flat_bounds, rope_table, rows, widths
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu


def _same_bounds(cache, bounds, block, lens):
    fresh = flat_bounds(kvq.block_bounds(cache, block))
    for s, L in enumerate(lens):
        nb = -(-L // block)
        assert torch.equal(flat_bounds(bounds)[s, ..., :nb], fresh[s, ..., :nb]), s


# ------------------------------------------------------------------ bounds
@pytest.mark.parametrize("block,page", [(16, 0), (64, 4096), (128, 0)])
@pytest.mark.parametrize("by", ["truncate", "positions"])
def test_bounds_of_a_sequence_rolled_back_without_new_tokens(block, page, by):
    lens, D = [400, 300, 131, 128, 5], 64
    f = Filled(lens, 2, D, page=page, seed=9, capacity=[500] * 5)
    f.k[20:40] *= 20                                           # (extremes that a cut may drop)
    table = rope_table(500, D)
    bounds = kvq.block_bounds(f.cache, block)
    for i, (back, new) in enumerate([([395, 300, 130, 3, 4], [0, 2, 0, 0, 0]), ([1, 256, 128, 0, -1], [0, 0, 0, 0, 1]),
                                     ([0, 255, 127, -1, 2], [0, 0, 0, 3, 0])]):
        pos, n = torch.tensor(back, dtype=torch.int32, device="cuda"), sum(new)
        k, v, bits = rows(n, 2, D, i), rows(n, 2, D, i + 5), widths(n, 2, i)
        if by == "truncate":
            f.cache.truncate(pos)
            kvq.kvq_write(k, v, bits, cu_of(new), f.cache)
        else:
            kvq.kvq_write_rope(None, k, v, bits, cu_of(new), f.cache, table, positions=pos)
        lens = [(min(L, b) if b >= 0 else L) + m for L, b, m in zip(lens, back, new)]
        kvq.block_bounds(f.cache, block, cu_of(new), out=bounds)
        f.cache.check()
        assert f.cache.lengths().tolist() == lens
        _same_bounds(f.cache, bounds, block, lens)


def test_bounds_after_a_refused_write():
    """A roll-back stands although the write behind it is refused: the bounds follow."""
    D, block = 64, 32
    f = Filled([100, 40], 2, D, seed=2, capacity=[120, 60])
    bounds = kvq.block_bounds(f.cache, block)
    n = 130
    pos = torch.tensor([50, 33], dtype=torch.int32, device="cuda")
    kvq.kvq_write_rope(None, rows(n, 2, D, 1), rows(n, 2, D, 2), widths(n, 2, 3), cu_of([90, 40]), f.cache, rope_table(500, D),
                       positions=pos)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_CAPACITY
    kvq.block_bounds(f.cache, block, cu_of([90, 40]), out=bounds)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK
    assert f.cache.lengths().tolist() == [50, 33]
    _same_bounds(f.cache, bounds, block, [50, 33])


# ------------------------------------------------------------------ rotating write
@pytest.mark.parametrize("n_new", [1, 30, 400])                # one launch; both forms of the scan
def test_a_sequence_without_new_tokens_may_be_longer_than_the_table(n_new):
    B, H, D = 3, 2, 64
    lens = [500, 20, 0]
    f = Filled(lens, H, D, seed=4, capacity=[600, 600, 600])
    counts = [0, n_new, 1]
    n = sum(counts)
    kvq.kvq_write_rope(None, rows(n, H, D, 1), rows(n, H, D, 2), widths(n, H, 3), cu_of(counts), f.cache,
                       rope_table(20 + n_new, D))
    f.cache.check()                                            # nothing was refused
    assert f.cache.lengths().tolist() == [500, 20 + n_new, 1]
    kvq.kvq_write_rope(None, rows(n, H, D, 1), rows(n, H, D, 2), widths(n, H, 3), cu_of(counts), f.cache,
                       rope_table(20 + n_new, D))              # sequence 1 would pass the table's end now
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_CAPACITY
    assert f.cache.lengths().tolist() == [500, 20 + n_new, 2]


def test_an_empty_write_is_captured():
    """No tokens: nothing without positions, the roll-back alone with them."""
    B, H, D = 2, 2, 64
    f = Filled([50, 40], H, D, seed=4)
    pos = torch.tensor([30, -1], dtype=torch.int32, device="cuda")
    none, x, bits, table = cu_of([0] * B), rows(0, H, D, 1), widths(0, H, 1), rope_table(50, D)
    q = rows(0, H, D, 2)
    kvq.kvq_write_rope(q, x, x, bits, none, f.cache, table, positions=torch.full((B,), -1, dtype=torch.int32, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_write_rope(None, x, x, bits, none, f.cache, table)
        out = kvq.kvq_write_rope(q, x, x, bits, none, f.cache, table, positions=pos)
    assert out.shape == (0, H, D) and f.cache.lengths().tolist() == [50, 40]
    graph.replay()
    f.cache.check()
    assert f.cache.lengths().tolist() == [30, 40]
    pos.copy_(torch.tensor([29, 7], dtype=torch.int32))
    graph.replay()
    f.cache.check()
    assert f.cache.lengths().tolist() == [29, 7]


@pytest.mark.parametrize("cu", [[0, 1, 2, 7], [0, 10, 20, 99], [0, 100, 200, 260], [0, 0, 0, 5]])
def test_inconsistent_ranges_are_not_rolled_back(cu):
    """Sequence 2's range ends behind the call's rows: it keeps its tokens, in every launch form."""
    n = {7: 3, 99: 40, 260: 250, 5: 0}[cu[-1]]
    B, H, D = 3, 2, 64
    f = Filled([50, 40, 30], H, D, seed=4, capacity=[400] * B)
    before = f.cache.export(2, 1, 0, 30)
    pos = torch.tensor([20, 5, 10], dtype=torch.int32, device="cuda")
    kvq.kvq_write_rope(None, rows(n, H, D, 1), rows(n, H, D, 2), widths(n, H, 3), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                       f.cache, rope_table(400, D), positions=pos)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK
    assert f.cache.lengths().tolist() == [20 + cu[1] - cu[0], 5 + cu[2] - cu[1], 30]
    assert all(torch.equal(a, b) for a, b in zip(f.cache.export(2, 1, 0, 30), before))


# ------------------------------------------------------------------ attention over chosen blocks
@pytest.mark.parametrize("G", [1, 4, 9, 20])
@pytest.mark.parametrize("entry", [2, 30])                     # within the sequence's number of blocks, and behind it
def test_bad_entries_are_reported_whichever_query_reads_them(G, entry):
    f = Filled([100], 1, 64, G=G, seed=4)
    ids = torch.full((1, 1, 40), -1, dtype=torch.int32, device="cuda")
    ids[..., 0], ids[..., entry] = 1, 50                       # 7 blocks
    q = rows(1, G, 64, 2)
    for g in {0, G // 2, G - 1}:
        modes = torch.zeros((1, G), dtype=torch.uint8, device="cuda")
        modes[0, g] = 2
        kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, modes, 0)
        with pytest.raises(kvq.KVQError) as e:
            f.cache.check()
        assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK
    kvq.routed_attn_decode_blocks(q, f.cache, ids, 16, torch.ones((1, G), dtype=torch.uint8, device="cuda"), 3)
    f.cache.check()                                            # no full query: the list is not read


@pytest.mark.parametrize("width", [521, 520])
def test_one_row_of_a_projection_of_any_width(width):
    """A single token's q, k and v as column ranges of one row: its stride does not matter."""
    H, G, D = 1, 2, 128
    f, plain = (Filled([3], H, D, G=G, seed=1, capacity=[9]) for _ in range(2))
    x = rows(1, 1, width, 2).flatten().as_strided((1, G + 2, D), (width, D, 1))
    q, k, v = x[:, :G], x[:, G:G + 1], x[:, G + 1:]
    assert x.stride(0) == width
    table, bits = rope_table(9, D), widths(1, H, 1)
    out = kvq.kvq_write_rope(q, k, v, bits, cu_of([1]), f.cache, table)
    want = kvq.kvq_write_rope(*(t.clone(memory_format=torch.contiguous_format) for t in (q, k, v)), bits, cu_of([1]),
                              plain.cache, table)
    f.cache.check()
    assert torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip(f.cache.export(0, 0, 0, 4), plain.cache.export(0, 0, 0, 4)))
