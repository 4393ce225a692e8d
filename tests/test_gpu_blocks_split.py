"""Attention over chosen blocks by many CTAs a KV head: partial states in the caller's scratch and a
second launch (more than 16 of them), clusters (2 to 16), both captured into graphs and on
streams of their own."""
import pytest
import torch

from blocks_testlib import Filled, assert_attention, attention64, choose, rows, scores64
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu


def _ids(lens, H, block, k, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.full((len(lens), H, k), -1, dtype=torch.int32)
    for s, L in enumerate(lens):
        nb = -(-L // block)
        for h in range(H):
            n = max(min(1, nb), min(k, nb) - h)
            ids[s, h, :n] = torch.randperm(nb, generator=g)[:n].sort().values.to(torch.int32)
    return ids.cuda()


def _modes(B, HQ, seed):
    m = torch.randint(0, 3, (B, HQ), generator=torch.Generator().manual_seed(seed)).to(torch.uint8)
    m[:, -1] = 2
    return m.cuda()


def _scratch(f, k, block, w):
    return kvq.load_library().routed_attn_decode_blocks_scratch(f.cache.handle, k, block, w)


SCRATCH = [
    # lens, H, G, D, block, k, w, page
    ([20000], 1, 3, 64, 128, 140, 300, 0),
    ([20000, 17], 1, 5, 128, 128, 140, 9000, 4096),
    ([18000], 1, 20, 64, 64, 280, 100, 65536),
    ([18000], 2, 20, 128, 128, 141, 12000, 0),
    ([20000, 9000], 2, 4, 128, 64, 300, 5000, 4096),
    ([30000], 1, 8, 64, 16, 1200, 0, 0),
    ([20000, 1, 0], 3, 2, 64, 128, 150, 20000, 0),
]


@pytest.mark.parametrize("case", range(len(SCRATCH)))
def test_partial_states_of_shared_heads(case):
    lens, H, G, D, block, k, w, page = SCRATCH[case]
    f = Filled(lens, H, D, G=G, page=page, seed=case)
    assert _scratch(f, k, block, w) > 0
    ids, q = _ids(lens, H, block, k, case), rows(len(lens), H * G, D, 30 + case)
    for modes in (torch.full((len(lens), H * G), 2, dtype=torch.uint8, device="cuda"), _modes(len(lens), H * G, case)):
        got = kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w)
        f.cache.check()
        ref, tol = attention64(f, q, ids, block, modes, w)
        assert_attention(got, ref, tol, f"case {case}")
        assert torch.equal(kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w), got)


def test_the_most_blocks_of_a_very_long_context():
    L, block, k = 600000, 128, 4096
    f = Filled([L], 1, 64, seed=5)
    q = rows(1, 1, 64, 5)
    ids = _ids([L], 1, block, k, 3)
    modes = torch.full((1, 1), 2, dtype=torch.uint8, device="cuda")
    assert _scratch(f, k, block, 0) > 0
    got = kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, 0)
    f.cache.check()
    assert_attention(got, *attention64(f, q, ids, block, modes, 0))


CAPTURED = [
    # lens, H, G, D, block, k, w, page: clusters in both kernels; scratch; one CTA a unit
    ([9000, 4000], 2, 4, 128, 64, 60, 200, 0),
    ([20000], 1, 5, 64, 64, 280, 9000, 4096),
    ([700] * 80, 8, 1, 128, 32, 8, 100, 0),
]


@pytest.mark.parametrize("case", range(len(CAPTURED)))
def test_choice_and_attention_in_graphs(case):
    """Two graphs of one memory pool, replayed in turn with new inputs, against eager calls."""
    lens, H, G, D, block, k, w, page = CAPTURED[case]
    B, HQ = len(lens), H * G
    f = Filled(lens, H, D, G=G, page=page, seed=case)
    assert (_scratch(f, k, block, w) > 0) == (case == 1)
    bounds = kvq.block_bounds(f.cache, block)
    q, modes = rows(B, HQ, D, 1), _modes(B, HQ, 1)

    def step():
        ids, _ = kvq.select_blocks(q, f.cache, bounds, block, k, modes)
        return ids, kvq.routed_attn_decode_blocks(q, f.cache, ids, block, modes, w)

    step()
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs = step()
        graphs.append((graph, outs))
    for i in range(4):
        q.copy_(rows(B, HQ, D, 50 + i))
        modes.copy_(_modes(B, HQ, 60 + i))
        graph, (ids, out) = graphs[i % 2]
        graph.replay()
        ids, out = ids.clone(), out.clone()
        want_ids, want = step()
        f.cache.check()
        assert torch.equal(ids, want_ids) and torch.equal(out, want)
    assert torch.equal(ids.cpu(), choose(scores64(q, bounds, modes, lens, block, G).float(), lens, block, k, 1, 1))
    ref, tol = attention64(f, q, ids, block, modes, w)
    assert_attention(out, ref, tol)


def test_scratch_of_two_streams_and_of_one_behind_pending_work():
    lens, H, G, D, block, k, w, page = SCRATCH[1]
    f = Filled(lens, H, D, G=G, page=page, seed=1)
    ids, q = _ids(lens, H, block, k, 1), [rows(len(lens), H * G, D, i) for i in range(2)]
    modes = _modes(len(lens), H * G, 2)
    want = [kvq.routed_attn_decode_blocks(x, f.cache, ids, block, modes, w) for x in q]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(6):
        torch.cuda._sleep(2_000_000)
        got = [kvq.routed_attn_decode_blocks(q[i % 2], f.cache, ids, block, modes, w, stream=st[i % 2]) for i in range(6)]
        here = kvq.routed_attn_decode_blocks(q[0], f.cache, ids, block, modes, w)
        torch.cuda.synchronize()
        f.cache.check()
        assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got)) and torch.equal(here, want[0])
