"""Calls on a stream of their own, while work on the caller's stream still reads a tensor that it has
already let go: the results must not take that tensor's memory."""
import pytest
import torch

from blocks_testlib import Filled, cu_of, rope_table, rows, widths
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu

B, H, G, D, BLOCK, K = 2, 2, 2, 128, 16, 9


def _calls():
    """name -> the call, on a cache of its own."""
    f = Filled([300, 200], H, D, G=G, seed=3, capacity=[400, 400])
    q, kv, bits = rows(B, H * G, D, 1), rows(B, H, D, 2), widths(B, H, 4)
    modes = torch.full((B, H * G), 2, dtype=torch.uint8, device="cuda")
    bounds, table, one, tail = kvq.block_bounds(f.cache, BLOCK), rope_table(400, D), cu_of([1, 1]), cu_of([200, 150])
    ids, _ = kvq.select_blocks(q, f.cache, bounds, BLOCK, K, modes)
    back = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    return f, {
        "kvq_write_rope": lambda **s: kvq.kvq_write_rope(q, kv, kv, bits, one, f.cache, table, positions=back, **s),
        "kvq_read": lambda **s: kvq.kvq_read(f.cache, tail, 350, torch.float32, **s),
        "block_bounds": lambda **s: kvq.block_bounds(f.cache, BLOCK, **s),
        "select_blocks": lambda **s: kvq.select_blocks(q, f.cache, bounds, BLOCK, K, modes, **s),
        "routed_attn_decode_blocks": lambda **s: kvq.routed_attn_decode_blocks(q, f.cache, ids, BLOCK, modes, 4, **s),
    }


@pytest.mark.parametrize("name", ["kvq_write_rope", "kvq_read", "block_bounds", "select_blocks", "routed_attn_decode_blocks"])
def test_pending_reads_of_a_freed_tensor(name):
    side = torch.cuda.Stream()
    f, calls = _calls()
    want = calls[name]()
    want = want if isinstance(want, tuple) else (want,)
    torch.cuda.synchronize()
    shapes = [(t.shape, t.dtype) for t in want]
    for _ in range(4):
        held = [torch.full(s, 5, dtype=t, device="cuda") for s, t in shapes]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)                       # about 20 ms: the copies below are pending meanwhile
        copies = [t.clone() for t in held]
        del held
        got = calls[name](stream=side)
        got = got if isinstance(got, tuple) else (got,)
        side.synchronize()
        torch.cuda.synchronize()
        f.cache.check()
        assert all(bool((c == 5).all()) for c in copies)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
