"""Results of a call given a stream belong to that stream: they are allocated while it is the current
one, so that the memory they get was last used on it, and are marked as used by the caller's
stream. Without a GPU: the library, the streams and the device are stand-ins."""
import contextlib
import types

import pytest
import torch
from torch.overrides import TorchFunctionMode

from mixed_precision_kv_write_b200 import kvq

HERE, SIDE = types.SimpleNamespace(cuda_stream=11), types.SimpleNamespace(cuda_stream=22)
MADE_BY = {torch.empty, torch.zeros, torch.Tensor.new_empty, torch.Tensor.new_zeros}


class _Watch(TorchFunctionMode):
    """Which stream was current at each allocation, and which streams each result is marked for."""

    def __init__(self):
        super().__init__()
        self.current, self.made, self.marked = HERE, [], []

    def __torch_function__(self, func, types_, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func in MADE_BY:
            self.made.append((out.data_ptr(), self.current))
        return out


class _Library:
    """Every call succeeds and notes the stream it was given (a call's last argument)."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            if name == "routed_attn_decode_blocks_scratch":
                return 4096
            self.streams.append(args[-1])
            return kvq.KVQ_OK
        return call


@pytest.fixture
def watch(monkeypatch):
    w, lib = _Watch(), _Library()

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream if stream is not None else w.current
        yield
        w.current = before

    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, stream: w.marked.append((t.data_ptr(), stream)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: w.current.cuda_stream, raising=False)
    monkeypatch.setattr(kvq, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(kvq, "load_library", lambda: lib)
    w.lib = lib
    return w


class _OnGpu(torch.Tensor):
    """route_argmax takes logits on a GPU alone."""
    device = types.SimpleNamespace(type="cuda", index=0)


B, H, G, D, BLOCK = 2, 2, 2, 64, 16


def _calls():
    cache = types.SimpleNamespace(device=torch.device("cpu"), batch=B, heads=H, head_dim=D, query_group=G, query_heads=H * G,
                                  capacity=[40] * B, handle=None, _h=None, _scratch={})
    q, kv = torch.zeros((B, H * G, D), dtype=torch.float16), torch.zeros((B, H, D), dtype=torch.float16)
    bits, cu = torch.full((B, H), 4, dtype=torch.uint8), torch.tensor([0, 1, 2], dtype=torch.int32)
    modes = torch.full((B, H * G), 2, dtype=torch.uint8)
    bounds = torch.zeros((B, H, 1, 2, D, 64), dtype=torch.float16)
    ids, table = torch.zeros((B, H, 3), dtype=torch.int32), torch.zeros((40, D))
    logits = torch.zeros((B, H, 3)).as_subclass(_OnGpu)
    return {
        "kvq_write_rope": lambda **s: kvq.kvq_write_rope(q, kv, kv, bits, cu, cache, table, **s),
        "kvq_read": lambda **s: kvq.kvq_read(cache, cu, 2, **s),
        "block_bounds": lambda **s: kvq.block_bounds(cache, BLOCK, **s),
        "select_blocks": lambda **s: kvq.select_blocks(q, cache, bounds, BLOCK, 3, modes, **s),
        "routed_attn_prefill": lambda **s: kvq.routed_attn_prefill(q, cache, modes, 4, cu, **s),
        "routed_attn_decode": lambda **s: kvq.routed_attn_decode(q, cache, modes, 4, **s),
        "routed_attn_decode_noalloc": lambda **s: kvq.routed_attn_decode_noalloc(q, cache, modes, 4, **s),
        "decode_step": lambda **s: kvq.decode_step(q, kv, kv, bits, cu, cache, modes, 4, **s),
        "lengths": lambda **s: kvq.KVQCache.lengths(cache, **s),
        "export": lambda **s: kvq.KVQCache.export(cache, 0, 0, 0, 1, **s),
        "route_argmax": lambda **s: kvq.route_argmax(logits, None, **s),
        "routed_attn_decode_blocks": lambda **s: kvq.routed_attn_decode_blocks(q, cache, ids, BLOCK, modes, 4, **s),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_results_belong_to_the_stream_of_the_call(name, watch):
    call = _calls()[name]
    with watch:
        results = call(stream=SIDE)
    results = [r for r in (results if isinstance(results, tuple) else (results,)) if r is not None]
    assert watch.lib.streams == [SIDE.cuda_stream]
    assert watch.made and all(stream is SIDE for _, stream in watch.made)
    for r in results:
        assert (r.data_ptr(), HERE) in watch.marked           # the caller goes on with it on this stream


@pytest.mark.parametrize("name", sorted(_calls()))
def test_results_without_a_stream(name, watch):
    call = _calls()[name]
    with watch:
        call()
    assert watch.lib.streams == [HERE.cuda_stream]
    assert watch.made and all(stream is HERE for _, stream in watch.made) and not watch.marked
