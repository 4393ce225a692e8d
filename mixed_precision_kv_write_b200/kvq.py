"""Thin ctypes binding of libkvq.so (C ABI in include/kvq.h).

Argument marshalling only: every step of the write and attention paths runs in the CUDA
library. Tensors must be CUDA tensors on the cache's device; the current torch stream is
passed to every call unless `stream` is given. With `stream`, tensors that the call makes are
that stream's memory; the order of the two streams (inputs before the call, results after
it) is the caller's. There is no CPU fallback: if the library is missing or a tensor is on the
CPU, the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

KVQ_OK, KVQ_ERR_ARG, KVQ_ERR_BITS, KVQ_ERR_MODE, KVQ_ERR_CAPACITY, KVQ_ERR_CUDA, \
    KVQ_ERR_DEVICE_CHECK, KVQ_ERR_NOMEM = range(8)
MODE_SKIP, MODE_LOCAL, MODE_FULL = 0, 1, 2
BLOCK_TILE = 64                  # blocks per tile of the bounds layout
_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

# every symbol include/kvq.h declares
EXPORTS = ("kvq_cache_create", "kvq_cache_create_gqa", "kvq_cache_create_paged", "kvq_cache_destroy", "kvq_cache_reset", "kvq_cache_truncate",
           "kvq_cache_lengths", "kvq_write", "routed_attn_prefill", "routed_attn_decode",
           "routed_attn_decode_noalloc", "kvq_decode_step", "kvq_cache_export", "kvq_check", "kvq_set_profile_events",
           "kvq_write_rope", "kvq_read", "kvq_block_bounds", "kvq_select_blocks", "routed_attn_decode_blocks",
           "routed_attn_decode_blocks_scratch",
           "kvq_route_argmax", "kvq_test_fail_alloc", "kvq_test_bounded_wait", "kvq_last_error")

_lib = None
_HERE = contextlib.nullcontext()


class KVQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvq status {code}: {msg}")
        self.code = code


def load_library(path: str = LIB_PATH):
    """Load libkvq.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m mixed_precision_kv_write_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    sig = {
        "kvq_cache_create": ([ctypes.POINTER(vp), i32, i32, i32, vp, vp], i32),
        "kvq_cache_create_gqa": ([ctypes.POINTER(vp), i32, i32, i32, i32, vp, vp], i32),
        "kvq_cache_create_paged": ([ctypes.POINTER(vp), i32, i32, i32, i32, vp, i64, i64, vp], i32),
        "kvq_cache_destroy": ([vp], i32),
        "kvq_cache_reset": ([vp, vp], i32),
        "kvq_cache_truncate": ([vp, vp, vp], i32),
        "kvq_cache_lengths": ([vp, vp, vp], i32),
        "kvq_write": ([vp, vp, vp, vp, i64, vp, vp], i32),
        "routed_attn_prefill": ([vp, vp, vp, i32, vp, i64, vp, vp], i32),
        "routed_attn_decode": ([vp, vp, vp, i32, vp, vp], i32),
        "routed_attn_decode_noalloc": ([vp, vp, vp, i32, vp, vp], i32),
        "kvq_decode_step": ([vp, vp, vp, vp, vp, i64, vp, vp, i32, vp, vp, vp], i32),
        "kvq_cache_export": ([vp, i32, i32, i64, i64, vp, vp, vp, vp, vp], i32),
        "kvq_check": ([vp, vp], i32),
        "kvq_set_profile_events": ([vp, vp], i32),
        "kvq_route_argmax": ([vp, vp, i64, vp, vp, vp], i32),
        "kvq_write_rope": ([vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, i32, vp, vp, vp, vp], i32),
        "kvq_read": ([vp, vp, i64, i32, vp, vp, vp], i32),
        "kvq_block_bounds": ([vp, i32, vp, vp, vp], i32),
        "kvq_select_blocks": ([vp, vp, vp, i32, vp, i32, i32, i32, vp, vp, vp], i32),
        "routed_attn_decode_blocks_scratch": ([vp, i32, i32, i32], i64),
        "routed_attn_decode_blocks": ([vp, vp, vp, i32, i32, vp, i32, vp, i64, vp, vp], i32),
        "kvq_test_fail_alloc": ([i32], i32),
        "kvq_test_bounded_wait": ([vp, i64, vp], i32),
        "kvq_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _raise(code: int):
    if code != KVQ_OK:
        raise KVQError(code, load_library().kvq_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    # the handle alone: building a torch.cuda.Stream takes as long as a short kernel
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _on(device):
    """The cache's device as the current one, for the call."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _result(stream, like, shape, dtype):
    """A tensor of the call's own, next to the tensor `like` or on that device. When the call runs on
    another stream, the memory is taken while that one is current: what it held before was last
    used there, so the call does not overwrite a tensor that work pending on the caller's stream
    still reads. The caller goes on with it on the current stream, so it is not handed out again
    before that has passed."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype) if isinstance(like, torch.Tensor) else \
            torch.empty(shape, dtype=dtype, device=like)
    with torch.cuda.stream(stream):
        t = _result(None, like, shape, dtype)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _check(t, name, dtype, device, shape=None):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous() and \
            (shape is None or t.shape == shape):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.device.index != device.index:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


class KVQCache:
    """Owning handle of a routed mixed-precision KV cache (kvq_cache_create/destroy)."""

    def __init__(self, batch: int, heads: int, head_dim: int, capacity, device=None, stream=None,
                 query_group: int = 1, page_bytes: int = 0, pool_pages: int = 0):
        lib = load_library()
        dev = torch.device("cuda") if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"the cache lives on a CUDA device (got {dev})")
        self.device = dev if dev.index is not None else \
            torch.device("cuda", torch.cuda.current_device())
        cap = [int(capacity)] * batch if isinstance(capacity, int) else [int(x) for x in capacity]
        if len(cap) != batch:
            raise ValueError("capacity must be an int or have one entry per sequence")
        self.batch, self.heads, self.head_dim, self.capacity = batch, heads, head_dim, cap
        self.query_group = int(query_group)
        self.query_heads = heads * self.query_group      # heads of q / modes / out
        arr = (ctypes.c_int64 * batch)(*cap)
        h = ctypes.c_void_p()
        self.page_bytes, self.pool_pages = int(page_bytes), int(pool_pages)
        with torch.cuda.device(self.device):
            _raise(lib.kvq_cache_create_paged(ctypes.byref(h), batch, heads, self.query_group, head_dim,
                                              ctypes.cast(arr, ctypes.c_void_p), self.page_bytes,
                                              self.pool_pages, _stream(stream, self.device)))
        self._h = h
        self._scratch = {}               # bytes of routed_attn_decode_blocks by (k, block, w)

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            with torch.cuda.device(self.device):
                load_library().kvq_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self, stream=None):
        _raise(load_library().kvq_cache_reset(self._h, _stream(stream, self.device)))

    def truncate(self, lengths: torch.Tensor, stream=None):
        _check(lengths, "lengths", torch.int32, self.device, (self.batch,))
        _raise(load_library().kvq_cache_truncate(self._h, _ptr(lengths), _stream(stream, self.device)))

    def lengths(self, stream=None) -> torch.Tensor:
        out = _result(stream, self.device, (self.batch,), torch.int32)
        _raise(load_library().kvq_cache_lengths(self._h, _ptr(out), _stream(stream, self.device)))
        return out

    def check(self, stream=None):
        """Synchronize and raise KVQError if a device-side check failed."""
        _raise(load_library().kvq_check(self._h, _stream(stream, self.device)))

    def export(self, seq: int, head: int, first: int, count: int, stream=None):
        """(k_codes uint16 [count, D], v_codes, side fp32 [count, 4], bits uint8 [count])."""
        D = self.head_dim
        kc = _result(stream, self.device, (count, D), torch.int16)
        vc = _result(stream, self.device, (count, D), torch.int16)
        sd = _result(stream, self.device, (count, 4), torch.float32)
        bt = _result(stream, self.device, (count,), torch.uint8)
        _raise(load_library().kvq_cache_export(self._h, seq, head, first, count, _ptr(kc), _ptr(vc),
                                               _ptr(sd), _ptr(bt), _stream(stream, self.device)))
        return kc, vc, sd, bt


def kvq_set_profile_events(before=None, after=None):
    """Record torch.cuda.Event pairs around the main kernel of the following calls."""
    for e in (before, after):
        if e is not None and e.cuda_event == 0:
            e.record()          # torch creates the CUDA event on first record
    b = None if before is None else ctypes.c_void_p(before.cuda_event)
    a = None if after is None else ctypes.c_void_p(after.cuda_event)
    _raise(load_library().kvq_set_profile_events(b, a))


def kvq_write(k, v, bits, cu_seqlens, cache: KVQCache, stream=None):
    """Quantize-on-write of k, v [n_tok, H, D] fp16 at widths bits [n_tok, H] (Eq. 4)."""
    dev = cache.device
    n = k.shape[0]
    _check(k, "k", torch.float16, dev, (n, cache.heads, cache.head_dim))
    _check(v, "v", torch.float16, dev, (n, cache.heads, cache.head_dim))
    _check(bits, "bits", torch.uint8, dev, (n, cache.heads))
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
    _raise(load_library().kvq_write(_ptr(k), _ptr(v), _ptr(bits), _ptr(cu_seqlens), n, cache.handle,
                                    _stream(stream, dev)))


def routed_attn_prefill(q, cache: KVQCache, modes, w: int, cu_seqlens, out=None, stream=None):
    """Routed causal attention (Eq. 2) of q [n_tok, H, D] over the cache; returns fp32 out."""
    dev = cache.device
    n = q.shape[0]
    _check(q, "q", torch.float16, dev, (n, cache.query_heads, cache.head_dim))
    _check(modes, "modes", torch.uint8, dev, (n, cache.query_heads))
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
    if out is None:
        out = _result(stream, q, (n, cache.query_heads, cache.head_dim), torch.float32)
    _check(out, "out", torch.float32, dev, (n, cache.query_heads, cache.head_dim))
    _raise(load_library().routed_attn_prefill(_ptr(q), cache.handle, _ptr(modes), int(w),
                                              _ptr(cu_seqlens), n, _ptr(out), _stream(stream, dev)))
    return out


def routed_attn_decode(q, cache: KVQCache, modes, w: int, out=None, stream=None):
    """Routed decode attention (Eq. 2), q [B, H, D] at t = len - 1; returns fp32 out."""
    dev = cache.device
    shape = (cache.batch, cache.query_heads, cache.head_dim)
    _check(q, "q", torch.float16, dev, shape)
    _check(modes, "modes", torch.uint8, dev, shape[:2])
    if out is None:
        out = _result(stream, q, shape, torch.float32)
    _check(out, "out", torch.float32, dev, shape)
    _raise(load_library().routed_attn_decode(_ptr(q), cache.handle, _ptr(modes), int(w), _ptr(out),
                                             _stream(stream, dev)))
    return out


def decode_step(q, k, v, bits, cu_seqlens, cache: KVQCache, modes, w: int, positions=None, out=None,
                stream=None):
    """One decode step (kvq_decode_step): append k, v [n_tok, H, D] at widths bits (Eq. 4),
    optionally after rolling each sequence back to `positions` [B] (int32), then routed
    decode attention (Eq. 2) of q [B, HQ, D]; returns fp32 out [B, HQ, D]."""
    dev = cache.device
    n = k.shape[0]
    shape = (cache.batch, cache.query_heads, cache.head_dim)
    _check(q, "q", torch.float16, dev, shape)
    _check(modes, "modes", torch.uint8, dev, shape[:2])
    _check(k, "k", torch.float16, dev, (n, cache.heads, cache.head_dim))
    _check(v, "v", torch.float16, dev, (n, cache.heads, cache.head_dim))
    _check(bits, "bits", torch.uint8, dev, (n, cache.heads))
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
    if positions is not None:
        _check(positions, "positions", torch.int32, dev, (cache.batch,))
    if out is None:
        out = _result(stream, q, shape, torch.float32)
    _check(out, "out", torch.float32, dev, shape)
    _raise(load_library().kvq_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(bits), _ptr(cu_seqlens), n,
                                          _ptr(positions), _ptr(modes), int(w), cache.handle, _ptr(out),
                                          _stream(stream, dev)))
    return out


def routed_attn_decode_noalloc(q, cache: KVQCache, modes, w: int, out=None, stream=None):
    """routed_attn_decode without any device allocation in the call: its scratch is the
    library's static device array (see include/kvq.h). Pass a preallocated `out` to keep
    the whole call allocation-free; the first call on a device should precede any stream
    capture, and calls that overlap on the GPU race on the shared scratch."""
    dev = cache.device
    shape = (cache.batch, cache.query_heads, cache.head_dim)
    _check(q, "q", torch.float16, dev, shape)
    _check(modes, "modes", torch.uint8, dev, shape[:2])
    if out is None:
        out = _result(stream, q, shape, torch.float32)
    _check(out, "out", torch.float32, dev, shape)
    _raise(load_library().routed_attn_decode_noalloc(_ptr(q), cache.handle, _ptr(modes), int(w),
                                                     _ptr(out), _stream(stream, dev)))
    return out


def _rows(t, name, heads, head_dim, device, n=None):
    """Checks fp16 rows [n, heads, head_dim] whose heads are contiguous; returns the row stride."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.float16 and t.device == device:
        shape, st = t.shape, t.stride()
        if len(shape) == 3 and shape[1] == heads and shape[2] == head_dim and (n is None or shape[0] == n) and \
                st[2] == 1 and (st[1] == head_dim or heads == 1):
            return st[0] if shape[0] > 1 else heads * head_dim       # (the stride of a single row says nothing)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be {torch.float16} (got {t.dtype})")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != head_dim or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must have shape {(n, heads, head_dim)} (got {tuple(t.shape)})")
    raise ValueError(f"{name}: the heads of a row must be contiguous (strides {t.stride()})")


def kvq_write_rope(q, k, v, bits, cu_seqlens, cache: KVQCache, cos_sin, interleaved: bool = False, positions=None,
                   q_out=None, stream=None):
    """Rotate q and k by position, append k and v at widths bits (kvq_write_rope); returns the
    rotated q [n_tok, HQ, D].

    q [n_tok, HQ, D], k, v [n_tok, H, D]: fp16, row strides free (heads of a row contiguous),
    q may be None. cos_sin: fp32 [max_pos, rot_dim], row t the cosines of position t, then its
    sines; rot_dim is its width. positions: int32 [B], roll the sequences back first."""
    dev, H, D = cache.device, cache.heads, cache.head_dim
    n = k.shape[0]
    ks, vs = _rows(k, "k", H, D, dev), _rows(v, "v", H, D, dev, n)
    qs = 0
    if q is not None:
        qs = _rows(q, "q", cache.query_heads, D, dev, n)
        if q_out is None:
            q_out = _result(stream, k, (n, cache.query_heads, D), torch.float16)
        _check(q_out, "q_out", torch.float16, dev, (n, cache.query_heads, D))
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(bits, "bits", torch.uint8, dev, (n, H))
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
    _check(cos_sin, "cos_sin", torch.float32, dev)
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin must be [max_pos, rot_dim] (got {tuple(cos_sin.shape)})")
    if positions is not None:
        _check(positions, "positions", torch.int32, dev, (cache.batch,))
    with _on(dev):
        _raise(load_library().kvq_write_rope(_ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(bits), _ptr(cu_seqlens), n,
                                             _ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1], int(interleaved),
                                             _ptr(positions), cache.handle, _ptr(q_out), _stream(stream, dev)))
    return q_out


def kvq_read(cache: KVQCache, cu_seqlens, n_rows: int, dtype=torch.float16, k_out=None, v_out=None, stream=None):
    """The last cu_seqlens[s+1] - cu_seqlens[s] tokens of each sequence as K and V rows
    [n_rows, H, D] of `dtype` (float16, bfloat16, float32); n_rows = cu_seqlens[-1]."""
    dev = cache.device
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be one of {tuple(_DTYPES)} (got {dtype})")
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
    shape = (int(n_rows), cache.heads, cache.head_dim)
    if k_out is None:
        k_out = _result(stream, cu_seqlens, shape, dtype)
    if v_out is None:
        v_out = _result(stream, cu_seqlens, shape, dtype)
    _check(k_out, "k_out", dtype, dev, shape)
    _check(v_out, "v_out", dtype, dev, shape)
    with _on(dev):
        _raise(load_library().kvq_read(cache.handle, _ptr(cu_seqlens), shape[0], _DTYPES[dtype], _ptr(k_out),
                                       _ptr(v_out), _stream(stream, dev)))
    return k_out, v_out


def block_tiles(cache: KVQCache, block: int) -> int:
    """Tiles of 64 blocks per (sequence, head) in the bounds of `block`-key blocks."""
    if block not in (16, 32, 64, 128):
        raise ValueError(f"block must be 16, 32, 64 or 128 (got {block})")
    return -(-(-(-max(cache.capacity) // block)) // BLOCK_TILE)


def block_bounds(cache: KVQCache, block: int, cu_seqlens=None, out=None, stream=None):
    """Per block of `block` keys, each channel's minimum and maximum of the dequantized keys
    (kvq_block_bounds): fp16 [B, H, nt, 2, D, 64]. With cu_seqlens, only the blocks that hold the
    newest tokens it counts are renewed in `out`; without it, every block."""
    dev = cache.device
    shape = (cache.batch, cache.heads, block_tiles(cache, block), 2, cache.head_dim, BLOCK_TILE)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.batch + 1,))
        if out is None:
            raise ValueError("cu_seqlens renews blocks of an `out` that holds the others")
    if out is None:
        with torch.cuda.stream(stream):                  # (zeroed on the stream that writes it)
            out = torch.zeros(shape, dtype=torch.float16, device=dev)
        if stream is not None:                           # (and the caller goes on with it on the current one)
            out.record_stream(torch.cuda.current_stream(dev))
    _check(out, "out", torch.float16, dev, shape)
    with _on(dev):
        _raise(load_library().kvq_block_bounds(cache.handle, block, _ptr(cu_seqlens), _ptr(out), _stream(stream, dev)))
    return out


def select_blocks(q, cache: KVQCache, bounds, block: int, k: int, modes=None, first: int = 1, last: int = 1, scores=None,
                  ids=None, stream=None):
    """Choose k blocks per (sequence, KV head) for the full queries of q [B, HQ, D]
    (kvq_select_blocks); returns (ids int32 [B, H, k] ascending then -1, scores fp32
    [B, H, nt * 64])."""
    dev, B, H = cache.device, cache.batch, cache.heads
    nt = block_tiles(cache, block)
    _check(q, "q", torch.float16, dev, (B, cache.query_heads, cache.head_dim))
    _check(bounds, "bounds", torch.float16, dev, (B, H, nt, 2, cache.head_dim, BLOCK_TILE))
    if modes is not None:
        _check(modes, "modes", torch.uint8, dev, (B, cache.query_heads))
    if scores is None:
        scores = _result(stream, q, (B, H, nt * BLOCK_TILE), torch.float32)
    if ids is None:
        ids = _result(stream, q, (B, H, k), torch.int32)
    _check(scores, "scores", torch.float32, dev, (B, H, nt * BLOCK_TILE))
    _check(ids, "ids", torch.int32, dev, (B, H, k))
    with _on(dev):
        _raise(load_library().kvq_select_blocks(_ptr(q), cache.handle, _ptr(bounds), block, _ptr(modes), int(k),
                                                int(first), int(last), _ptr(scores), _ptr(ids), _stream(stream, dev)))
    return ids, scores


def routed_attn_decode_blocks(q, cache: KVQCache, ids, block: int, modes, w: int, out=None, stream=None):
    """Routed decode attention (Eq. 2) whose full queries read the blocks of ids [B, H, k]
    (as select_blocks returns them); q [B, HQ, D] at t = len - 1; returns fp32 out."""
    dev = cache.device
    shape = (cache.batch, cache.query_heads, cache.head_dim)
    _check(q, "q", torch.float16, dev, shape)
    _check(modes, "modes", torch.uint8, dev, shape[:2])
    _check(ids, "ids", torch.int32, dev)
    if ids.dim() != 3 or ids.shape[:2] != (cache.batch, cache.heads):
        raise ValueError(f"ids must be [{cache.batch}, {cache.heads}, k] (got {tuple(ids.shape)})")
    if out is None:
        out = _result(stream, q, shape, torch.float32)
    _check(out, "out", torch.float32, dev, shape)
    k, w, lib = ids.shape[2], int(w), load_library()
    with _on(dev):
        need = cache._scratch.get((k, block, w))
        if need is None:
            need = cache._scratch[k, block, w] = lib.routed_attn_decode_blocks_scratch(cache.handle, k, block, w)
        scratch = None
        if need > 0:                 # this call's own: allocated for the stream that runs it
            with torch.cuda.stream(stream):
                scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        _raise(lib.routed_attn_decode_blocks(_ptr(q), cache.handle, _ptr(ids), k, block, _ptr(modes), w,
                                             _ptr(scratch), max(need, 0), _ptr(out), _stream(stream, dev)))
    return out


def route_argmax(z_attn=None, z_bits=None, stream=None):
    """Router hard argmax (Eq. 5 heads): modes uint8 [...] from z_attn fp32 [..., 3] and
    bits uint8 [...] in {2, 4, 8, 16} from z_bits fp32 [..., 4]; either may be None."""
    ref = z_attn if z_attn is not None else z_bits
    if ref is None:
        raise ValueError("route_argmax: pass z_attn, z_bits or both")
    dev = ref.device
    if dev.type != "cuda":
        raise ValueError(f"route_argmax: logits must be on a CUDA device (got {dev})")
    outs, n = [], None
    for z, k in ((z_attn, 3), (z_bits, 4)):
        if z is None:
            outs.append(None)
            continue
        if z.dtype != torch.float32 or not z.is_contiguous() or z.shape[-1] != k or z.device != dev:
            raise ValueError(f"route_argmax: expected contiguous fp32 [..., {k}] on {dev}")
        rows = z.numel() // k
        if n is not None and rows != n:
            raise ValueError("route_argmax: z_attn and z_bits have different row counts")
        n = rows
        outs.append(_result(stream, z, z.shape[:-1], torch.uint8))
    _raise(load_library().kvq_route_argmax(_ptr(z_attn) if z_attn is not None else None,
                                           _ptr(z_bits) if z_bits is not None else None, n,
                                           _ptr(outs[0]) if outs[0] is not None else None,
                                           _ptr(outs[1]) if outs[1] is not None else None,
                                           _stream(stream, dev)))
    return outs[0], outs[1]
