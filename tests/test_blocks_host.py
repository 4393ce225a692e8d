"""Host-side refusals of the rotating write, the read-back and block-sparse decoding, without a
GPU: every call refuses a missing cache before it touches the device, and says so."""
import types

import pytest

from mixed_precision_kv_write_b200 import build, kvq


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load_library()


def test_calls_refuse_a_null_cache(lib):
    assert lib.kvq_write_rope(None, 0, None, 0, None, 0, None, None, 0, None, 0, 64, 0, None, None, None, None) == \
        kvq.KVQ_ERR_ARG
    assert b"kvq_write_rope" in lib.kvq_last_error()
    assert lib.kvq_read(None, None, 0, 0, None, None, None) == kvq.KVQ_ERR_ARG
    assert b"kvq_read" in lib.kvq_last_error()
    assert lib.kvq_block_bounds(None, 64, None, None, None) == kvq.KVQ_ERR_ARG
    assert lib.kvq_select_blocks(None, None, None, 64, None, 4, 1, 1, None, None, None) == kvq.KVQ_ERR_ARG
    assert lib.routed_attn_decode_blocks(None, None, None, 4, 64, None, 0, None, 0, None, None) == kvq.KVQ_ERR_ARG
    assert b"routed_attn_decode_blocks" in lib.kvq_last_error()
    assert lib.routed_attn_decode_blocks_scratch(None, 4, 64, 0) == -1


@pytest.mark.parametrize("capacity,block,tiles", [([1], 16, 1), ([1024, 7], 16, 1), ([1025], 16, 2), ([8192], 64, 2),
                                                  ([8193], 64, 3), ([8388607], 128, 1024)])
def test_tiles_of_the_bounds(capacity, block, tiles):
    assert kvq.block_tiles(types.SimpleNamespace(capacity=capacity), block) == tiles


@pytest.mark.parametrize("block", [0, 8, 48, 256, -16])
def test_other_blocks_are_refused(block):
    with pytest.raises(ValueError):
        kvq.block_tiles(types.SimpleNamespace(capacity=[100]), block)


@pytest.mark.parametrize("heads,stride,n,want", [(2, 128, 3, 128), (2, 400, 3, 400), (1, 72, 5, 72), (2, 404, 1, 128),
                                                 (2, 7, 1, 128), (2, 0, 1, 128), (1, 1, 0, 64), (3, 193, 0, 192)])
def test_row_strides(heads, stride, n, want):
    """The stride of several rows is theirs; that of one row or none, which nothing reads, the row's size."""
    import torch
    flat = torch.zeros(3000, dtype=torch.float16)
    x = flat.as_strided((n, heads, 64), (stride, 64, 1))
    assert kvq._rows(x, "k", heads, 64, flat.device) == want
