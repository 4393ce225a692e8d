"""Read-back of the newest tokens (kvq_read): fp32 rows bit for bit fl(fl(code * s) + z), fp16 and
bf16 rows their rounding, within rounding of the 64-bit values."""
import pytest
import torch

from blocks_testlib import U16, U32, UB16, Filled, cu_of, values32, values64
from mixed_precision_kv_write_b200 import kvq

pytestmark = pytest.mark.gpu
STEP = {torch.float32: U32, torch.float16: U16, torch.bfloat16: UB16}


def _tail_rows(f, tails):
    return torch.tensor([f.start[s] + f.lens[s] - t + i for s, t in enumerate(tails) for i in range(t)],
                        dtype=torch.long, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,tails,H,D,page", [
    ([1], [1], 1, 64, 0),
    ([5, 0, 130, 1], [5, 0, 130, 1], 3, 128, 0),
    ([700, 33, 64], [1, 33, 0], 2, 64, 4096),
    ([900, 2, 1500], [257, 2, 1499], 5, 128, 4096),
])
def test_rows(dtype, lens, tails, H, D, page):
    f = Filled(lens, H, D, page=page, seed=11)
    k, v = kvq.kvq_read(f.cache, cu_of(tails), sum(tails), dtype=dtype)
    f.cache.check()
    r = _tail_rows(f, tails)
    for got, x in ((k, f.k), (v, f.v)):
        want = values32(x[r], f.bits[r])
        assert torch.equal(got, want.to(dtype))
        wide = values64(x[r], f.bits[r])
        # product and sum in fp32 (magnitudes up to (2^b - 1) s + |z| <= 4 max|x|), then half a step of dtype
        tol = 12 * U32 * x[r].double().abs().amax(-1, keepdim=True) + STEP[dtype] * wide.abs() + 2.0 ** -25
        assert bool(((got.double() - wide).abs() <= tol).all())


def test_many_rows():
    f = Filled([20000, 1, 900], 8, 64, seed=6)                 # more pairs than start the larger CTAs
    k, v = kvq.kvq_read(f.cache, f.cu, 20901)
    f.cache.check()
    assert torch.equal(k, values32(f.k, f.bits).half()) and torch.equal(v, values32(f.v, f.bits).half())


def test_one_output_rows_behind_and_too_many_rows():
    f = Filled([40, 7], 2, 64, seed=3)
    k = torch.full((60, 2, 64), 9.0, device="cuda")
    v = torch.full((60, 2, 64), 9.0, device="cuda")
    kvq.kvq_read(f.cache, cu_of([10, 7]), 60, dtype=torch.float32, k_out=k, v_out=v)
    f.cache.check()
    assert bool((k[17:] == 9.0).all()) and bool((v[17:] == 9.0).all())
    r = _tail_rows(f, [10, 7])
    assert torch.equal(k[:17], values32(f.k[r], f.bits[r]))
    # sequence 1 holds 7 tokens: rows of tokens before its first are zeros, and reported
    k, v = kvq.kvq_read(f.cache, cu_of([1, 9]), 10, dtype=torch.float32)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK
    assert bool((k[1:3] == 0).all()) and torch.equal(v[3:], values32(f.v[40:], f.bits[40:]))
    lib, p = kvq.load_library(), lambda t: t.data_ptr()
    only = torch.full((17, 2, 64), 9.0, device="cuda")
    assert lib.kvq_read(f.cache.handle, p(cu_of([10, 7])), 17, 2, None, p(only), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(only, values32(f.v[r], f.bits[r]))


def test_broken_cu_seqlens_are_reported():
    f = Filled([40, 7, 9], 1, 64, seed=3)
    cu = torch.tensor([0, 12, 3, 20], dtype=torch.int32, device="cuda")
    kvq.kvq_read(f.cache, cu, 20)
    with pytest.raises(kvq.KVQError) as e:
        f.cache.check()
    assert e.value.code == kvq.KVQ_ERR_DEVICE_CHECK


def test_widths_one_at_a_time_and_outliers():
    for b in (2, 4, 8, 16):
        f = Filled([77], 2, 128, seed=b, widths_of=b)
        k, _ = kvq.kvq_read(f.cache, f.cu, 77, dtype=torch.float32)
        assert torch.equal(k, values32(f.k, f.bits))
    n = 16
    x = torch.zeros((n, 1, 64), dtype=torch.float16, device="cuda")
    x[::2, 0, 5], x[::4, 0, 9] = 65504.0, -65504.0
    cache = kvq.KVQCache(1, 1, 64, n)
    bits = torch.tensor([2, 4, 8, 16] * 4, dtype=torch.uint8, device="cuda")[:, None].contiguous()
    kvq.kvq_write(x, x, bits, cu_of([n]), cache)
    k, v = kvq.kvq_read(cache, cu_of([n]), n)
    assert torch.equal(k, values32(x, bits).half()) and torch.equal(v, k) and bool(k.isfinite().all())


def test_refusals():
    f = Filled([4], 1, 64)
    with pytest.raises(TypeError):
        kvq.kvq_read(f.cache, f.cu, 4, dtype=torch.float64)
    with pytest.raises(ValueError):
        kvq.kvq_read(f.cache, f.cu.cpu(), 4)
    with pytest.raises(ValueError):
        kvq.kvq_read(f.cache, f.cu, 4, k_out=torch.zeros((3, 1, 64), dtype=torch.float16, device="cuda"))
    lib, p = kvq.load_library(), f.cu.data_ptr()
    assert lib.kvq_read(f.cache.handle, p, 4, 0, None, None, None) == kvq.KVQ_ERR_ARG
    assert lib.kvq_read(f.cache.handle, p, -1, 0, None, None, None) == kvq.KVQ_ERR_ARG
    assert lib.kvq_read(f.cache.handle, p, 4, 7, p, None, None) == kvq.KVQ_ERR_ARG
    assert lib.kvq_read(f.cache.handle, p, 4, 0, p + 4, None, None) == kvq.KVQ_ERR_ARG
