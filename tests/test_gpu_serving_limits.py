"""Row counts at the end of 32 bits: n_max is an upper bound, the sequences' counts are on the device."""
import ctypes

import pytest
import torch

import test_gpu_serving as base
import test_gpu_serving_loop as loop
from test_gpu_serving import DEV, bits, gen, randn

pytestmark = pytest.mark.gpu

ST3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


@pytest.mark.parametrize("n_max", [2**31 - 1, 2**31 - 33, 2**30 + 1, 2**24])
@pytest.mark.parametrize("d,kind", [(128, 0), (64, 0), (256, 0), (128, 1)])
def test_read_of_few_rows_of_many(tq, d, kind, n_max):
    B, H, cap, n = 1, 1, 64, 40
    g = gen(d)
    seg = base.random_segment(tq, g, B, H, d, cap, 3, 4) if kind == 0 else tq.Fp16Segment(
        B, H, d, cap, k=randn(g, B, H, cap, d, dtype=torch.float16), v=randn(g, B, H, cap, d, dtype=torch.float16))
    rot = tq.tq_make_rotation(d, 5)
    first, count = (torch.tensor([x], dtype=torch.int32, device=DEV) for x in (-2, n))
    out = torch.full((B, H, n + 9, d), 7.0, dtype=torch.float16, device=DEV)
    st = tq._lib.tq_read(seg.reference(), ctypes.byref(rot), n_max, first.data_ptr(), count.data_ptr(), tq.TQ_DTYPE_F16,
                         out.data_ptr(), ST3(d, d, d), None, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    want = tq.tq_read(seg, rot, first + 2, n - 2, out=[torch.empty(B, H, n - 2, d, dtype=torch.float16, device=DEV), None])[0]
    assert torch.equal(bits(out[:, :, 2:n].contiguous()), bits(want))
    assert (out[:, :, :2] == 7).all() and (out[:, :, n:] == 7).all()


@pytest.mark.parametrize("n_max", [2**31 - 1, 2**31 - 33, 2**24])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("d,kind", [(128, 0), (64, 0), (128, 1)])
def test_append_of_few_rows_of_many(tq, d, kind, gather, n_max):
    B, H, cap, n, S = 1, 1, 64, 40, 50
    g = gen(d)
    K, V = (randn(g, B, H, S, d, dtype=torch.float16) for _ in range(2))
    rot = tq.tq_make_rotation(d, 5)
    make = (lambda: base.filled_segment(tq, B, H, d, cap, 3, 4)) if kind == 0 else (lambda: tq.Fp16Segment(B, H, d, cap))
    seg, want = make(), make()
    first, count = (torch.tensor([x], dtype=torch.int32, device=DEV) for x in (11, n))
    index = torch.randint(0, S, (1, n), generator=g, device=DEV, dtype=torch.int32) if gather else None
    st = tq._lib.tq_append(seg.reference(), ctypes.byref(rot), None, None, 0, K.data_ptr(), ST3(S * d, S * d, d), V.data_ptr(),
                           ST3(S * d, S * d, d), S, n_max, first.data_ptr(), count.data_ptr(),
                           index.data_ptr() if gather else None, n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    tq.tq_append(want, rot, K, V, first, n_new=count, index=index)
    torch.cuda.synchronize()
    for name in (base.BUFS if kind == 0 else ("k", "v")):
        assert torch.equal(getattr(seg, name).view(torch.uint8), getattr(want, name).view(torch.uint8)), name


# ------------------------------------------------------------------ many rows of many widths
@pytest.mark.parametrize("B,S,n,gather,layout,r", [(1, 4100, 4100, False, 0, 128), (3, 1500, 1400, True, 1, 64)])
def test_append_of_many_rows_of_every_width(tq, B, S, n, gather, layout, r):
    loop.test_large_append_is_compress(tq, 8, loop.MIXED, loop.MIXED[::-1], B, S, n, gather, layout, r, 0, 0)


@pytest.mark.parametrize("d,B,n", [(128, 1, 4200), (64, 2, 4200)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_read_of_many_rows_of_every_width(tq, d, B, n, dtype):
    loop.test_large_read_is_dequantize(tq, dtype, d, B, n, 0, False, 0, True)
