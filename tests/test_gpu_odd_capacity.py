"""Packed segments whose capacity is no multiple of 16: heads then begin off the boundaries that records of
their own width would have."""
import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import DEV, bits, gen, randn
from test_gpu_serving_loop import records, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def same(seg, want, n):
    """The first n rows of each head, whatever the capacities."""
    L = seg.layout
    for b in range(L.batch):
        for which in "kv":
            x, y = records(seg, which, b), records(want, which, b)
            for h in range(L.n_heads):
                assert torch.equal(x[h][:n], y[h][:n]), (which, b, h)
                assert torch.equal(bits(scales(seg, which, b)[h][:n]), bits(scales(want, which, b)[h][:n]))


# 16 dims: records of 2 b bytes, so that heads begin at 2 mod 4 behind an odd capacity of an odd width
# (or, behind an odd sum of widths, in every other sequence)
@pytest.mark.parametrize("widths", [([1, 2, 8, 3, 4], [3, 2, 5, 4, 8]), ([2, 1], [4, 3])])
@pytest.mark.parametrize("cap", [7, 9, 10, 13])
def test_16_dims(tq, cap, widths):
    d, B, H, n = 16, 3, len(widths[0]), 6
    g = gen(cap)
    K, V = (randn(g, B, H, n, d, dtype=torch.float16) for _ in range(2))
    rot = tq.tq_make_rotation(d, 3)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    make = lambda c: base.filled_segment(tq, B, H, d, c, *widths)  # noqa: E731
    want, written, compressed = make(16), make(cap), make(cap)
    tq.tq_compress(want, rot, K, V, 0)
    tq.tq_append(written, rot, K, V, zero)
    tq.tq_compress(compressed, rot, K, V, 0)
    torch.cuda.synchronize()
    same(written, want, n)
    same(compressed, want, n)
    for use in (rot, None):
        got = tq.tq_read(written, use, zero, n, dtype=torch.float32)
        ref = tq.tq_dequantize(want, 0, n, rot, rotated=use is None, original=use is not None)
        for x, y in zip(got, ref[2:] if use is not None else ref[:2]):
            assert torch.equal(bits(x), bits(y))


# 64 dims: records of 8 b bytes, two of which are stored at once where 16-byte boundaries allow
@pytest.mark.parametrize("cap", [33, 47])
def test_64_dims(tq, cap):
    d, B, H, n = 64, 3, 5, 30
    widths = ([1, 2, 8, 3, 4], [3, 2, 5, 4, 7])
    g = gen(cap)
    K, V = (randn(g, B, H, n, d, dtype=torch.float16) for _ in range(2))
    rot = tq.tq_make_rotation(d, 3)
    make = lambda c: base.filled_segment(tq, B, H, d, c, *widths)  # noqa: E731
    want, written, compressed = make(48), make(cap), make(cap)
    tq.tq_compress(want, rot, K, V, 0)
    tq.tq_compress(compressed, rot, K, V, 0)
    tq.tq_append(written, rot, K, V, torch.zeros(B, dtype=torch.int32, device=DEV))
    same(compressed, want, n)
    same(written, want, n)
    ref = tq.tq_dequantize(want, 0, n, rot, rotated=False, original=True)[2:]
    for m in (n, 700):  # small and large reads (rows behind the capacity are not read)
        zero = torch.zeros(B, dtype=torch.int32, device=DEV)
        got = tq.tq_read(written, rot, zero, m, n_read=zero + n, dtype=torch.float32)
        for x, y in zip(got, ref):
            assert torch.equal(bits(x[:, :, :n].contiguous()), bits(y)) and not x[:, :, n:].any()
