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


# ------------------------------------------------------------------ offsets beyond 32 bits
@pytest.mark.parametrize("d,cap,kb,vb", [(128, 40_000_000, 8, 8), (64, 80_000_000, 8, 2), (256, 20_000_000, 8, 1)])
def test_records_beyond_four_gigabytes(tq, d, cap, kb, vb):
    """Rows at the end of a segment of more than 2^32 bytes of keys, beside one at its beginning."""
    B, H, n = 1, 1, 96
    g = gen(d)
    K, V = (randn(g, B, H, n, d, dtype=torch.float16) for _ in range(2))
    rot = tq.tq_make_rotation(d, 21)
    big = tq.PackedSegment(tq.make_layout(B, H, d, cap, kb, vb), n_tokens=cap)
    assert big.kcodes.numel() > 1 << 32
    small = tq.PackedSegment(tq.make_layout(B, H, d, n, kb, vb), n_tokens=n)
    at = torch.tensor([cap - n], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    tq.tq_append(big, rot, K, V, at)
    tq.tq_append(small, rot, K, V, zero)
    assert torch.equal(big.kcodes[-n * d * kb // 8:], small.kcodes) and torch.equal(big.vcodes[-n * d * vb // 8:], small.vcodes)
    for m in (n, 20000):  # small and large reads
        got = tq.tq_read(big, rot, at, m, n_read=zero + n)
        want = tq.tq_read(small, rot, zero, n)
        for x, y in zip(got, want):
            assert torch.equal(bits(x[:, :, :n].contiguous()), bits(y))
    # Attention over all of it: records of zero bits have every rotated coordinate at the lowest level, which
    # points against a query whose rotated coordinates sum to much; at that scale they get no weight.
    R = base.rotation64(tq, d, 21)[1]
    lead = torch.ones(d, dtype=torch.float64, device=DEV) @ R
    q = (lead * (1 + torch.rand(1, 5, 2, 1, generator=g, device=DEV))).half()
    k, v = (randn(g, B, H, 5, d, dtype=torch.float16) for _ in range(2))
    big.kscale[:cap - n] = 100.0
    out, want = (base.run_tree(tq, q, k, v, [s]) for s in (big, small))
    if d != 256:
        base.check_tree(out, base.tree_ref(tq, q, k, v, None, [small], [None], R))
    assert (out.double() - want.double()).norm() <= 2.0**-10 * want.double().norm()


def test_cache_without_sinks(tq):
    """Prompts and a verified step of a cache whose tokens all lie in the packed segment, fewer drafts than it takes."""
    from rotated_quantized_kv_gb300.model_cache import SpeculativeCache
    B, H, Hq, d, N, S, cap = 2, 2, 4, 128, 3, 30, 64
    g = gen(1)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 100))
    c = SpeculativeCache(1, B, H, Hq, d, cap, rope, 4, 4, sinks=0, drafts=8)
    K, V = (randn(g, B, H, S, d, dtype=torch.float16) for _ in range(2))
    n = torch.tensor([30, 0], dtype=torch.int32, device=DEV)
    c.prefill(0, K, V, n, torch.arange(S, dtype=torch.int32, device=DEV))
    c.advance(n)
    q, (k, v) = randn(g, B, N, Hq, d, dtype=torch.float16), (randn(g, B, H, N, d, dtype=torch.float16) for _ in range(2))
    at = c.length[:, None] + torch.arange(N, dtype=torch.int32, device=DEV)
    out = torch.empty(B, N, Hq, d, dtype=torch.float16, device=DEV)
    turned = base.rope_ref(K, rope.table, torch.arange(S, device=DEV).expand(B, S), d // 2, False, False, torch.float16)
    stored = tq.PackedSegment(c.body[0].layout, n_tokens=cap)
    tq.tq_append(stored, c.rot[0], turned, V, torch.zeros_like(n), n_new=n)
    c.attend(0, q, k, v, at, out)
    _, R = base.rotation64(tq, d, 42)
    base.check_tree(out, base.tree_ref(tq, q, k, v, None, [stored], [n], R))
    took = torch.tensor([1, 3], dtype=torch.int32, device=DEV)
    path = torch.arange(N, dtype=torch.int32, device=DEV).expand(B, N).contiguous()
    c.commit(0, k, v, path, took)
    c.advance(took)
    assert c.length.tolist() == [31, 3] and c.body_at.tolist() == [31, 3] and c.body_len.tolist() == [31, 3]
    tq.tq_append(stored, c.rot[0], k, v, n, n_new=took)
    for x, y in zip(c.read(0, torch.zeros_like(n), 40), tq.tq_read(stored, c.rot[0], torch.zeros_like(n), 40, n_read=c.length)):
        assert torch.equal(bits(x), bits(y))
