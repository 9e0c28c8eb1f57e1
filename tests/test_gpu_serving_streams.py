"""Calls that are given a stream while another one is current, and busy."""
import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import DEV, bits, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


class Behind:
    """Keeps the current stream busy, so that work put there by mistake comes too late (and what such work
    would leave in freed memory is written over at once)."""

    def __enter__(self):
        torch.cuda.synchronize()
        torch.cuda._sleep(1_000_000_000)  # about half a second
        self.after = torch.cuda.Event()
        self.after.record()

    def __exit__(self, kind, *_):
        if kind is None:
            assert not self.after.query()  # the other stream's results were there while this one slept
        torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("d,kb,vb", [(128, 3, 3), (64, 4, 2)])
def test_cache_on_a_stream_that_is_not_current(tq, d, kb, vb, raw):
    from rotated_quantized_kv_gb300.model_cache import SpeculativeCache
    B, H, Hq, N, sinks, cap, S = 3, 2, 8, 5, 16, 96, 60
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 256))
    g = gen(d)
    K, V = (randn(g, B, H, S, d, dtype=torch.float16) for _ in range(2))
    pos = torch.arange(S, dtype=torch.int32, device=DEV)
    n0 = torch.tensor([5, 60, 16], dtype=torch.int32, device=DEV)
    took = torch.tensor([2, 0, 3], dtype=torch.int32, device=DEV)
    path = torch.tensor([[0, 2, 0, 0, 0], [0] * 5, [0, 1, 4, 0, 0]], dtype=torch.int32, device=DEV)
    at = n0[:, None] + torch.arange(N, dtype=torch.int32, device=DEV)
    first = torch.tensor([0, 10, 14], dtype=torch.int32, device=DEV)
    qkv = randn(g, B, N, Hq + 2 * H, d, dtype=torch.float16)

    def loop(c, stream):
        x = qkv.clone() if stream is None else mine
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + H].transpose(1, 2), x[:, :, Hq + H:].transpose(1, 2)
        out = torch.zeros(B, N, Hq, d, dtype=torch.float16, device=DEV) if stream is None else place
        c.prefill(0, K, V, n0, pos, stream=stream)
        c.advance(n0, stream=stream)
        c.attend(0, q, k, v, at, out, stream=stream)
        c.commit(0, k, v, path, took, stream=stream)
        c.advance(took, stream=stream)
        return [out, c.length, c.body_at] + c.read(0, first, 50, stream=stream) + c.read(0, first, 7, torch.float32, stream=stream)

    make = lambda: SpeculativeCache(1, B, H, Hq, d, cap, rope, kb, vb, sinks, N)  # noqa: E731
    want = loop(make(), None)
    mine, place = qkv.clone(), torch.zeros(B, N, Hq, d, dtype=torch.float16, device=DEV)
    c = make()
    side = torch.cuda.Stream()
    side_now = side.cuda_stream if raw else side
    loop(make(), side_now)  # (memory of both streams is cached from here on)
    mine.copy_(qkv)
    place.zero_()
    with Behind():
        got = loop(c, side_now)
        junk = [torch.full((B,), -1, dtype=torch.int32, device=DEV) for _ in range(64)]  # into memory that is free by now
        side.synchronize()
    assert all(int(x.sum()) == -B for x in junk)
    for x, y in zip(got, want):
        assert torch.equal(bits(x) if x.is_floating_point() else x, bits(y) if y.is_floating_point() else y)


@pytest.mark.parametrize("raw", [False, True])
def test_results_that_a_call_allocates(tq, raw):
    """Tables and rows read back, while the current stream is busy: their zeros come first."""
    B, H, d, cap, n = 2, 4, 128, 64, 40
    g = gen(3)
    seg = base.random_segment(tq, g, B, H, d, cap, 3, 4)
    rot = tq.tq_make_rotation(d, 5)
    spec = tq.tq_make_rope(d)
    first, count = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([3, 20], [40, 11]))
    calls = (lambda s: tq.tq_read(seg, rot, first, n, n_read=count, stream=s),
             lambda s: [tq.tq_rope_table(spec, 300, stream=s)],
             lambda s: list(tq.tq_dequantize(seg, 0, cap, rot, original=True, stream=s)))
    want = [f(None) for f in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    host = [[torch.empty_like(t, device="cpu", pin_memory=True) for t in w] for w in want]
    with Behind():
        got = [f(side.cuda_stream if raw else side) for f in calls]
        with torch.cuda.stream(side):
            for h, x in zip(host, got):
                for a, b in zip(h, x):
                    a.copy_(b, non_blocking=True)
        side.synchronize()
    for w, h, x in zip(want, host, got):
        for a, b, c in zip(w, h, x):
            assert torch.equal(bits(a.cpu()), bits(b)) and torch.equal(bits(a), bits(c))


def test_null_handle_is_the_default_stream(tq):
    g = gen(4)
    seg = base.random_segment(tq, g, 1, 2, 64, 16, 3, 3)
    first = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = tq.tq_read(seg, None, first, 16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = tq.tq_read(seg, None, first, 16, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want))


@pytest.mark.parametrize("raw", [False, True])
def test_captured_calls_that_name_their_stream(tq, raw):
    """Results that a captured call allocates belong to the graph, whether the stream is current or named."""
    from rotated_quantized_kv_gb300.model_cache import SpeculativeCache
    B, H, Hq, d, S, cap = 2, 2, 4, 128, 30, 64
    g = gen(6)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 100))
    caches = [SpeculativeCache(1, B, H, Hq, d, cap, rope, 3, 4, sinks=16, drafts=4) for _ in range(2)]
    K, V = (torch.zeros(B, H, S, d, dtype=torch.float16, device=DEV) for _ in range(2))
    n, first = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)

    def calls(c, stream):
        c.length.zero_()
        c.prefill(0, K, V, n, pos, stream=stream)
        c.advance(n, stream=stream)
        return c.read(0, first, 20, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls(caches[0], None)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = calls(caches[0], side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for lens, at in (([30, 4], [10, 0]), ([17, 29], [0, 16])):
        K.copy_(randn(g, *K.shape, dtype=torch.float16)), V.copy_(randn(g, *V.shape, dtype=torch.float16))
        n.copy_(torch.tensor(lens)), first.copy_(torch.tensor(at))
        torch.cuda.synchronize()
        graph.replay()
        want = calls(caches[1], None)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(bits(x), bits(y)) and bool((x != 0).any())
