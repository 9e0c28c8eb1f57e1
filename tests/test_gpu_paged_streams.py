"""The calls on pages and drafts on a stream that is not the current one, and in graphs, against plain references."""
import numpy as np
import pytest
import torch

import test_gpu_pages as pages
import test_gpu_verify as verify
from test_gpu_serving import DEV, bits, gen, randn
from test_gpu_serving_streams import Behind

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    for n_max in (3, 40):  # (a kernel's first launch loads it, which waits for what runs)
        args = [torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((1, 2), 1, 1, 4, 1)]
        T.tq_page_tables(*args, 16, n_max)
        T.tq_page_release(*args, 16)
    x = verify.verify_case(1, 1, 9, torch.float32, "chain", True, 0, 1)
    T.tq_verify(x[0], x[3], x[5], draft=x[4])
    return T


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def same(got, want):
    return all(np.array_equal(x.cpu().numpy(), np.asarray(y)) for x, y in zip(got, want))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("n_max", [7, 40])
def test_tables_behind_other_work(tq, n_max, raw):
    B, P, M, n_pages = 9, 16, 12, 200
    table, length, count, free, n_free = pages.pages_case(B, P, M, n_pages, 60, n_max, 3, False)
    side = torch.cuda.Stream()
    args, keep = [i32(a) for a in (table, length, count, free, [n_free])], i32(length)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # (memory of both streams is cached from here on)
        [torch.empty(B * n_max, dtype=torch.int32, device=DEV) for _ in range(8)]
    with Behind():
        out = tq.tq_page_tables(*args, P, n_max, stream=side.cuda_stream if raw else side)
        side.synchronize()
    want = pages.place(table, length, count, free, n_free, P, n_max, n_pages)
    assert same((*out, args[4][0], args[0], args[1], args[3]), (*want, table, length, free))
    with Behind():
        tq.tq_page_release(args[0], args[1], keep, args[3], args[4], P, stream=side.cuda_stream if raw else side)
        side.synchronize()
    assert torch.equal(args[1], keep) and int(args[4]) == n_free and np.array_equal(args[3].cpu().numpy()[:n_free], free[:n_free])


@pytest.mark.parametrize("raw", [False, True])
def test_verification_behind_other_work(tq, raw):
    tokens, parents, par, target, draft, uniform = verify.verify_case(4, 5, 999, torch.float32, "tree", True, 0, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with Behind():
        got = tq.tq_verify(tokens, target, uniform, draft=draft, parents=par, stream=side.cuda_stream if raw else side)
        side.synchronize()
    verify.check(got, tokens, parents, target, draft, uniform)


@pytest.mark.parametrize("n_max", [3, 300])
def test_captured_tables(tq, n_max):
    """Tables, slots and release in one graph, replayed on other lengths and counts."""
    B, P, M, n_pages = 20, 16, 30, 700
    args = [i32(a) for a in (np.zeros((B, M)), np.zeros(B), np.zeros(B), np.zeros(n_pages), [0])]
    keep = i32(np.zeros(B))
    out = (i32(np.zeros((B, n_max))), i32(np.zeros((B, n_max))), i32(np.zeros(B)))
    behind = [torch.zeros_like(a) for a in args]  # what the first call left
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        tq.tq_page_tables(*args, P, n_max, out=out)
        for x, y in zip(behind, args):
            x.copy_(y)
        tq.tq_page_release(args[0], args[1], keep, args[3], args[4], P)
    for seed, spare in ((1, 700), (2, 90), (3, 0)):
        table, length, count, free, n_free = pages.pages_case(B, P, M, n_pages, spare, n_max, seed, False)
        for x, y in zip((*args, keep), (table, length, count, free, [n_free], length)):
            x.copy_(i32(y))
        before = length.copy()
        graph.replay()
        torch.cuda.synchronize()
        want = pages.place(table, length, count, free, n_free, P, n_max, n_pages)
        assert same((*out, behind[4][0], behind[0], behind[1]), (*want, table, length))
        assert same((args[1], args[4][0], args[3][:n_free]), (before, n_free, free[:n_free]))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("d,kb,vb", [(128, 3, 4), (64, None, None)])
def test_paged_cache_on_a_stream_that_is_not_current(tq, d, kb, vb, raw):
    from rotated_quantized_kv_gb300.model_cache import PagedCache
    B, H, Hq, S, P = 3, 2, 8, 50, 16
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 256))
    g = gen(d)
    K, V = (randn(g, B, H, S, d, dtype=torch.float16) for _ in range(2))
    q0 = randn(g, B, Hq, d, dtype=torch.float16)
    n, keep = i32([50, 0, 17]), i32([20, 0, 16])
    one = i32([1, 1, 0])
    at = [i32([49, -1, 16]), i32([20, 0, 15])]

    def loop(c, q, outs, stream):
        slots, positions, granted = c.grow(n, S, stream=stream)
        c.write(0, K, V, slots, positions, stream=stream)
        c.attend(0, q[0], at[0], outs[0], stream=stream)
        c.release(keep, stream=stream)
        s2, p2, g2 = c.grow(one, 1, stream=stream)
        c.write(0, K, V, s2, p2, stream=stream)
        c.attend(0, q[1], at[1], outs[1], stream=stream)
        return [*outs, *q, slots, positions, granted, s2, p2, g2, c.length, c.table, c.n_free] + c.read(0, slots, torch.float32, stream=stream)

    make = lambda: PagedCache(1, B, H, Hq, d, 20, 6, rope, kb, vb, page=P)  # noqa: E731
    place = lambda: ([q0.clone(), q0.clone()], [torch.zeros_like(q0) for _ in range(2)])  # noqa: E731
    want = loop(make(), *place(), None)
    side = torch.cuda.Stream()
    side_now = side.cuda_stream if raw else side
    loop(make(), *place(), side_now)
    c, mine = make(), place()
    with Behind():
        got = loop(c, *mine, side_now)
        side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(bits(x) if x.is_floating_point() else x, bits(y) if y.is_floating_point() else y)
    assert want[0].abs().sum() > 0 and want[6].tolist() == [50, 0, 17] and want[10].tolist() == [21, 1, 16]
