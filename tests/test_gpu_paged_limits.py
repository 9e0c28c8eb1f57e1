"""Attention over paged segments at the ends of its ranges."""
import pytest
import torch

import test_gpu_paged as paged
from test_gpu_serving import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def attend(tq, rot, q, segs, tables, lens):
    B, Hq, d = q.shape
    view = tq.layer_view(rot, segs)
    H = segs[0].layout.n_heads
    ws = torch.full((tq.tq_paged_workspace_size(view, B, H, Hq, d),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((B, Hq, d), float("nan"), dtype=torch.float16, device=DEV)
    return tq.tq_paged_attention(view, q, out, ws, tables, lens)


# d, key and value bits (None: fp16 rows), bytes a token of what passes 2^32 bytes: keys, values, or the scales
LARGE = [(128, None, None, 256), (64, None, None, 128), (128, 8, 1, 128), (128, 1, 8, 128), (64, 8, 2, 64), (64, 1, 1, 4), (256, 8, 1, 256)]


@pytest.mark.parametrize("d,kb,vb,row", LARGE)
def test_segment_without_a_table_beyond_four_gigabytes(tq, d, kb, vb, row):
    """Rows behind 2^32 bytes of one head, in a segment that holds its sequence in one piece: all others have keys and values of
    zero, so that their weight is nothing beside that of the last rows, which the query points along."""
    H, n, g = 1, 96, gen(d)
    cap = (1 << 32) // row + (1 << 32) // (row * 64)  # (some workers' shares begin behind the border)
    cap -= cap % 64
    k, v = (randn(g, 1, H, n, d, dtype=torch.float16) for _ in range(2))
    lead = torch.randn(d, generator=g, device=DEV)
    k = (k.float() + 3.0 * lead).half()
    q = (2.0 * lead[None, None] + torch.randn(1, 4, d, generator=g, device=DEV)).half()
    rot = tq.tq_make_rotation(d, 21)
    segs = []
    for size in (cap, n):
        at = torch.tensor([size - n], dtype=torch.int32, device=DEV)
        if kb is None:
            seg = tq.Fp16Segment(1, H, d, size, n_tokens=size, k=torch.zeros(1, H, size, d, dtype=torch.float16, device=DEV),
                                 v=torch.zeros(1, H, size, d, dtype=torch.float16, device=DEV))
        else:
            seg = tq.PackedSegment(tq.make_layout(1, H, d, size, kb, vb), n_tokens=size)
            seg.kscale.zero_()
            seg.vscale.zero_()
        tq.tq_append(seg, None if kb is None else rot, k, v, at)
        segs.append(seg)
    out, want = (attend(tq, rot, q, [s], [None], [None]) for s in segs)
    assert want.abs().max() > 0.1
    # (other workers' shares, so other roundings: each result is off by half a step, and by 2^-11 of a level)
    assert (out.double() - want.double()).norm() <= 2.0**-10 * want.double().norm()


INF = float("inf")


def infinite_case(tq, d, seed, kinds, lens, gqa=4):
    B, H = len(lens), 2
    c = paged.Case(tq, d, H, gqa, B, [(k, 32, max(lens)) for k in kinds], seed=seed, lens=[lens] * len(kinds))
    c.q[:, :, 0] = c.q[:, :, 0].abs() + 0.5          # the sign of an infinite coordinate is that of the score
    return c


def place(c, i, b, t):
    """Pages of segment i, and places on them, of tokens t of sequence b."""
    P = c.parts[i].layout.capacity
    return c.tables[i][b].long()[t // P], t % P


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("beside", [False, True])
def test_keys_at_minus_infinity(tq, d, beside):
    """Tokens whose score is minus infinity have no weight, wherever a worker's share begins; a row of nothing else is zeros."""
    lens = [40000, 33, 16, 70000, 64]                # (a share is several stages)
    c = infinite_case(tq, d, d + 1, ["fp16", (4, 4)] if beside else ["fp16"], lens)
    gone = {(0, 0): range(30000), (0, 1): range(0, 40000, 3), (1, 1): range(33), (2, 0): range(16), (2, 1): range(1, 16),
            (3, 0): range(16, 70000), (3, 1): range(69950)}
    for (b, h), t in gone.items():
        t = torch.tensor(list(t), device=DEV)
        page, at = place(c, 0, b, t)
        c.parts[0].k[page, h, at, 0] = -INF
        c.rows[0][b][0][h, t, 0] = -INF
    out = c.run()
    want, size, reach = c.reference()
    if not beside:
        for b, h in ((1, 1), (2, 0)):
            assert torch.isnan(want[b, 4 * h:4 * h + 4]).all()  # (0 / 0 of the definition)
            assert (out[b, 4 * h:4 * h + 4] == 0).all()
            want[b, 4 * h:4 * h + 4] = size[b, 4 * h:4 * h + 4] = 0.0
    assert torch.isfinite(out).all()
    # (Case.check's bound; the largest finite score is below 40 here)
    err = (out.double() - want).norm(dim=-1)
    tol = 2.0**-11 * 1.01 * want.norm(dim=-1) + ((2.0**-11 if beside else 0.0) + 2.0**-18 + 80 * 2.0**-19) * size + 1e-7
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("beside", [False, True])
def test_infinite_values(tq, d, beside):
    """An infinite coordinate of an fp16 value makes that coordinate of the outputs infinite, and no other."""
    lens = [40, 3, 130]
    c = infinite_case(tq, d, d + 3, ["fp16", (4, 4)] if beside else ["fp16"], lens)
    c.q *= 0.25                                      # (weights near one another)
    for b, h, t, e, x in ((0, 0, 7, 5, INF), (0, 1, 20, d - 1, -INF), (1, 0, 0, 3, INF), (1, 0, 1, 3, -INF), (2, 1, 129, 0, INF),
                          (2, 1, 0, 9, -INF), (2, 1, 100, 9, -INF)):
        page, at = place(c, 0, b, t)
        c.parts[0].v[page, h, at, e] = x
        c.rows[0][b][1][h, t, e] = x
    out = c.run().double()
    want, _, _ = c.reference()
    assert torch.isinf(want).sum() == 4 * 4 and torch.isnan(want).sum() == 4
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out[torch.isinf(want)], want[torch.isinf(want)])
    assert (out - want)[~odd].abs().max() < 0.01


def test_query_heads_beyond_24_bits(tq):
    """More blocks of query rows than 2^23, all with the same query: every row is what one row alone is."""
    d, Hq, n = 64, (1 << 24) + 10, 30
    g = gen(3)
    rot = tq.tq_make_rotation(d, 21)
    seg = tq.PackedSegment(tq.make_layout(1, 1, d, 32, 4, 4), n_tokens=n)
    k, v = (randn(g, 1, 1, n, d, dtype=torch.float16) for _ in range(2))
    tq.tq_append(seg, rot, k, v, torch.zeros(1, dtype=torch.int32, device=DEV))
    q = randn(g, 1, 1, d, dtype=torch.float16)
    want = attend(tq, rot, q, [seg], [None], [None])
    out = attend(tq, rot, q.expand(1, Hq, d), [seg], [None], [None])
    assert want.abs().max() > 0.01
    for part in out[0].split(1 << 22):
        assert torch.equal(part, want[0].expand(len(part), d))


@pytest.mark.parametrize("Hq", [1, 4, 40])
def test_view_without_segments(tq, Hq):
    """No segment, no token: zeros, for any number of query heads, eager and in a graph behind other work."""
    d, B = 128, 3
    q = randn(gen(1), B, Hq, d, dtype=torch.float16)
    view = tq.layer_view(tq.tq_make_rotation(d, 1), [])
    ws = torch.empty(max(tq.tq_paged_workspace_size(view, B, 1, Hq, d), 1), dtype=torch.uint8, device=DEV)
    out = torch.full((B, Hq, d), 7.0, dtype=torch.float16, device=DEV)
    tq.tq_paged_attention(view, q, out, ws, [], [])
    assert (out == 0).all()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out.zero_()
        out.add_(3.0)
        tq.tq_paged_attention(view, q, out, ws, [], [])
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 0).all()


@pytest.mark.parametrize("spread", [0.02, 2.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [(4, 1), (3, 1), (3, 2), (4, 3), (8, 4), (2, 5), (1, 8), "fp16"])
def test_long_sums_are_as_good_as_their_rounding(tq, d, kind, spread):
    """40000 tokens of 8 heads (some twenty tiles a worker), vectors of one size, scores of standard deviation `spread`: a
    mean far smaller than its values, and weights far apart.  The error of the whole is that of rounding the result (uniform in a
    step: step / sqrt(12) each), once more that of the levels above 4 bits (independent of it, at most as large: sqrt(2)),
    0.3 of it up to 4 bits (levels are scaled to round well: sqrt(1.09)), and a tenth for all else: 4096 and more
    roundings, whose squares' mean is within 5 x 1.4% of its expectation, and sums and weights of 22 bits."""
    H = 8
    c = paged.Case(tq, d, H, 4, 2, [(kind, 64, 40000)], seed=5, scale=0.25, lens=[[40000, 39000]])
    if kind != "fp16":
        for i, scale in enumerate((c.parts[0].kscale, c.parts[0].vscale)):
            own = scale[:c.parts[0].layout.batch * H * 64].view(-1, H, 64)
            for b in range(2):
                page, at = place(c, 0, b, torch.arange(int(c.lens[0][b]), device=DEV))
                c.rows[0][b][i] = c.rows[0][b][i] / own[page, :, at].t()[:, :, None].double()
            scale[~torch.isnan(scale)] = 1.0
    x = torch.cat([(c.q[b].double().view(H, 4, d) @ c.rows[0][b][0].transpose(1, 2)).flatten() for b in range(2)]) / d**0.5
    c.q *= spread / float(x.std())
    out = c.run().double()
    want, _, _ = c.reference()
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-14))) - 10)
    some = 1.41 if kind != "fp16" and kind[1] > 4 else 1.05
    far = float((out - want).norm() / (step.norm() / 12**0.5))
    assert far <= 1.1 * some, far
