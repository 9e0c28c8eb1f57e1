"""Tree attention where the values of a sequence differ widely in size."""
import math

import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def check(out, ref, largest):
    """check_tree's bound, the weights' half steps counted in a row's 2-norm: each weight is off by 2^-11 of
    itself or, below 2^-14 of the row's largest weighted value, by 2^-25 of that (its share: `largest`)."""
    want, size, reach = ref
    err = (out.double() - want).norm(dim=-1)
    tol = 2.0**-11 * want.norm(dim=-1) * 1.01 + (2 * 2.0**-11 + 2 * reach * 2.0**-19) * size + largest + 1e-7
    assert bool(torch.isfinite(out).all())
    assert bool((err <= tol).all()), float((err / tol).max())
    # independent roundings, in squares over the whole output: sqrt(3) half steps, as in check_tree
    bound = (3 * 2.0**-11 + 2 * reach.max() * 2.0**-19) * want.norm() + largest.norm() / 16
    assert err.norm() <= bound, float(err.norm() / bound)


def one_direction(tq, d, H, gqa, B, N, kb, vb, n, seed):
    """Queries that are positive multiples of one vector (and a little besides), so that a token whose key points
    against it gets little weight from every row.  (q, k, v, segment, the tokens' scores for that vector, R)"""
    g = gen(seed)
    cap = -(-n // 16) * 16
    seg = base.random_segment(tq, g, B, H, d, cap, [kb] * H, [vb] * H, n=n)
    seg.kscale.fill_(1.0)
    seg.vscale.fill_(1.0)
    lead = randn(g, 1, 1, 1, d)
    q = (lead * (1 + 0.2 * torch.rand(B, N, H * gqa, 1, generator=g, device=DEV)) + 0.02 * randn(g, B, N, H * gqa, d)).half()
    k, v = (randn(g, B, H, N, d, dtype=torch.float16) for _ in range(2))
    _, R = base.rotation64(tq, d, 21)
    score = torch.einsum("bhtd,d->bht", base.stored64(tq, seg, R)[0], lead[0, 0, 0].double()) / math.sqrt(d)
    return q, k, v, seg, score, R


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", [3, 14])
@pytest.mark.parametrize("power", [12, 16, 20, 24, 30])
@pytest.mark.parametrize("where", ["first", "later", "both"])
def test_large_value_of_little_weight(tq, d, N, power, where):
    """A token whose value is 2^power times the others' and whose weight is 2^-(power + 12): it adds 2^-12 of the
    others' size, and must not cost them their precision."""
    H, gqa, B, n = 1, 4, 1, 700
    q, k, v, seg, score, R = one_direction(tq, d, H, gqa, B, N, 4, 4, n, seed=d + N)
    usual = base.tree_ref(tq, q, k, v, None, [seg], [None], R)[2]  # the scores that have weight
    for lo, hi in {"first": [(0, 128)], "later": [(256, 384)], "both": [(0, 128), (384, 512)]}[where]:
        t = lo + int(score[0, 0, lo:hi].argmin())
        assert score[0, 0, t] < -0.2
        seg.vscale[t] = 2.0**power
        seg.kscale[t] = (power + 12) * math.log(2) / -float(score[0, 0, t])
    out = base.run_tree(tq, q, k, v, [seg])
    ref = base.tree_ref(tq, q, k, v, None, [seg], [None], R)
    # the largest weighted value of a row is at most its sum; n tokens of 2^-25 of it (in squares: sqrt(n) of them)
    check(out, (ref[0], ref[1], usual), (n + N) * 2.0**-25 * ref[1])


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_zero_size_first(tq, d):
    """Whole tiles of zero values, then values of 2^-6: the scale of the first is not kept for the others."""
    H, gqa, B, N, n = 1, 4, 1, 5, 700
    q, k, v, seg, score, R = one_direction(tq, d, H, gqa, B, N, 4, 4, n, seed=d)
    seg.vscale[:n] = 2.0**-6
    seg.vscale[:300] = 0.0
    v.zero_()
    seg.kscale[300:n] = 12.0  # a few tokens have most of the weight
    out = base.run_tree(tq, q, k, v, [seg])
    ref = base.tree_ref(tq, q, k, v, None, [seg], [None], R)
    check(out, ref, (n + N) * 2.0**-25 * ref[1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_coordinate_of_a_stored_value(tq, d, bad):
    """One coordinate of one fp16 row: it reaches that coordinate of the result alone."""
    H, gqa, B, N, at = 2, 2, 2, 6, 37
    q, k, v, parts, lens, rng = base.tree_case(tq, d, H, gqa, B, N, [((4, 3), 300), ("fp16", 150)], False, seed=d)
    parts[0].kscale.nan_to_num_(0.0)
    parts[0].vscale.nan_to_num_(0.0)
    want = base.run_tree(tq, q, k, v, parts)
    parts[1].v[1, :, 70, at] = bad
    got = base.run_tree(tq, q, k, v, parts)
    rest = [i for i in range(d) if i != at]
    assert torch.equal(base.bits(got[0]), base.bits(want[0]))
    assert torch.equal(base.bits(got[1][..., rest]), base.bits(want[1][..., rest]))
    hit = got[1][..., at].float()
    assert bool(torch.isnan(hit).all()) if math.isnan(bad) else bool((hit == bad).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [3, 14])
def test_large_fp16_value_of_little_weight(tq, d, N):
    """An fp16 row near fp16's end, 2^24 times the others' size, at a weight of 2^-26 of theirs: a hundredth of the
    result's size, by a weight that one fp16 beside the row's largest does not hold."""
    H, gqa, B, n, at = 1, 4, 1, 300, 170
    g = gen(d + N)
    lead = randn(g, 1, 1, 1, d)
    q = (lead * (1 + 0.01 * torch.rand(B, N, H * gqa, 1, generator=g, device=DEV))).half()
    seg = tq.Fp16Segment(B, H, d, 304, n_tokens=n, k=(0.1 * randn(g, B, H, 304, d)).half(),
                         v=(2.0**-8 * randn(g, B, H, 304, d)).half())
    k, v = ((s * randn(g, B, H, N, d)).half() for s in (0.1, 2.0**-8))
    usual = base.tree_ref(tq, q, k, v, None, [seg], [None], torch.eye(d, device=DEV).double())[2]
    x = lead[0, 0, 0].half()
    seg.k[0, 0, at] = (-26 * math.log(2) * math.sqrt(d) / float((x.float() ** 2).sum()) * x.float()).half()
    seg.v[0, 0, at] = (60000 * torch.sign(randn(g, d))).half()
    out = base.run_tree(tq, q, k, v, [seg])
    ref = base.tree_ref(tq, q, k, v, None, [seg], [None], torch.eye(d, device=DEV).double())
    # half a step of 2^-35 of the row's largest weight, which is a hundredth of their sum at most, for the large
    # row, and half a step of fp16's smallest, 2^-24, for each coordinate of the result
    check(out, (ref[0], ref[1], usual), math.sqrt(d) * (2.0**-36 * 60000 / 100 + 2.0**-25) * torch.ones_like(usual))
    share = (ref[0] - base.tree_ref(tq, q, k, v, None, [without(tq, seg, at)], [None], torch.eye(d, device=DEV).double())[0])
    assert share.norm() > 0.003 * ref[0].norm()  # (what the test is about)


def without(tq, seg, at):
    keep = [t for t in range(seg.k.shape[2]) if t != at]
    return tq.Fp16Segment(1, 1, seg.k.shape[3], len(keep), n_tokens=seg.n_tokens - 1, k=seg.k[:, :, keep].contiguous(),
                          v=seg.v[:, :, keep].contiguous())


def level_error(tq, bits):
    """Root mean square error of fp16(s c) / s over the levels c, of their own, s in [1, 2) the scale in steps of
    1/4096 at which the levels' errors, weighted by the share of N(0, 1) in their cells, are smallest."""
    c = tq.tq_fit_codebook(bits)[0].double()
    edge = torch.cat([torch.tensor([-math.inf]).double(), (c[1:] + c[:-1]) / 2, torch.tensor([math.inf]).double()])
    mass = torch.special.ndtr(edge[1:]) - torch.special.ndtr(edge[:-1])
    s = (1 + torch.arange(4096) / 4096.0)[:, None]
    e = ((s * c.float()).half().double() / s.double() - c) ** 2
    return float(e[(e * mass).sum(1).argmin()].mean().sqrt() / (c**2).mean().sqrt())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [4, 8, 16, 40])
@pytest.mark.parametrize("vb", range(1, 9))
def test_weights_round_no_further_than_the_result(tq, d, N, vb):
    """Weights of 22 bits, and levels whose rounding is known: beside it the error is that of rounding the result to
    fp16."""
    H, gqa, B, n = 2, 4, 1, 1500
    q, k, v, parts, lens, rng = base.tree_case(tq, d, H, gqa, B, N, [((4, vb), n)], False, seed=vb + N)
    parts[0].kscale.nan_to_num_(0.0).clamp_(max=0.5)
    parts[0].vscale.nan_to_num_(0.0)
    out = base.run_tree(tq, q, k, v, parts)
    _, R = base.rotation64(tq, d, 21)
    want, _, reach = base.tree_ref(tq, q, k, v, None, parts, lens, R)
    best = (want.half().double() - want).norm() / want.norm()
    # random codes: the levels' errors are as independent as the values; scores as in check_tree; a tenth
    # more for the samples' spread (rows of one cache share its tokens)
    bound = 1.1 * math.hypot(float(best), level_error(tq, vb)) + float(2 * reach.max()) * 2.0**-19
    assert float((out.double() - want).norm() / want.norm()) <= bound


@pytest.mark.parametrize("d,N,widths", [(64, 5, (3, 4)), (128, 5, (3, 4)), (128, 16, (8, 8)), (128, 8, (5, 6))])
@pytest.mark.parametrize("polls", [0, 1, 2, 3, 5, 8, 16, 64])
def test_a_wait_that_ran_out_is_reported(tq, d, N, widths, polls):
    """Few polls a wait: some roles go on and others give up.  Either the flag says so or the output is whole."""
    q, k, v, parts, lens, rng = base.tree_case(tq, d, 2, 4, 2, N, [(widths, 1500), ((8, 1), 300), ("fp16", 200)], False, seed=N)
    want = base.run_tree(tq, q, k, v, parts)
    lv = tq.layer_view(tq.tq_make_rotation(d, 21), parts)
    ws = torch.empty(tq.tq_tree_workspace_size(lv, 2, 2, 8, N, d), dtype=torch.uint8, device=DEV)
    flags = 0
    for _ in range(4):
        out = torch.zeros_like(want)
        try:
            tq.tq_set_decode_wait_polls(polls)
            tq.tq_tree_attention(lv, q, k, v, out, ws)
            flag = tq.tq_decode_error_flag(ws)
        finally:
            tq.tq_set_decode_wait_polls(tq.TQ_WAIT_POLLS_DEFAULT)
        flags += flag != 0
        assert flag != 0 or torch.equal(base.bits(out), base.bits(want))
    assert flags == 4 or polls > 0
    assert torch.equal(base.bits(base.run_tree(tq, q, k, v, parts, ws=ws)), base.bits(want))
