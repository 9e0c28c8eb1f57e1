"""Attention of one new token over paged segments against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import DEV, MIXED, bits, gen, randn
from test_gpu_serving_streams import Behind

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Case:
    """Segments whose tokens lie on pages in any order (or, page None, one after another), and what the attention
    has to see of them; every other place holds NaN scales or rows."""

    def __init__(self, tq, d, H, gqa, B, segs, seed, scale=1.0, lens=None):
        self.g, self.rng = gen(seed), np.random.RandomState(seed)
        rng = self.rng
        self.tq, self.d, self.H, self.B = tq, d, H, B
        self.parts, self.tables, self.lens, self.rows = [], [], [], []
        self.rot, self.R = base.rotation64(tq, d, 21)
        for i, (kind, page, most) in enumerate(segs):
            n = rng.randint(0, most + 1, size=B) if lens is None else np.array(lens[i])
            if lens is None:
                n[rng.randint(B)] = most
                if B > 2:
                    n[rng.randint(B)] = rng.choice([0, 1])
            P = page or -(-max(most, 1) // 16) * 16
            M = -(-max(most, 1) // P)
            n_pages = B if page is None else B * M + 3
            table = np.arange(B)[:, None] if page is None else rng.permutation(n_pages)[:B * M].reshape(B, M)
            law = 0
            if kind == "fp16":
                s = tq.Fp16Segment(n_pages, H, d, P, n_tokens=min(P, most), k=randn(self.g, n_pages, H, P, d, dtype=torch.float16),
                                   v=randn(self.g, n_pages, H, P, d, dtype=torch.float16))
                x = [s.k.double(), s.v.double()]
            else:
                kb, vb = kind[:2]
                law = kind[2] if len(kind) > 2 else 0
                s = base.random_segment(tq, self.g, n_pages, H, d, P, kb, vb, law, n=min(P, most))
                s.kscale.clamp_(max=4.0)
                x = base.stored64(tq, s, self.R)
            seen = torch.zeros(n_pages, P, dtype=torch.bool, device=DEV)
            rows = []
            for b in range(B):
                t = np.arange(n[b])
                at = torch.tensor(table[b, t // P], device=DEV), torch.tensor(t % P, device=DEV)
                seen[at] = True
                rows.append([y.transpose(1, 2)[at].transpose(0, 1) for y in x])  # [H][n][d]
            if kind == "fp16":
                s.k.masked_fill_(~seen[:, None, :, None], float("nan"))
                s.v.masked_fill_(~seen[:, None, :, None], float("inf"))
            else:
                for y in (s.kscale, s.vscale):
                    y[:n_pages * H * P].view(n_pages, H, P).masked_fill_(~seen[:, None], float("nan"))
            self.parts.append(s)
            self.tables.append(None if page is None else i32(table))
            self.lens.append(i32(n))
            self.rows.append(rows)
        self.q = (scale * randn(self.g, B, H * gqa + 2, d)).half()[:, :H * gqa]
        self.view = tq.layer_view(self.rot, self.parts)

    def workspace(self):
        size = self.tq.tq_paged_workspace_size(self.view, self.B, self.H, self.q.shape[1], self.d)
        return torch.full((size,), 255, dtype=torch.uint8, device=DEV)

    def run(self, ws=None, out=None, **kw):
        ws = self.workspace() if ws is None else ws
        out = torch.full(self.q.shape, float("nan"), dtype=torch.float16, device=DEV) if out is None else out
        self.tq.tq_paged_attention(self.view, self.q, out, ws, self.tables, self.lens, **kw)
        return out

    def reference(self):
        """64 bits: (output, sum of p ||v|| a row, largest |q| |k| / sqrt(d))."""
        B, Hq, d = self.q.shape
        g = Hq // self.H
        out, size, reach = (torch.zeros(s, dtype=torch.float64, device=DEV) for s in ((B, Hq, d), (B, Hq), (B, Hq)))
        for b in range(B):
            K, V = (torch.cat([r[b][i] for r in self.rows] + [torch.zeros(self.H, 0, d, dtype=torch.float64, device=DEV)], 1)
                    for i in range(2))
            if K.shape[1] == 0:
                continue
            q = self.q[b].double().view(self.H, g, d)
            p = torch.softmax(q @ K.transpose(1, 2) / math.sqrt(d), -1)
            out[b] = (p @ V).flatten(0, 1)
            size[b] = (p @ V.norm(dim=-1, keepdim=True)).flatten()
            reach[b] = (q.norm(dim=-1) * K.norm(dim=-1).amax(-1, keepdim=True) / math.sqrt(d)).flatten()
        return out, size, reach

    def check(self, out, wide=None):
        """The result rounds by half a step (2^-11).  Operands of the scores carry 22 bits, their binary32
        sums 2^-20 of |q| |k| at most (256 additions with truncation), which moves a weight by that much of itself and its
        normaliser likewise; weights and sums carry 2^-20 too (32 tiles of truncated additions: 32 x 2 x 2^-24, besides 22 bits).  Levels of the value
        codebook as fp16: 2^-11 of a level.  In the 2-norm of a row (rotations keep it)."""
        want, size, reach = self.reference()
        err = (out.double() - want).norm(dim=-1)
        packed = any(p.kind == 0 for p in self.parts)
        levels = 2.0**-11 if packed else 0.0
        tol = 2.0**-11 * want.norm(dim=-1) * 1.01 + (levels + 2.0**-18 + 2 * reach * 2.0**-19) * size + 1e-7
        assert bool(torch.isfinite(out).all())
        assert bool((err <= tol).all()), float((err / tol).max())
        if want.abs().sum() > 0:  # in squares: the roundings are independent of the values and of each other
            wide = any(p.layout.vbits[h] > 4 for p in self.parts if p.kind == 0 for h in range(self.H))
            some = (1.0 + (1.0 if wide else 0.25 if packed else 0.0)) * 2.0**-11
            assert err.norm() <= (some + 2 * reach.max() * 2.0**-19) * want.norm(), float(err.norm() / want.norm())
        return out


# d, H, query heads a KV head, sequences, segments (bits or fp16, page (None: no pages), most tokens)
PAGED = [
    (128, 2, 4, 1, [((4, 4), 64, 900)]),
    (128, 2, 4, 3, [((3, 3), 16, 333)]),
    (128, 1, 1, 1, [((3, 3), 64, 1)]),
    (128, 2, 2, 2, [((3, 3), 64, 0)]),                                       # nothing at all
    (128, 8, 1, 3, [((MIXED, MIXED[::-1]), 48, 260)]),                       # every width
    (128, 8, 4, 2, [((MIXED[::-1], MIXED), 16, 700), ((MIXED, [3] * 8), 128, 127)]),
    (128, 2, 8, 4, [("fp16", None, 128), ((4, 4), 64, 1500), ("fp16", 32, 70)]),
    (128, 1, 4, 2, [((2, 1), 256, 5000)]),
    (128, 2, 3, 40, [((3, 2), 32, 400), ("fp16", 16, 9)]),                   # many sequences
    (128, 1, 16, 1, [((8, 8), 64, 1000)]),
    (128, 1, 5, 2, [((6, 7), 32, 600), ("fp16", None, 128)]),
    (128, 1, 33, 2, [((4, 3), 64, 300), ("fp16", 64, 200)]),                 # three blocks of rows
    (128, 4, 4, 2, [((5, 5, 1), 64, 500)]),                                  # the sphere law
    (128, 4, 4, 700, [((4, 4), 16, 40)]),
    (128, 2, 4, 5, [("fp16", 1, 37), ("fp16", 5, 41)]),                      # odd pages
    (128, 4, 2, 2, [("fp16", 128, 3001)]),
    (64, 2, 2, 3, [("fp16", None, 128), ((8, 3), 16, 700), ("fp16", 32, 61)]),
    (64, 8, 1, 2, [((MIXED, MIXED[::-1]), 64, 301)]),
    (64, 8, 4, 2, [((MIXED[::-1], MIXED), 128, 1023)]),
    (64, 1, 8, 3, [((3, 3), 48, 999), ((1, 1), 16, 129)]),
    (64, 1, 3, 2, [((4, 4), 64, 515), ("fp16", 16, 515)]),
    (64, 2, 20, 2, [((2, 2), 64, 4000)]),
    (256, 2, 2, 2, [((3, 4), 32, 200), ("fp16", 16, 30)]),
    (256, 1, 5, 1, [((8, 8), 64, 150)]),
    (512, 1, 2, 2, [((4, 2), 16, 70), ("fp16", None, 5)]),
    (16, 2, 4, 3, [((5, 3), 16, 300), ("fp16", 16, 20)]),
    (32, 1, 1, 2, [((2, 6), 64, 90)]),
    (1024, 1, 1, 1, [((3, 3), 16, 40)]),
]


@pytest.mark.parametrize("d,H,gqa,B,segs", PAGED)
def test_attention(tq, d, H, gqa, B, segs):
    c = Case(tq, d, H, gqa, B, segs, seed=d + 7 * B + H)
    ws = c.workspace()
    out = c.check(c.run(ws))
    assert tq.tq_decode_error_flag(ws) == 0
    none = torch.stack(c.lens).sum(0) == 0
    assert (out[none] == 0).all()
    assert torch.equal(bits(c.run(ws)), bits(out))  # nothing depends on an order of arrival
    # a longer table, strides, queries at odd places
    c.tables = [t if t is None else torch.cat([t, torch.full((B, 3), 1 << 30, dtype=torch.int32, device=DEV)], 1)[:, :t.shape[1] + 1]
                for t in c.tables]
    odd = torch.zeros(B * H * gqa * (d + 1) + 1, dtype=torch.float16, device=DEV)[1:].view(B, H * gqa, d + 1)
    odd[:, :, :d] = c.q
    c.q = odd[:, :, :d]
    assert torch.equal(bits(c.run(ws, out=torch.empty(B, H * gqa, d, dtype=torch.float16, device=DEV))), bits(out))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_and_pages_that_are_not_there(tq, d):
    """Lengths outside the table's reach count as the nearest inside; tokens on a page outside the pool are left out."""
    B, H, gqa, P = 5, 2, 4, 32
    c = Case(tq, d, H, gqa, B, [((4, 3), P, 200), ("fp16", P, 150)], seed=d, lens=[[200, 77, 0, 130, 200], [150, 150, 3, 64, 0]])
    for i, b, gone in ((0, 0, [1]), (0, 3, [0, 1]), (1, 0, [2]), (1, 3, [0])):
        n = int(c.lens[i][b])
        keep = torch.ones(n, dtype=torch.bool, device=DEV)
        for k, page in enumerate(gone):
            keep[page * P:(page + 1) * P] = False
            c.tables[i][b, page] = (-1, c.parts[i].layout.batch, 1 << 30)[(b + i + k) % 3]
        c.rows[i][b] = [x[:, keep] for x in c.rows[i][b]]
    assert c.tables[0].shape[1] * P > 200
    c.lens[0][4] = 2**31 - 1  # (its 200th token is not the table's last: the rest has to be there)
    c.parts[0].kscale.nan_to_num_(0.5)
    c.parts[0].vscale.nan_to_num_(0.5)
    x = base.stored64(tq, c.parts[0], c.R)
    pages = c.tables[0][4].long()
    c.rows[0][4] = [y[pages].transpose(0, 1).flatten(1, 2) for y in x]
    c.lens[0][2], c.lens[1][4] = -4, -(1 << 31)
    c.check(c.run())


@pytest.mark.parametrize("d,kb,vb", [(128, 4, 4), (128, 1, 8), (64, 3, 3), (256, 4, 4)])
def test_scores_and_values_of_any_size(tq, d, kb, vb):
    """Large scores, values of which one is far larger than the rest and has no weight, vectors of zeros."""
    c = Case(tq, d, 2, 4, 3, [((kb, vb), 64, 700)], seed=d + kb, scale=6.0)
    c.check(c.run())
    s, n = c.parts[0], 0
    L = s.layout
    for b in range(3):
        m = int(c.lens[0][b])
        if m < 4:
            continue
        K, q = c.rows[0][b][0], c.q[b].double()
        x = torch.einsum("hgd,htd->hgt", q.view(2, 4, d), K).amax(1)  # [H][m]
        low = x.argmin(1)
        for h in range(2):
            for t, f in ((int(low[h]), 2.0**24), (int(x[h].argsort()[m // 2]), 0.0)):
                page, at = int(c.tables[0][b, t // 64]), t % 64
                i = (page * 2 + h) * 64 + at
                s.vscale[i] *= f
                c.rows[0][b][1][h, t] *= f
                n += 1
        s.kscale[(int(c.tables[0][b, 0]) * 2) * 64] = 0.0
        c.rows[0][b][0][0, 0] = 0.0
    assert n
    want, size, reach = c.reference()
    out = c.run().double()
    # the large value's own weight: 2^-36 of the largest weighted value is dropped, else as everywhere
    tol = 2.0**-11 * want.norm(dim=-1) * 1.01 + (2.0**-11 + 2.0**-18 + 2 * reach * 2.0**-19) * size + 1e-6
    assert bool(((out - want).norm(dim=-1) <= tol).all())


def test_long_context(tq):
    """A context whose scores grow along it, over many stages of one worker and many workers of one head."""
    for d, kb, vb, B in ((128, 3, 3, 1), (64, 4, 2, 2)):
        c = Case(tq, d, 1, 4, B, [((kb, vb), 64, 40000)], seed=d, lens=[[40000] + [17000] * (B - 1)])
        c.check(c.run())
        s = c.parts[0]
        for b in range(B):
            n = int(c.lens[0][b])
            grow = torch.linspace(0.01, 4.0, n, device=DEV, dtype=torch.float64)
            t = np.arange(n)
            at = torch.tensor(c.tables[0].cpu().numpy()[b, t // 64] * 64 + t % 64, device=DEV)
            f = (grow / s.kscale[at].double()).float()
            s.kscale[at] = s.kscale[at] * f
            c.rows[0][b][0] = c.rows[0][b][0] * f.double()[None, :, None]
        c.check(c.run())


def test_many_workers_share_few_tokens_and_one_shares_many(tq):
    """More workers than stages, and long runs of empty sequences between those that hold something."""
    lens = np.zeros(300, int)
    lens[[3, 170, 171, 299]] = [1, 500, 16, 64]
    c = Case(tq, 128, 2, 2, 300, [((4, 4), 16, 500)], seed=9, lens=[lens])
    out = c.check(c.run())
    assert (out[4:170] == 0).all()


def test_captured_and_replayed_on_other_lengths(tq):
    B, H, gqa, d = 4, 2, 4, 128
    segs = [((3, 4), 32, 500), ("fp16", None, 64)]
    a, b = (Case(tq, d, H, gqa, B, segs, seed=s) for s in (5, 6))
    ws, out = a.workspace(), torch.zeros(B, H * gqa, d, dtype=torch.float16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a.run(ws, out)
    side.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that share a workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a.run(ws, out)
        graphs.append(graph)
    want = [a.run().clone(), b.run().clone()]
    for step in range(4):
        if step == 2:  # the other case's numbers in the captured buffers
            for x, y in zip(a.parts, b.parts):
                for name in ("kcodes", "vcodes", "kscale", "vscale", "k", "v"):
                    if hasattr(x, name):
                        getattr(x, name).copy_(getattr(y, name))
            for x, y in zip([a.q] + a.lens + [t for t in a.tables if t is not None], [b.q] + b.lens + [t for t in b.tables if t is not None]):
                x.copy_(y)
        graphs[step & 1].replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want[step // 2]))


@pytest.mark.parametrize("raw", [False, True])
def test_on_a_stream_that_is_not_current(tq, raw):
    c = Case(tq, 128, 2, 4, 3, [((3, 3), 64, 300), ("fp16", 32, 40)], seed=12)
    ws, place = c.workspace(), torch.zeros_like(c.q, memory_format=torch.contiguous_format)
    want = c.run(ws).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with Behind():
        c.run(ws, place, stream=side.cuda_stream if raw else side)
        side.synchronize()
    assert torch.equal(bits(place), bits(want))


def test_page_tables_and_drafts_on_a_stream_that_is_not_current(tq):
    import test_gpu_pages as pages
    import test_gpu_verify as verify
    table, length, count, free, n_free = pages.pages_case(9, 16, 12, 200, 60, 40, 3, False)
    x = verify.verify_case(4, 5, 999, torch.float32, "tree", True, 0, 3)
    want = verify.reference
    side = torch.cuda.Stream()
    args = [i32(a) for a in (table, length, count, free, [n_free])]
    again = [a.clone() for a in args]
    one = tq.tq_page_tables(*args, 16, 40)
    two = tq.tq_verify(x[0], x[3], x[5], draft=x[4], parents=x[2])
    tq.tq_page_release(args[0], args[1], i32(length), args[3], args[4], 16)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # (memory of both streams is cached from here on)
        [torch.empty(9 * 40, dtype=torch.int32, device=DEV) for _ in range(8)]
    keep = i32(length)
    with Behind():
        got = tq.tq_page_tables(*again, 16, 40, stream=side)
        sec = tq.tq_verify(x[0], x[3], x[5], draft=x[4], parents=x[2], stream=side)
        tq.tq_page_release(again[0], again[1], keep, again[3], again[4], 16, stream=side)
        side.synchronize()
    assert want and all(torch.equal(a, b) for a, b in zip((*one, *two, *args), (*got, *sec, *again)))


def test_table_without_entries(tq):
    """A table of no columns is a table: no sequence holds a token, however many pages the pool has."""
    B, H, d = 4, 2, 128
    c = Case(tq, d, H, 2, B, [((4, 4), 64, 64)], seed=9, lens=[[64, 1, 0, 64]])
    c.tables = [t[:, :0] for t in c.tables]
    out = c.run(c.workspace())
    assert (out == 0).all()


@pytest.mark.parametrize("d,kind", [(128, (4, 4)), (64, (3, 3)), (128, "fp16")])
def test_no_wait_to_run_out(tq, d, kind):
    """The limit of the waits of other calls' kernels has no part in this one: nothing in it polls for another part."""
    c = Case(tq, d, 2, 4, 3, [(kind, 64, 700)], seed=3)
    ws = c.workspace()
    want = c.run(ws).clone()
    out = torch.full_like(want, float("nan"))
    try:
        tq.tq_set_decode_wait_polls(0)
        c.run(ws, out)
        assert tq.tq_decode_error_flag(ws) == 0
    finally:
        tq.tq_set_decode_wait_polls(tq.TQ_WAIT_POLLS_DEFAULT)
    assert torch.equal(bits(out), bits(want))


def test_offsets_past_32_bits(tq):
    """A pool beyond 2^32 bytes, its last pages in use."""
    d, H, P = 128, 16, 64
    n_pages = (1 << 32) // (H * P * d) + 40
    pool = tq.PackedSegment(tq.make_layout(n_pages, H, d, P, 8, 1))
    K, V = (randn(gen(1), 1, H, 2 * P, d, dtype=torch.float16) for _ in range(2))
    last = np.array([[n_pages - 1, n_pages - 2]])
    slots = i32(last.repeat(P, 1) * P + np.tile(np.arange(P), 2))
    rot, _ = base.rotation64(tq, d, 21)
    tq.tq_paged_append(pool, rot, K, V, slots)
    small = tq.PackedSegment(tq.make_layout(2, H, d, P, 8, 1))
    tq.tq_paged_append(small, rot, K, V, i32(np.arange(2 * P)[None]))
    q, n = randn(gen(2), 1, 2 * H, d, dtype=torch.float16), i32([2 * P - 3])
    outs = []
    for s, t in ((pool, last), (small, [[0, 1]])):
        view = tq.layer_view(rot, [s])
        ws = torch.empty(tq.tq_paged_workspace_size(view, 1, H, 2 * H, d), dtype=torch.uint8, device=DEV)
        outs.append(tq.tq_paged_attention(view, q, torch.empty_like(q), ws, [i32(t)], [n]))
    assert torch.equal(bits(outs[0]), bits(outs[1])) and outs[0].abs().sum() > 0


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("d,kb,vb", [(128, 4, 3), (64, 3, 3), (128, None, None)])
def test_paged_cache_serves_sequences_that_come_and_go(tq, d, kb, vb):
    """Prompts enter, tokens are added, sequences end and others take their places and pages: after every step the attention
    is that of the tokens each sequence wrote."""
    from rotated_quantized_kv_gb300.model_cache import PagedCache
    B, H, Hq, P, layers = 3, 2, 8, 16, 2
    g, rng = gen(d), np.random.RandomState(d)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 512))
    c = PagedCache(layers, B, H, Hq, d, n_pages=17, max_pages=8, rope=rope, kbits=kb, vbits=vb, page=P)
    told = [[None] * layers for _ in range(B)]   # K (rotated), V of each sequence, as written
    for step in range(14):
        length = c.length.cpu().numpy()
        if step % 4 == 3:                        # some end, one is cut
            keep = [0 if rng.rand() < 0.4 else int(length[b]) for b in range(B)]
            b = int(rng.randint(B))
            keep[b] = min(keep[b], int(rng.randint(0, length[b] + 1)))
            c.release(i32(keep))
            told = [[None if x is None else [y[:, :keep[b]] for y in x] for x in told[b]] for b in range(B)]
            length = c.length.cpu().numpy()
        S = int(rng.choice([1, 1, 40]))
        n = [min(S, 1 if length[b] else int(rng.randint(1, S + 1))) for b in range(B)]
        slots, positions, granted = c.grow(i32(n), S)
        got = granted.cpu().numpy()
        pages = sum(-(-int(x) // P) for x in c.length.cpu())
        assert int(c.n_free) == 17 - pages and (got <= n).all()
        used = c.table.cpu().numpy()
        used = np.concatenate([used[b, :-(-int(c.length[b]) // P)] for b in range(B)] + [c.free[:int(c.n_free)].cpu().numpy()])
        assert np.array_equal(np.sort(used), np.arange(17))     # every page is somewhere, once
        for l in range(layers):
            K, V = (randn(g, B, S, H, d, dtype=torch.float16).transpose(1, 2) for _ in range(2))
            c.write(l, K, V, slots, positions)
            rot_k = base.rope_ref(K, rope.table, positions, d // 2, False, False, torch.float16)
            back = c.read(l, slots, torch.float32)
            for b in range(B):
                m = int(got[b])
                one = [x[b, :, :m].double() for x in back]
                if kb is None:
                    assert torch.equal(back[0][b, :, :m], rot_k[b, :, :m].float()) and torch.equal(back[1][b, :, :m], V[b, :, :m].float())
                old = told[b][l]
                told[b][l] = one if old is None else [torch.cat([x, y], 1) for x, y in zip(old, one)]
            q = randn(g, B, Hq, d, dtype=torch.float16)
            at = (c.length - 1).clamp(min=0)
            want_q = base.rope_ref(q[:, :, None], rope.table, at[:, None], d // 2, False, False, torch.float16)[:, :, 0]
            out = torch.full_like(q, float("nan"))
            c.attend(l, q, at, out)
            assert torch.equal(q, want_q)
            for b in range(B):
                K64, V64 = told[b][l]
                assert K64.shape[1] == int(c.length[b])
                if not K64.shape[1]:
                    assert (out[b] == 0).all()
                    continue
                x = q[b].double().view(H, -1, d) @ K64.transpose(1, 2) / math.sqrt(d)
                p = torch.softmax(x, -1)
                want = (p @ V64).flatten(0, 1)
                size = (p @ V64.norm(dim=-1, keepdim=True)).flatten(0, 1)
                err = (out[b].double() - want).norm(dim=-1, keepdim=True)
                # (the rows read back in binary32: 2^-20 besides what Case.check counts)
                assert (err <= 2.0**-11 * 1.01 * want.norm(dim=-1, keepdim=True) + (2.0**-11 + 2.0**-12) * size + 1e-6).all()


def test_captured_serving_step(tq):
    """grow, write, attend in one graph, replayed while the sequences grow: the same bits as calls one by one."""
    from rotated_quantized_kv_gb300.model_cache import PagedCache
    B, H, Hq, d = 4, 2, 4, 128
    g = gen(8)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 256))
    caches = [PagedCache(1, B, H, Hq, d, 24, 8, rope, 4, 4, page=16) for _ in range(2)]
    prompt, K0, V0 = i32([3, 40, 0, 16]), *(randn(g, B, H, 40, d, dtype=torch.float16) for _ in range(2))
    for c in caches:
        slots, positions, _ = c.grow(prompt, 40)
        c.write(0, K0, V0, slots, positions)
    n, at = i32([1, 1, 0, 1]), torch.zeros(B, dtype=torch.int32, device=DEV)
    K, V, q = (torch.zeros(B, h, 1, d, dtype=torch.float16, device=DEV) for h in (H, H, Hq))
    out = torch.zeros(B, Hq, d, dtype=torch.float16, device=DEV)

    def step(c, K, V, q, out):
        slots, positions, _ = c.grow(n, 1)
        c.write(0, K, V, slots, positions)
        torch.sub(c.length, 1, out=at)
        c.attend(0, q, at, out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(caches[0], K, V, q[:, :, 0], out)
    for _ in range(20):
        for t in (K, V, q):
            t.copy_(randn(g, *t.shape, dtype=torch.float16))
        q2, out2 = q[:, :, 0].clone(), torch.zeros_like(out)
        step(caches[1], K, V, q2, out2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(out2)) and torch.equal(caches[0].length, caches[1].length)
    assert caches[0].length.tolist() == [23, 60, 0, 36]


def test_drafted_verified_committed(tq):
    """A speculative step from the drafts to the cache: the accepted path is what the cache holds behind it."""
    from rotated_quantized_kv_gb300.model_cache import SpeculativeCache
    B, H, Hq, d, N, V = 3, 2, 4, 64, 6, 40
    g, rng = gen(2), np.random.RandomState(2)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 128))
    c = SpeculativeCache(1, B, H, Hq, d, 64, rope, 8, 8, sinks=16, drafts=N)
    n0 = i32([5, 20, 17])
    K, Vv = (randn(g, B, H, 20, d, dtype=torch.float16) for _ in range(2))
    c.prefill(0, K, Vv, n0, torch.arange(20, dtype=torch.int32, device=DEV))
    c.advance(n0)
    for _ in range(3):
        parents = i32([[rng.randint(-1, i) if i else -1 for i in range(N)] for _ in range(B)])
        qkv = randn(g, B, N, Hq + 2 * H, d, dtype=torch.float16)
        q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H].transpose(1, 2), qkv[:, :, Hq + H:].transpose(1, 2)
        before = c.length.clone()
        out = torch.empty(B, N, Hq, d, dtype=torch.float16, device=DEV)
        c.attend(0, q, k, v, before[:, None] + torch.arange(N, dtype=torch.int32, device=DEV), out, mask=tq.tree_mask(parents))
        target = torch.softmax(3 * torch.randn(B, N + 1, V, generator=g, device=DEV), -1)
        tokens = torch.randint(0, V, (B, N), generator=g, device=DEV, dtype=torch.int32)
        target[0, :, :] = 1e-3
        target[0].scatter_(1, tokens[:1].repeat(N + 1, 1).long(), 1.0)  # one sequence accepts all it can
        uniform = 0.98 * torch.rand(B, N + 1, generator=g, device=DEV)
        accepted, count, token = c.verify(tokens, target, uniform, parents=parents)
        c.commit(0, k, v, accepted, count)
        c.advance(count)
        assert torch.equal(c.length, before + count) and int(count[0]) > 0 and (token >= 0).all()
        got = c.read(0, before, N, torch.float32)
        for b in range(B):
            path = accepted[b, :int(count[b])].tolist()
            walk = [-1] + path
            assert all(int(parents[b, j]) == i for i, j in zip(walk, path))
            for x, y in zip(got, (k, v)):
                rows = y[b][:, path].float()
                err = (x[b, :, :len(path)] - rows).norm(dim=-1)
                assert (err <= 0.03 * rows.norm(dim=-1) + 1e-3).all()     # 8 bits: 2^-8 of the largest coordinate each
                assert (x[b, :, len(path):] == 0).all()
