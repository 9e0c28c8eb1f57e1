"""The serving calls as they are used together, and where calls meet: large
ragged writes and reads, streams, captured graphs, bounded waits."""
import ctypes

import numpy as np
import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import DEV, bits, gen, randn

pytestmark = pytest.mark.gpu
MIXED = [1, 2, 3, 4, 5, 6, 7, 8]


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def records(seg, which, b):
    """Views [capacity][bytes] of sequence b's records, head by head."""
    L = seg.layout
    codes, widths = (seg.kcodes, L.kbits) if which == "k" else (seg.vcodes, L.vbits)
    H, d, cap = L.n_heads, L.head_dim, L.capacity
    per = [d * widths[h] // 8 * cap for h in range(H)]
    block = codes[b * sum(per):(b + 1) * sum(per)]
    at = np.concatenate([[0], np.cumsum(per)])
    return [block[at[h]:at[h + 1]].view(cap, -1) for h in range(H)]


def scales(seg, which, b):
    L = seg.layout
    s = seg.kscale if which == "k" else seg.vscale
    return s[:L.batch * L.n_heads * L.capacity].view(L.batch, L.n_heads, L.capacity)[b]


# H, kbits, vbits, B, source rows, rows, gather, pair layout (None: no positions), rotary dims, law, element offset
MANY = [
    (8, MIXED, MIXED[::-1], 1, 1100, 1100, False, 0, 128, 0, 0),
    (8, [4] * 8, [4] * 8, 4, 300, 290, True, 1, 64, 0, 0),
    (4, [3] * 4, [5] * 4, 3, 760, 750, True, 0, 40, 1, 0),
    (8, [2] * 8, [1] * 8, 2, 600, 577, False, 1, 36, 0, 0),
    (8, [6] * 8, [8, 7] * 4, 2, 600, 600, False, None, 0, 0, 0),
    (8, [4] * 8, [3] * 8, 2, 600, 600, False, 0, 128, 0, 1),     # rows not 16-byte aligned
    (1, [8], [2], 1, 8300, 8300, False, 1, 128, 0, 0),
]


@pytest.mark.parametrize("H,kb,vb,B,S,n,gather,layout,r,law,off", MANY)
def test_large_append_is_compress(tq, H, kb, vb, B, S, n, gather, layout, r, law, off):
    d, g, rng = 128, gen(S + n), np.random.RandomState(n)
    cap = 16 * (n // 16 + 4)
    kv = randn(g, 2 * B * S * H * d + off, dtype=torch.float16)[off:].view(2, B, S, H, d)
    K, V = (2 * kv[0]).transpose(1, 2) if not off else kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    count = torch.tensor([n] + [rng.randint(n // 2, n + 3) for _ in range(B - 1)], dtype=torch.int32, device=DEV)
    first = torch.tensor([rng.randint(0, cap - n + 1) for _ in range(B)], dtype=torch.int32, device=DEV)
    if B > 1:
        first[-1] = 40  # the last rows do not fit
    index = torch.tensor(rng.randint(-1, S + 1, size=(B, n)), dtype=torch.int32, device=DEV) if gather else None
    rope = pos = None
    want_k = K
    if layout is not None:
        rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(r), 500), layout)
        pos = torch.randint(-1, 502, (B, S), generator=g, device=DEV, dtype=torch.int32)
        want_k = base.rope_ref(K, rope.table, pos, r // 2, layout == 1, False, torch.float16)
    rot = tq.tq_make_rotation(d, 9)
    seg = base.filled_segment(tq, B, H, d, cap, kb, vb, law)
    before = {x: getattr(seg, x).clone() for x in base.BUFS}
    tq.tq_append(seg, rot, K, V, first, n_new=count, index=index, n_max=n, rope=rope, positions=pos)
    old = base.filled_segment(tq, B, H, d, cap, kb, vb, law)
    for x in base.BUFS:
        assert torch.equal(getattr(old, x).view(torch.uint8), before[x].view(torch.uint8))
    rows = torch.arange(n, device=DEV)
    for b in range(B):
        src = index[b].long() if gather else rows
        at = rows + int(first[b])
        ok = (rows < min(int(count[b]), n)) & (src >= 0) & (src < S) & (at < cap)
        one = tq.PackedSegment(tq.make_layout(1, H, d, cap, kb, vb, value_law=law))
        take = src[ok]
        tq.tq_compress(one, rot, want_k[b:b + 1][:, :, take].contiguous(), V[b:b + 1][:, :, take].contiguous(), 0)
        hit = at[ok]
        rest = torch.ones(cap, dtype=torch.bool, device=DEV)
        rest[hit] = False
        for which in "kv":
            for h in range(H):
                got, new, was = records(seg, which, b)[h], records(one, which, 0)[h], records(old, which, b)[h]
                assert torch.equal(got[hit], new[:len(hit)]), (which, b, h)
                assert torch.equal(got[rest], was[rest]), (which, b, h)
                x, y, z = scales(seg, which, b)[h], scales(one, which, 0)[h], scales(old, which, b)[h]
                assert torch.equal(bits(x[hit]), bits(y[:len(hit)])) and torch.equal(bits(x[rest]), bits(z[rest]))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,B,n,law,token_major,off,rotate", [
    (128, 1, 900, 0, False, 0, True), (128, 3, 333, 1, True, 0, True), (128, 2, 500, 0, True, 1, True),
    (128, 2, 450, 0, False, 0, False), (64, 1, 1701, 0, False, 0, True), (64, 3, 555, 0, True, 0, True),
    (64, 2, 900, 0, True, 1, True), (64, 2, 801, 0, False, 0, False)])
def test_large_read_is_dequantize(tq, dtype, d, B, n, law, token_major, off, rotate):
    H, rng = 8, np.random.RandomState(n)
    cap, g = 16 * (n // 16 + 5), gen(n)
    seg = base.random_segment(tq, g, B, H, d, cap, MIXED, MIXED[::-1], law)
    rot = tq.tq_make_rotation(d, 4)
    count = torch.tensor([n] + [rng.randint(n // 2, n + 3) for _ in range(B - 1)], dtype=torch.int32, device=DEV)
    first = torch.tensor([rng.randint(0, cap - n + 1) for _ in range(B)], dtype=torch.int32, device=DEV)
    if B > 1:
        first[-1] = 60
        first[0] = -3
    shape = (2, B, n, H, d) if token_major else (2, B, H, n, d)
    flat = torch.full((int(np.prod(shape)) + off,), 7.0, dtype=dtype, device=DEV)
    out = [x.transpose(1, 2) if token_major else x for x in flat[off:].view(shape)]
    tq.tq_read(seg, rot if rotate else None, first, n, n_read=count, out=out)
    four = tq.tq_dequantize(seg, 0, cap, rot, rotated=not rotate, original=rotate)
    whole = four[2:] if rotate else four[:2]
    for b in range(B):
        m = min(int(count[b]), n)
        for x, w in zip(out, whole):
            for j0, j1, keep in ((0, m, True), (m, n, False)):
                at = torch.arange(j0, j1, device=DEV) + int(first[b])
                ok = (at >= 0) & (at < cap) & keep
                got = x[b][:, j0:j1]
                assert torch.equal(bits(got[:, ok].contiguous()), bits(w[b][:, at[ok]].to(dtype)))
                assert (got[:, ~ok] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_large_calls_captured(tq, d):
    """Several launches a call, replayed on other rows and lengths, between other work of the stream."""
    B, H, S, cap, g = 2, 8, 1200, 1216, gen(d)
    kb, vb = [3, 4] * 4, [2, 4] * 4
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), cap))
    rot = tq.tq_make_rotation(d, 5)
    src, kv = torch.zeros(2, B, H, S, d, dtype=torch.float16, device=DEV), torch.zeros(2, B, H, S, d, dtype=torch.float16, device=DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)
    n, first = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    segs = [base.filled_segment(tq, B, H, d, cap, kb, vb) for _ in range(2)]
    outs = [[torch.zeros(B, H, S, d, dtype=torch.float16, device=DEV) for _ in range(2)] for _ in range(2)]

    def calls(i):
        kv.copy_(src)  # a kernel before, which writes what the call reads
        tq.tq_append(segs[i], rot, kv[0], kv[1], first, n_new=n, rope=rope, positions=pos)
        tq.tq_read(segs[i], rot, first, S, n_read=n, out=outs[i])
        kv.zero_()     # and one behind, which overwrites it

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls(0)
    torch.cuda.synchronize()
    for lens, at in (([1200, 1200], [0, 16]), ([700, 1133], [333, 0])):
        src.copy_(randn(g, *src.shape, dtype=torch.float16))
        n.copy_(torch.tensor(lens)), first.copy_(torch.tensor(at))
        torch.cuda.synchronize()
        graph.replay()
        calls(1)
        torch.cuda.synchronize()
        for name in base.BUFS:
            assert torch.equal(getattr(segs[0], name).view(torch.uint8), getattr(segs[1], name).view(torch.uint8)), name
        for x, y in zip(*outs):
            assert torch.equal(bits(x), bits(y)) and bool((x != 0).any())


# ------------------------------------------------------------------ the loop of a server
@pytest.mark.parametrize("d,kb,vb", [(128, 3, 3), (64, 4, 2), (256, 4, 4)])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(tq, d, kb, vb, captured):
    from rotated_quantized_kv_gb300.model_cache import SpeculativeCache
    L, B, H, Hq, N, sinks, cap, S = 2, 3, 2, 8, 7, 16, 96, 40
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(d), 256))
    g, rng = gen(d), np.random.RandomState(d)
    c = SpeculativeCache(L, B, H, Hq, d, cap, rope, kb, vb, sinks, N)
    n0 = torch.tensor([5, 40, 16], dtype=torch.int32, device=DEV)
    kept = [[[], [], []] for _ in range(L)]  # rotated fp16 rows of a sequence: [2][H][t][d]
    for l in range(L):
        K, V = (randn(g, B, H, S, d, dtype=torch.float16) for _ in range(2))
        pos = torch.arange(S, dtype=torch.int32, device=DEV)
        c.prefill(l, K, V, n0, pos)
        turned = base.rope_ref(K, rope.table, pos.expand(B, S), d // 2, False, False, torch.float16)
        for b in range(B):
            kept[l][b].append(torch.stack([turned[b], V[b]])[:, :, :int(n0[b])])
    c.advance(n0)

    qkv = torch.zeros(L, B, N, Hq + 2 * H, d, dtype=torch.float16, device=DEV)
    out = torch.zeros(L, B, N, Hq, d, dtype=torch.float16, device=DEV)
    depth, mask = torch.zeros(B, N, dtype=torch.int32, device=DEV), torch.zeros(B, N, 1, dtype=torch.int32, device=DEV)
    path, took = torch.zeros(B, N, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        at = c.length[:, None] + depth
        for l in range(L):
            x = qkv[l].clone()
            q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + H].transpose(1, 2), x[:, :, Hq + H:].transpose(1, 2)
            c.attend(l, q, k, v, at, out[l], mask=mask)
            c.commit(l, k, v, path, took)
        c.advance(took)

    run = step
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # accepts nothing: took is zero
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        torch.cuda.synchronize()
        run = graph.replay
    for _ in range(4):
        qkv.copy_(randn(g, *qkv.shape, dtype=torch.float16))
        par = np.array([[-1] + [rng.randint(0, i) for i in range(1, N)] for _ in range(B)])
        dep = np.zeros((B, N), int)
        see = np.zeros((B, N, N), bool)
        for b in range(B):
            for i in range(N):
                if par[b, i] >= 0:
                    see[b, i], dep[b, i] = see[b, par[b, i]], dep[b, par[b, i]] + 1
                see[b, i, i] = True
        mask.copy_(tq.tree_mask(torch.tensor(par, device=DEV)))
        assert torch.equal(mask, base.mask_words(see))
        depth.copy_(torch.tensor(dep))
        ends = [rng.randint(0, N) for _ in range(B)]
        walks = [np.flatnonzero(see[b, ends[b]])[:rng.randint(0, N + 1)] for b in range(B)]
        took.copy_(torch.tensor([len(w) for w in walks]))
        path.zero_()
        for b, w in enumerate(walks):
            path[b, :len(w)] = torch.tensor(w, dtype=torch.int32)
        length = c.length.clone()
        lens = [c.head_len.clone(), c.body_len.clone()]
        stored = []
        for l in range(L):
            s, p = tq.Fp16Segment(B, H, d, sinks, n_tokens=sinks, k=c.head[l].k.clone(), v=c.head[l].v.clone()), c.body[l]
            t = tq.PackedSegment(p.layout, n_tokens=cap)
            for name in base.BUFS:
                getattr(t, name).copy_(getattr(p, name))
            stored.append([s, t])
        run()
        torch.cuda.synchronize()
        assert tq.tq_decode_error_flag(c.workspace) == 0
        at = length[:, None] + depth
        for l in range(L):
            x = qkv[l].transpose(1, 2)  # [B][heads][N][d]
            turned = base.rope_ref(x[:, :Hq + H], rope.table, at, d // 2, False, False, torch.float16)
            q, k, v = turned[:, :Hq].transpose(1, 2), turned[:, Hq:], x[:, Hq + H:]
            _, R = base.rotation64(tq, d, 42 + l)
            base.check_tree(out[l], base.tree_ref(tq, q, k, v, see, stored[l], lens, R))
            for b, w in enumerate(walks):
                if len(w):
                    kept[l][b].append(torch.stack([k[b], v[b]])[:, :, torch.tensor(w, device=DEV)])
    # the caches hold what was accepted, each row as the library compresses it
    for l in range(L):
        for b in range(B):
            rows = torch.cat(kept[l][b], 2)
            n = rows.shape[2]
            assert int(c.length[b]) == n and int(c.head_len[b]) == min(n, sinks) and int(c.body_len[b]) == max(n - sinks, 0)
            m = min(n, sinks)
            assert torch.equal(bits(c.head[l].k[b, :, :m]), bits(rows[0][:, :m]))
            assert torch.equal(bits(c.head[l].v[b, :, :m]), bits(rows[1][:, :m]))
            if n > sinks:
                one = tq.PackedSegment(tq.make_layout(1, H, d, cap, [kb] * H, [vb] * H))
                tq.tq_compress(one, c.rot[l], rows[0][None, :, sinks:].contiguous(), rows[1][None, :, sinks:].contiguous(), 0)
                for which in "kv":
                    for h in range(H):
                        assert torch.equal(records(c.body[l], which, b)[h][:n - sinks], records(one, which, 0)[h][:n - sinks])
                        assert torch.equal(bits(scales(c.body[l], which, b)[h][:n - sinks]), bits(scales(one, which, 0)[h][:n - sinks]))
    # and back: sinks verbatim, packed rows as a read of the segment gives them
    first = torch.tensor([0, 10, 14], dtype=torch.int32, device=DEV)
    got = c.read(0, first, 50)
    packed = tq.tq_read(c.body[0], c.rot[0], c.zero, cap)
    for b in range(B):
        for i in range(2):
            for j in range(50):
                t = int(first[b]) + j
                if t >= int(c.length[b]):
                    assert (got[i][b, :, j] == 0).all()
                elif t < sinks:
                    assert torch.equal(got[i][b, :, j], (c.head[0].k, c.head[0].v)[i][b, :, t])
                else:
                    assert torch.equal(got[i][b, :, j], packed[i][b, :, t - sinks])


def small_tree(tq, seed, d=128, B=2, N=5, scale=1.0, segs=(((3, 4), 700), ("fp16", 60))):
    q, k, v, parts, lens, rng = base.tree_case(tq, d, 2, 4, B, N, list(segs), False, seed=seed, scale=scale)
    see = base.random_tree(rng, B, N)
    return q, k, v, parts, see, base.mask_words(see)


def clean(parts):
    for s in parts:
        if s.kind == 0:
            s.kscale.nan_to_num_(0.0)
            s.vscale.nan_to_num_(0.0)
    return parts


@pytest.mark.parametrize("d", [64, 128, 256])
def test_tree_on_two_streams(tq, d):
    """Two calls at once, each with its workspace, on streams of their own."""
    cases = [small_tree(tq, s, d) for s in (1, 2)]
    want = [base.run_tree(tq, *c[:4], mask=c[5]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces, outs = [], [[], []]
    for c in cases:
        lv = tq.layer_view(tq.tq_make_rotation(d, 21), c[3])
        spaces.append(torch.empty(tq.tq_tree_workspace_size(lv, 2, 2, 8, 5, d), dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    for _ in range(10):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(base.run_tree(tq, *c[:4], mask=c[5], stream=streams[i].cuda_stream, ws=spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(bits(o), bits(want[i]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("polls", [0, 1])
def test_tree_wait_that_runs_out(tq, d, polls):
    q, k, v, parts, see, mask = small_tree(tq, 5, d, segs=(((3, 4), 1500), ((8, 1), 300), ("fp16", 200)))
    want = base.run_tree(tq, q, k, v, parts, mask)
    lv = tq.layer_view(tq.tq_make_rotation(d, 21), parts)
    ws = torch.empty(tq.tq_tree_workspace_size(lv, 2, 2, 8, 5, d), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(want)
    try:
        tq.tq_set_decode_wait_polls(polls)
        tq.tq_tree_attention(lv, q, k, v, out, ws, mask=mask)
        flag = tq.tq_decode_error_flag(ws)
    finally:
        tq.tq_set_decode_wait_polls(tq.TQ_WAIT_POLLS_DEFAULT)
    if polls == 0:
        f = ctypes.c_int()
        assert flag != 0 and tq._lib.tq_decode_error_flag(ws.data_ptr(), ctypes.byref(f), None) == tq.TQ_ERR_TIMEOUT
    again = base.run_tree(tq, q, k, v, parts, mask, ws=ws)  # the next call clears the flag
    assert torch.equal(bits(again), bits(want))


@pytest.mark.parametrize("d,N,gqa,kb,vb", [
    (128, 16, 4, 8, 8), (128, 16, 4, 8, 5), (128, 16, 4, 7, 5), (128, 16, 4, 4, 4), (128, 16, 4, 2, 6), (128, 5, 4, 5, 7),
    (128, 4, 4, 8, 6), (64, 16, 4, 8, 8), (64, 8, 4, 6, 5), (64, 3, 2, 3, 7)])
def test_tree_over_many_tiles(tq, d, N, gqa, kb, vb):
    """Several tiles a worker, with every depth of the record ring and both forms of the weights."""
    B, H, n = 2, 8, 5000
    q, k, v, parts, lens, rng = base.tree_case(tq, d, H, gqa, B, N, [((kb, vb), n), ("fp16", 128)], False, seed=kb + 9 * vb)
    out = base.run_tree(tq, q, k, v, parts)
    _, R = base.rotation64(tq, d, 21)
    ref = base.tree_ref(tq, q, k, v, None, clean(parts), [None] * 2, R)
    base.check_tree(out, ref)
    if vb >= 6:
        # the levels' half steps alone (and the result's): sqrt(2 / 3) of a half step, where the
        # weights' half steps would make it sqrt(3 / 3); a tenth more for the fewer samples
        assert (out.double() - ref[0]).norm() <= 1.1 * (2 / 3) ** 0.5 * 2.0**-11 * ref[0].norm()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_tree_of_one_unseen_draft_is_decode(tq, d):
    """A draft that does not see itself attends to the cache alone: what a decode step computes."""
    B, H, Hq = 2, 2, 8
    q, k, v, parts, _, _ = small_tree(tq, 9, d, N=1)
    clean(parts)
    none = torch.zeros(B, 1, 1, dtype=torch.int32, device=DEV)
    got = base.run_tree(tq, q, k, v, parts, none)
    lv = tq.layer_view(tq.tq_make_rotation(d, 21), parts)
    want = torch.empty(1, B, Hq, d, device=DEV)
    ws = torch.empty(tq.tq_decode_workspace_size([lv], B, H, Hq, d), dtype=torch.uint8, device=DEV)
    tq.tq_decode_attention([lv], q[:, 0][None].contiguous(), want, ws, H)
    _, R = base.rotation64(tq, d, 21)
    ref = base.tree_ref(tq, q, k, v, np.zeros((B, 1, 1), bool), parts, [None] * len(parts), R)
    base.check_tree(got, ref)
    # the decode path's bound is 2e-3 of the reach of the values (its operands are fp16 throughout)
    err = (want[0].double() - ref[0][:, 0]).norm(dim=-1)
    assert bool((err <= 2e-3 * ref[1][:, 0] * (1 + ref[2][:, 0])).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 12.0, 60.0])
def test_tree_flat_and_sharp_weights(tq, d, scale):
    """Weights that are all alike, and scores of hundreds that keep growing along the cache."""
    q, k, v, parts, see, mask = small_tree(tq, 31, d, N=9, scale=scale, segs=(((4, 4), 1500), ("fp16", 260)))
    ramp = torch.linspace(0.05, 1.0, parts[0].layout.capacity, device=DEV)
    n = parts[0].layout.batch * parts[0].layout.n_heads * parts[0].layout.capacity
    parts[0].kscale[:n] *= ramp.repeat(n // len(ramp))
    out = base.run_tree(tq, q, k, v, parts, mask)
    _, R = base.rotation64(tq, d, 21)
    base.check_tree(out, base.tree_ref(tq, q, k, v, see, clean(parts), [None] * 2, R))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(tq, d, bad):
    """A query of another row, and a draft that the row does not see, may hold anything."""
    B, N = 2, 6
    q, k, v, parts, see, _ = small_tree(tq, 77, d, B, N)
    see[:] = np.eye(N, dtype=bool)  # no draft sees another
    mask = base.mask_words(see)
    want = base.run_tree(tq, q, k, v, parts, mask)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[0, 2], k2[0, :, 2], v2[0, :, 2] = bad, bad, bad
    v2[1, :, 4] = bad
    got = base.run_tree(tq, q2, k2, v2, parts, mask)
    rows = torch.ones(B, N, dtype=torch.bool, device=DEV)
    rows[0, 2] = rows[1, 4] = False
    assert torch.equal(bits(got[rows]), bits(want[rows]))
    assert not torch.isfinite(got[0, 2].float()).any()
