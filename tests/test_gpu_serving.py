"""Serving calls on the GPU against plain implementations in 64 bits, and
against the library's own compression, bit for bit."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF_STEP = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def bits(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------------ rotary positions
def rope_ref(x, table, pos, half, inter, inverse, out_dtype):
    """Elementwise binary32 products and sums, rounded once; rows of positions
    outside the table unchanged."""
    ok = (pos >= 0) & (pos < table.shape[0])
    cs = table[pos.clamp(0, table.shape[0] - 1).long()][:, None]
    c, s = cs[..., 0, :], cs[..., 1, :]
    s = -s if inverse else s
    z = x.to(table.dtype).clone()
    i = slice(0, 2 * half, 2) if inter else slice(0, half)
    j = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    a, b = z[..., i].clone(), z[..., j].clone()
    z[..., i] = a * c - b * s
    z[..., j] = b * c + a * s
    return torch.where(ok[:, None, :, None], z.to(out_dtype), x.to(out_dtype))


ROPE = [  # dtype, B, T, heads, d, rotary_dim, interleaved, token-major, element offset
    (torch.float16, 1, 1, (32, 8), 128, 128, False, True, 0),
    (torch.float16, 2, 37, (8, 2), 128, 128, True, True, 0),
    (torch.float16, 3, 129, (5,), 256, 96, False, False, 0),
    (torch.float16, 2, 17, (4, 4, 1), 64, 64, False, True, 1),     # rows not 16-byte aligned
    (torch.bfloat16, 3, 21, (6, 2), 80, 20, True, False, 0),       # pairs that fill no vector
    (torch.bfloat16, 1, 1025, (4, 1), 128, 32, True, True, 0),
    (torch.bfloat16, 2, 9, (3,), 64, 48, False, False, 0),
    (torch.float32, 2, 65, (4, 2), 64, 64, False, True, 0),
    (torch.float32, 1, 3, (2, 2, 2, 2), 12, 8, True, False, 0),
    (torch.float32, 2, 5, (3,), 7, 6, False, False, 0),
    (torch.float16, 1, 3, (2,), 1024, 1024, True, False, 0),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype,B,T,heads,d,r,inter,token_major,off", ROPE)
def test_rope(tq, dtype, B, T, heads, d, r, inter, token_major, off, inverse):
    g = gen(B * 1000 + T)
    n_pos = 500
    spec = tq.tq_make_rope(r, 10000.0, tq.TQ_ROPE_SCALE_TURNS, 4.0, 64.0, 8.0, 1.0, amplitude=1.25)
    table = tq.tq_rope_table(spec, n_pos)
    rope = tq.Rope(table, tq.TQ_ROPE_INTERLEAVED if inter else tq.TQ_ROPE_HALF)
    pos = torch.randint(-2, n_pos + 2, (B, T), generator=g, device=DEV, dtype=torch.int32)
    H = sum(heads)
    if token_major:
        buf = randn(g, B * T * H * d + off, dtype=dtype)[off:].view(B, T, H, d).transpose(1, 2)
    else:
        buf = randn(g, B * T * H * d + off, dtype=dtype)[off:].view(B, H, T, d)
    xs = list(torch.split(buf, heads, 1))
    keep = buf.clone()
    out = [torch.full((B, h, T, d), 7.0, dtype=dtype, device=DEV) for h in heads]
    got = tq.tq_rope(rope, pos, xs, out=out, inverse=inverse)
    assert torch.equal(bits(buf), bits(keep))
    for x, y in zip(xs, got):
        ref = rope_ref(x, table, pos, r // 2, inter, inverse, dtype)
        assert torch.equal(bits(y), bits(ref))
        # 64 bits: three binary32 roundings of terms of at most |a| + |b| times the amplitude, one of the type
        ref = rope_ref(x, table.double(), pos, r // 2, inter, inverse, torch.float64)
        size = x.double().abs().amax(-1, keepdim=True) * 2 * 1.25
        assert ((y.double() - ref).abs() <= HALF_STEP[dtype] * ref.abs() * 1.001 + 3 * 2.0**-24 * size).all()
    # in place, one tensor, positions of one row for all sequences
    x = xs[0].clone()
    ref = rope_ref(x, table, pos[:1].expand(B, T), r // 2, inter, inverse, dtype)
    assert tq.tq_rope(rope, pos[0], x, inverse=inverse) is x
    assert torch.equal(bits(x), bits(ref))


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(tq, inter):
    """inverse = the gradient: against the formula differentiated by autograd in
    64 bits, and against differences of the call itself."""
    g = gen(5)
    table = tq.tq_rope_table(tq.tq_make_rope(32, amplitude=1.5), 40)
    rope = tq.Rope(table, int(inter))
    pos = torch.arange(3, 9, device=DEV, dtype=torch.int32)
    x, dy = randn(g, 2, 3, 6, 48), randn(g, 2, 3, 6, 48)
    dx = tq.tq_rope(rope, pos, dy, out=torch.empty_like(dy), inverse=True)
    xd = x.double().requires_grad_()
    y = rope_ref(xd, table.double(), pos.expand(2, 6), 16, inter, False, torch.float64)
    (y * dy.double()).sum().backward()
    # three roundings of terms of at most 2 max|dy| 1.5
    assert (dx.double() - xd.grad).abs().max() <= 4 * 2.0**-24 * 3 * dy.abs().max()
    # the call is linear: its difference along v is its value at v
    v = randn(g, 2, 3, 6, 48)
    f = lambda z: (tq.tq_rope(rope, pos, z, out=torch.empty_like(z)).double() * dy.double()).sum()  # noqa: E731
    # each of the 1728 terms of either sum is off by at most 4 roundings of about 3 |x| 2 |dy|
    assert abs((f(x + v) - f(x - v)) / 2 - (dx.double() * v.double()).sum()) <= 1728 * 4 * 2.0**-24 * 3 * 25


def test_rope_table_of_far_positions(tq):
    for first, base, amp in ((0, 10000.0, 1.0), (1 << 20, 1e6, 1.1), (2**31 - 1 - 64, 10000.0, 0.7)):
        spec = tq.tq_make_rope(64, base, amplitude=amp)
        t = tq.tq_rope_table(spec, 64, first).double().cpu().numpy()
        w = tq.tq_rope_frequencies(spec).astype(np.longdouble)
        a = (np.arange(64, dtype=np.longdouble) + first)[:, None] * w
        # binary64 angle: 2^-53 of itself; cosine and product a few 2^-53; one binary32 rounding
        tol = amp * (2.0**-24 + float(a.max()) * 2.0**-53 + 2.0**-50)
        assert np.abs(t[:, 0] - amp * np.cos(a)).max() <= tol
        assert np.abs(t[:, 1] - amp * np.sin(a)).max() <= tol


# ------------------------------------------------------------------ ragged writes
def filled_segment(tq, B, H, d, cap, kb, vb, value_law=0):
    seg = tq.PackedSegment(tq.make_layout(B, H, d, cap, kb, vb, value_law=value_law))
    for t in (seg.kcodes, seg.vcodes):
        t.fill_(0xA5)
    for t in (seg.kscale, seg.vscale):
        t.fill_(-3.0)
    return seg


BUFS = ("kcodes", "vcodes", "kscale", "vscale")
MIXED = [1, 2, 3, 4, 5, 6, 7, 8]
APPEND = [  # d, H, kbits, vbits, batch, source rows, n_max, gathered, rope layout (None: none), rotary_dim, law, offset
    (128, 8, MIXED, MIXED[::-1], 3, 20, 16, True, None, 0, 0, 0),
    (128, 8, 3, 3, 2, 300, 300, False, 0, 128, 0, 0),
    (128, 4, [4, 4, 8, 2], [4, 3, 4, 5], 2, 67, 40, True, 1, 96, 0, 0),
    (128, 2, [2, 1], [3, 4], 1, 33, 33, False, 0, 64, 1, 0),
    (128, 1, 8, 3, 5, 7, 5, True, 0, 128, 0, 3),                 # rows not 16-byte aligned
    (64, 8, MIXED, MIXED[::-1], 3, 37, 37, False, 0, 64, 0, 0),
    (64, 3, 5, 2, 2, 130, 129, True, 0, 20, 0, 0),
    (256, 2, [3, 8], [4, 1], 2, 50, 41, True, 0, 256, 0, 0),
    (512, 2, [2, 6], [7, 3], 1, 18, 18, False, 1, 512, 0, 0),
    (16, 3, [1, 3, 8], [5, 2, 1], 2, 70, 70, False, 1, 8, 0, 0),
    (32, 2, [7, 2], [3, 6], 2, 9, 9, True, 0, 32, 0, 1),
    (1024, 1, 4, 4, 1, 6, 6, False, 0, 1024, 0, 0),
]


@pytest.mark.parametrize("d,H,kb,vb,B,S,n,gather,layout,r,law,off", APPEND)
def test_append_is_compress_at_each_position(tq, d, H, kb, vb, B, S, n, gather, layout, r, law, off):
    g = gen(d + S)
    cap = 16 * (n // 16 + 3)
    # token-major rows of a wider buffer
    kv = randn(g, 2 * B * S * H * d * 2 + off, dtype=torch.float16)[off:].view(2, B, S, 2 * H, d)[:, :, :, :H]
    K, V = (3 * kv[0]).transpose(1, 2), kv[1].transpose(1, 2)
    K[0, 0, 0] = 0  # an all-zero vector
    rng = np.random.RandomState(S)
    count = torch.tensor([n] + [rng.randint(-1, n + 3) for _ in range(B - 1)], dtype=torch.int32, device=DEV)
    first = torch.tensor([rng.randint(0, cap - n + 1) for _ in range(B)], dtype=torch.int32, device=DEV)
    if B > 1:
        first[-1] = cap - 2  # rows that do not fit are dropped
    index = None
    if gather:
        index = torch.tensor(rng.randint(-1, S + 1, size=(B, n + 2)), dtype=torch.int32, device=DEV)
    rope = pos = None
    want_k = K
    if layout is not None:
        rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(r), 64), layout)
        pos = torch.randint(-1, 66, (B, S), generator=g, device=DEV, dtype=torch.int32)
        want_k = rope_ref(K, rope.table, pos, r // 2, layout == 1, False, torch.float16)
    rot = tq.tq_make_rotation(d, 9)
    seg, want = (filled_segment(tq, B, H, d, cap, kb, vb, law) for _ in range(2))
    tq.tq_append(seg, rot, K, V, first, n_new=count, index=index, n_max=n, rope=rope, positions=pos)
    # one sequence and row at a time through tq_compress
    for b in range(B):
        sub, m = {}, min(int(count[b]), n)
        one = tq.PackedSegment(tq.make_layout(1, H, d, cap, kb, vb, value_law=law))
        for name in BUFS:
            whole = getattr(want, name)
            sub[name] = whole.view(B, -1)[b] if whole.numel() % B == 0 and B > 1 else whole
            setattr(one, name, sub[name])
        for j in range(max(m, 0)):
            s, t = int(index[b, j]) if gather else j, int(first[b]) + j
            if 0 <= s < S and t < cap:
                x = torch.stack([want_k[b:b + 1, :, s:s + 1], V[b:b + 1, :, s:s + 1]])
                tq.tq_compress(one, rot, x[0], x[1], t)
    for name in BUFS:
        x, y = getattr(seg, name), getattr(want, name)
        assert torch.equal(bits(x), bits(y)) if x.dtype == torch.float32 else torch.equal(x, y), name


def test_append_matches_the_oracle(tq):
    """The stored codes against the CPU oracle's compression of the same rows."""
    from oracle import oracle as O
    B, H, d, S, cap = 2, 4, 128, 50, 64
    kb, vb = [4, 3, 8, 1], [4, 2, 3, 6]
    g = gen(77)
    K, V = randn(g, B, H, S, d, dtype=torch.float16), randn(g, B, H, S, d, dtype=torch.float16)
    seg = tq.PackedSegment(tq.make_layout(B, H, d, cap, kb, vb))
    tq.tq_append(seg, tq.tq_make_rotation(d, 42), K, V, torch.zeros(B, dtype=torch.int32, device=DEV))
    ref = O.PackedSegment(B, H, d, cap, kb, vb)
    O.compress(ref, K.cpu().numpy().view(np.uint16), V.cpu().numpy().view(np.uint16), O.signs(d, 42))
    assert np.array_equal(seg.kcodes.cpu().numpy(), ref.kcodes) and np.array_equal(seg.vcodes.cpu().numpy(), ref.vcodes)
    assert np.array_equal(seg.kscale.cpu().numpy(), ref.kscale) and np.array_equal(seg.vscale.cpu().numpy(), ref.vscale)


def test_append_to_fp16_rows(tq):
    B, H, d, S, cap, n = 3, 2, 64, 30, 40, 12
    g = gen(8)
    K, V = (randn(g, B, S, H, d, dtype=torch.float16).transpose(1, 2) for _ in range(2))
    seg = tq.Fp16Segment(B, H, d, cap)
    seg.k.fill_(5.0)
    seg.v.fill_(6.0)
    rope = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(32), 64))
    pos = torch.randint(0, 64, (B, S), generator=g, device=DEV, dtype=torch.int32)
    first = torch.tensor([0, 39, 20], dtype=torch.int32, device=DEV)
    count = torch.tensor([12, 5, 7], dtype=torch.int32, device=DEV)
    index = torch.randint(0, S, (B, n), generator=g, device=DEV, dtype=torch.int32)
    tq.tq_append(seg, None, K, V, first, n_new=count, index=index, rope=rope, positions=pos)
    kr = rope_ref(K, rope.table, pos, 16, False, False, torch.float16)
    want_k, want_v = torch.full_like(seg.k, 5.0), torch.full_like(seg.v, 6.0)
    for b in range(B):
        for j in range(int(count[b])):
            t = int(first[b]) + j
            if t < cap:
                want_k[b, :, t], want_v[b, :, t] = kr[b, :, index[b, j]], V[b, :, index[b, j]]
    assert torch.equal(bits(seg.k), bits(want_k)) and torch.equal(bits(seg.v), bits(want_v))
    # and back, in another type
    got = tq.tq_read(seg, None, first, n, n_read=count, dtype=torch.float32)
    for b in range(B):
        m = min(int(count[b]), cap - int(first[b]))
        assert torch.equal(got[0][b, :, :m], want_k[b, :, int(first[b]):int(first[b]) + m].float())
        assert (got[1][b, :, m:] == 0).all()


# ------------------------------------------------------------------ reading back
def rotation64(tq, d, seed):
    rot = tq.tq_make_rotation(d, seed)
    s = torch.tensor([-1.0 if (rot.sign_bits[i >> 5] >> (i & 31)) & 1 else 1.0 for i in range(d)], dtype=torch.float64)
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return rot, (s[:, None] * h * s[None] / math.sqrt(d)).to(DEV)


def stored64(tq, seg, R):
    """(k, v) that a packed segment stands for, 64 bits [B][H][cap][d] (R None: rotated space)."""
    L = seg.layout
    B, H, d, cap = L.batch, L.n_heads, L.head_dim, L.capacity
    out = []
    for codes, scale, widths, value in ((seg.kcodes, seg.kscale, L.kbits, False), (seg.vcodes, seg.vscale, L.vbits, True)):
        per = d * sum(widths[h] for h in range(H)) // 8 * cap
        data = codes[:B * per].view(B, per)
        at, heads = 0, []
        for h in range(H):
            w = widths[h]
            rec = data[:, at:at + cap * d * w // 8].reshape(B, cap, d * w // 8)
            at += cap * d * w // 8
            stream = (rec[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
            code = (stream.flatten(-2).view(B, cap, d, w).long() << torch.arange(w, device=DEV)).sum(-1)
            if value:
                fit = tq.tq_fit_codebook_sphere(w, 128) if L.value_law else tq.tq_fit_codebook(w)
                y = fit[0].double().to(DEV)[code]
            else:
                y = (2 * code + 1).double() / 2**w - 1
            heads.append(y)
        y = torch.stack(heads, 1) * scale[:B * H * cap].view(B, H, cap, 1).double()
        out.append(y if R is None else y @ R)
    return out


READ = [  # d, H, kbits, vbits, B, cap, n, type, law, token-major
    (128, 8, MIXED, MIXED[::-1], 2, 64, 40, torch.float16, 0, False),
    (128, 3, 3, 3, 1, 400, 333, torch.float32, 0, True),
    (128, 2, [4, 8], [3, 4], 4, 32, 9, torch.bfloat16, 1, False),
    (64, 8, MIXED, MIXED[::-1], 3, 48, 33, torch.float16, 0, True),
    (256, 2, [3, 5], [2, 8], 2, 32, 32, torch.float32, 0, False),
    (512, 1, 6, 4, 1, 16, 7, torch.float16, 0, False),
    (16, 4, [1, 3, 5, 7], [7, 5, 3, 1], 2, 80, 70, torch.float32, 0, False),
    (32, 2, 2, 5, 3, 16, 1, torch.bfloat16, 0, True),
    (1024, 1, 4, 3, 2, 16, 5, torch.float32, 0, False),
]


def random_segment(tq, g, B, H, d, cap, kb, vb, law=0, n=None):
    """Random codes (every byte string is a record) and scales of both small and large size."""
    seg = tq.PackedSegment(tq.make_layout(B, H, d, cap, kb, vb, value_law=law), n_tokens=cap if n is None else n)
    for t in (seg.kcodes, seg.vcodes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in (seg.kscale, seg.vscale):
        t.copy_(torch.exp(randn(g, t.numel())))
    return seg


@pytest.mark.parametrize("d,H,kb,vb,B,cap,n,dtype,law,token_major", READ)
def test_read(tq, d, H, kb, vb, B, cap, n, dtype, law, token_major):
    g = gen(d + n)
    seg = random_segment(tq, g, B, H, d, cap, kb, vb, law)
    rng = np.random.RandomState(n)
    first = torch.tensor([rng.randint(0, cap - n + 1) for _ in range(B)], dtype=torch.int32, device=DEV)
    count = torch.tensor([n + 1] + [rng.randint(-1, n + 1) for _ in range(B - 1)], dtype=torch.int32, device=DEV)
    if B > 1:
        first[-1], count[-1] = cap - 1, n  # rows behind the segment are not read
    rot, R = rotation64(tq, d, 11)
    for use in (rot, None):
        out = [torch.full((B, n, H, d) if token_major else (B, H, n, d), 9.0, dtype=dtype, device=DEV) for _ in "kv"]
        if token_major:
            out = [o.transpose(1, 2) for o in out]
        tq.tq_read(seg, use, first, n, n_read=count, out=out)
        want = stored64(tq, seg, R if use is not None else None)
        for x, y in zip(out, want):
            for b in range(B):
                m = max(0, min(int(count[b]), n, cap - int(first[b])))
                ref = y[b, :, int(first[b]):int(first[b]) + m]
                # level, scale product and log2(d) + 1 butterfly steps in binary32, each relative to the
                # vector's norm at most; then the type's rounding
                tol = HALF_STEP[dtype] * ref.abs() * 1.01 + (math.log2(d) + 4) * 2.0**-24 * ref.norm(dim=-1, keepdim=True)
                assert ((x[b, :, :m].double() - ref).abs() <= tol).all()
                assert (x[b, :, m:] == 9.0).all()
    only = tq.tq_read(seg, rot, first, n, out=[None, torch.zeros(B, H, n, d, dtype=dtype, device=DEV)])
    assert only[0] is None and only[1].abs().sum() > 0


# ------------------------------------------------------------------ tree attention
def tree_ref(tq, q, k, v, mask, segs, lens, R):
    """64 bits: (output [B][N][Hq][d], sum of p ||v|| per row, largest |q| |k| / sqrt(d) of the row's tokens)."""
    B, N, Hq, d = q.shape
    H = k.shape[1]
    g = Hq // H
    out = torch.zeros(B, N, Hq, d, dtype=torch.float64, device=DEV)
    size, reach = torch.zeros(B, N, Hq, dtype=torch.float64, device=DEV), torch.zeros(B, N, Hq, dtype=torch.float64, device=DEV)
    rows = [stored64(tq, s, R) if s.kind == 0 else (s.k.double(), s.v.double()) for s in segs]
    for b in range(B):
        n = [int(l[b]) if l is not None else s.n_tokens for s, l in zip(segs, lens)]
        n = [max(0, min(x, s.n_tokens)) for x, s in zip(n, segs)]
        for i in range(N):
            see = [j for j in range(N) if (mask is None and j <= i) or (mask is not None and mask[b][i][j])]
            for h in range(H):
                ks = torch.cat([r[0][b, h, :m] for r, m in zip(rows, n)] + [k[b, h, see].double()])
                vs = torch.cat([r[1][b, h, :m] for r, m in zip(rows, n)] + [v[b, h, see].double()])
                if not len(ks):
                    continue
                x = q[b, i, h * g:(h + 1) * g].double() @ ks.T / math.sqrt(d)
                p = torch.softmax(x, -1)
                out[b, i, h * g:(h + 1) * g] = p @ vs
                size[b, i, h * g:(h + 1) * g] = p @ vs.norm(dim=-1)
                reach[b, i, h * g:(h + 1) * g] = q[b, i, h * g:(h + 1) * g].double().norm(dim=-1) * ks.norm(dim=-1).max() / math.sqrt(d)
    return out, size, reach


def check_tree(out, ref):
    """fp16 operands: the weights and the value levels round by half a step (2^-11
    of the term) each, the result by half a step; the scores' operands carry
    22 bits, their binary32 sums 2^-20 of |q| |k| at most (256 additions with
    truncation), which moves a weight by that much of itself and its normaliser
    likewise.  In the 2-norm of a row (rotations keep it)."""
    want, size, reach = ref
    err = (out.double() - want).norm(dim=-1)
    tol = 2.0**-11 * want.norm(dim=-1) * 1.01 + (2 * 2.0**-11 + 2 * reach * 2.0**-19) * size + 1e-7
    assert bool(torch.isfinite(out).all())
    assert bool((err <= tol).all()), float((err / tol).max())
    # the roundings are independent of each other and of the values: over the whole output they
    # add up in squares to at most sqrt(3) half steps, and the scores' share
    if want.abs().sum() > 0:
        assert err.norm() <= (3 * 2.0**-11 + 2 * reach.max() * 2.0**-19) * want.norm()


def random_tree(rng, B, N, empty=False):
    see = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N):
            par = rng.randint(-1, i) if i else -1
            if par >= 0:
                see[b, i] = see[b, par]
            see[b, i, i] = True
        if empty:
            see[b, rng.randint(N)] = False
    return see


def mask_words(see):
    B, N, _ = see.shape
    W = -(-N // 32)
    full = np.zeros((B, N, 32 * W), np.uint64)
    full[:, :, :N] = see
    w = (full.reshape(B, N, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.tensor(w.view(np.int32), device=DEV)


def run_tree(tq, q, k, v, segs, mask=None, lens=None, seed=21, stream=None, ws=None):
    B, N, Hq, d = q.shape
    lv = tq.layer_view(tq.tq_make_rotation(d, seed), segs)
    out = torch.full((B, N, Hq, d), float("nan"), dtype=torch.float16, device=DEV)
    if ws is None:
        ws = torch.full((tq.tq_tree_workspace_size(lv, B, k.shape[1], Hq, N, d),), 255, dtype=torch.uint8, device=DEV)
    tq.tq_tree_attention(lv, q, k, v, out, ws, mask=mask, seg_len=lens, stream=stream)
    if stream is None:
        assert tq.tq_decode_error_flag(ws) == 0
    return out


# d, H, gqa, B, N, segments (kind/bits, tokens), ragged, mask
TREE = [
    (128, 2, 4, 1, 8, [("fp16", 128), ((4, 4), 900), ("fp16", 17)], False, "tree"),
    (128, 2, 4, 1, 1, [((3, 3), 1)], False, "chain"),
    (128, 1, 1, 2, 3, [], False, "tree"),                                       # drafts alone
    (128, 1, 2, 2, 5, [((3, 3), 0), ("fp16", 0)], False, "empty"),              # rows that see nothing
    (128, 8, 1, 3, 7, [((MIXED, MIXED[::-1]), 260)], True, "tree"),             # every width
    (128, 8, 2, 2, 33, [((MIXED[::-1], MIXED), 129), ((MIXED, [3] * 8), 127)], True, "empty"),
    (128, 2, 8, 2, 16, [((3, 2), 1000), ((4, 4), 300), ("fp16", 200)], True, "tree"),
    (128, 1, 4, 1, 64, [((2, 1), 2000)], False, "chain"),
    (128, 2, 3, 40, 2, [((3, 3), 130), ("fp16", 9)], True, "tree"),             # many sequences
    (128, 1, 16, 1, 9, [((8, 8), 128)], False, "tree"),
    (128, 1, 1, 1, 256, [((5, 5), 640)], False, "chain"),
    (128, 1, 5, 2, 70, [((6, 7), 100), ("fp16", 128)], True, "tree"),
    (64, 2, 2, 3, 13, [("fp16", 128), ((8, 3), 700), ("fp16", 61)], True, "tree"),
    (64, 8, 1, 2, 4, [((MIXED, MIXED[::-1]), 300)], False, "chain"),
    (64, 1, 8, 2, 21, [((3, 3), 127), ((1, 1), 129)], True, "empty"),
    (256, 2, 2, 2, 6, [((3, 4), 200), ("fp16", 30)], True, "tree"),
    (256, 1, 4, 1, 40, [((8, 8), 150)], False, "chain"),
    (512, 1, 2, 1, 3, [((4, 2), 70), ("fp16", 5)], False, "tree"),
    (16, 2, 4, 2, 5, [((5, 3), 300), ("fp16", 20)], True, "tree"),
    (32, 1, 1, 2, 40, [((2, 6), 90)], True, "tree"),
    (1024, 1, 1, 1, 2, [((3, 3), 40)], False, "chain"),
]


def tree_case(tq, d, H, gqa, B, N, segs, ragged, seed, scale=1.0):
    g, rng = gen(seed), np.random.RandomState(seed)
    parts, lens = [], []
    for kind, n in segs:
        cap = -(-max(n, 1) // 16) * 16
        if kind == "fp16":
            s = tq.Fp16Segment(B, H, d, cap, n_tokens=n, k=randn(g, B, H, cap, d, dtype=torch.float16),
                               v=randn(g, B, H, cap, d, dtype=torch.float16))
            s.k[:, :, n:], s.v[:, :, n:] = float("nan"), float("nan")  # behind the tokens: anything
        else:
            s = random_segment(tq, g, B, H, d, cap, *kind, n=n)
            s.kscale.clamp_(max=4.0)
            for t in (s.kscale, s.vscale):
                t[:B * H * cap].view(B * H, cap)[:, n:] = float("nan")
        parts.append(s)
        l = rng.randint(-1, n + 3, size=B) if ragged else None
        if ragged and n > 127:
            l[0] = n
            l[-1] = rng.choice([0, 1, 127, 128])
        lens.append(None if l is None else torch.tensor(l, dtype=torch.int32, device=DEV))
        if l is not None:  # what is behind a sequence's own length is not read as a number either
            for b in range(B):
                m = max(0, min(int(l[b]), n))
                if kind == "fp16":
                    s.k[b, :, m:], s.v[b, :, m:] = float("nan"), float("inf")
                else:
                    for t in (s.kscale, s.vscale):
                        t[:B * H * cap].view(B, H, cap)[b, :, m:] = float("nan")
    qkv = randn(g, B, N, H * gqa + 2 * H, d, dtype=torch.float16)
    q = (scale * qkv[:, :, :H * gqa].float()).half()
    k, v = qkv[:, :, H * gqa:H * gqa + H].transpose(1, 2), qkv[:, :, H * gqa + H:].transpose(1, 2)
    return q, k, v, parts, lens, rng


@pytest.mark.parametrize("d,H,gqa,B,N,segs,ragged,kind", TREE)
def test_tree_attention(tq, d, H, gqa, B, N, segs, ragged, kind):
    q, k, v, parts, lens, rng = tree_case(tq, d, H, gqa, B, N, segs, ragged, seed=d + 7 * N + H)
    see = None if kind == "chain" else random_tree(rng, B, N, kind == "empty")
    mask = None if see is None else mask_words(see)
    out = run_tree(tq, q, k, v, parts, mask, lens if ragged else None)
    _, R = rotation64(tq, d, 21)
    clean = []
    for s in parts:  # the reference multiplies what it then leaves out
        if s.kind == 0:
            s.kscale.nan_to_num_(0.0)
            s.vscale.nan_to_num_(0.0)
        clean.append(s)
    check_tree(out, tree_ref(tq, q, k, v, see, clean, lens, R))
    if see is not None and not any(s.n_tokens for s in parts):
        for b, i in zip(*np.where(~see.any(-1))):
            assert (out[b, i] == 0).all()
    again = run_tree(tq, q, k, v, parts, mask, lens if ragged else None)
    assert torch.equal(bits(out), bits(again))  # nothing depends on an order of arrival
