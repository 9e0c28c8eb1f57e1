"""Host side of the serving calls (no GPU): rotary frequencies, tree masks,
workspace sizes, and every refusal, which comes before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import build
    build.build()
    from rotated_quantized_kv_gb300 import tq as T
    return T


def test_frequencies(tq):
    r, base, s, L = 96, 500000.0, 8.0, 8192.0
    m = np.arange(r // 2)
    w = base ** (-2.0 * m / r)
    f = tq.tq_rope_frequencies
    np.testing.assert_allclose(f(tq.tq_make_rope(r, base)), w, rtol=1e-14)
    np.testing.assert_allclose(f(tq.tq_make_rope(r, base, tq.TQ_ROPE_SCALE_LINEAR, s)), w / s, rtol=1e-14)
    wide = f(tq.tq_make_rope(r, base, tq.TQ_ROPE_SCALE_BASE, s))
    np.testing.assert_allclose([wide[0], wide[-1]], [1.0, w[-1] / s], rtol=1e-12)
    assert np.all(np.diff(wide) < 0)
    # turns over the original length: kept from `fast` on, divided by s up to `slow`, linear between
    got = f(tq.tq_make_rope(r, base, tq.TQ_ROPE_SCALE_TURNS, s, L, fast=4.0, slow=1.0))
    turns = L * w / (2 * math.pi)
    for i in range(r // 2):
        u = 1.0 if turns[i] >= 4 else 0.0 if turns[i] <= 1 else (turns[i] - 1) / 3
        assert got[i] == pytest.approx(u * w[i] + (1 - u) * w[i] / s, rel=1e-13)
    assert 0 < (got == w).sum() < r // 2 and got[-1] == pytest.approx(w[-1] / s)
    # linear in the index between the pairs with 32 and with 1 turn
    got = f(tq.tq_make_rope(r, base, tq.TQ_ROPE_SCALE_INDEX, s, L, fast=32.0, slow=1.0))
    lo = math.floor(next(x for x in np.arange(0, r, 1e-3) if L * base ** (-2 * x / r) / (2 * math.pi) <= 32))
    hi = math.ceil(next(x for x in np.arange(0, r, 1e-3) if L * base ** (-2 * x / r) / (2 * math.pi) <= 1))
    for i in range(r // 2):
        u = 1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert got[i] == pytest.approx(u * w[i] + (1 - u) * w[i] / s, rel=1e-12)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=1026), dict(base=1.0), dict(base=math.inf),
    dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.0), dict(scaling=2, factor=2.0, rotary_dim=2),
    dict(scaling=3, factor=2.0, original_len=100.0, fast=1.0, slow=1.0),
    dict(scaling=4, factor=2.0, original_len=0.0, fast=2.0, slow=1.0),
    dict(scaling=3, factor=2.0, original_len=100.0, fast=2.0, slow=math.nan), dict(amplitude=0.0),
])
def test_frequency_refusals(tq, kw):
    with pytest.raises(tq.TQError) as e:
        tq.tq_make_rope(**{"rotary_dim": 64, **kw})
    assert e.value.status == -1


def test_tree_mask(tq):
    rng = np.random.RandomState(3)
    for N in (1, 2, 31, 32, 33, 70):
        par = np.array([[rng.randint(-1, i) if i else -1 for i in range(N)] for _ in range(3)])
        got = tq.tree_mask(torch.tensor(par)).numpy().view(np.uint32)
        assert got.shape == (3, N, -(-N // 32))
        for b in range(3):
            for i in range(N):
                seen, j = set(), i
                while j >= 0:
                    seen.add(j)
                    j = par[b, j]
                bits = {j for j in range(32 * got.shape[2]) if got[b, i, j // 32] >> (j % 32) & 1}
                assert bits == seen
        one = tq.tree_mask(torch.tensor(par[1])).numpy().view(np.uint32)
        assert np.array_equal(one, got[1])


P = ctypes.c_void_p
A = 4096  # an aligned address: these calls never reach the device


def _seg(tq, B=2, H=4, d=128, cap=64, n=40, kind=0, kb=3, vb=3, **kw):
    s = tq.tq_segment()
    s.kind, s.n_tokens, s.layout = kind, n, tq.make_layout(B, H, d, cap, kb, vb, **kw)
    s.packed = tq.tq_packed_bufs(A, A, A, A, A, A, A, A)
    s.k16 = s.v16 = A
    return s


def _rope(tq, d=128, layout=0, table=A, n_pos=100):
    return tq.tq_rope_view(d, layout, n_pos, table)


def test_rope_refusals(tq):
    def call(view=None, dtype=0, B=2, T=3, d=128, pos=A, n=1, x=None, **kw):
        t = (tq.tq_rope_tensor * 4)()
        for i in range(4):
            t[i].in_, t[i].out, t[i].n_heads = A, 2 * A, 4
            t[i].in_stride = t[i].out_stride = (ctypes.c_int64 * 3)(4 * 3 * d, 3 * d, d)
            for k, v in kw.items():
                setattr(t[i], k, v)
        return tq._lib.tq_rope(ctypes.byref(view or _rope(tq)), dtype, B, T, d, pos, T, t if x is None else x, n, 0,
                               None)
    st3 = ctypes.c_int64 * 3
    assert call(dtype=3) == -1 and call(d=0) == -1 and call(d=1025) == -1 and call(n=5) == -1
    assert call(view=_rope(tq, 7)) == -1 and call(view=_rope(tq, 130)) == -1 and call(view=_rope(tq, layout=2)) == -1
    assert call(view=_rope(tq, table=None)) == -1 and call(view=_rope(tq, table=A + 8)) == -3
    assert call(pos=None) == -1 and call(pos=A + 2) == -3
    assert call(in_=None) == -1 and call(in_=A + 1) == -3 and call(dtype=2, out=A + 2) == -3
    assert call(n_heads=-1) == -1 and call(n_heads=70000) == -2
    assert call(out_stride=st3(1536, 384, 64)) == -1          # rows overlap
    assert call(out=A, in_stride=st3(1536, 384, 128), out_stride=st3(1536, 128, 512)) == -1  # in place, other strides
    assert tq._lib.tq_rope(None, 0, 1, 1, 128, A, 1, None, 0, 0, None) == -1
    assert call(B=0) == 0 and call(T=0) == 0 and call(n=0) == 0 and call(n_heads=0) == 0  # nothing to do
    spec = tq.tq_make_rope(64)
    tab = tq._lib.tq_rope_table
    assert tab(ctypes.byref(spec), -1, 4, A, None) == -1 and tab(ctypes.byref(spec), 0, -1, A, None) == -1
    assert tab(ctypes.byref(spec), 2, 0x7fffffff, A, None) == -1 and tab(ctypes.byref(spec), 0, 4, None, None) == -1
    assert tab(ctypes.byref(spec), 0, 4, A + 4, None) == -3 and tab(ctypes.byref(spec), 0, 0, None, None) == 0


def test_append_and_read_refusals(tq):
    st3 = ctypes.c_int64 * 3
    ok = st3(4 * 8 * 128, 8 * 128, 128)
    rot = tq.tq_make_rotation(128, 1)

    def app(seg=None, rot=rot, rope=None, pos=A, K=A, ks=ok, V=A, vs=ok, S=8, n=8, t0=A, cnt=None, idx=None):
        sg = seg or _seg(tq)
        return tq._lib.tq_append(ctypes.byref(sg), ctypes.byref(rot) if rot else None,
                                 ctypes.byref(rope) if rope else None, pos, 8, K, ks, V, vs, S, n, t0, cnt, idx, 8, None)
    assert app(seg=_seg(tq, kb=9)) == -1 and app(seg=_seg(tq, kind=2)) == -1 and app(rot=None) == -1
    assert app(rot=tq.tq_make_rotation(64, 1)) == -1 and app(ks=None) == -1 and app(S=-1) == -1 and app(n=-1) == -1
    assert app(K=None) == -1 and app(t0=None) == -1 and app(K=A + 1) == -3 and app(t0=A + 1) == -3
    assert app(cnt=A + 2) == -3 and app(idx=A + 2) == -3
    assert app(rope=_rope(tq), pos=None) == -1 and app(rope=_rope(tq, 256)) == -1
    assert app(seg=_seg(tq, qjl=[1, 0, 0, 0])) == -2 and app(seg=_seg(tq, qjl_v=[1, 0, 0, 0])) == -2
    r64 = tq.tq_make_rotation(64, 1)
    assert app(seg=_seg(tq, d=64, value_law=1), rot=r64) == -2
    dense = tq.tq_make_rotation(128, 1)
    dense.dense = A
    assert app(rot=dense) == -2
    bad = _seg(tq)
    bad.packed.kcodes = A + 8
    assert app(seg=bad) == -3
    bad.packed.kcodes = None
    assert app(seg=bad) == -1
    half = _seg(tq, kind=1)
    half.v16 = A + 2
    assert app(seg=half) == -3
    assert app(S=0) == 0 and app(n=0) == 0 and app(seg=_seg(tq, cap=0)) == 0

    def read(seg=None, rot=rot, n=8, t0=A, cnt=None, dtype=0, K=A, ks=ok, V=A, vs=ok):
        sg = seg or _seg(tq)
        return tq._lib.tq_read(ctypes.byref(sg), ctypes.byref(rot) if rot else None, n, t0, cnt, dtype, K, ks, V, vs, None)
    assert read(dtype=3) == -1 and read(n=-1) == -1 and read(t0=None) == -1 and read(ks=None) == -1
    assert read(rot=r64) == -1 and read(rot=dense) == -2 and read(seg=_seg(tq, d=64, value_law=1), rot=r64) == -2
    assert read(K=A + 1) == -3 and read(dtype=2, V=A + 2) == -3 and read(t0=A + 2) == -3
    assert read(ks=st3(4 * 8 * 128, 8 * 128, 64)) == -1       # rows overlap
    assert read(K=None, V=None) == 0 and read(n=0) == 0


def test_tree_refusals_and_workspace(tq):
    def view(*segs, d=128):
        lv = tq.tq_layer_view()
        lv.rot, lv.n_segments = tq.tq_make_rotation(d, 1), len(segs)
        for i, s in enumerate(segs):
            lv.seg[i] = s
        return lv

    def size(lv, B=2, H=4, Hq=8, N=5, d=128):
        try:
            return tq.tq_tree_workspace_size(lv, B, H, Hq, N, d)
        except tq.TQError as e:
            return e.status
    v = view(_seg(tq))
    assert size(v) > 0 and size(view()) > 0
    assert size(v, N=0) == -1 and size(v, N=257) == -1 and size(v, Hq=6) == -1 and size(v, H=3, Hq=6) == -1
    assert size(v, B=3) == -1 and size(v, d=64) == -1 and size(v, d=100) == -1
    assert size(view(_seg(tq, n=65))) == -4 and size(view(_seg(tq, n=-1))) == -4
    assert size(view(_seg(tq, cap=40, n=4))) == -3
    assert size(view(_seg(tq, qjl=[0, 1, 0, 0]))) == -2 and size(view(_seg(tq, qjl_v=[0, 1, 0, 0]))) == -2
    assert size(view(_seg(tq, d=64, value_law=1), d=64), d=64) == -2
    mass = _seg(tq)
    mass.attn_mass = A
    assert size(view(mass)) == -2
    dense = view(_seg(tq))
    dense.rot.dense = A
    assert size(dense) == -2

    def call(lv=v, ws=A, n=1 << 30, N=5, **kw):
        t = tq.tq_tree()
        t.n_drafts, t.q, t.k, t.v, t.out = N, A, A, A, A
        for k, x in kw.items():
            setattr(t, k, x)
        return tq._lib.tq_tree_attention(ctypes.byref(lv), 2, 4, 8, 128, ctypes.byref(t), ws, n, None)
    assert call(q=None) == -1 and call(k=None) == -1 and call(v=None) == -1 and call(out=None) == -1
    assert call(ws=None) == -1 and call(mask_stride_b=-1) == -1
    assert call(q=A + 1) == -3 and call(out=A + 8) == -3 and call(ws=A + 8) == -3 and call(mask=A + 2) == -3
    lens = (ctypes.c_void_p * 8)()
    lens[0] = A + 2
    assert call(seg_len=lens) == -3
    assert call(n=size(v) - 1) == -4
    assert tq._lib.tq_tree_attention(ctypes.byref(v), 2, 4, 8, 128, None, A, 1 << 30, None) == -1


def test_binding_refusals(tq):
    """What the binding checks itself: types, shapes, devices."""
    rope = tq.Rope(torch.zeros(10, 2, 8))
    pos = torch.zeros(1, 3, dtype=torch.int32)
    x = torch.zeros(1, 2, 3, 16)
    for bad in (lambda: tq.Rope(torch.zeros(10, 2, 8, dtype=torch.float64)),
                lambda: tq.Rope(torch.zeros(10, 16)),
                lambda: tq.Rope(torch.zeros(10, 2, 8), 2),
                lambda: tq.tq_rope(rope, pos.long(), x),
                lambda: tq.tq_rope(rope, pos[:, :2], x),
                lambda: tq.tq_rope(rope, pos, x.double()),
                lambda: tq.tq_rope(rope, pos, x.transpose(2, 3)),
                lambda: tq.tq_rope(rope, pos, [x] * 5),
                lambda: tq.tq_rope(rope, pos, [x, x.half()]),
                lambda: tq.tq_rope(rope, pos, x)):  # not on a GPU
        with pytest.raises(tq.TQError) as e:
            bad()
        assert e.value.status == -1
    seg = tq.PackedSegment(tq.make_layout(1, 2, 16, 16, 3, 3), device="cpu")
    rot = tq.tq_make_rotation(16, 1)
    kv = torch.zeros(1, 2, 3, 16, dtype=torch.float16)
    at = torch.zeros(1, dtype=torch.int32)
    for bad in (lambda: tq.tq_append(seg, rot, kv.float(), kv.float(), at),
                lambda: tq.tq_append(seg, rot, kv[:, :1], kv[:, :1], at),
                lambda: tq.tq_append(seg, rot, kv, kv, at.long()),
                lambda: tq.tq_append(seg, rot, kv, kv, at, index=pos[:, :2], n_max=3),
                lambda: tq.tq_append(seg, rot, kv, kv, at, rope=rope),
                lambda: tq.tq_append(seg, rot, kv, kv, at),
                lambda: tq.tq_read(seg, rot, at, 4, out=[kv, kv]),
                lambda: tq.tq_read(seg, rot, at, 3, out=[kv, kv.float()]),
                lambda: tq.tq_read(seg, rot, at, 3)):
        with pytest.raises(tq.TQError) as e:
            bad()
        assert e.value.status == -1
    lv = tq.layer_view(rot, [seg])
    q = torch.zeros(1, 3, 4, 16, dtype=torch.float16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (lambda: tq.tq_tree_attention(lv, q, kv, kv, q.float(), ws),
                lambda: tq.tq_tree_attention(lv, q, kv[:, :, :2], kv[:, :, :2], q.clone(), ws),
                lambda: tq.tq_tree_attention(lv, q, kv, kv, q.clone(), ws, mask=torch.zeros(3, 2, dtype=torch.int32)),
                lambda: tq.tq_tree_attention(lv, q, kv, kv, q.clone(), ws, seg_len=[at, at]),
                lambda: tq.tq_tree_attention(lv, q, kv, kv, q.clone(), ws)):
        with pytest.raises(tq.TQError) as e:
            bad()
        assert e.value.status == -1
