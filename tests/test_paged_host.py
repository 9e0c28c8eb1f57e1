"""Host side of the calls on pages and drafts (no GPU): workspace sizes, and every refusal,
which comes before anything is launched."""
import ctypes

import pytest
import torch

from test_serving_host import A, _seg


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import build
    build.build()
    from rotated_quantized_kv_gb300 import tq as T
    return T


def test_page_refusals(tq):
    def tables(B=2, P=16, M=4, n=8, table=A, stride=4, length=A, new=A, n_max=3, free=A, n_free=A, slots=A, pos=A, granted=A):
        return tq._lib.tq_page_tables(B, P, M, n, table, stride, length, new, n_max, free, n_free, slots, pos, granted, None)

    def release(B=2, P=16, M=4, n=8, table=A, stride=4, length=A, keep=A, free=A, n_free=A):
        return tq._lib.tq_page_release(B, P, M, n, table, stride, length, keep, free, n_free, None)
    for call in (tables, release):
        assert call(B=-1) == -1 and call(P=0) == -1 and call(M=-1) == -1 and call(n=-1) == -1
        assert call(stride=3) == -1 and call(stride=-4) == -1
        assert call(table=None) == -1 and call(length=None) == -1 and call(free=None) == -1 and call(n_free=None) == -1
        assert call(M=1 << 27, stride=1 << 27) == -2 and call(n=1 << 27) == -2  # 2^31 tokens
        assert call(table=A + 2) == -3 and call(length=A + 1) == -3 and call(free=A + 2) == -3 and call(n_free=A + 2) == -3
        assert call(B=0) == 0
    assert tables(n_max=-1) == -1 and tables(new=None) == -1 and tables(granted=None) == -1 and release(keep=None) == -1
    assert tables(slots=A + 2) == -3 and tables(pos=A + 2) == -3 and tables(granted=A + 2) == -3


def test_slot_refusals(tq):
    st3 = ctypes.c_int64 * 3
    ok = st3(4 * 8 * 128, 8 * 128, 128)
    rot, r64 = tq.tq_make_rotation(128, 1), tq.tq_make_rotation(64, 1)

    def app(seg=None, rot=rot, K=A, ks=ok, V=A, B=3, S=8, n=8, slots=A, cnt=None, idx=None):
        sg = _seg(tq) if seg is None else seg
        return tq._lib.tq_paged_append(ctypes.byref(sg) if sg else None, ctypes.byref(rot) if rot else None, None, None, 0, K, ks, V,
                                       ok, B, S, n, slots, 8, cnt, idx, 8, None)

    def read(seg=None, rot=rot, B=3, n=8, slots=A, cnt=None, dtype=0, K=A, ks=ok, V=A):
        sg = _seg(tq) if seg is None else seg
        return tq._lib.tq_paged_read(ctypes.byref(sg) if sg else None, ctypes.byref(rot) if rot else None, B, n, slots, 8, cnt, dtype,
                                     K, ks, V, ok, None)
    huge = dict(B=1 << 20, cap=1 << 12)
    for call in (app, read):
        assert call(seg=0) == -1 and call(B=-1) == -1 and call(n=-1) == -1 and call(slots=None) == -1 and call(ks=None) == -1
        assert call(slots=A + 2) == -3 and call(cnt=A + 2) == -3 and call(K=A + 1) == -3
        assert call(rot=r64) == -1 and call(seg=_seg(tq, kb=9)) == -1
        assert call(seg=_seg(tq, **huge)) == -2  # slots past 32 bits
        assert call(B=0) == 0 and call(n=0) == 0 and call(seg=_seg(tq, cap=0)) == 0
    assert app(rot=None) == -1 and app(seg=_seg(tq, qjl=[1, 0, 0, 0])) == -2 and app(S=-1) == -1 and app(S=0) == 0
    assert app(idx=A + 1) == -3 and read(dtype=3) == -1 and read(K=None, V=None) == 0


def _view(tq, *segs, d=128):
    lv = tq.tq_layer_view()
    lv.rot, lv.n_segments = tq.tq_make_rotation(d, 1), len(segs)
    for i, s in enumerate(segs):
        lv.seg[i] = s
    return lv


def test_attention_refusals_and_workspace(tq):
    def size(lv, B=2, H=4, Hq=8, d=128):
        n = ctypes.c_size_t()
        st = tq._lib.tq_paged_workspace_size(ctypes.byref(lv) if lv else None, B, H, Hq, d, ctypes.byref(n))
        return n.value if st == 0 else st
    pool = _seg(tq, B=9)
    assert size(None) == -1 and size(_view(tq, pool), B=0) == -1 and size(_view(tq, pool), H=5, Hq=5) == -1
    assert size(_view(tq, pool), Hq=6) == -1 and size(_view(tq, pool), Hq=2) == -1 and size(_view(tq, pool), d=96) == -1
    assert size(_view(tq, pool, d=64)) == -1 and size(_view(tq, _seg(tq, B=9, d=64))) == -1
    assert size(_view(tq, _seg(tq, qjl=[0, 1, 0, 0]))) == -2 and size(_view(tq, _seg(tq, qjl_v=[0, 1, 0, 0]))) == -2
    assert size(_view(tq, _seg(tq, d=64, value_law=1), d=64), d=64) == -2 and size(_view(tq, _seg(tq, cap=40, n=1))) == -3
    mass, dense = _seg(tq), _view(tq, pool)
    mass.attn_mass, dense.rot.dense = A, A
    assert size(_view(tq, mass)) == -2 and size(dense) == -2
    assert size(_view(tq, pool), B=1 << 29) == -2  # query rows past 32 bits
    assert 0 < size(_view(tq, pool)) < size(_view(tq, pool), B=64) < size(_view(tq, pool, _seg(tq, kind=1)), B=64)
    assert size(_view(tq, pool)) == size(_view(tq, _seg(tq, B=90000, cap=128)))  # no matter how many pages

    def call(lv=None, pages=None, B=2, q=A, out=A, ws=A, bytes_=1 << 40, qs=True, **kw):
        p = (tq.tq_pages * 8)()
        for i in range(8):
            p[i] = tq.tq_pages(A, 4, 4, A)
            for k, v in kw.items():
                setattr(p[i], k, v)
        lv = _view(tq, pool) if lv is None else lv
        return tq._lib.tq_paged_attention(ctypes.byref(lv), None if pages is False else p, B, 4, 8, 128, q,
                                          (ctypes.c_int64 * 2)(1024, 128) if qs else None, out, ws, bytes_, None)
    assert call(pages=False) == -1 and call(q=None) == -1 and call(qs=False) == -1 and call(out=None) == -1 and call(ws=None) == -1
    assert call(q=A + 1) == -3 and call(out=A + 8) == -3 and call(ws=A + 8) == -3
    assert call(table=A + 2) == -3 and call(len=A + 2) == -3
    assert call(max_pages=-1) == -1 and call(table_stride_b=3) == -1 and call(table_stride_b=-4) == -1 and call(len=None) == -1
    assert call(max_pages=1 << 26, table_stride_b=1 << 26) == -2 and call(bytes_=100) == -4
    assert call(table=None) == -1                                   # its batch is not the call's
    assert call(table=None, lv=_view(tq, _seg(tq, n=65))) == -4 and call(table=None, lv=_view(tq, _seg(tq, n=-1))) == -4


def test_verify_refusals(tq):
    def call(**kw):
        v = tq.tq_verification(2, 3, 100, 0, A, 3, A, 3, A, (ctypes.c_int64 * 2)(400, 100), A, (ctypes.c_int64 * 2)(400, 100), A, 4,
                               A, A, A)
        for k, x in kw.items():
            setattr(v, k, x)
        return tq._lib.tq_verify(ctypes.byref(v), None)
    assert tq._lib.tq_verify(None, None) == -1
    assert call(batch=-1) == -1 and call(n_drafts=-1) == -1 and call(n_drafts=257) == -1 and call(vocab=0) == -1 and call(dtype=3) == -1
    assert call(vocab=(1 << 30) + 1) == -2 and call(batch=(1 << 24) + 1) == -2
    for name in ("target", "uniform", "n_accepted", "token", "tokens", "accepted"):
        assert call(**{name: None}) == -1
    for name in ("target", "draft"):
        assert call(**{name: A + 1}) == -3 and call(**{name: A + 2, "dtype": 2}) == -3
    for name in ("tokens", "parents", "uniform", "accepted", "n_accepted", "token"):
        assert call(**{name: A + 2}) == -3
    assert call(batch=0) == 0


def test_binding_refusals(tq):
    i32, f16 = dict(dtype=torch.int32), dict(dtype=torch.float16)
    B, N, V = 2, 3, 50
    tok, tgt, u = torch.zeros(B, N, **i32), torch.zeros(B, N + 1, V), torch.zeros(B, N + 1)

    def refused(f, *a, **kw):
        with pytest.raises(tq.TQError) as e:
            f(*a, **kw)
        assert e.value.status == -1
    v = tq.tq_verify
    refused(v, tok.long(), tgt, u)
    refused(v, tok, tgt[:, :N], u)
    refused(v, tok, tgt.double(), u)
    refused(v, tok, tgt, u[:, :N])
    refused(v, tok, tgt, u, draft=tgt[:, :2])
    refused(v, tok, tgt, u, draft=tgt.half())
    refused(v, tok, tgt, u, parents=tok[:, :2])
    refused(v, tok, tgt, u, out=(tok, tok[:, 0].contiguous(), tok[:1, 0]))
    refused(v, tok, tgt, u)                    # not on a CUDA device
    pool = tq.PackedSegment(tq.make_layout(5, 2, 64, 16, 3, 3), device="cpu")
    rot = tq.tq_make_rotation(64, 1)
    kv, slots = torch.zeros(B, 2, 4, 64, **f16), torch.zeros(B, 4, **i32)
    refused(tq.tq_paged_append, pool, rot, kv.float(), kv, slots)
    refused(tq.tq_paged_append, pool, rot, kv, kv, slots[0])
    refused(tq.tq_paged_append, pool, rot, kv, kv, slots, n_max=5)
    refused(tq.tq_paged_append, pool, rot, kv, kv, slots, index=slots.long())
    refused(tq.tq_paged_append, pool, rot, kv, kv, slots)
    refused(tq.tq_paged_read, pool, rot, slots.long(), out=[kv, kv])
    refused(tq.tq_paged_read, pool, rot, slots, out=[kv[:, :, :3], kv])
    refused(tq.tq_paged_read, pool, rot, slots)
    view = tq.layer_view(rot, [pool])
    q, ws = torch.zeros(B, 4, 64, **f16), torch.zeros(tq.tq_paged_workspace_size(view, B, 2, 4, 64), dtype=torch.uint8)
    table, n = torch.zeros(B, 3, **i32), torch.zeros(B, **i32)
    for kw in (dict(q=q.float()), dict(out=q[:, :2]), dict(tables=[]), dict(lens=[None]), dict(tables=[table[0]]), dict(lens=[n.long()]), {}):
        a = {**dict(q=q, out=torch.zeros_like(q), tables=[table], lens=[n]), **kw}
        refused(tq.tq_paged_attention, view, a["q"], a["out"], ws, a["tables"], a["lens"])
    one = torch.ones(1, **i32)
    for bad in (dict(table=table.long()), dict(length=n[:1]), dict(n_free=n)):
        a = {**dict(table=table, length=n, n_free=one), **bad}
        refused(tq.tq_page_tables, a["table"], a["length"], n, slots[0], a["n_free"], 16, 3, out=(None, None, n))
        refused(tq.tq_page_release, a["table"], a["length"], n, slots[0], a["n_free"], 16)
    refused(tq.tq_page_tables, table, n, n, slots[0], one, 16, 3, out=(slots, None, n))
    refused(tq.tq_page_tables, table, n, n, slots[0], one, 16, 3)
