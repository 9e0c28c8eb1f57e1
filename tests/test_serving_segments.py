"""What the serving calls are handed of a segment (no GPU): it follows the segment's fields, and leaves nothing on it."""
import copy
import ctypes
import pickle
import threading

import pytest


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import build
    build.build()
    from rotated_quantized_kv_gb300 import tq as T
    return T


def segments(tq):
    return [tq.PackedSegment(tq.make_layout(2, 4, 64, 32, [1, 2, 3, 4], 5), device="cpu", n_tokens=7),
            tq.Fp16Segment(2, 4, 64, 32, device="cpu", n_tokens=9)]


def handed(tq, seg):
    ref = seg.reference()
    return tq.tq_segment.from_buffer_copy(ref if isinstance(ref, bytes) else ref._obj)


def test_fields(tq):
    for seg in segments(tq):
        for n in (7, 20):
            seg.n_tokens = n
            got, want = handed(tq, seg), seg.segment()
            assert (got.kind, got.n_tokens, bytes(got.layout)) == (want.kind, n, bytes(want.layout))
            for name in ("kcodes", "vcodes", "kscale", "vscale"):
                assert getattr(got.packed, name) == getattr(want.packed, name)
            assert (got.k16, got.v16) == (want.k16, want.v16)


@pytest.mark.parametrize("how", [copy.deepcopy, lambda s: pickle.loads(pickle.dumps(s))])
def test_copy_of_a_used_segment(tq, how):
    for seg in segments(tq):
        seg.reference()
        other = how(seg)
        x, y = handed(tq, seg), handed(tq, other)
        assert bytes(x.layout) == bytes(y.layout) and x.n_tokens == y.n_tokens
        assert (x.packed.kcodes, x.k16) != (y.packed.kcodes, y.k16)  # its own memory


def test_shallow_copy_shares_nothing_that_a_call_sets(tq):
    for seg in segments(tq):
        first = seg.reference()
        other = copy.copy(seg)
        other.n_tokens = 3
        second = other.reference()
        assert second is not first
        assert handed(tq, seg).n_tokens == seg.n_tokens != 3 and handed(tq, other).n_tokens == 3
        kept = tq.tq_segment.from_buffer_copy(first if isinstance(first, bytes) else first._obj)
        assert kept.n_tokens == seg.n_tokens  # what one call holds is not another call's to change


def test_two_threads_at_once(tq):
    """Each call has what it was given, while another thread works on the same segment."""
    seg = segments(tq)[0]
    held, gate = [], threading.Barrier(2)

    def work(n):
        gate.wait()
        for _ in range(200):
            ref = seg.reference()
            assert ref is not None
            held.append(ref)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert len(held) == 400
    size = ctypes.sizeof(tq.tq_segment)
    seg.n_tokens = 30
    seg.reference()
    assert all(len(bytes(r if isinstance(r, bytes) else r._obj)) == size for r in held)
    assert all(tq.tq_segment.from_buffer_copy(r if isinstance(r, bytes) else r._obj).n_tokens == 7 for r in held)


def test_tree_mask_of_parents_that_are_none(tq):
    """A parent that is not before its draft is none: the draft is a root, and nothing is read out of bounds."""
    import torch
    p = torch.tensor([[-1, 0, 2, 7, 100, -5, 5, 2**31 - 1]], dtype=torch.int32)
    want = torch.tensor([[-1, 0, -1, -1, -1, -1, 5, -1]], dtype=torch.int32)
    assert torch.equal(tq.tree_mask(p), tq.tree_mask(want))
    for t in (torch.int8, torch.int16, torch.int32, torch.int64):
        assert torch.equal(tq.tree_mask(want.to(t)), tq.tree_mask(want))
    assert tq.tree_mask(want)[0, :, 0].tolist() == [1, 3, 4, 8, 16, 32, 96, 128]


@pytest.mark.parametrize("d", [64, 16])
def test_tree_over_a_segment_at_the_end_of_32_bits(tq, d):
    """Token counts that rounded up to whole tiles pass 2^31 - 1 are refused; the largest others are counted."""
    lv = tq.tq_layer_view()
    lv.rot, lv.n_segments = tq.tq_make_rotation(d, 1), 1
    for n, ok in ((2**31 - 16, False), (2**31 - 127, False), (2**31 - 128, True)):
        s = tq.tq_segment()
        s.kind, s.n_tokens, s.layout = tq.TQ_SEG_PACKED, n, tq.make_layout(1, 1, d, 2**31 - 16, 1, 1)
        lv.seg[0] = s
        if ok:
            assert tq.tq_tree_workspace_size(lv, 1, 1, 1, 1, d) > 0
        else:
            with pytest.raises(tq.TQError) as e:
                tq.tq_tree_workspace_size(lv, 1, 1, 1, 1, d)
            assert e.value.status == -2
