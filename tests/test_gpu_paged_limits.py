"""Attention over paged segments at the ends of its ranges."""
import pytest
import torch

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
