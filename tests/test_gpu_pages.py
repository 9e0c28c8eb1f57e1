"""Page tables and writes and reads by slot on the GPU, against plain Python and the library's own
ragged calls, bit for bit."""
import numpy as np
import pytest
import torch

import test_gpu_serving as base
from test_gpu_serving import BUFS, DEV, MIXED, bits, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ tables
def place(table, length, count, free, n_free, P, n_max, n_pages):
    """Sequence by sequence, page by page (numpy, in place): slots, positions, granted, n_free."""
    B, M = table.shape
    slots, positions, granted = np.full((B, n_max), -1), np.full((B, n_max), -1), np.zeros(B, int)
    top = min(max(n_free, 0), n_pages)
    asked = 0
    taken = 0
    for b in range(B):
        length[b] = min(max(length[b], 0), M * P)
        want = min(min(max(count[b], 0), n_max), M * P - length[b])
        held = -(-length[b] // P)
        need = -(-(length[b] + want) // P) - held
        got = min(max(top - asked, 0), need)
        asked += need
        for k in range(got):
            table[b, held + k] = free[top - 1 - taken]
            taken += 1
        granted[b] = min(want, (held + got) * P - length[b])
        for j in range(granted[b]):
            t = length[b] + j
            page = table[b, t // P]
            positions[b, j] = t
            slots[b, j] = page * P + t % P if 0 <= page < n_pages else -1
        length[b] += granted[b]
    return slots, positions, granted, top - taken


def pages_case(B, P, M, n_pages, spare, n_max, seed, odd):
    r = np.random.RandomState(seed)
    length = r.randint(0, M * P + 1, size=B)
    length[r.rand(B) < 0.3] = 0
    if odd and B > 3:
        length[1], length[2], length[3] = -5, M * P + 7, M * P
    count = r.randint(-1 if odd else 0, n_max + 2, size=B)
    table = r.randint(0, max(n_pages, 1), size=(B, M))
    if odd:
        table[r.rand(B, M) < 0.1] = -3
        table[r.rand(B, M) < 0.1] = n_pages
    free = r.permutation(n_pages)
    return table, length, count, free, min(spare, n_pages)


PAGES = [  # B, page, entries, pages, free, n_max, odd values
    (1, 16, 4, 20, 20, 1, False), (1, 16, 4, 20, 20, 200, False), (5, 1, 7, 40, 40, 5, True), (33, 64, 9, 500, 40, 1, True),
    (32, 16, 33, 3000, 1100, 32, True), (64, 48, 20, 3000, 50, 33, True), (7, 128, 100, 900, 901, 2500, False),
    (1000, 16, 3, 4000, 1500, 3, True), (1200, 16, 5, 9000, 2500, 60, False), (3, 16, 0, 10, 10, 4, False), (4, 16, 4, 0, 0, 4, False),
    (9, 16, 8, 100, 0, 20, True), (2, 16, 8, 100, 100, 0, False),
]


@pytest.mark.parametrize("B,P,M,n_pages,spare,n_max,odd", PAGES)
def test_tables(tq, B, P, M, n_pages, spare, n_max, odd):
    table, length, count, free, n_free = pages_case(B, P, M, n_pages, spare, n_max, B + M, odd)
    wide = torch.full((B, M + 3), 77, dtype=torch.int32, device=DEV)  # rows apart, with others' entries between
    wide[:, :M] = i32(table).reshape(B, M)
    dt, dl, dn = wide[:, :M], i32(length), i32([n_free])
    df = i32(free)
    if spare > n_pages:
        dn.fill_(spare)
    slots, positions, granted = tq.tq_page_tables(dt, dl, i32(count), df, dn, P, n_max)
    want = place(table, length, count, free, n_free, P, n_max, n_pages)
    for got, ref in zip((slots, positions, granted, dn[0], dt, dl, df), (*want, table, length, free)):
        assert np.array_equal(got.cpu().numpy(), np.asarray(ref))
    assert (wide[:, M:] == 77).all()


@pytest.mark.parametrize("B,P,M,n_pages,spare,n_max,odd", PAGES)
def test_release_undoes_a_call(tq, B, P, M, n_pages, spare, n_max, odd):
    table, length, count, free, n_free = pages_case(B, P, M, n_pages, spare, n_max, B + M, False)
    dt, dl, df, dn = i32(table).reshape(B, M), i32(length), i32(free), i32([n_free])
    tq.tq_page_tables(dt, dl, i32(count), df, dn, P, n_max, out=(None, None, i32(length)))
    df[int(dn):] = -9  # (what was taken is above the stack)
    tq.tq_page_release(dt, dl, i32(length), df, dn, P)
    assert np.array_equal(dl.cpu().numpy(), length) and int(dn) == n_free
    assert np.array_equal(df.cpu().numpy()[:n_free], free[:n_free])


def test_release_cuts_and_ends(tq):
    P, M, n_pages = 16, 6, 40
    length, keep = np.array([90, 33, 0, 16, 50, 20]), np.array([17, 0, 5, 16, -4, 99])
    table = np.arange(36).reshape(6, M)
    df, dn, dl = i32(np.full(n_pages, -1)), i32([3]), i32(length)
    tq.tq_page_release(i32(table), dl, i32(keep), df, dn, P)
    back = []
    for b in range(6):
        kept = min(length[b], max(keep[b], 0))
        back += list(table[b, -(-kept // P):-(-length[b] // P)])
    assert np.array_equal(dl.cpu().numpy(), np.minimum(length, np.maximum(keep, 0)))
    assert int(dn) == 3 + len(back) and df[3:int(dn)].tolist() == back[::-1]
    # a stack that is too full: what does not fit is dropped, nothing behind it is written
    guard = i32(np.full(n_pages + 8, -1))
    dn.fill_(38)
    tq.tq_page_release(i32(table), i32(length), i32(np.zeros(6)), guard[:n_pages], dn, P)
    assert int(dn) == n_pages and (guard[n_pages:] == -1).all()


# ------------------------------------------------------------------ writes and reads by slot
# d, H, kbits, vbits, page, sequences, rows, gathered, rotary dims (0: none), law, fp16 pool
SLOTS = [
    (128, 8, MIXED, MIXED[::-1], 16, 3, 20, True, 0, 0, False),
    (128, 4, 3, 3, 64, 2, 300, False, 128, 0, False),
    (128, 8, 4, 4, 64, 4, 700, False, 96, 0, False),           # a thread a vector
    (128, 8, [2, 5] * 4, 1, 48, 3, 900, True, 40, 1, False),
    (64, 8, 3, 4, 16, 2, 1000, False, 64, 0, False),           # pairs of vectors on other pages
    (64, 3, [1, 7, 8], [5, 2, 3], 7, 2, 40, True, 0, 0, False),  # an odd page
    (16, 2, [1, 3], [2, 5], 16, 2, 33, False, 16, 0, False),
    (256, 2, 3, 6, 32, 2, 50, False, 64, 0, False),
    (1024, 1, 2, 2, 16, 1, 9, False, 0, 0, False),
    (128, 4, 1, 1, 64, 3, 100, True, 128, 0, True),
    (32, 2, 1, 1, 5, 2, 12, False, 32, 0, True),
]


@pytest.mark.parametrize("d,H,kb,vb,P,B,n,gather,r,law,half", SLOTS)
def test_slots_are_ragged_writes(tq, d, H, kb, vb, P, B, n, gather, r, law, half):
    g, rng = gen(d + n), np.random.RandomState(d + n)
    S = n + 5 if gather else n
    K, V = (randn(g, B, S, H, d, dtype=torch.float16).transpose(1, 2) for _ in range(2))
    index = i32(rng.randint(-1, S + 1, size=(B, n))) if gather else None
    count = i32(rng.randint(n // 2, n + 3, size=B))
    n_pages = B * (n // P + 2) + 3
    # contiguous places, and the pages in any order that hold them
    cap = P * (n // P + 2)
    first = i32(rng.randint(0, P, size=B))
    order = rng.permutation(n_pages)[:B * cap // P].reshape(B, -1)
    t = np.arange(n) + first.cpu().numpy()[:, None]
    slots = np.take_along_axis(order, t // P, 1) * P + t % P
    slots[rng.rand(B, n) < 0.05] = -1
    slots[rng.rand(B, n) < 0.05] = n_pages * P
    kw = dict(n_new=count, index=index, n_max=n)
    if r:
        kw["rope"] = tq.Rope(tq.tq_rope_table(tq.tq_make_rope(r), 400))
        kw["positions"] = torch.randint(-1, 402, (B, S), generator=g, device=DEV, dtype=torch.int32)
    rot = tq.tq_make_rotation(d, 5)
    if half:
        make = lambda b, c: tq.Fp16Segment(b, H, d, c, k=torch.full((b, H, c, d), 3.0, dtype=torch.float16, device=DEV),  # noqa: E731
                                           v=torch.full((b, H, c, d), 3.0, dtype=torch.float16, device=DEV))
    else:
        make = lambda b, c: base.filled_segment(tq, b, H, d, c, kb, vb, law)  # noqa: E731
    pool, flat = make(n_pages, P), make(B, cap)
    tq.tq_paged_append(pool, None if half else rot, K, V, i32(slots), **kw)
    tq.tq_append(flat, None if half else rot, K, V, first, **kw)

    def rows(seg):  # [batch][H][capacity][bytes and scale] of both, head by head
        L = seg.layout
        if half:
            return [[x[:, h] for h in range(H)] for x in (seg.k, seg.v)]
        out = []
        for codes, scale, w in ((seg.kcodes, seg.kscale, L.kbits), (seg.vcodes, seg.vscale, L.vbits)):
            per = [d * w[h] // 8 * L.capacity for h in range(H)]
            at = np.concatenate([[0], np.cumsum(per)])
            data = codes[:L.batch * at[-1]].view(L.batch, -1)
            s = scale[:L.batch * H * L.capacity].view(L.batch, H, L.capacity, 1).view(torch.uint8)
            out.append([torch.cat([data[:, at[h]:at[h + 1]].reshape(L.batch, L.capacity, -1), s[:, h]], -1) for h in range(H)])
        return out
    stored = (slots >= 0) & (slots < n_pages * P) & (np.arange(n) < count.cpu().numpy()[:, None])
    b_at, j_at = (torch.tensor(x, device=DEV) for x in np.nonzero(stored))
    t_at = torch.tensor(t, device=DEV)[b_at, j_at]
    s_at = torch.tensor(slots, device=DEV)[b_at, j_at]
    untouched = torch.ones(n_pages * P, dtype=torch.bool, device=DEV)
    untouched[s_at] = False
    for x, y, z in zip(rows(pool), rows(flat), rows(make(n_pages, P))):
        for h in range(H):
            got = x[h].flatten(0, 1)
            assert torch.equal(got[s_at], y[h][b_at, t_at])
            assert torch.equal(got[untouched], z[h].flatten(0, 1)[untouched])
    # and back
    for dtype in (torch.float16, torch.float32):
        new = [torch.full((B, n, H, d), 9.0, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2)]
        got = tq.tq_paged_read(pool, None if half else rot, i32(slots), n_read=count, out=new)
        want = tq.tq_read(flat, None if half else rot, first, n, dtype=dtype)
        hit = torch.tensor(stored, device=DEV)[:, None, :, None]
        for x, y in zip(got, want):
            assert torch.equal(x, torch.where(hit, y, torch.full_like(y, 9.0)))
    only = tq.tq_paged_read(pool, None if half else rot, i32(slots), out=[None, torch.zeros(B, H, n, d, dtype=torch.float16, device=DEV)])
    assert only[0] is None and only[1].abs().sum() > 0


def test_records_past_32_bits(tq):
    """A pool whose codes and rows lie beyond 2^32 bytes."""
    d, H, P = 128, 16, 64
    n_pages = (1 << 32) // (H * P * d) + 40     # 8-bit keys: 4 GB and some
    pool = tq.PackedSegment(tq.make_layout(n_pages, H, d, P, 8, 1))
    g = gen(1)
    K, V = (randn(g, 2, H, 40, d, dtype=torch.float16) for _ in range(2))
    slots = i32(np.stack([np.arange(40) + (n_pages - 1) * P, np.arange(40)]))
    rot = tq.tq_make_rotation(d, 5)
    tq.tq_paged_append(pool, rot, K, V, slots)
    got = tq.tq_paged_read(pool, rot, slots, dtype=torch.float32)
    one = tq.PackedSegment(tq.make_layout(2, H, d, P, 8, 1))
    tq.tq_compress(one, rot, K, V)
    want = tq.tq_read(one, rot, i32([0, 0]), 40, dtype=torch.float32)
    for x, y in zip(got, want):
        assert torch.equal(bits(x), bits(y))
