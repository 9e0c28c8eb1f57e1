"""Cases of the operators of a server whose sequences share pools of pages and whose
drafts are verified on the GPU: page tables and slot maps, writes by slot, attention
of one new token over paged segments, verification of drafted tokens.

``prepare`` makes the inputs a caller holds, ``run`` makes one pass, either in
plain torch operations (``own`` false) or through the library (``own`` true),
``exact`` computes the same in 64 bits from the definitions, ``work`` counts
the bytes and operations a pass cannot do without.

A pool is a segment whose batch axis counts pages: record (page, head, token of the
page).  Token t of sequence b lies on page table[b][t // size] at t % size; its slot
is page * size + t % size.
"""
import math

import numpy as np
import torch

own = False

SEED = 42          # rotation seed of the cache
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 32 sequences: one token each, now and then a new page; pure latency
        dict(name="pages_decode_b32", op="pages", batch=32, page=64, width=512, spare=64, most=1, drop=0.0),
        # prompts enter a running batch, short of pages for the last of them; some sequences hold nothing yet
        dict(name="pages_prompts_b64", op="pages", batch=64, page=16, width=2048, spare=20000, most=8192, drop=0.5),
        # the new token of each of 32 sequences, keys rotated as they are written
        dict(name="write_decode_b32", op="write", batch=32, tokens=1, page=64, pages=600, kv_heads=8, head_dim=128,
             kbits=3, vbits=3, rope=True),
        # a chunk of ragged prompts, pages of 128 tokens, head_dim 64, odd widths
        dict(name="write_chunk_d64", op="write", batch=7, tokens=333, page=128, pages=64, kv_heads=4, head_dim=64,
             kbits=5, vbits=2, rope=False),
        # a padded batch of prompts, keys rotated as they are written
        dict(name="write_prompt_b4_8k", op="write", batch=4, tokens=8192, page=64, pages=1024, kv_heads=8,
             head_dim=128, kbits=4, vbits=4, rope=True),
        # one sequence on a short context: latency
        dict(name="attend_b1_1k", op="attend", batch=1, q_heads=32, kv_heads=8, head_dim=128, page=64, sinks=0,
             bits="K4V4", longest=1000),
        # one sequence on a 64K context, split over its length
        dict(name="attend_b1_64k", op="attend", batch=1, q_heads=32, kv_heads=8, head_dim=128, page=64, sinks=128,
             bits="K3V3", longest=65408),
        # a batch of 32 unequal sequences, fp16 sinks beside the packed pages
        dict(name="attend_b32_ragged_16k", op="attend", batch=32, q_heads=32, kv_heads=8, head_dim=128, page=64,
             sinks=128, bits="K4V4", longest=16384),
        # head_dim 64, group of two, small pages, wide keys
        dict(name="attend_d64_b16_9k", op="attend", batch=16, q_heads=16, kv_heads=8, head_dim=64, page=16, sinks=0,
             bits="K8V3", longest=9001),
        # pages that are not compressed
        dict(name="attend_fp16_b8_4k", op="attend", batch=8, q_heads=32, kv_heads=8, head_dim=128, page=32, sinks=0,
             bits="fp16", longest=4096),
        # a chain of four drafts of one sequence that a lookup proposed (no draft distribution)
        dict(name="verify_chain4_b1", op="verify", batch=1, drafts=4, vocab=32000, dtype="fp32", tree=False,
             draft=False),
        # trees of 16 drafts of 32 sequences with the distributions they were drawn from
        dict(name="verify_tree16_b32", op="verify", batch=32, drafts=16, vocab=131072, dtype="bf16", tree=True,
             draft=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("pages", "write", "attend", "attend", "attend", "verify", "verify"))
    if op == "pages":
        batch, page = _spread(rng, 1, 256), rng.choice((16, 32, 48, 64, 128))
        most = _spread(rng, 1, max(1, 524288 // batch))
        return dict(op="pages", batch=batch, page=page, width=rng.randint(1, 1024), spare=_spread(rng, 1, 16384),
                    most=min(most, 16384), drop=rng.choice((0.0, 0.3)))
    kv = rng.choice((1, 2, 4, 8))
    if op == "write":
        d = rng.choice((64, 128, 128, 256))
        batch, page = _spread(rng, 1, 64), rng.choice((16, 48, 64, 128))
        tokens = max(1, min(_spread(rng, 1, 8192), 8192 * 4 * 8 * 128 // (batch * kv * d)))
        return dict(op="write", batch=batch, tokens=tokens, page=page,
                    pages=batch * -(-tokens // page) + batch + rng.randint(0, 100), kv_heads=kv, head_dim=d,
                    kbits=rng.randint(1, 8), vbits=rng.randint(1, 8), rope=rng.random() < 0.5)
    if op == "attend":
        d = rng.choice((64, 128, 128))
        batch = _spread(rng, 1, 64)
        longest = max(1, min(_spread(rng, 1, 65408), 32 * 16384 * 8 * 128 // (batch * kv * d)))
        return dict(op="attend", batch=batch, q_heads=kv * rng.choice((1, 2, 3, 4, 8)), kv_heads=kv, head_dim=d,
                    page=rng.choice((16, 32, 48, 64, 128, 256)), sinks=rng.choice((0, 128)), longest=longest,
                    bits=rng.choice(("fp16", f"K{rng.randint(1, 8)}V{rng.randint(1, 8)}",
                                     f"K{rng.randint(2, 4)}V{rng.randint(2, 4)}")))
    vocab = _spread(rng, 1000, 131072)
    drafts = _spread(rng, 1, 32)
    batch = max(1, min(_spread(rng, 1, 64), 32 * 16 * 131072 // (vocab * drafts)))
    return dict(op="verify", batch=batch, drafts=drafts, vocab=vocab, dtype=rng.choice(("fp16", "bf16", "fp32")),
                tree=rng.random() < 0.5, draft=rng.random() < 0.6)


def _bits(c):
    return None if c["bits"] == "fp16" else (int(c["bits"][1]), int(c["bits"][3]))


def work(c):
    if c["op"] == "pages":
        # lengths, counts and grants, an entry of the table and of the free list a page taken, a slot and a position a
        # token; half of the largest count a sequence
        tokens = c["batch"] * (c["most"] + 1) / 2
        pages = min(c["spare"], tokens / c["page"] + c["batch"] / 2)
        return {"bytes": 4 * (6 * c["batch"] + 2 * pages + 2 * c["batch"] * c["most"]), "flops": tokens}
    d = c["head_dim"] if "head_dim" in c else 0
    if c["op"] == "write":
        vectors = 2 * c["batch"] * c["tokens"] * c["kv_heads"] * 0.75
        record = d * (c["kbits"] + c["vbits"]) / 16 + 4
        # fp16 rows in, records written, records read back, fp16 rows out
        return {"bytes": vectors * (4 * d + 2 * record) + 16 * c["batch"] * c["tokens"],
                "flops": vectors * 2 * (d * math.log2(d) + 3 * d)}
    if c["op"] == "attend":
        kv = _bits(c)
        row = 4 * d if kv is None else d * sum(kv) / 8 + 8
        mean = (0.75 * c["longest"]) if c["batch"] > 1 else c["longest"]  # of the lengths drawn in prepare()
        heads = c["batch"] * c["kv_heads"]
        q = 4 * c["batch"] * c["q_heads"] * d  # queries in, results out
        return {"bytes": heads * (mean * row + c["sinks"] * 4 * d) + q + 4 * c["batch"] * mean / c["page"],
                "flops": 4.0 * c["batch"] * c["q_heads"] * d * (mean + c["sinks"])}
    # the rows of the node where the drafts end, and what the tests on the way there look up
    size = 4 if c["dtype"] == "fp32" else 2
    rows = 2 if c["draft"] else 1
    return {"bytes": c["batch"] * (rows * c["vocab"] * size + c["drafts"] * (20 + rows * size)),
            "flops": c["batch"] * rows * 2 * c["vocab"]}


# ------------------------------------------------------------------ the format
def _signs(d, seed=SEED):
    """The rotation's sign diagonal: top bits of the SplitMix64 stream."""
    m, out, state = (1 << 64) - 1, [], seed
    for _ in range(d):
        state = (state + 0x9E3779B97F4A7C15) & m
        z = ((state ^ (state >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return np.array(out)


def _hadamard(d):
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h


def _rotation(d):
    """R = D H D / sqrt(d) (symmetric, R R = 1), 64 bits."""
    s = _signs(d)
    return s[:, None] * _hadamard(d) * s[None, :] / math.sqrt(d)


_codebooks = {}


def _codebook(bits):
    """Levels and thresholds of the Lloyd-Max quantizer of N(0, 1): the upper half solves c_k = mean of the normal law
    between its thresholds, by Newton's iteration behind some sweeps of Lloyd's."""
    if bits not in _codebooks:
        half = 1 << (bits - 1)
        tail = np.vectorize(lambda x: 0.5 * math.erfc(x / math.sqrt(2)))
        dens = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731

        def means(c):
            e = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1])])
            f, t = dens(e), tail(e)
            den = t - np.append(t[1:], 0.0)
            return (f - np.append(f[1:], 0.0)) / den, e, f, den

        c = np.linspace(0.5, half - 0.5, half) * (3.2 / half if bits < 6 else 4.2 / half)
        for _ in range(400):
            c = means(c)[0]
        for _ in range(40):
            g, e, f, den = means(c)
            lo = f * (g - e) / den                                     # d mean_k / d edge_k
            hi = np.append(f[1:] * (e[1:] - g[:-1]) / den[:-1], 0.0)  # d mean_k / d edge_(k+1)
            lo[0] = 0.0                                                # the middle edge stays at 0
            J = np.eye(half)
            for k in range(half):  # d edge_k = (dc_(k-1) + dc_k) / 2
                J[k, k] -= 0.5 * (lo[k] + (hi[k] if k + 1 < half else 0.0))
                if k:
                    J[k, k - 1] -= 0.5 * lo[k]
                if k + 1 < half:
                    J[k, k + 1] -= 0.5 * hi[k]
            step = np.linalg.solve(J, g - c)
            c = c + step
            if np.max(np.abs(step)) < 1e-14:
                break
        level = np.concatenate([-c[::-1], c])
        _codebooks[bits] = (level.astype(np.float32), (0.5 * (level[1:] + level[:-1])).astype(np.float32))
    return _codebooks[bits]


def _pack(codes, bits):
    """[..., d] codes to [..., d bits / 8] bytes, least significant bit first."""
    w = codes.to(torch.int64).reshape(*codes.shape[:-1], -1, 8)
    w = (w << (bits * torch.arange(8, device=w.device))).sum(-1, keepdim=True)
    return ((w >> (8 * torch.arange(bits, device=w.device))) & 255).to(torch.uint8).flatten(-2)


def _unpack(data, bits):
    w = data.reshape(*data.shape[:-1], -1, bits).to(torch.int64)
    w = (w << (8 * torch.arange(bits, device=w.device))).sum(-1, keepdim=True)
    return ((w >> (bits * torch.arange(8, device=w.device))) & ((1 << bits) - 1)).flatten(-2)


def _rope_table(max_pos, rotary_dim, dev, base=10000.0):
    """[max_pos][2][rotary_dim / 2]: cosines and sines, the angles in 64 bits."""
    w = base ** (-2 * torch.arange(rotary_dim // 2, dtype=torch.float64, device=dev) / rotary_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * w
    return torch.stack([a.cos(), a.sin()], 1).float()


# ------------------------------------------------------------------ prepare
def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    return {"pages": _prepare_pages, "write": _prepare_write, "attend": _prepare_attend,
            "verify": _prepare_verify}[c["op"]](c, g, r, "cuda")


def _i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def _prepare_pages(c, g, r, dev):
    B, P, M = c["batch"], c["page"], c["width"]
    length = r.randint(0, M * P + 1, size=B)
    length[r.rand(B) < c["drop"]] = 0
    count = r.randint(1, c["most"] + 1, size=B)
    held = -(-length // P)
    total = B * M + c["spare"]  # (the pages that no sequence holds and that are not free are someone else's)
    order = r.permutation(total)
    table = np.full((B, M), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(total, -1)
    free[:c["spare"]] = order[at:at + c["spare"]]
    return dict(op="pages", P=P, most=c["most"], total=total, table=_i32(table, dev), length=_i32(length, dev),
                before=_i32(length, dev), count=_i32(count, dev), free=_i32(free, dev), n_free=_i32([c["spare"]], dev),
                slots=torch.empty(B, c["most"], dtype=torch.int32, device=dev),
                positions=torch.empty(B, c["most"], dtype=torch.int32, device=dev),
                granted=torch.empty(B, dtype=torch.int32, device=dev))


def _prepare_write(c, g, r, dev):
    B, H, d, S, P, n_pages = c["batch"], c["kv_heads"], c["head_dim"], c["tokens"], c["page"], c["pages"]
    scale = torch.ones(2, 1, 1, H, d, device=dev)
    for i in range(2 * H):  # four channels of each head ten times as large
        scale[i // H, 0, 0, i % H, torch.tensor(r.permutation(d)[:4], device=dev)] = 10.0
    kv = (torch.randn(2, B, S, H, d, generator=g, device=dev) * scale).half().transpose(2, 3)
    # each sequence goes on somewhere in its pages; the rows behind its last one have no slot
    count = r.randint((S + 1) // 2, S + 1, size=B)
    pages = iter(r.permutation(n_pages))
    slots = np.full((B, S), -1)
    for b in range(B):
        first = r.randint(0, P)
        own_pages = np.array([next(pages) for _ in range((first + count[b] - 1) // P + 1)])
        t = first + np.arange(count[b])
        slots[b, :count[b]] = own_pages[t // P] * P + t % P
    s = dict(op="write", K=kv[0], V=kv[1], d=d, H=H, P=P, kbits=c["kbits"], vbits=c["vbits"], slots=_i32(slots, dev),
             table=None)
    if c["rope"]:
        s["table"] = _rope_table(max(S, 32768), d, dev)
        start = torch.tensor(r.randint(0, s["table"].shape[0] - S + 1, size=B), device=dev)
        s["positions"] = (start[:, None] + torch.arange(S, device=dev)).int()
    s["R"] = torch.tensor(_rotation(d), dtype=torch.float32, device=dev)
    s["level"], s["bound"] = (torch.tensor(t, device=dev) for t in _codebook(c["vbits"]))
    if own:
        from rotated_quantized_kv_gb300 import tq
        s["rot"] = tq.tq_make_rotation(d, SEED)
        s["pool"] = tq.PackedSegment(tq.make_layout(n_pages, H, d, P, c["kbits"], c["vbits"]))
        s["rope"] = tq.Rope(s["table"], tq.TQ_ROPE_HALF) if c["rope"] else None
        s["out"] = [torch.zeros(B, H, S, d, dtype=torch.float16, device=dev) for _ in range(2)]
    return s


def _packed_pool(g, n_pages, H, P, d, kbits, vbits, dev):
    """Pages of rotated keys and values N(0, 4), some pages at a time: max |y| and RMS as scales, midrise cells and
    nearest levels as codes."""
    pool = dict(kbits=kbits, vbits=vbits, P=P,
                kcodes=torch.empty(n_pages, H, P, d * kbits // 8, dtype=torch.uint8, device=dev),
                vcodes=torch.empty(n_pages, H, P, d * vbits // 8, dtype=torch.uint8, device=dev),
                kscale=torch.empty(n_pages, H, P, device=dev), vscale=torch.empty(n_pages, H, P, device=dev))
    step = max(1, (1 << 26) // (H * P * d))
    for i in range(0, n_pages, step):
        at = slice(i, min(i + step, n_pages))
        for kind, bits in (("k", kbits), ("v", vbits)):
            y = 2 * torch.randn(at.stop - i, H, P, d, generator=g, device=dev)
            if kind == "k":
                scale = y.abs().amax(-1, keepdim=True)
                codes = torch.clamp(torch.floor((y / scale + 1) * 2 ** (bits - 1)), 0, 2**bits - 1)
            else:
                scale = y.square().mean(-1, keepdim=True).sqrt()
                codes = torch.bucketize(y / scale, torch.tensor(_codebook(bits)[1], device=dev))
            pool[kind + "codes"][at] = _pack(codes, bits)
            pool[kind + "scale"][at] = scale[..., 0]
    return pool


def _fp16_pool(g, n_pages, H, P, d, dev):
    k, v = ((2 * torch.randn(n_pages, H, P, d, generator=g, device=dev)).half() for _ in range(2))
    return dict(P=P, k=k, v=v)


def _prepare_attend(c, g, r, dev):
    B, Hq, H, d, P = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    length = r.randint((c["longest"] + 1) // 2, c["longest"] + 1, size=B) if B > 1 else np.array([c["longest"]])
    if B > 2:
        length[r.randint(B)] = r.randint(0, 2)  # one that has just begun
    held = -(-length // P)
    n_pages = int(held.sum()) + 5
    order, M = r.permutation(n_pages), -(-c["longest"] // P)
    table = np.full((B, M), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    kv = _bits(c)
    pools = [_fp16_pool(g, n_pages, H, P, d, dev) if kv is None else _packed_pool(g, n_pages, H, P, d, *kv, dev)]
    tables, lens = [_i32(table, dev)], [_i32(length, dev)]
    if c["sinks"]:  # the first positions in fp16, a row of the segment a sequence
        pools.insert(0, _fp16_pool(g, B, H, c["sinks"], d, dev))
        tables.insert(0, None)
        lens.insert(0, _i32(np.full(B, c["sinks"]), dev))
    # the queries as the projection leaves them, keys and values behind them
    q = torch.randn(B, Hq + 2 * H, d, generator=g, device=dev).half()[:, :Hq]
    s = dict(op="attend", q=q, pools=pools, tables=tables, lens=lens, H=H, d=d,
             R=torch.tensor(_rotation(d), dtype=torch.float32, device=dev),
             level=None if kv is None else torch.tensor(_codebook(kv[1])[0], device=dev))
    if own:
        from rotated_quantized_kv_gb300 import tq
        parts = []
        for p in pools:
            if "k" in p:
                parts.append(tq.Fp16Segment(p["k"].shape[0], H, d, p["P"], n_tokens=p["P"], k=p["k"], v=p["v"]))
            else:
                seg = tq.PackedSegment(tq.make_layout(n_pages, H, d, P, *kv), n_tokens=P)
                seg.kcodes, seg.vcodes, seg.kscale, seg.vscale = (p[k] for k in ("kcodes", "vcodes", "kscale", "vscale"))
                parts.append(seg)
        s["parts"], s["view"] = parts, tq.layer_view(tq.tq_make_rotation(d, SEED), parts)
        s["out"] = torch.empty(B, Hq, d, dtype=torch.float16, device=dev)
        s["ws"] = torch.empty(tq.tq_paged_workspace_size(s["view"], B, H, Hq, d), dtype=torch.uint8, device=dev)
    return s


def _prepare_verify(c, g, r, dev):
    B, N, V, dt = c["batch"], c["drafts"], c["vocab"], DTYPES[c["dtype"]]
    parents = np.tile(np.arange(-1, N - 1), (B, 1))
    if c["tree"]:  # any earlier node: siblings as well as chains
        for b in range(B):
            for i in range(1, N):
                parents[b, i] = r.randint(max(-1, i - 4), i)
    target = torch.empty(B, N + 1, V, dtype=dt, device=dev)
    draft = torch.empty(B, N + 1, V, dtype=dt, device=dev) if c["draft"] else None
    tokens = torch.empty(B, N, dtype=torch.int32, device=dev)
    up = torch.tensor(parents + 1, device=dev)
    for b in range(B):  # a draft model that is near the target
        z = 2.5 * torch.randn(N + 1, V, generator=g, device=dev)
        p, q = torch.softmax(z, -1), torch.softmax(z + 0.7 * torch.randn(N + 1, V, generator=g, device=dev), -1)
        target[b] = p.to(dt)
        if draft is not None:
            draft[b] = q.to(dt)
        cum = (q if draft is not None else p).cumsum(-1)  # a lookup's guess is a likely token too
        x = torch.rand(N, 1, generator=g, device=dev) * cum[up[b], -1:]
        tokens[b] = torch.searchsorted(cum[up[b]], x, right=True)[:, 0].clamp(max=V - 1).int()
    s = dict(op="verify", target=target, draft=draft, tokens=tokens, chain=not c["tree"], parents=_i32(parents, dev),
             uniform=torch.rand(B, N + 1, generator=g, device=dev))
    if own:
        s["out"] = [torch.empty(B, N, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev),
                    torch.empty(B, dtype=torch.int32, device=dev)]
    return s


# ------------------------------------------------------------------ run
def run(s):
    if own:
        return _run_own(s)
    return {"pages": _pages_plain, "write": _write_plain, "attend": _attend_plain, "verify": _verify_plain}[s["op"]](s)


def _run_own(s):
    from rotated_quantized_kv_gb300 import tq
    if s["op"] == "pages":
        # the step's tokens get their places, and are taken back (as drafts that were not accepted are)
        tq.tq_page_tables(s["table"], s["length"], s["count"], s["free"], s["n_free"], s["P"], s["most"],
                          out=(s["slots"], s["positions"], s["granted"]))
        tq.tq_page_release(s["table"], s["length"], s["before"], s["free"], s["n_free"], s["P"])
        return [s["slots"], s["positions"], s["granted"], s["table"], s["length"], s["free"], s["n_free"]]
    if s["op"] == "write":
        tq.tq_paged_append(s["pool"], s["rot"], s["K"], s["V"], s["slots"], rope=s["rope"],
                           positions=s["positions"] if s["rope"] else None)
        return tq.tq_paged_read(s["pool"], s["rot"], s["slots"], out=s["out"])
    if s["op"] == "attend":
        return tq.tq_paged_attention(s["view"], s["q"], s["out"], s["ws"], tables=s["tables"], lens=s["lens"])
    return tq.tq_verify(s["tokens"], s["target"], s["uniform"], draft=s["draft"],
                        parents=None if s["chain"] else s["parents"], out=s["out"])


def _pages_plain(s):
    P, M, n = s["P"], s["table"].shape[1], s["most"]
    dev = s["table"].device
    length, free = s["length"].long(), s["n_free"].long()
    want = torch.minimum(s["count"].long().clamp(0, n), M * P - length)
    held = (length + P - 1) // P
    need = (length + want + P - 1) // P - held
    base = need.cumsum(0) - need
    got = torch.minimum((free - base).clamp(min=0), need)
    granted = torch.minimum(want, (held + got) * P - length)
    k = torch.arange(M, device=dev) - held[:, None]
    new = (k >= 0) & (k < got[:, None])
    at = torch.where(new, free - 1 - base[:, None] - k, torch.zeros_like(k))
    s["table"].copy_(torch.where(new, s["free"][at], s["table"]))
    j = torch.arange(n, device=dev)
    t = length[:, None] + j
    fits = j < granted[:, None]
    page = s["table"].gather(1, torch.where(fits, t // P, torch.zeros_like(t))).long()
    slots = torch.where(fits & (page >= 0) & (page < s["total"]), page * P + t % P, torch.full_like(t, -1)).int()
    positions = torch.where(fits, t, torch.full_like(t, -1)).int()
    # what the release of the same tokens leaves: lengths and free list as they were, the table's entries stale
    return [slots, positions, granted.int(), s["table"], s["length"], s["free"], s["n_free"]]


def _rope_plain(x, table, positions):
    half = table.shape[2]
    c, t = (z[:, None] for z in table[positions.long()].unbind(2))
    a, b = x.float()[..., :half], x.float()[..., half:]
    return torch.cat([a * c - b * t, b * c + a * t], -1).to(x.dtype)


def _write_plain(s):
    K, V = s["K"], s["V"]
    if s["table"] is not None:
        K = _rope_plain(K, s["table"], s["positions"])
    k, v = K.float() @ s["R"], V.float() @ s["R"]
    m = k.abs().amax(-1, keepdim=True)
    code = torch.clamp(torch.floor((k / m + 1) * 2 ** (s["kbits"] - 1)), 0, 2 ** s["kbits"] - 1)
    sd = v.square().mean(-1, keepdim=True).sqrt()
    back = [(((2 * code + 1) / 2 ** s["kbits"] - 1) * m) @ s["R"],
            (s["level"][torch.bucketize(v / sd, s["bound"])] * sd) @ s["R"]]
    stored = (s["slots"] >= 0)[:, None, :, None]
    return [torch.where(stored, x, 0.0).half() for x in back]


def _rows_plain(s, p, table, kind):
    """[B][H][tokens][d] of a pool in the order of each sequence (rows behind its last are others')."""
    B = s["q"].shape[0]
    if table is None:
        take = lambda x: x  # noqa: E731
    else:
        at = table.long().clamp(min=0)
        take = lambda x: x[at].transpose(1, 2).flatten(2, 3)  # noqa: E731
    if "k" in p:
        return take(p[kind]).float()
    codes = _unpack(take(p[kind + "codes"]), p[kind + "bits"])
    y = (2 * codes + 1).float() / 2 ** p["kbits"] - 1 if kind == "k" else s["level"][codes]
    return (y * take(p[kind + "scale"]).reshape(B, s["H"], -1, 1)) @ s["R"]


def _attend_plain(s):
    q, H, d = s["q"].float(), s["H"], s["d"]
    B, Hq, _ = q.shape
    K = torch.cat([_rows_plain(s, p, t, "k") for p, t in zip(s["pools"], s["tables"])], 2)
    V = torch.cat([_rows_plain(s, p, t, "v") for p, t in zip(s["pools"], s["tables"])], 2)
    seen = torch.cat([torch.arange(p["P"] * (1 if t is None else t.shape[1]), device=q.device) < n[:, None]
                      for p, t, n in zip(s["pools"], s["tables"], s["lens"])], 1)[:, None, None]
    w = (q.view(B, H, Hq // H, d) @ K.transpose(2, 3)).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, (w @ V) / total, 0.0).view(B, Hq, d).half()


def _verify_plain(s):
    """Draft by draft, all sequences at once: the node each has reached, the weights it has left there."""
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniform"].double()
    B, N, V = target.shape[0], tokens.shape[1], target.shape[2]
    dev = target.device
    b = torch.arange(B, device=dev)
    zero = torch.zeros(B, dtype=torch.long, device=dev)
    node, count = zero - 1, zero.clone()
    left, mass = target[:, 0].double(), torch.ones(B, dtype=torch.float64, device=dev)
    accepted = torch.full((B, N), -1, dtype=torch.long, device=dev)
    for i in range(N):
        here = s["parents"][:, i] == node
        t = tokens[:, i]
        q = draft[b, node + 1].double() if draft is not None else torch.zeros_like(left).scatter_(1, t[:, None], 1.0)
        take = here & (u[:, i] * q[b, t] * mass < left[b, t])
        lost = here & ~take
        if draft is not None:
            rest = (left - mass[:, None] * q).clamp(min=0)
        else:
            rest = left * (1 - q)
        rest_mass = rest.sum(-1)
        row = target[b, torch.where(take, i, node) + 1].double()
        empty = rest_mass == 0  # nothing left: the target's own weights
        left = torch.where((take | (lost & empty))[:, None], row, torch.where(lost[:, None], rest, left))
        mass = torch.where(take, 1.0, torch.where(lost, torch.where(empty, row.sum(-1), rest_mass), mass))
        accepted[b, count.clamp(max=N - 1)] = torch.where(take, i, accepted[b, count.clamp(max=N - 1)])
        count, node = count + take, torch.where(take, i, node)
    cum = left.cumsum(-1)
    token = (cum > u[:, N:] * cum[:, -1:]).to(torch.uint8).argmax(-1)
    token = torch.where(cum[:, -1] > 0, token, -1)
    return [accepted.int(), count.int(), token.int()]


# ------------------------------------------------------------------ exact
def exact(c, seed):
    """What run() returns, in 64 bits, from the operators' definitions."""
    s = prepare(c, seed)
    return {"pages": _exact_pages, "write": _exact_write, "attend": _exact_attend, "verify": _exact_verify}[c["op"]](c, s)


def _exact_pages(c, s):
    """Sequence after sequence, page after page, with a list for the free ones."""
    P, B, M = c["page"], c["batch"], c["width"]
    table, free = s["table"].cpu().numpy(), s["free"].cpu().numpy()[:c["spare"]].tolist()
    length, count = s["length"].cpu().numpy(), s["count"].cpu().numpy()
    slots, positions = np.full((B, c["most"]), -1), np.full((B, c["most"]), -1)
    granted = np.zeros(B, int)
    wanted_before = 0
    for b in range(B):
        end = min(length[b] + count[b], M * P)
        pages = list(range(-(-length[b] // P), -(-end // P)))
        share = max(c["spare"] - wanted_before, 0)  # a sequence short of pages does not give way to a later one
        wanted_before += len(pages)
        for m in pages[:share]:
            table[b, m] = free.pop()
        end = min(end, (-(-length[b] // P) + min(share, len(pages))) * P)
        granted[b] = max(end - length[b], 0)
        t = np.arange(length[b], length[b] + granted[b])
        slots[b, :granted[b]] = table[b, t // P] * P + t % P
        positions[b, :granted[b]] = t
    dev = s["table"].device
    return [_i32(slots, dev), _i32(positions, dev), _i32(granted, dev), _i32(table, dev), s["length"], s["free"],
            s["n_free"]]


def _exact_write(c, s):
    B, H, S, d = s["K"].shape
    R = torch.tensor(_rotation(d), dtype=torch.float64, device="cuda")
    level, bound = (torch.tensor(t, dtype=torch.float64, device="cuda") for t in _codebook(c["vbits"]))
    K = s["K"]
    if c["rope"]:
        t = s["table"].double()[s["positions"].long()][:, None]
        z = torch.complex(K[..., :d // 2].double(), K[..., d // 2:].double()) * torch.complex(t[:, :, :, 0], t[:, :, :, 1])
        K = torch.cat([z.real, z.imag], -1).half()
    out = [torch.zeros(B, H, S, d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for b in range(B):
        at = torch.nonzero(s["slots"][b] >= 0)[:, 0]
        y = torch.einsum("htd,de->hte", K[b][:, at].double(), R)
        top = y.abs().amax(-1, keepdim=True)
        cell = torch.floor((y / top + 1) * 2.0 ** (c["kbits"] - 1)).clamp(0, 2 ** c["kbits"] - 1)
        out[0][b][:, at] = torch.einsum("htd,de->hte", ((cell + 0.5) * 2.0 ** (1 - c["kbits"]) - 1) * top, R)
        y = torch.einsum("htd,de->hte", s["V"][b][:, at].double(), R)
        rms = (y * y).mean(-1, keepdim=True).sqrt()
        cell = torch.zeros_like(y, dtype=torch.long)
        for t in bound:
            cell += y / rms > t
        out[1][b][:, at] = torch.einsum("htd,de->hte", level[cell] * rms, R)
    return out


def _exact_rows(p, kind, pages, n):
    """The first n rotated (or fp16) rows of a list of pages, 64 bits: bit j of code i is bit (i bits + j) of the record."""
    if "k" in p:
        return p[kind][pages].double().transpose(0, 1).flatten(1, 2)[:, :n]
    bits = p[kind + "bits"]
    data = p[kind + "codes"][pages].transpose(0, 1).flatten(1, 2)[:, :n]
    stream = (data[..., None] >> torch.arange(8, device=data.device, dtype=torch.uint8)) & 1
    stream = stream.flatten(-2).unflatten(-1, (-1, bits))
    code = (stream.to(torch.int32) << torch.arange(bits, device=data.device, dtype=torch.int32)).sum(-1)
    scale = p[kind + "scale"][pages].transpose(0, 1).flatten(1, 2)[:, :n, None].double()
    if kind == "k":
        return scale * ((code.double() + 0.5) * 2.0 ** (1 - bits) - 1)
    return scale * torch.tensor(_codebook(bits)[0], dtype=torch.float64, device=data.device)[code]


def _exact_attend(c, s):
    B, Hq, H, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    R = torch.tensor(_rotation(d), dtype=torch.float64, device="cuda")
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    for b in range(B):
        ks, vs = [], []
        for p, table, lens in zip(s["pools"], s["tables"], s["lens"]):
            n = int(lens[b])
            pages = torch.tensor([b], device="cuda") if table is None else table[b, :-(-n // p["P"])].long()
            for rows, kind in ((ks, "k"), (vs, "v")):
                x = _exact_rows(p, kind, pages, n)
                rows.append(x if "k" in p else torch.einsum("htd,de->hte", x, R))
        K, V = torch.cat(ks, 1), torch.cat(vs, 1)
        if K.shape[1]:
            z = torch.einsum("hgd,htd->hgt", s["q"][b].double().unflatten(0, (H, -1)), K) / math.sqrt(d)
            out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), V).flatten(0, 1)
    return out


def _exact_verify(c, s):
    """Sequence by sequence, child by child."""
    B, N = c["batch"], c["drafts"]
    tokens, parents, u = s["tokens"].tolist(), s["parents"].tolist(), s["uniform"].double().tolist()
    accepted, counts, drawn = np.full((B, N), -1), np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        node, path, going = -1, [], True
        while going:
            p, going = s["target"][b, node + 1].double(), False
            left, mass = p, 1.0
            for i in [i for i in range(N) if parents[b][i] == node]:
                t = tokens[b][i]
                q = float(s["draft"][b, node + 1, t]) if s["draft"] is not None else 1.0
                if u[b][i] * q * mass < float(left[t]):
                    node, going = i, True
                    path.append(i)
                    break
                if s["draft"] is not None:
                    rest = torch.relu(left - mass * s["draft"][b, node + 1].double())
                else:
                    rest = left.clone()
                    rest[t] = 0.0
                left = rest if float(rest.sum()) > 0 else p
                mass = float(left.sum())
        accepted[b, :len(path)], counts[b] = path, len(path)
        cum = torch.cumsum(left, 0)
        drawn[b] = int(torch.searchsorted(cum, cum[-1] * u[b][N], right=True)) if float(cum[-1]) > 0 else -1
    dev = s["tokens"].device
    return [_i32(accepted, dev), _i32(counts, dev), _i32(drawn, dev)]
