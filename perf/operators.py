"""Cases of the operators around the compressed cache: rotary positions, the
ragged write into a packed segment, the read back, and attention of a tree of
drafted tokens over the cache.

``prepare`` makes the inputs a caller holds, ``run`` makes one pass, either in
plain torch operations (``own`` false) or through the library (``own`` true),
``exact`` computes the same in 64 bits from the definitions, ``work`` counts
the bytes and operations a pass cannot do without.
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
        # one token of one sequence before a decode step: pure latency
        dict(name="rope_decode_1", op="rope", dtype="fp16", batch=1, tokens=1, q_heads=32, kv_heads=8, head_dim=128,
             rotary_dim=128, layout="half", inverse=False, token_major=True, max_pos=32768),
        # a prompt of 16K tokens, queries and keys as the projection leaves them (token-major)
        dict(name="rope_prompt_16k", op="rope", dtype="fp16", batch=1, tokens=16384, q_heads=32, kv_heads=8,
             head_dim=128, rotary_dim=128, layout="half", inverse=False, token_major=True, max_pos=131072),
        # interleaved pairs on a part of a wide head, bf16, an odd length, head-major: the transpose (gradient) direction
        dict(name="rope_part_inverse", op="rope", dtype="bf16", batch=3, tokens=1021, q_heads=16, kv_heads=4,
             head_dim=256, rotary_dim=96, layout="interleaved", inverse=True, token_major=False, max_pos=4096),
        # the accepted rows of 32 sequences' draft trees (up to 16 of 24) written at their own positions
        dict(name="write_accepted_b32", op="write", batch=32, tokens=16, source=24, capacity=4096, kv_heads=8,
             head_dim=128, kbits=3, vbits=3, rope=False, gather=True),
        # one 64-token chunk of one sequence, rotated by its positions as it is written
        dict(name="write_chunk_64", op="write", batch=1, tokens=64, source=64, capacity=16384, kv_heads=8,
             head_dim=128, kbits=8, vbits=3, rope=True, gather=False),
        # a padded batch of prompts, keys rotated as they are written
        dict(name="write_prompt_b4_8k", op="write", batch=4, tokens=8192, source=8192, capacity=8192, kv_heads=8,
             head_dim=128, kbits=4, vbits=4, rope=True, gather=False),
        # head_dim 64, odd widths, a ragged chunk
        dict(name="read_d64_ragged", op="read", batch=5, tokens=777, capacity=2048, kv_heads=8, head_dim=64, kbits=5,
             vbits=2, dtype="bf16"),
        # the whole of a 64K context back in fp16 (handing a cache over, a prefill over stored keys)
        dict(name="read_64k", op="read", batch=1, tokens=65408, capacity=65408, kv_heads=8, head_dim=128, kbits=3,
             vbits=3, dtype="fp16"),
        # a small tree of one sequence on a short context: latency
        dict(name="tree_8_b1_1k", op="tree", batch=1, drafts=8, q_heads=32, kv_heads=8, head_dim=128, sinks=128,
             packed="K4V4:895", window=17, ragged=False),
        # 16 drafts over the 64K context of one sequence
        dict(name="tree_16_b1_64k", op="tree", batch=1, drafts=16, q_heads=32, kv_heads=8, head_dim=128, sinks=128,
             packed="K3V3:65408", window=33, ragged=False),
        # 64 drafts over age tiers (fp16 / K4V4 / K3V2) of a batch of unequal sequences
        dict(name="tree_64_tiers_ragged", op="tree", batch=4, drafts=64, q_heads=32, kv_heads=8, head_dim=128, sinks=0,
             packed="K3V2:24576,K4V4:7168", window=1024, ragged=True),
        # head_dim 64, group of two, a batch of 16, odd counts
        dict(name="tree_13_d64_b16", op="tree", batch=16, drafts=13, q_heads=16, kv_heads=8, head_dim=64, sinks=128,
             packed="K8V3:9001", window=61, ragged=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "tree", "tree"))
    if op == "rope":
        d = rng.choice((64, 128, 256))
        batch = _spread(rng, 1, 32)
        hq = rng.choice((8, 16, 32))
        tokens = max(1, min(_spread(rng, 1, 16384), 16384 * 32 * 128 // (batch * hq * d)))
        return dict(op="rope", dtype=rng.choice(("fp16", "bf16", "fp32")), batch=batch, tokens=tokens, q_heads=hq,
                    kv_heads=rng.choice((1, 2, 4, 8)), head_dim=d,
                    rotary_dim=rng.choice((d, d, d // 2, 3 * d // 4, 2 * rng.randint(1, d // 2))),
                    layout=rng.choice(("half", "interleaved")), inverse=rng.random() < 0.3,
                    token_major=rng.random() < 0.6, max_pos=max(tokens, rng.choice((4096, 32768, 131072))))
    kv = rng.choice((1, 4, 8))
    d = rng.choice((64, 128, 128, 256))
    if op == "write":
        batch = _spread(rng, 1, 32)
        tokens = max(1, min(_spread(rng, 1, 8192), 8192 * 4 * 8 * 128 // (batch * kv * d)))
        gather = tokens <= 64 and rng.random() < 0.6
        source = tokens + rng.randint(0, 16) if gather else tokens
        return dict(op="write", batch=batch, tokens=tokens, source=source,
                    capacity=-(-(tokens + rng.randint(0, 500)) // 16) * 16, kv_heads=kv, head_dim=d,
                    kbits=rng.randint(1, 8), vbits=rng.randint(1, 8), rope=rng.random() < 0.5, gather=gather)
    if op == "read":
        batch = _spread(rng, 1, 16)
        tokens = max(1, min(_spread(rng, 1, 65408), 65408 * 8 * 128 // (batch * kv * d)))
        return dict(op="read", batch=batch, tokens=tokens, capacity=-(-(tokens + rng.randint(0, 300)) // 16) * 16,
                    kv_heads=kv, head_dim=d, kbits=rng.randint(1, 8), vbits=rng.randint(1, 8),
                    dtype=rng.choice(("fp16", "bf16", "fp32")))
    d = rng.choice((64, 128, 128))
    gqa = rng.choice((1, 2, 4, 8))
    drafts = _spread(rng, 1, 64)
    batch = _spread(rng, 1, 16)
    most = 4 * 64 * 32 * 32768 * 128  # operations of the largest listed tree, about
    cached = max(1, min(_spread(rng, 1, 65408), most // (batch * drafts * kv * gqa * d), 524288 // batch))
    two = cached > 64 and rng.random() < 0.4
    a = rng.randint(1, cached - 1) if two else cached
    widths = [f"K{rng.randint(1, 8)}V{rng.randint(1, 8)}:{n}" for n in ((a, cached - a) if two else (cached,))]
    return dict(op="tree", batch=batch, drafts=drafts, q_heads=kv * gqa, kv_heads=kv, head_dim=d,
                sinks=rng.choice((0, 128)), packed=",".join(widths), window=rng.randint(0, 64),
                ragged=rng.random() < 0.5)


def work(c):
    if c["op"] == "rope":
        n = c["batch"] * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["head_dim"]
        r = c["rotary_dim"] / c["head_dim"]
        size = 4 if c["dtype"] == "fp32" else 2
        table = min(c["batch"] * c["tokens"], c["max_pos"]) * c["rotary_dim"] * 4
        return {"bytes": 2 * n * size + table + 4 * c["batch"] * c["tokens"], "flops": 3 * n * r}
    d = c["head_dim"]
    if c["op"] == "tree":
        rows = c["drafts"] * c["q_heads"] // c["kv_heads"]
        heads = c["batch"] * c["kv_heads"]
        packed = [(k, v, n) for k, v, n in _segments(c)]
        fp16 = c["sinks"] + c["window"] + c["drafts"]
        share = 0.75 if c["ragged"] else 1.0  # mean of the lengths drawn in prepare()
        total = sum(n for _, _, n in packed) * share + fp16
        size = sum(n * (d * (k + v) / 8 + 8) for k, v, n in packed) * share + fp16 * 4 * d + rows * 4 * d
        return {"bytes": heads * size, "flops": 4.0 * heads * rows * d * total}
    vectors = 2 * c["batch"] * c["tokens"] * c["kv_heads"]
    record = d * (c["kbits"] + c["vbits"]) / 16 + 4
    out = (4 if c.get("dtype") == "fp32" else 2) * d
    rotate = d * math.log2(d)
    if c["op"] == "read":
        return {"bytes": vectors * (record + out), "flops": vectors * (rotate + 2 * d)}
    # fp16 rows in, records written, records read back, fp16 rows out
    return {"bytes": vectors * 0.75 * (4 * d + 2 * record), "flops": vectors * 0.75 * 2 * (rotate + 3 * d)}


def _segments(c):
    parts = [p.split(":") for p in c["packed"].split(",")]
    return [(int(w[1]), int(w[3]), int(n)) for w, n in parts]


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
    """Levels and thresholds of the Lloyd-Max quantizer of N(0, 1): Newton's iteration on the centroid condition of
    the upper half, after some sweeps of Lloyd's."""
    if bits not in _codebooks:
        half = 1 << (bits - 1)
        tail = np.vectorize(lambda x: 0.5 * math.erfc(x / math.sqrt(2)))
        dens = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731

        def means(c):
            e = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1])])
            f, t = dens(e), tail(e)
            num = f - np.append(f[1:], 0.0)
            den = t - np.append(t[1:], 0.0)
            return num / den, e, f, den

        c = np.linspace(0.5, half - 0.5, half) * (3.2 / half if bits < 6 else 4.2 / half)
        for _ in range(400):
            c = means(c)[0]
        for _ in range(40):
            g, e, f, den = means(c)
            lo = f * (g - e) / den                                     # d mean_k / d edge_k
            hi = np.append(f[1:] * (e[1:] - g[:-1]) / den[:-1], 0.0)  # d mean_k / d edge_(k+1)
            lo[0] = 0.0                                                # the middle edge stays at 0
            J = np.eye(half)
            for k in range(half):
                # d edge_k = (dc_(k-1) + dc_k) / 2
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


def _store(y, kind, bits):
    """Codes and scale of rotated vectors, as a cache of this format holds them."""
    if kind == "k":
        m = y.abs().amax(-1, keepdim=True)
        return torch.clamp(torch.floor((y / m + 1) * 2 ** (bits - 1)), 0, 2**bits - 1), m[..., 0]
    s = y.square().mean(-1, keepdim=True).sqrt()
    return torch.bucketize(y / s, torch.tensor(_codebook(bits)[1], device=y.device)), s[..., 0]


def _packed_segment(g, B, H, n, d, kbits, vbits, dev):
    """A packed segment with n stored tokens: rotated keys and values N(0, 4) (four channels of 128 ten times as large
    spread to that by the rotation), made and packed one sequence at a time."""
    cap = -(-n // 16) * 16
    seg = dict(kbits=kbits, vbits=vbits, n=n, cap=cap,
               kcodes=torch.zeros(B, H, cap, d * kbits // 8, dtype=torch.uint8, device=dev),
               vcodes=torch.zeros(B, H, cap, d * vbits // 8, dtype=torch.uint8, device=dev),
               kscale=torch.zeros(B, H, cap, device=dev), vscale=torch.zeros(B, H, cap, device=dev))
    for b in range(B):
        for kind, bits in (("k", kbits), ("v", vbits)):
            y = 2 * torch.randn(H, n, d, generator=g, device=dev)
            codes, scale = _store(y, kind, bits)
            seg[kind + "codes"][b, :, :n] = _pack(codes, bits)
            seg[kind + "scale"][b, :, :n] = scale
    return seg


def _handle(seg, B, H, d):
    """The library's segment over the same bytes."""
    from rotated_quantized_kv_gb300 import tq
    p = tq.PackedSegment(tq.make_layout(B, H, d, seg["cap"], seg["kbits"], seg["vbits"]), n_tokens=seg["n"])
    p.kcodes, p.vcodes, p.kscale, p.vscale = (seg[k] for k in ("kcodes", "vcodes", "kscale", "vscale"))
    return p


def _rope_table(max_pos, rotary_dim, dev, base=10000.0):
    """[max_pos][2][rotary_dim / 2]: cosines and sines, the angles in 64 bits."""
    w = base ** (-2 * torch.arange(rotary_dim // 2, dtype=torch.float64, device=dev) / rotary_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * w
    return torch.stack([a.cos(), a.sin()], 1).float()


# ------------------------------------------------------------------ prepare
def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    return {"rope": _prepare_rope, "write": _prepare_write, "read": _prepare_read, "tree": _prepare_tree}[c["op"]](
        c, g, r, dev)


def _prepare_rope(c, g, r, dev):
    B, T, d, dt = c["batch"], c["tokens"], c["head_dim"], DTYPES[c["dtype"]]
    H = c["q_heads"] + c["kv_heads"]
    # queries and keys are slices of one projection's output, the values behind them
    if c["token_major"]:
        x = torch.randn(B, T, H + c["kv_heads"], d, generator=g, device=dev).to(dt).transpose(1, 2)
    else:
        x = torch.randn(B, H + c["kv_heads"], T, d, generator=g, device=dev).to(dt)
    first = torch.tensor(r.randint(0, c["max_pos"] - T + 1, size=B), device=dev)
    s = dict(op="rope", q=x[:, :c["q_heads"]], k=x[:, c["q_heads"]:H], layout=c["layout"], inverse=c["inverse"],
             positions=(first[:, None] + torch.arange(T, device=dev)).int(),
             table=_rope_table(c["max_pos"], c["rotary_dim"], dev))
    if own:
        from rotated_quantized_kv_gb300 import tq
        s["rope"] = tq.Rope(s["table"], getattr(tq, "TQ_ROPE_" + c["layout"].upper()))
        s["out"] = [torch.empty_like(s["q"], memory_format=torch.preserve_format),
                    torch.empty_like(s["k"], memory_format=torch.preserve_format)]
    return s


def _prepare_write(c, g, r, dev):
    B, H, d, S, n = c["batch"], c["kv_heads"], c["head_dim"], c["source"], c["tokens"]
    scale = torch.ones(2, 1, 1, H, d, device=dev)
    for i in range(2 * H):  # four channels of each head ten times as large
        scale[i // H, 0, 0, i % H, torch.tensor(r.permutation(d)[:4], device=dev)] = 10.0
    kv = (torch.randn(2, B, S, H, d, generator=g, device=dev) * scale).half().transpose(2, 3)
    count = r.randint((n + 1) // 2, n + 1, size=B)
    first = np.array([r.randint(0, c["capacity"] - m + 1) for m in count])
    s = dict(op="write", K=kv[0], V=kv[1], n=n, d=d, H=H, cap=c["capacity"], kbits=c["kbits"], vbits=c["vbits"],
             count=torch.tensor(count, dtype=torch.int32, device=dev),
             first=torch.tensor(first, dtype=torch.int32, device=dev), index=None, table=None)
    if c["gather"]:
        rows = np.stack([np.sort(r.permutation(S)[:n]) for _ in range(B)])
        s["index"] = torch.tensor(rows, dtype=torch.int32, device=dev)
    if c["rope"]:
        s["table"] = _rope_table(max(c["capacity"], S), d, dev)
        start = torch.tensor(r.randint(0, s["table"].shape[0] - S + 1, size=B), device=dev)
        s["positions"] = (start[:, None] + torch.arange(S, device=dev)).int()
    s["R"] = torch.tensor(_rotation(d), dtype=torch.float32, device=dev)
    s["level"], s["bound"] = (torch.tensor(t, device=dev) for t in _codebook(c["vbits"]))
    if own:
        from rotated_quantized_kv_gb300 import tq
        s["rot"] = tq.tq_make_rotation(d, SEED)
        s["seg"] = tq.PackedSegment(tq.make_layout(B, H, d, c["capacity"], c["kbits"], c["vbits"]))
        s["rope"] = tq.Rope(s["table"], tq.TQ_ROPE_HALF) if c["rope"] else None
        s["out"] = [torch.zeros(B, H, n, d, dtype=torch.float16, device=dev) for _ in range(2)]
    return s


def _prepare_read(c, g, r, dev):
    B, H, d, n = c["batch"], c["kv_heads"], c["head_dim"], c["tokens"]
    seg = _packed_segment(g, B, H, c["capacity"], d, c["kbits"], c["vbits"], dev)
    first = torch.tensor([r.randint(0, c["capacity"] - n + 1) for _ in range(B)], dtype=torch.int32, device=dev)
    s = dict(op="read", seg=seg, first=first, n=n, d=d, dtype=DTYPES[c["dtype"]],
             R=torch.tensor(_rotation(d), dtype=torch.float32, device=dev),
             level=torch.tensor(_codebook(c["vbits"])[0], device=dev))
    if own:
        from rotated_quantized_kv_gb300 import tq
        s["rot"], s["handle"] = tq.tq_make_rotation(d, SEED), _handle(seg, B, H, d)
        s["out"] = [torch.empty(B, H, n, d, dtype=s["dtype"], device=dev) for _ in range(2)]
    return s


def _prepare_tree(c, g, r, dev):
    B, N, Hq, H, d = c["batch"], c["drafts"], c["q_heads"], c["kv_heads"], c["head_dim"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    seg = [_packed_segment(g, B, H, n, d, k, v, dev) for k, v, n in _segments(c)]
    fp16 = lambda n: dict(k=(2 * rand(B, H, n, d)).half(), v=(2 * rand(B, H, n, d)).half(), n=n, cap=n)  # noqa: E731
    segs = ([fp16(c["sinks"])] if c["sinks"] else []) + seg + ([fp16(c["window"])] if c["window"] else [])
    # unequal sequences: each packed and window segment is filled to half at least
    lens = [torch.tensor([r.randint((p["n"] + 1) // 2, p["n"] + 1) if c["ragged"] and i >= (c["sinks"] > 0) else p["n"]
                          for _ in range(B)], dtype=torch.int32, device=dev) for i, p in enumerate(segs)]
    # draft trees: the parent of node i is one of the nodes before it (-1: the last cached token), and a node sees
    # itself and its ancestors
    see = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N):
            parent = r.randint(max(-1, i - 4), i) if i else -1
            see[b, i] = see[b, parent] if parent >= 0 else False
            see[b, i, i] = True
    words = -(-N // 32)
    bits = np.zeros((B, N, words * 32), np.int64)
    bits[:, :, :N] = see
    mask = (bits.reshape(B, N, words, 32) << np.arange(32)).sum(-1).astype(np.uint32).view(np.int32)
    # queries, keys and values of the drafts as the projection leaves them, token-major
    qkv = rand(B, N, Hq + 2 * H, d).half()
    s = dict(op="tree", q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + H].transpose(1, 2), v=qkv[:, :, Hq + H:].transpose(1, 2),
             segs=segs, lens=lens, mask=torch.tensor(mask, device=dev), H=H, d=d,
             R=torch.tensor(_rotation(d), dtype=torch.float32, device=dev),
             levels={p["vbits"]: torch.tensor(_codebook(p["vbits"])[0], device=dev) for p in seg})
    if own:
        from rotated_quantized_kv_gb300 import tq
        parts = [_handle(p, B, H, d) if "kbits" in p else
                 tq.Fp16Segment(B, H, d, p["cap"], n_tokens=p["n"], k=p["k"], v=p["v"]) for p in segs]
        s["parts"] = parts
        s["view"] = tq.layer_view(tq.tq_make_rotation(d, SEED), parts)
        s["out"] = torch.empty(B, N, Hq, d, dtype=torch.float16, device=dev)
        s["ws"] = torch.empty(tq.tq_tree_workspace_size(s["view"], B, H, Hq, N, d), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ run
def run(s):
    if s["op"] == "rope":
        if own:
            from rotated_quantized_kv_gb300 import tq
            return tq.tq_rope(s["rope"], s["positions"], [s["q"], s["k"]], out=s["out"], inverse=s["inverse"])
        return [_rope_plain(x, s["table"], s["positions"], s["layout"], s["inverse"]) for x in (s["q"], s["k"])]
    if s["op"] == "write":
        if own:
            from rotated_quantized_kv_gb300 import tq
            tq.tq_append(s["seg"], s["rot"], s["K"], s["V"], s["first"], n_new=s["count"], index=s["index"], n_max=s["n"],
                         rope=s["rope"], positions=s["positions"] if s["rope"] else None)
            return tq.tq_read(s["seg"], s["rot"], s["first"], s["n"], n_read=s["count"], out=s["out"])
        return _write_plain(s)
    if s["op"] == "read":
        if own:
            from rotated_quantized_kv_gb300 import tq
            return tq.tq_read(s["handle"], s["rot"], s["first"], s["n"], out=s["out"])
        return _read_plain(s)
    if own:
        from rotated_quantized_kv_gb300 import tq
        return tq.tq_tree_attention(s["view"], s["q"], s["k"], s["v"], s["out"], s["ws"], mask=s["mask"],
                                    seg_len=s["lens"])
    return _tree_plain(s)


def _rope_plain(x, table, positions, layout, inverse):
    half = table.shape[2]
    c, t = table[positions.long()].unbind(2)          # [B][T][half]
    c, t = c[:, None], (-t if inverse else t)[:, None]
    y = x.float()
    if layout == "half":
        a, b = y[..., :half], y[..., half:2 * half]
        z = torch.cat([a * c - b * t, b * c + a * t], -1)
    else:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        z = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    return torch.cat([z, y[..., 2 * half:]], -1).to(x.dtype)


def _levels(codes, kind, bits, level):
    """The value each code stands for, before its scale."""
    return (2 * codes + 1).float() / 2**bits - 1 if kind == "k" else level[codes]


def _write_plain(s):
    K, V = s["K"], s["V"]
    if s["table"] is not None:
        K = _rope_plain(K, s["table"], s["positions"], "half", False)
    if s["index"] is not None:
        at = s["index"].long()[:, None, :, None].expand(-1, s["H"], -1, s["d"])
        K, V = K.gather(2, at), V.gather(2, at)
    else:
        K, V = K[:, :, :s["n"]], V[:, :, :s["n"]]
    k, v = K.float() @ s["R"], V.float() @ s["R"]
    m = k.abs().amax(-1, keepdim=True)
    code = torch.clamp(torch.floor((k / m + 1) * 2 ** (s["kbits"] - 1)), 0, 2 ** s["kbits"] - 1).long()
    sd = v.square().mean(-1, keepdim=True).sqrt()
    back = [(_levels(code, "k", s["kbits"], None) * m) @ s["R"],
            (s["level"][torch.bucketize(v / sd, s["bound"])] * sd) @ s["R"]]
    new = torch.arange(s["n"], device=k.device) < s["count"][:, None]
    return [torch.where(new[:, None, :, None], x, 0.0).half() for x in back]


def _stored(seg, kind, R, level):
    """The rows a packed segment stands for: R (scale level(code))."""
    codes = _unpack(seg[kind + "codes"], seg[kind + "bits"])
    return (_levels(codes, kind, seg[kind + "bits"], level) * seg[kind + "scale"][..., None]) @ R


def _read_plain(s):
    at = s["first"].long()[:, None] + torch.arange(s["n"], device=s["first"].device)
    b = torch.arange(at.shape[0], device=at.device)[:, None]
    seg = {k: (v[b, :, at].transpose(1, 2) if isinstance(v, torch.Tensor) else v) for k, v in s["seg"].items()}
    return [_stored(seg, kind, s["R"], s["level"]).to(s["dtype"]) for kind in ("k", "v")]


def _tree_plain(s):
    q, H, d = s["q"], s["H"], s["d"]
    B, N, Hq, _ = q.shape
    dev = q.device
    rows = [(_stored(p, "k", s["R"], None), _stored(p, "v", s["R"], s["levels"][p["vbits"]])) if "kbits" in p else
            (p["k"].float(), p["v"].float()) for p in s["segs"]] + [(s["k"].float(), s["v"].float())]
    K, V = torch.cat([k for k, _ in rows], 2), torch.cat([v for _, v in rows], 2)
    seen = [(torch.arange(p["cap"], device=dev) < n[:, None])[:, None].expand(B, N, -1)
            for p, n in zip(s["segs"], s["lens"])]
    j = torch.arange(N, device=dev)
    seen.append((s["mask"][:, :, j // 32] >> (j % 32)) & 1 > 0)
    g = Hq // H
    seen = torch.cat(seen, 2).repeat_interleave(g, 1)[:, None]   # query rows (draft, head of the group)
    x = q.float().view(B, N, H, g, d).permute(0, 2, 1, 3, 4).reshape(B, H, N * g, d)
    w = (x @ K.transpose(2, 3)).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    o = (w @ V) / w.sum(-1, keepdim=True)
    return o.view(B, H, N, g, d).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d).half()


# ------------------------------------------------------------------ exact
def exact(c, seed):
    """What run() returns, in 64 bits, from the operators' definitions."""
    s = prepare(c, seed)
    if c["op"] == "rope":
        return [_exact_rope(x, s, c["layout"], c["inverse"]) for x in (s["q"], s["k"])]
    R = torch.tensor(_rotation(c["head_dim"]), dtype=torch.float64, device="cuda")
    if c["op"] == "write":
        return _exact_write(c, s, R)
    if c["op"] == "read":
        out = []
        for kind in ("k", "v"):
            y = torch.stack([_exact_rows(s["seg"], kind, b, int(s["first"][b]), c["tokens"]) for b in
                             range(c["batch"])])
            out.append(torch.einsum("bhtd,de->bhte", y, R))
        return out
    return _exact_tree(c, s, R)


def _exact_rope(x, s, layout, inverse):
    B, H, T, d = x.shape
    z = x.double().clone()
    t = s["table"].double()[s["positions"].long()]
    half = t.shape[-2:][1]
    first, step = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2),
                                                                                  slice(1, 2 * half, 2))
    turn = torch.complex(t[:, None, :, 0], t[:, None, :, 1])
    w = torch.complex(z[..., first], z[..., step]) * (turn.conj() if inverse else turn)
    z[..., first], z[..., step] = w.real, w.imag
    return z


def _exact_write(c, s, R):
    n, d = c["tokens"], c["head_dim"]
    level, bound = (torch.tensor(t, dtype=torch.float64, device="cuda") for t in _codebook(c["vbits"]))
    out = [torch.zeros(c["batch"], c["kv_heads"], n, d, dtype=torch.float64, device="cuda") for _ in range(2)]
    K = _exact_rope(s["K"], s, "half", False).half() if c["rope"] else s["K"]
    for b in range(c["batch"]):
        m = int(s["count"][b])
        at = s["index"][b, :m].long() if c["gather"] else torch.arange(m, device="cuda")
        y = torch.einsum("htd,de->hte", K[b][:, at].double(), R)
        top = y.abs().amax(-1, keepdim=True)
        cell = torch.floor((y / top + 1) * 2.0 ** (c["kbits"] - 1)).clamp(0, 2 ** c["kbits"] - 1)
        out[0][b, :, :m] = torch.einsum("htd,de->hte", ((cell + 0.5) * 2.0 ** (1 - c["kbits"]) - 1) * top, R)
        y = torch.einsum("htd,de->hte", s["V"][b][:, at].double(), R)
        rms = (y * y).mean(-1, keepdim=True).sqrt()
        u = y / rms
        cell = torch.zeros_like(u, dtype=torch.long)
        for t in bound:
            cell += u > t
        out[1][b, :, :m] = torch.einsum("htd,de->hte", level[cell] * rms, R)
    return out


def _exact_rows(seg, kind, b, t0, n):
    """Rotated rows [t0, t0 + n) of sequence b, 64 bits: bit j of code i is bit (i bits + j) of the record."""
    bits = seg[kind + "bits"]
    data = seg[kind + "codes"][b, :, t0:t0 + n]
    stream = (data[..., None] >> torch.arange(8, device=data.device, dtype=torch.uint8)) & 1
    stream = stream.flatten(-2).unflatten(-1, (-1, bits))
    code = (stream.to(torch.int32) << torch.arange(bits, device=data.device, dtype=torch.int32)).sum(-1)
    scale = seg[kind + "scale"][b, :, t0:t0 + n, None].double()
    if kind == "k":
        return scale * ((code.double() + 0.5) * 2.0 ** (1 - bits) - 1)
    return scale * torch.tensor(_codebook(bits)[0], dtype=torch.float64, device=data.device)[code]


def _exact_tree(c, s, R):
    B, N, Hq, H, d = c["batch"], c["drafts"], c["q_heads"], c["kv_heads"], c["head_dim"]
    if 4.0 * B * N * Hq * d * sum(p["n"] for p in s["segs"]) > 4e12:
        return None
    g, out = Hq // H, torch.zeros(B, N, Hq, d, dtype=torch.float64, device="cuda")
    tree = s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        ks, vs = [], []
        for p, n in zip(s["segs"], s["lens"]):
            n = int(n[b])
            if "kbits" in p:
                ks.append(torch.einsum("htd,de->hte", _exact_rows(p, "k", b, 0, n), R))
                vs.append(torch.einsum("htd,de->hte", _exact_rows(p, "v", b, 0, n), R))
            else:
                ks.append(p["k"][b, :, :n].double())
                vs.append(p["v"][b, :, :n].double())
        K, V = torch.cat(ks + [s["k"][b].double()], 1), torch.cat(vs + [s["v"][b].double()], 1)
        dark = torch.tensor([[not (int(tree[b, i, j // 32]) >> (j % 32)) & 1 for j in range(N)] for i in range(N)],
                            device="cuda")
        for h in range(Hq):
            z = s["q"][b, :, h].double() @ K[h // g].T / math.sqrt(d)
            z[:, -N:].masked_fill_(dark, -math.inf)
            out[b, :, h] = torch.softmax(z, -1) @ V[h // g]
    return out
