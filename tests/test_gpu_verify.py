"""Verification of drafted tokens on the GPU against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from test_gpu_serving import DEV, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from rotated_quantized_kv_gb300 import tq as T
    return T


def weights(row):
    x = row.double().cpu().numpy()
    return np.where((x > 0) & (x < 2.0**90), x, 0.0)


def reference(tokens, parents, u, target, draft):
    """One sequence: (path, token, how close the closest comparison was, relative to its sides)."""
    N, V = len(tokens), target.shape[1]
    node, path, margin = -1, [], np.inf

    def less(a, b):
        nonlocal margin
        if max(a, b) > 0:
            margin = min(margin, abs(a - b) / max(a, b))
        return a < b
    going = True
    while going:
        p, going = weights(target[node + 1]), False
        left, mass = p, 1.0
        for i in range(node + 1, N):
            par = parents[i] if parents is not None else i - 1
            if par != node or not 0 <= tokens[i] < V:
                continue
            t = tokens[i]
            q = weights(draft[node + 1]) if draft is not None else None
            if less(u[i] * (q[t] if q is not None else 1.0) * mass, left[t]):
                node, going = i, True
                path.append(i)
                break
            if q is not None:
                rest = np.maximum(left - mass * q, 0)
            else:
                rest = left.copy()
                rest[t] = 0
            left = rest if rest.sum() > 0 else p
            mass = left.sum()
    cum = np.cumsum(left)
    if not cum[-1] > 0:
        return path, -1, margin
    goal = u[N] * cum[-1]
    token = int(np.searchsorted(cum, goal, side="right"))
    token = min(token, int(np.nonzero(left)[0][-1]))
    return path, token, min(margin, np.abs(cum - goal).min() / cum[-1])


# B, N, V, dtype, tree, draft rows, element offset of the rows
CASES = [
    (1, 0, 1, torch.float32, "chain", False, 0), (2, 1, 1, torch.float16, "chain", True, 0),
    (40, 4, 7, torch.float32, "chain", True, 0), (40, 4, 33, torch.bfloat16, "chain", False, 0),
    (30, 9, 500, torch.float32, "tree", True, 0), (30, 9, 501, torch.float16, "tree", True, 0),
    (30, 9, 502, torch.bfloat16, "star", True, 1), (30, 9, 503, torch.float32, "star", False, 3),
    (16, 16, 5001, torch.float32, "tree", False, 0), (9, 12, 20000, torch.bfloat16, "tree", True, 0),
    (3, 5, 50257, torch.float32, "tree", True, 1), (2, 3, 131072, torch.float16, "star", True, 0),
    (2, 256, 300, torch.float32, "tree", True, 0), (1, 2, 1 << 20, torch.float32, "star", True, 0),
]


def verify_case(B, N, V, dtype, kind, with_draft, off, seed):
    g, r = gen(seed), np.random.RandomState(seed)
    parents = None
    if kind == "tree":
        parents = np.array([[r.randint(max(-1, i - 3), i) for i in range(N)] for _ in range(B)])
    elif kind == "star":  # many children of few nodes: rejections in turn
        parents = np.array([[-1 if i < (N + 1) // 2 else 0 for i in range(N)] for _ in range(B)])

    def rows(scale, shift=None):
        flat = torch.empty(B * (N + 1) * V + off, dtype=dtype, device=DEV)
        x = flat[off:].view(B, N + 1, V)
        z = scale * torch.randn(B, N + 1, V, generator=g, device=DEV)
        if shift is not None:
            z += shift
        x.copy_(torch.softmax(z, -1))
        return x, z
    target, z = rows(2.0)
    draft, _ = rows(0.7, z) if with_draft else (None, None)
    source = draft if with_draft else target
    up = torch.zeros(B, N, dtype=torch.long) if parents is None else torch.tensor(parents + 1)
    if parents is None:
        up = torch.arange(N).expand(B, N)
    tokens = torch.empty(B, N, dtype=torch.int32, device=DEV)
    for b in range(B):
        for i in range(N):
            cum = source[b, up[b, i]].double().cumsum(-1)
            tokens[b, i] = int(torch.searchsorted(cum, cum[-1] * r.rand(), right=True).clamp(max=V - 1))
    uniform = torch.tensor(r.rand(B, N + 1), dtype=torch.float32, device=DEV)
    par = None if parents is None else torch.tensor(parents, dtype=torch.int32, device=DEV)
    return tokens, parents, par, target, draft, uniform


def check(got, tokens, parents, target, draft, uniform, least=1e-9):
    """Comparisons closer than the arithmetic's own error could fall either way: a difference r - s q of
    weights is rounded to 2^-24 of itself and of its operands, sums to 2^-44; the cases have none so near."""
    accepted, count, token = (x.cpu().numpy() for x in got)
    B, N = tokens.shape
    tk, u = tokens.cpu().numpy(), uniform.double().cpu().numpy()
    for b in range(B):
        path, want, margin = reference(tk[b], None if parents is None else parents[b], u[b], target[b],
                                       None if draft is None else draft[b])
        assert margin > least, (b, margin)
        assert count[b] == len(path) and list(accepted[b]) == path + [-1] * (N - len(path)), b
        assert token[b] == want, b
    return count


@pytest.mark.parametrize("B,N,V,dtype,kind,with_draft,off", CASES)
def test_verify(tq, B, N, V, dtype, kind, with_draft, off):
    tokens, parents, par, target, draft, uniform = verify_case(B, N, V, dtype, kind, with_draft, off, B + N + V)
    got = tq.tq_verify(tokens, target, uniform, draft=draft, parents=par)
    count = check(got, tokens, parents, target, draft, uniform)
    if B >= 30:
        assert 0 < count.sum() < B * N
    again = tq.tq_verify(tokens, target, uniform, draft=draft, parents=par)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    # rows anywhere: between others, and the draft's without the last
    wide = torch.full((B, N + 2, V + 5), 7.0, dtype=dtype, device=DEV)
    wide[:, :N + 1, :V] = target
    less = None if draft is None else draft[:, :max(N, 1)].clone()
    again = tq.tq_verify(tokens, wide[:, :N + 1, :V], uniform, draft=less, parents=par)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_rows_with_nothing_and_odd_entries(tq):
    B, N, V = 6, 2, 70
    g = gen(4)
    target = torch.softmax(torch.randn(B, N + 1, V, generator=g, device=DEV), -1)
    draft = torch.softmax(torch.randn(B, N + 1, V, generator=g, device=DEV), -1)
    target[0] = 0.0                                   # no weight at all
    target[1, :, ::2], target[1, :, 1] = float("nan"), float("inf")
    target[2, :, 5:] = -1.0
    draft[3] = target[3]                              # nothing left behind a rejection that rounding makes
    draft[4] = float("nan")                           # q = 0: what has a weight is accepted
    target[5, :, 1:] = 3.0e38                         # (no weights either)
    target[5, :, 0] = 2.0**89
    tokens = torch.randint(0, 5, (B, N), generator=g, device=DEV, dtype=torch.int32)
    uniform = torch.full((B, N + 1), 0.99, device=DEV)
    uniform[3, 0] = 1.5                               # (as if the test had failed)
    for d in (draft, None):
        got = tq.tq_verify(tokens, target, uniform, draft=d)
        check(got, tokens, None, target, d, uniform, 0.0)
        assert got[2][0] == -1 and got[1][0] == 0


def test_drafts_that_are_none(tq):
    """Tokens outside the vocabulary, parents that are not before their draft: skipped, and what hangs on them."""
    V, g = 50, gen(5)
    target = torch.softmax(torch.randn(1, 6, V, generator=g, device=DEV), -1)
    target[:, :, 7] = 5.0                             # (a draft of 7 is always accepted)
    tokens = torch.tensor([[-1, V, 7, 7, 7]], dtype=torch.int32, device=DEV)
    par = torch.tensor([[-1, -1, 0, 4, -1]], dtype=torch.int32, device=DEV)
    uniform = torch.full((1, 6), 0.5, device=DEV)
    accepted, count, token = tq.tq_verify(tokens, target, uniform, parents=par)
    assert accepted.tolist() == [[4, -1, -1, -1, -1]] and count.tolist() == [1]
    shared = tq.tq_verify(tokens.expand(3, -1).contiguous(), target.expand(3, -1, -1), uniform.expand(3, -1), parents=par[0])
    assert shared[0].tolist() == [[4, -1, -1, -1, -1]] * 3 and shared[2].tolist() == token.tolist() * 3
    chain = tq.tq_verify(tokens, target, uniform)     # its first is none: the others cannot be reached
    assert chain[1].tolist() == [0]


def test_distribution(tq):
    """What comes out first is distributed as the target's row, whatever the drafts: 200000 sequences in one
    call, each cell within five standard deviations."""
    B, N, V, g = 200000, 3, 6, gen(6)
    p = torch.softmax(torch.randn(N + 1, V, generator=g, device=DEV), -1)
    q = torch.softmax(torch.randn(N + 1, V, generator=g, device=DEV), -1)
    par = torch.full((N,), -1, dtype=torch.int32, device=DEV)  # three children of the root, drawn from q's first row
    tokens = torch.multinomial(q[0], B * N, replacement=True, generator=g).view(B, N).int()
    uniform = torch.rand(B, N + 1, generator=g, device=DEV)
    accepted, count, token = tq.tq_verify(tokens, p.expand(B, -1, -1), uniform, draft=q.expand(B, -1, -1), parents=par)
    first = torch.where(count > 0, tokens.gather(1, accepted[:, :1].clamp(min=0).long())[:, 0], token)
    share = torch.bincount(first.long(), minlength=V).double() / B
    want = p[0].double() / p[0].double().sum()
    assert ((share - want).abs() < 5 * (want * (1 - want) / B).sqrt()).all()
    assert 0.3 < float((count > 0).double().mean()) < 1.0


def test_captured_with_new_numbers(tq):
    B, N, V = 5, 6, 3001
    tokens, parents, par, target, draft, uniform = verify_case(B, N, V, torch.float32, "tree", True, 0, 77)
    out = tuple(torch.empty(s, dtype=torch.int32, device=DEV) for s in ((B, N), (B,), (B,)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        tq.tq_verify(tokens, target, uniform, draft=draft, parents=par, out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tq.tq_verify(tokens, target, uniform, draft=draft, parents=par, out=out)
    for seed in (78, 79):
        new = verify_case(B, N, V, torch.float32, "tree", True, 0, seed)
        for x, y in zip((tokens, par, target, draft, uniform), (new[0], new[2], new[3], new[4], new[5])):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        check(out, tokens, new[1], target, draft, uniform)
