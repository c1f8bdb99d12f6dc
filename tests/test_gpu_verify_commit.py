"""kv_verify_tree against the definition in exact integers (tokens must be equal), its distribution
against the target's, and kv_tree_commit against moving the rows by hand."""

import numpy as np
import pytest
import torch

from tests import spec_ref

pytestmark = pytest.mark.gpu


def _kvq():
    import bit_rotated_kv_gb300 as m
    return m


def _cfg(batch, **kw):
    base = dict(n_q_heads=1, n_kv_heads=1, batch=batch, max_pages_per_seq=1, num_pages=1, ring_cap=272)
    base.update(kw)
    return _kvq().KVConfig(**base)


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _inputs(rng, counts, vocab, dist, kind="random", noise=0.7):
    rows = int(np.sum(counts))
    lp = 2.0 * rng.standard_normal((rows, vocab))
    p, q = _softmax(lp), _softmax(lp + noise * rng.standard_normal((rows, vocab)))
    parent = np.concatenate([spec_ref.random_tree(rng, n, kind) for n in counts]).astype(np.int32) if rows else np.zeros(0, np.int32)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    token = np.zeros(rows, np.int32)
    for b in range(len(counts)):
        for i in range(1, counts[b]):
            row = q[cu[b] + parent[cu[b] + i]].astype(np.float64)
            token[cu[b] + i] = rng.choice(vocab, p=row / row.sum()) if dist else np.argsort(-row)[i % min(4, vocab)]
    return cu, parent, token, p, q if dist else None, rng.random(rows).astype(np.float32)


def _run(cu, parent, token, p, q, u, pad=0, status_ok=True):
    kvq = _kvq()
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    def rows(a):
        if a is None:
            return None
        wide = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device="cuda")
        wide[:, :a.shape[1]] = dev(a)
        return wide[:, :a.shape[1]]
    batch = len(cu) - 1
    path = torch.full((len(token),), 77, dtype=torch.int32, device="cuda")
    acc = torch.full((batch,), 77, dtype=torch.int32, device="cuda")
    nxt = torch.full((batch,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kv_verify_tree(_cfg(batch), dev(cu), dev(parent), dev(token), rows(p), rows(q), dev(u), path, acc, nxt, status)
    torch.cuda.synchronize()
    if status_ok:
        assert int(status.item()) == 0
    return path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("dist", [False, True])
@pytest.mark.parametrize("counts,vocab,kind,pad", [
    ([8], 1000, "random", 0), ([1, 1, 1], 37, "random", 3), ([5, 0, 17, 2], 513, "random", 0),
    ([128], 300, "random", 0), ([40], 4099, "star", 1), ([30, 12], 8192, "chain", 0), ([6, 6], 2, "star", 0),
    ([3], 1, "random", 0), ([20], 40000, "random", 0),
])
def test_verify(dist, counts, vocab, kind, pad):
    for seed in range(3):
        rng = np.random.default_rng([seed, vocab, len(counts)])
        cu, parent, token, p, q, u = _inputs(rng, counts, vocab, dist, kind)
        path, acc, nxt, _ = _run(cu, parent, token, p, q, u, pad)
        for b, n in enumerate(counts):
            s = slice(cu[b], cu[b + 1])
            if n == 0:
                assert (acc[b], nxt[b]) == (0, -1)
                continue
            want, last = spec_ref.verify(parent[s], token[s], p[s], None if q is None else q[s], u[s])
            assert acc[b] == len(want), (seed, b)
            assert path[s].tolist() == want + [-1] * (n - len(want))
            assert nxt[b] == last, (seed, b)


def test_edges_of_the_numbers():
    # u = 0 accepts whatever has weight; u just below 1 rejects unless the target is sure
    p = np.array([[0.25, 0.25, 0.5, 0.0]] * 3, np.float32)
    parent, token, cu = np.array([-1, 0, 0], np.int32), np.array([0, 3, 2], np.int32), np.array([0, 3], np.int32)
    below = np.float32(1) - np.float32(2.0 ** -24)
    for u in ([0.0, 0.0, 0.0], [below, below, below], [below, 0.0, 0.5], [0.0, 0.0, 0.4999]):
        u = np.array(u, np.float32)
        want, last = spec_ref.verify(parent, token, p, None, u)
        path, acc, nxt, _ = _run(cu, parent, token, p, None, u)
        assert path[:acc[0]].tolist() == want and nxt[0] == last and p[0][last] > 0
    # a residual that is empty (the draft is the target and u is 1): the draw is from the target
    u = np.array([0.6, 1.0, 1.0], np.float32)
    path, acc, nxt, _ = _run(cu, parent, np.array([0, 0, 2], np.int32), p, p, u)
    assert acc[0] in (1, 2) and p[0][nxt[0]] > 0


@pytest.mark.parametrize("dist", [False, True])
def test_probabilities_at_the_ends_of_their_range(dist):
    """Ones, values a step below, at and under the unit 2^-60, denormals, both zeros, more than 1 -- with misses."""
    ends = np.array([0.0, -0.0, 1.0, np.nextafter(np.float32(1), np.float32(0)), 2.0 ** -23, 2.0 ** -24, 2.0 ** -36, 1.9999999 * 2.0 ** -37,
                     1.5 * 2.0 ** -46, 2.0 ** -60, 1.5 * 2.0 ** -60, 2.0 ** -61, 2.0 ** -126, 2.0 ** -149, 0.3, 1.5], np.float32)
    below = np.float32(1) - np.float32(2.0 ** -24)
    for seed in range(12):
        rng = np.random.default_rng(seed)
        n, vocab = 7, 300
        p, q = np.zeros((n, vocab), np.float32), np.zeros((n, vocab), np.float32)
        for m in (p, q):
            for r in range(n):                       # at most two of the large ones a row: its sum stays under 4
                at = rng.choice(vocab, 60, replace=False)
                m[r, at] = rng.choice(ends[[0, 1, *range(4, 14)]], 60)
                m[r, at[:2]] = rng.choice(ends[[2, 3, 14, 15]], 2)
        parent = np.array([-1, 0, 0, 0, 0, 3, 3], np.int32)
        token = np.array([0] + [int(rng.choice(np.nonzero(q[max(0, parent[i])])[0])) for i in range(1, n)], np.int32)
        u = rng.choice(np.array([0.0, 0.5, below, 2.0 ** -40], np.float32), n)
        want, last = spec_ref.verify(parent, token, p, q if dist else None, u)
        path, acc, nxt, _ = _run(np.array([0, n], np.int32), parent, token, p, q if dist else None, u, pad=seed % 4)
        assert path[:acc[0]].tolist() == want and nxt[0] == last, seed


def test_sums_over_a_vocabulary_of_many_chunks():
    # 700,003 tokens: 43 chunks of 128 a warp; a draft that is missed once, and twice
    rng = np.random.default_rng(3)
    vocab, below = 700003, np.float32(1) - np.float32(2.0 ** -24)
    p, q = (_softmax(rng.standard_normal((3, vocab))) for _ in range(2))
    token = np.array([0, int(np.argmax(q[0] - 9 * p[0])), int(np.argmax(q[0] - 5 * p[0]))], np.int32)
    parent, cu = np.array([-1, 0, 0], np.int32), np.array([0, 3], np.int32)
    for us in ([0.37, below, below], [0.9999, below, 0.0], [below, 0.0, below]):
        u = np.array(us, np.float32)
        for draft in (None, q):
            want, last = spec_ref.verify(parent, token, p, draft, u)
            path, acc, nxt, _ = _run(cu, parent, token, p, draft, u, pad=1)
            assert path[:acc[0]].tolist() == want and nxt[0] == last


def test_tokens_are_distributed_as_the_target():
    """First new token over 20000 independent sequences with two sampled siblings: each of 5 tokens'
    frequency within 5 standard deviations of the target's probability."""
    rng = np.random.default_rng(11)
    B, V = 20000, 5
    p0 = np.array([0.05, 0.1, 0.4, 0.25, 0.2], np.float32)
    q0 = np.array([0.3, 0.3, 0.1, 0.1, 0.2], np.float32)
    p, q = np.tile(p0, (3 * B, 1)), np.tile(q0, (3 * B, 1))
    parent = np.tile(np.array([-1, 0, 0], np.int32), B)
    token = rng.choice(V, size=3 * B, p=q0.astype(np.float64) / q0.astype(np.float64).sum()).astype(np.int32)
    cu = (3 * np.arange(B + 1)).astype(np.int32)
    for dist in (True, False):
        path, acc, nxt, _ = _run(cu, parent, token, p, q if dist else None, rng.random(3 * B).astype(np.float32))
        first = np.where(acc > 1, token[cu[:-1] + path[np.minimum(cu[:-1] + 1, 3 * B - 1)].clip(0)], nxt)
        f = np.bincount(first, minlength=V) / B
        assert (np.abs(f - p0) <= 5 * np.sqrt(p0 * (1 - p0) / B)).all(), (dist, f)


def test_faults_of_verify():
    kvq = _kvq()
    rng = np.random.default_rng(2)
    cu, parent, token, p, q, u = _inputs(rng, [6, 6], 100, True)
    for edit in ("parent", "root", "token"):
        par, tok = parent.copy(), token.copy()
        if edit == "parent":
            par[3] = 5
        elif edit == "root":
            par[2] = -1
        else:
            tok[4] = 100
        path, acc, nxt, status = _run(cu, par, tok, p, q, u, status_ok=False)
        assert status == kvq.KVQ_ERR_BOUNDS
        assert (acc[0], nxt[0]) == (0, -1) and (path[:6] == -1).all()
        want, last = spec_ref.verify(parent[6:], token[6:], p[6:], q[6:], u[6:])
        assert acc[1] == len(want) and nxt[1] == last
    # more nodes than a tree may have
    cu, parent, token, p, q, u = _inputs(rng, [129], 10, True)
    _, acc, nxt, status = _run(cu, parent, token, p, q, u, status_ok=False)
    assert status == kvq.KVQ_ERR_BOUNDS and (acc[0], nxt[0]) == (0, -1)
    # rows that are no distributions
    for fill in (float("nan"), 0.0, 1.0):
        cu, parent, token, p, q, u = _inputs(rng, [1], 50, False)
        p[:] = fill
        _, acc, nxt, status = _run(cu, parent, token, p, q, u, status_ok=False)
        assert status == kvq.KVQ_ERR_NONFINITE and (acc[0], nxt[0]) == (1, -1)


# ---- commit -------------------------------------------------------------------------------------------
def _cache(batch, hkv, lens, edges, sink=5, cap=160, keep=48):
    kvq = _kvq()
    cfg = kvq.KVConfig(n_q_heads=hkv, n_kv_heads=hkv, batch=batch, max_pages_per_seq=8, num_pages=8, ring_cap=cap, s_sink=sink,
                       s_keep=keep, s_flush=8)
    c = kvq.KVCache(cfg)
    g = torch.Generator("cuda").manual_seed(4)
    for t in (c.sink_k, c.sink_v, c.ring_k, c.ring_v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    c.s_quant.copy_(torch.tensor(edges, dtype=torch.int32))
    return cfg, c


@pytest.mark.parametrize("hkv", [1, 8])
def test_commit(hkv):
    kvq = _kvq()
    sink, cap = 5, 160
    counts = [12, 1, 0, 30, 128, 9, 7]
    base = [300, 150, 40, 0, 159, 2, 88]                    # before the drafts: ring wrap, inside the sink, empty
    lens = [a + n for a, n in zip(base, counts)]
    edges = [max(sink, a // 8 * 8 - 40) for a in base]
    cfg, c = _cache(len(counts), hkv, lens, edges)
    rng = np.random.default_rng(0)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    path, acc = np.full(cu[-1], -1, np.int32), []
    for b, n in enumerate(counts):
        k = [5, 1, 0, 30, 90, 0, 3][b]
        path[cu[b]:cu[b] + k] = np.sort(rng.choice(n, k, replace=False)) if k else []
        acc.append(k)
    before = {k: getattr(c, k).clone() for k in ("sink_k", "sink_v", "ring_k", "ring_v")}
    want = {k: v.clone() for k, v in before.items()}
    for b, n in enumerate(counts):
        for j in range(acc[b]):
            s, d = base[b] + int(path[cu[b] + j]), base[b] + j
            for kv in ("k", "v"):
                row = before["sink_" + kv][b, :, s] if s < sink else before["ring_" + kv][b, :, s % cap]
                if d < sink:
                    want["sink_" + kv][b, :, d] = row
                else:
                    want["ring_" + kv][b, :, d % cap] = row
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    kvq.kv_tree_commit(cfg, c, dev(cu), dev(path), dev(acc), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for k, v in want.items():
        assert torch.equal(getattr(c, k).view(torch.int16), v.view(torch.int16)), k
    assert c.seq_len.tolist() == [a + k for a, k in zip(base, acc)]


@pytest.mark.parametrize("path,acc", [([0, 2, 2], 3), ([1, 0, 2], 2), ([0, 5, 6], 2), ([0, -1, -1], 2), ([0, 1, 2], 4), ([0, 1, 2], -1)])
def test_commit_refuses_what_is_no_path(path, acc):
    kvq = _kvq()
    cfg, c = _cache(2, 2, [103, 203], [60, 160])
    before = [t.clone() for t in (c.sink_k, c.sink_v, c.ring_k, c.ring_v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kvq.kv_tree_commit(cfg, c, dev([0, 3, 6]), dev(path + [0, 1, 2]), dev([acc, 1]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS
    assert c.seq_len.tolist() == [103, 201]
    for t, b in zip((c.sink_k, c.sink_v, c.ring_k, c.ring_v), before):
        assert torch.equal(t[0].view(torch.int16), b[0].view(torch.int16))


def test_commit_refuses_quantized_drafts():
    kvq = _kvq()
    cfg, c = _cache(1, 2, [103], [101])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kvq.kv_tree_commit(cfg, c, dev([0, 3]), dev([0, 2, -1]), dev([2]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS and c.seq_len.tolist() == [103]
