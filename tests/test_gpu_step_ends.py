"""A serving loop from the projections' rows to tokens, as a user's program runs it: prompts are taken in, drafted trees
come with their positions by depth, logits go through penalties, biases and masks, the drafts are checked against them, the kept
tokens stay in the cache and are counted.  Every part is compared with plain references; the whole step is captured too."""

import numpy as np
import pytest
import torch

import bit_rotated_kv_gb300 as kvq
import synth
from tests import harness, spec_ref, step_ref

pytestmark = pytest.mark.gpu

W = synth.WUSH_CHUNK_B16.replace(batch=3, chunk_queries=False, transform="orthogonal", value_transform="orthogonal", ctx_lo=90, ctx_hi=90, n_new=1,
                                 s_flush=8, s_keep=64, s_sink=16)
NODES, VOCAB = 7, 997


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def _depth(parent):
    d = np.zeros(len(parent), np.int64)
    for i, p in enumerate(parent):
        d[i] = d[p] + 1 if p >= 0 else 0
    return d


class Loop:
    def __init__(self):
        from bit_rotated_kv_gb300.runner import DecodeRunner
        self.cfg, table = harness.kv_config(W, np.full(W.batch, 400), 256, 0)
        self.tr, self.host_tr = harness.device_transform(W, torch.device("cuda"))
        self.r = DecodeRunner(self.cfg, self.tr, 400)
        self.r.set_page_table(table)
        rng = self.rng = np.random.default_rng(3)
        self.norms = [rng.uniform(0.5, 1.5, 128).astype(np.float32) for _ in range(2)]
        self.rope = kvq.Rope.make(kvq.KVQ_ROPE_HALF, 64, 1e4, kvq.KVQ_ROPE_YARN, 4.0, 32768.0, 32.0, 1.0, q_norm=torch.from_numpy(self.norms[0]).cuda(),
                                  k_norm=torch.from_numpy(self.norms[1]).cuda())

    def rows(self, n):
        hq, hkv = W.n_q_heads, W.n_kv_heads
        x = torch.from_numpy(self.rng.standard_normal((n, hq + 2 * hkv, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    def near(self, got, x, w, far, mats, gqa):
        angle = step_ref.phases(self.rope.freq.cpu().tolist(), far)
        y, m = step_ref.placed(x.double().cpu().numpy(), angle, False, self.rope.scale, w, self.rope.norm_eps)
        want, bound = step_ref.transformed(y, m, mats, gqa)
        assert step_ref.near(got.double().cpu().numpy(), want, bound).all()


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_serving_loop(graph):
    a = Loop()
    rng, B, hq, hkv = a.rng, W.batch, W.n_q_heads, W.n_kv_heads
    length = np.array([90, 57, 33])
    # prompts: their rows, and their tokens
    q, k, v = a.rows(int(length.sum()))
    seq, pos = np.repeat(np.arange(B), length), np.concatenate([np.arange(x) for x in length])
    a.r.rope_append(a.rope, k, v, _i32(seq), _i32(pos))
    a.r.flush(128)
    counts = torch.zeros((B, VOCAB + 1), dtype=torch.int16, device="cuda")
    said = rng.integers(0, VOCAB, int(length.sum())).astype(np.int32)
    a.r.count_prompts(counts, VOCAB, _i32(np.concatenate([[0], np.cumsum(length)])), _i32(said))
    tally = np.zeros((B, VOCAB + 1), np.int64)
    tally[seq, said] |= 0x8000
    # rules of each sequence
    host = {"temperature": np.array([0.8, 0.0, 1.2], np.float32), "repetition": np.array([1.2, 1.0, 1.1], np.float32),
            "frequency": np.array([0.2, 0.1, 0.0], np.float32), "presence": np.array([0.5, 0.0, 0.3], np.float32),
            "bias": {0: {3: 2.0, 500: -np.inf}, 1: {}, 2: {7: -1.5}}}
    n = NODES * B
    allowed = rng.random((n, 32 * 32)) < 0.6
    allowed[:, :5] = True
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    mask_row = np.where(np.arange(n) % 3 == 0, -1, np.arange(n)).astype(np.int32)
    rules = kvq.LogitRules(*(dev(host[x]) for x in ("temperature", "repetition", "frequency", "presence")), counts, _i32([0, 2, 2, 3]), _i32([3, 500, 7]),
                           torch.tensor([2.0, -np.inf, -1.5], device="cuda"), dev(np.packbits(allowed, axis=1, bitorder="little").view(np.int32)), dev(mask_row))
    proj = torch.from_numpy(rng.standard_normal((hq * 128, VOCAB)).astype(np.float32)).cuda() * 0.1
    ws = a.r.tree_workspace(n)
    ints = {x: torch.zeros(n, dtype=torch.int32, device="cuda") for x in ("idx", "pos", "far", "parent", "token", "path")}
    cu = _i32(np.arange(B + 1) * NODES)
    n_accept, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    fused = torch.zeros((n, hq + 2 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    u, p = torch.zeros(n, device="cuda"), torch.zeros((n, VOCAB), device="cuda")
    q_out, out = torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, hq, 128), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((n, VOCAB), dtype=torch.bfloat16, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        a.r.tree_step(q, k, v, ints["idx"], ints["pos"], cu, ints["parent"], q_out, out, ws, st, a.rope, ints["far"])
        logits.copy_(out.reshape(n, -1).float() @ proj)
        a.r.accept_logits(rules, cu, ints["parent"], ints["token"], logits, p, None, u, ints["path"], n_accept, nxt, NODES, st)

    captured = None
    for turn in range(4):
        parent = np.concatenate([spec_ref.random_tree(rng, NODES, "random") for _ in range(B)])
        token = rng.integers(0, VOCAB, n)
        depth = np.concatenate([_depth(parent[b * NODES:(b + 1) * NODES]) for b in range(B)])
        far = np.repeat(length, NODES) + depth
        rows = a.rows(n)
        for t, x in zip((q, k, v), rows):
            t.copy_(x)
        random = rng.random(n).astype(np.float32)
        random[rng.random(n) < 0.5] = 0.0                # (half of the drafts pass)
        random[::NODES] = rng.random(B)
        u.copy_(torch.from_numpy(random))
        for name, val in (("idx", np.repeat(np.arange(B), NODES)), ("pos", np.concatenate([x + np.arange(NODES) for x in length])), ("far", far),
                          ("parent", parent), ("token", token)):
            ints[name].copy_(_i32(val))
        before = tally.copy()
        if graph and turn == 1:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        captured.replay() if captured is not None else step()
        torch.cuda.synchronize()
        assert int(a.r.status.item()) == 0
        # queries as the formulas have them; keys of the kept nodes, where the cache holds them now
        a.near(q_out, q, a.norms[0], far, a.host_tr[1], hq // hkv)
        acc, path = n_accept.cpu().numpy(), ints["path"].cpu().numpy()
        ring, edge = a.r.cache.ring_k, a.r.cache.s_quant.cpu().numpy()
        for b in range(B):
            keep = path[b * NODES:b * NODES + acc[b]]
            live = [j for j in range(acc[b]) if length[b] + j >= edge[b]]     # (what is still a bf16 row)
            at = b * NODES + keep[live]
            slots = (length[b] + np.array(live)) % a.cfg.ring_cap
            a.near(ring[b][:, slots].transpose(0, 1), k[at.tolist()], a.norms[1], far[at], a.host_tr[0], 1)
        # probabilities, the check of the drafts, and the counts
        probs, lg = p.cpu().numpy(), logits.double().cpu().numpy()
        for b in range(B):
            rows_b = range(b * NODES, (b + 1) * NODES)
            for r in rows_b:
                above, i = [], r
                while parent[i] >= 0:
                    above.append(int(token[i]))
                    i = b * NODES + parent[i]
                m = None if mask_row[r] < 0 else allowed[mask_row[r], :VOCAB]
                x, size = step_ref.values(lg[r], before[b, :VOCAB], above, host, b, m)
                want, tol = step_ref.probabilities(x, size, float(host["temperature"][b]))
                assert (np.abs(probs[r] - want) <= tol).all()
            s = slice(b * NODES, (b + 1) * NODES)
            kept, last = spec_ref.verify(parent[s], token[s], probs[s], None, random[s])
            assert list(path[s][:acc[b]]) == kept and int(nxt[b]) == last
            for t in [*token[s][kept[1:]], last]:
                tally[b, t] += 1
            length[b] += acc[b]
        assert np.array_equal(counts.cpu().numpy().view(np.uint16), tally)
        assert a.r.cache.seq_len.tolist() == length.tolist()


def test_plain_steps():
    """One token a sequence and step: rope_step, next_tokens."""
    a = Loop()
    rng, B = a.rng, W.batch
    length = np.array([20, 75, 40])
    q, k, v = a.rows(int(length.sum()))
    a.r.rope_append(a.rope, k, v, _i32(np.repeat(np.arange(B), length)), _i32(np.concatenate([np.arange(x) for x in length])))
    a.r.flush(128)
    counts = torch.zeros((B, VOCAB + 1), dtype=torch.int16, device="cuda")
    rules = kvq.LogitRules(temperature=torch.tensor([1.0, 0.0, 0.7], device="cuda"), frequency=torch.full((B,), 50.0, device="cuda"), counts=counts)
    proj = torch.from_numpy(rng.standard_normal((W.n_q_heads * 128, VOCAB)).astype(np.float32)).cuda() * 0.2
    nxt, p = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros((B, VOCAB), device="cuda")
    seen = [[] for _ in range(B)]
    for _ in range(12):
        q, k, v = a.rows(B)
        a.r.rope_step(a.rope, q, k, v, _i32(np.arange(B)), _i32(length), _i32(length), 1)
        a.near(a.r.q_out, q, a.norms[0], length, a.host_tr[1], W.n_q_heads // W.n_kv_heads)
        length += 1
        logits = a.r.out.reshape(B, -1) @ proj
        random = rng.random(B).astype(np.float32)
        a.r.next_tokens(rules, logits, p, torch.from_numpy(random).cuda(), nxt)
        probs = p.cpu().numpy()
        for b in range(B):
            assert int(nxt[b]) == spec_ref.verify([-1], [0], probs[b:b + 1], None, random[b:b + 1])[1]
            seen[b].append(int(nxt[b]))
    assert int(a.r.status.item()) == 0 and a.r.cache.seq_len.tolist() == length.tolist()
    assert all(len(set(s)) == 12 for s in seen)          # (a penalty of 50 keeps every token from coming twice)
    want = np.zeros((B, VOCAB + 1), np.int64)
    for b in range(B):
        want[b, seen[b]] = 1
    assert np.array_equal(counts.cpu().numpy(), want)


def test_next_tokens_captured_first():
    """The runner's first call is captured; one beside the graph, before it has run, is right too."""
    a = Loop()
    rng, B = a.rng, W.batch
    logits = torch.from_numpy(rng.standard_normal((B, VOCAB)).astype(np.float32) * 3).cuda()
    random = rng.random(B).astype(np.float32)
    u = torch.from_numpy(random).cuda()
    p, p2 = (torch.zeros((B, VOCAB), device="cuda") for _ in range(2))
    nxt, nxt2 = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.r.next_tokens(None, logits, p, u, nxt, stream=torch.cuda.current_stream().cuda_stream)
    a.r.next_tokens(None, logits, p2, u, nxt2)
    torch.cuda.synchronize()
    want = [spec_ref.verify([-1], [0], p2.cpu().numpy()[b:b + 1], None, random[b:b + 1])[1] for b in range(B)]
    assert nxt2.tolist() == want and int(a.r.status.item()) == 0 and nxt.tolist() == [-7] * B
    graph.replay()
    torch.cuda.synchronize()
    assert nxt.tolist() == want and torch.equal(p, p2) and int(a.r.status.item()) == 0
