"""The speculative and page-pool calls together, as a serving loop runs them: a prompt is prefilled
into reserved pages and forked, every copy drafts a tree, the target checks it, the kept rows stay; in
between sequences leave, the pool is compacted and new ones come.  A second cache gets the kept tokens by
the ordinary append: codes, scales, windows, lengths and decode results are equal bit for bit."""

import numpy as np
import pytest
import torch

import synth
from tests import harness, spec_ref

pytestmark = pytest.mark.gpu

W = synth.WUSH_CHUNK_B16.replace(batch=6, chunk_queries=False, transform="orthogonal", ctx_lo=300, ctx_hi=300, n_new=1, s_flush=1)
NODES, VOCAB = 9, 501


class Loop:
    def __init__(self, seed, table=None):
        from bit_rotated_kv_gb300.runner import DecodeRunner
        self.cfg, full = harness.kv_config(W, np.full(W.batch, 700), 256, 0)
        self.dev = torch.device("cuda")
        tr, _ = harness.device_transform(W, self.dev)
        self.r = DecodeRunner(self.cfg, tr, 700, self.dev)
        if table == "full":
            self.r.set_page_table(full)
        self.rng = np.random.default_rng(seed)

    def i32(self, a):
        return torch.tensor(np.asarray(a, np.int32), device=self.dev)

    def append(self, k, v, seqs, lengths):
        """k, v: one [n, Hkv, d] tensor per entry of seqs, from lengths[i] on; then a flush."""
        idx = np.concatenate([np.full(len(x), b) for x, b in zip(k, seqs)])
        pos = np.concatenate([length + np.arange(len(x)) for x, length in zip(k, lengths)])
        self.r.append(torch.cat(k), torch.cat(v), self.i32(idx), self.i32(pos))
        self.r.flush(max(len(x) for x in k) + self.cfg.s_flush)


def _rand(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)


def _state(loop, b):
    """Everything that sequence b holds, by value."""
    c, cfg = loop.r.cache, loop.cfg
    L, e = int(c.seq_len[b]), int(c.s_quant[b])
    full, part = divmod(max(0, e - cfg.s_sink), 16)
    ids = c.page_table[b, :full + (part > 0)].cpu().tolist()
    snap = {"pages": c.pages.cpu().numpy()}
    from tests import layout
    out = [L, e]
    for h in range(cfg.n_kv_heads):
        u = layout.decode_unit(snap["pages"], np.asarray(ids + [0], np.int32), h, cfg.s_sink, e, cfg.group_size, bool(cfg.key_l2norm), 0)
        out += [np.asarray(u[k]) for k in ("codes_k", "codes_v", "delta_k", "zero_k", "delta_v", "zero_v")]
    slots = torch.arange(max(e, cfg.s_sink), L, device="cuda") % cfg.ring_cap
    for s, r in ((c.sink_k, c.ring_k), (c.sink_v, c.ring_v)):
        out += [harness.bits(s[b, :, :min(L, cfg.s_sink)]), harness.bits(r[b][:, slots])]
    return out


def _same(a, la, b, lb):
    for x, y in zip(_state(a, la), _state(b, lb)):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("drawn", [False, True], ids=["chosen", "drawn"])
def test_serving_loop(graph, drawn):
    a, b = Loop(1), Loop(1, "full")
    rng = np.random.default_rng(7)
    hkv, hq, d = W.n_kv_heads, W.n_q_heads, 128
    # a prompt of 300 tokens in sequence 0, forked to 1, 2, 4; 3 and 5 stay empty
    k0, v0 = _rand(rng, 300, hkv, d), _rand(rng, 300, hkv, d)
    a.r.reserve(a.i32([300, 0, 0, 0, 0, 0]))
    a.append([k0], [v0], [0], [0])
    a.r.fork(a.i32([0, 0, 0]), a.i32([1, 2, 4]))
    live = [0, 1, 2, 4]
    for s in live:
        b.append([k0], [v0], [s], [0])
    length = {s: 300 for s in live}
    ws, cws = a.r.tree_workspace(NODES * W.batch), a.r.compact_workspace()
    proj = _rand(rng, hq * d, VOCAB).float()
    # buffers that a captured step keeps
    n = NODES * len(live)
    bufs = dict(q=_rand(rng, n, hq, d), k=_rand(rng, n, hkv, d), v=_rand(rng, n, hkv, d), u=torch.zeros(n, device="cuda"),
                qp=torch.zeros(n, VOCAB, device="cuda"), p=torch.zeros(n, VOCAB, device="cuda"))
    ints = {x: torch.zeros(n, dtype=torch.int32, device="cuda") for x in ("idx", "pos", "parent", "token", "path")}
    cu = torch.zeros(W.batch + 1, dtype=torch.int32, device="cuda")
    n_accept, nxt = (torch.zeros(W.batch, dtype=torch.int32, device="cuda") for _ in range(2))
    q_out, out = torch.zeros_like(bufs["q"]), torch.zeros_like(bufs["q"])

    def step():
        st = torch.cuda.current_stream()
        a.r.tree_step(bufs["q"], bufs["k"], bufs["v"], ints["idx"], ints["pos"], cu, ints["parent"], q_out, out, ws, st)
        bufs["p"].copy_(torch.softmax(out.reshape(n, -1).float() @ proj * 0.05, -1))
        a.r.accept(cu, ints["parent"], ints["token"], bufs["p"], bufs["qp"] if drawn else None, bufs["u"], ints["path"], n_accept,
                   nxt, NODES, st)

    captured = None
    for turn in range(5):
        # every live sequence has a tree of NODES nodes
        a.r.reserve(a.i32([NODES if s in live else 0 for s in range(W.batch)]))
        counts = [NODES if s in live else 0 for s in range(W.batch)]
        cu.copy_(a.i32(np.concatenate([[0], np.cumsum(counts)])))
        parent = np.concatenate([spec_ref.random_tree(rng, NODES, "random") for _ in live]).astype(np.int32)
        token = rng.integers(0, VOCAB, n).astype(np.int32)
        u = rng.random(n).astype(np.float32)
        u[rng.random(n) < 0.5] = 0.0                 # (half of the drafts pass, whatever their probability)
        u[::NODES] = rng.random(len(live)).astype(np.float32)
        for name, val in (("q", _rand(rng, n, hq, d)), ("k", _rand(rng, n, hkv, d)), ("v", _rand(rng, n, hkv, d)),
                          ("u", torch.from_numpy(u).cuda()), ("qp", torch.softmax(_rand(rng, n, VOCAB).float(), -1))):
            bufs[name].copy_(val)
        for name, val in (("idx", np.repeat(live, NODES)), ("parent", parent), ("token", token),
                          ("pos", np.concatenate([length[s] + np.arange(NODES) for s in live]))):
            ints[name].copy_(a.i32(val))
        if graph and turn == 1:                      # (the first turn ran eagerly)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        if captured is not None:
            captured.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(a.r.status.item()) == 0
        acc, nx, path = n_accept.cpu().numpy(), nxt.cpu().numpy(), ints["path"].cpu().numpy()
        p, qp = bufs["p"].cpu().numpy(), bufs["qp"].cpu().numpy()
        for i, s in enumerate(live):
            rows = slice(i * NODES, (i + 1) * NODES)
            want = spec_ref.verify(parent[rows], token[rows], p[rows], qp[rows] if drawn else None, u[rows])
            keep = list(path[rows][:acc[s]])
            assert keep == list(want[0]) and nx[s] == want[1]
            at = [i * NODES + j for j in keep]
            b.append([bufs["k"][at]], [bufs["v"][at]], [s], [length[s]])
            length[s] += len(keep)
            _same(a, s, b, s)
        # decode from both caches
        qd = _rand(rng, W.batch, hq, d)
        for loop in (a, b):
            loop.r.append(None, None, None, None, qd, loop.r.q_out)
            loop.r.decode(loop.r.q_out, loop.r.out)
        torch.cuda.synchronize()
        for s in live:
            assert torch.equal(a.r.out[s], b.r.out[s])
        if turn == 2:                                # two leave, the pool closes up, one forks again into their places
            gone, stays = live[1:3], live[0]
            a.r.free(a.i32(gone))
            held = int(a.r.compact(cws).item())
            assert held == int((a.r.page_ref > 0).sum()) and bool((a.r.page_ref[:held] > 0).all())
            a.r.fork(a.i32([stays, stays]), a.i32([3, 1]))
            live = [0, 1, 3, 4]
            b.r.cache.seq_len[gone] = 0
            b.r.cache.s_quant[gone] = b.cfg.s_sink
            length[1] = length[3] = length[stays]
            for s in (1, 3):
                # (the ordinary cache is rebuilt from what sequence 0 holds: rows by value)
                cb, ca = b.r.cache, a.r.cache
                ids_a, ids_b = ca.page_table[stays].tolist(), cb.page_table[s].tolist()
                for x, y in zip(ids_a, ids_b):
                    if x >= 0 and y >= 0:
                        cb.pages[y] = ca.pages[x]
                for t, f in ((cb.sink_k, ca.sink_k), (cb.sink_v, ca.sink_v), (cb.ring_k, ca.ring_k), (cb.ring_v, ca.ring_v)):
                    t[s] = f[stays]
                cb.seq_len[s], cb.s_quant[s] = ca.seq_len[stays], ca.s_quant[stays]
            for s in live:
                _same(a, s, b, s)
    assert int(a.r.status.item()) == 0 and int(b.r.status.item()) == 0
