"""The page pool's calls against plain lists: tables, counts, lengths, page bytes and window rows
are equal bit for bit, over a random sequence of reserve / fork / free / compact."""

import numpy as np
import pytest
import torch

from tests import harness, spec_ref

pytestmark = pytest.mark.gpu


def _kvq():
    import bit_rotated_kv_gb300 as m
    return m


class Device:
    def __init__(self, batch=9, hkv=2, max_pages=20, num_pages=60, seed=0, **kw):
        kvq = _kvq()
        base = dict(n_q_heads=hkv, n_kv_heads=hkv, batch=batch, max_pages_per_seq=max_pages, num_pages=num_pages, ring_cap=96,
                    s_sink=5, s_keep=48, s_flush=1, group_size=64)
        base.update(kw)
        self.cfg = kvq.KVConfig(**base)
        self.c = kvq.KVCache(self.cfg)
        g = torch.Generator("cuda").manual_seed(seed)
        for t in (self.c.sink_k, self.c.sink_v, self.c.ring_k, self.c.ring_v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.c.pages.copy_(torch.randint(0, 256, self.c.pages.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.ref = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(max(256, kvq.kv_pages_compact_workspace_bytes(self.cfg)), dtype=torch.uint8, device="cuda")

    def dev(self, a):
        return torch.tensor(np.asarray(a, np.int32), device="cuda")

    def do(self, name, *args):
        kvq = _kvq()
        if name == "compact":
            kvq.kv_pages_compact(self.cfg, self.c, self.ref, self.n_live, self.ws, self.status)
        else:
            fn = {"reserve": kvq.kv_pages_reserve, "fork": kvq.kv_seq_fork, "free": kvq.kv_seq_free}[name]
            fn(self.cfg, self.c, self.ref, *[self.dev(a) for a in args], self.status)
        torch.cuda.synchronize()
        return int(self.status.item())

    def snap(self):
        c = self.c
        return {"pages": c.pages.cpu().numpy(), "seq_len": c.seq_len.cpu().numpy(), "s_quant": c.s_quant.cpu().numpy(),
                "sink_k": harness.bits(c.sink_k), "sink_v": harness.bits(c.sink_v), "ring_k": harness.bits(c.ring_k),
                "ring_v": harness.bits(c.ring_v)}

    def plain(self):
        return spec_ref.Pool(self.cfg, self.snap(), self.c.page_table.cpu().numpy(), self.ref.cpu().numpy())

    def grow(self, b, tokens):
        """Sequence b gets `tokens` more tokens, as appends and flushes would leave the lengths."""
        L = int(self.c.seq_len[b]) + tokens
        self.c.seq_len[b] = L
        self.c.s_quant[b] = max(int(self.c.s_quant[b]), max(self.cfg.s_sink, L - self.cfg.s_keep))

    def check(self, p):
        assert np.array_equal(self.c.page_table.cpu().numpy(), p.table)
        assert np.array_equal(self.ref.cpu().numpy(), p.ref)
        s = self.snap()
        for k in s:
            assert np.array_equal(s[k], p.s[k]), k
        assert (self.c.counters == 0).all()


@pytest.mark.parametrize("seed", range(4))
def test_random_sequence_of_calls(seed):
    rng = np.random.default_rng(seed)
    d = Device(batch=9, hkv=int(rng.choice([1, 2, 8])), seed=seed, group_size=int(rng.choice([32, 64, 128])))
    for _ in range(14):
        lens = d.c.seq_len.cpu().numpy()
        empty, used = np.nonzero(lens == 0)[0], np.nonzero(lens > 0)[0]
        op = rng.choice(["admit", "fork", "free", "compact"])
        p = d.plain()
        if op == "admit" and len(empty):
            b = int(rng.choice(empty))
            n = int(rng.integers(1, 250))
            tokens = np.zeros(d.cfg.batch, np.int32)
            tokens[b] = n
            if int((d.ref == 0).sum()) < 17:
                continue
            assert d.do("reserve", tokens) == 0
            p.reserve(tokens)
            d.check(p)
            d.grow(b, n)
        elif op == "fork" and len(empty) > 1 and len(used):
            dst = rng.permutation(empty)[:int(rng.integers(1, len(empty)))]
            src = rng.choice(used, len(dst))
            if int((d.ref == 0).sum()) < len(dst):
                continue
            assert d.do("fork", src, dst) == 0
            p.fork(src, dst)
            d.check(p)
        elif op == "free" and len(used):
            seqs = rng.choice(used, int(rng.integers(1, 4)))           # (twice the same one, at times)
            assert d.do("free", seqs) == 0
            p.free(seqs)
            d.check(p)
        elif op == "compact":
            assert d.do("compact") == 0
            n = p.compact()
            d.check(p)
            assert int(d.n_live.item()) == n
            held = d.ref.cpu().numpy() > 0
            assert held[:n].all() and not held[n:].any()


def test_reserve_stops_where_the_pool_ends():
    kvq = _kvq()
    d = Device(batch=4, num_pages=20, max_pages=12)
    p = d.plain()
    assert d.do("reserve", [100, 160, 100, 5]) == kvq.KVQ_ERR_BOUNDS     # 6, 10, 6 (too many), 0
    p.reserve([100, 160, 100, 5])
    d.check(p)
    assert (d.c.page_table[2] == -1).all()
    d.status.zero_()
    assert d.do("reserve", [0, -3, 33, 16]) == 0
    p.reserve([0, -3, 33, 16])
    d.check(p)
    assert d.do("reserve", [12 * 16 + 6, 0, 0, 0]) == kvq.KVQ_ERR_BOUNDS   # more than a row of the table
    d.check(p)


def test_needs_whose_sum_passes_32_bits():
    # 2,099 sequences that ask for 2^20 pages each, behind one that asks for 3
    kvq = _kvq()
    cfg = kvq.KVConfig(n_q_heads=1, n_kv_heads=1, batch=2100, max_pages_per_seq=1 << 20, num_pages=50, ring_cap=16, s_sink=0, s_keep=8,
                       s_flush=1)
    c = kvq.KVCache(cfg)
    ref, status = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (50, 1))
    want = torch.full((2100,), 16 << 20, dtype=torch.int32, device="cuda")
    want[0] = 48
    kvq.kv_pages_reserve(cfg, c, ref, want, status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS
    assert c.page_table[0, :4].tolist() == [0, 1, 2, -1] and int((c.page_table >= 0).sum()) == 3 and int(ref.sum()) == 3


def test_reserve_extends_what_a_sequence_holds():
    d = Device(batch=3, num_pages=64, max_pages=40)
    p = d.plain()
    for tokens in ([21, 0, 7], [37, 300, 0], [21, 40, 500], [600, 1, 1]):
        # the last call would bring the three to 38 + 19 + 31 = 88 pages of 64: its first sequence is
        # already one that cannot be served, so none is
        assert d.do("reserve", tokens) == (_kvq().KVQ_ERR_BOUNDS if tokens[0] == 600 else 0)
        p.reserve(tokens)
        d.check(p)


def test_pool_larger_than_one_scan():
    d = Device(batch=70, hkv=1, num_pages=30000, max_pages=900, group_size=128)
    p = d.plain()
    tokens = np.random.default_rng(1).integers(0, 4000, 70)
    assert d.do("reserve", tokens) == 0
    p.reserve(tokens)
    d.check(p)
    assert d.do("free", np.arange(0, 70, 2)) == 0
    p.free(range(0, 70, 2))
    d.check(p)
    assert d.do("compact") == 0
    p.compact()
    d.check(p)


def test_pages_beyond_4_gib():
    # six pages at the far end of a pool of more than 5 GiB: forked (the half-filled one is copied), then moved to its front
    kvq = _kvq()
    cfg = kvq.KVConfig(n_q_heads=8, n_kv_heads=8, batch=2, max_pages_per_seq=8, num_pages=1, ring_cap=96, s_sink=5, s_keep=48, s_flush=1,
                       group_size=64)
    cfg.num_pages = many = (5 << 30) // (8 * kvq.kvq_page_head_bytes(cfg))
    c = kvq.KVCache(cfg)
    ids = torch.arange(many - 6, many, dtype=torch.int32, device="cuda")
    c.pages[many - 6:] = torch.randint(0, 256, c.pages[:6].shape, device="cuda", dtype=torch.uint8)
    was = c.pages[many - 6:].clone()
    c.page_table[0, :6] = ids
    c.s_quant[0], c.seq_len[0] = 5 + 5 * 16 + 7, 5 + 5 * 16 + 7 + 48
    ref, status, n_live = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (many, 1, 1))
    ref[many - 6:] = 1
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    kvq.kv_seq_fork(cfg, c, ref, one(0), one(1), status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and c.page_table[1, :7].tolist() == [*ids[:5].tolist(), 0, -1]
    assert torch.equal(c.pages[0], was[5])
    ws = torch.zeros(kvq.kv_pages_compact_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    kvq.kv_pages_compact(cfg, c, ref, n_live, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and int(n_live.item()) == 7
    assert c.page_table[0, :6].tolist() == [1, 2, 3, 4, 5, 6] and c.page_table[1, :6].tolist() == [1, 2, 3, 4, 5, 0]
    assert torch.equal(c.pages[1:7], was) and ref[:8].tolist() == [1, 2, 2, 2, 2, 2, 1, 0] and int(ref.sum()) == 12


def test_fork_refusals():
    kvq = _kvq()
    d = Device()
    d.do("reserve", [100, 0, 40, 0, 0, 0, 0, 0, 0])
    d.grow(0, 100)
    d.grow(2, 40)
    p = d.plain()
    for src, dst in (([0], [2]), ([0], [0]), ([0], [9]), ([-1], [3]), ([0, 3], [3, 4])):
        d.status.zero_()
        assert d.do("fork", src, dst) == kvq.KVQ_ERR_BOUNDS, (src, dst)
        if (src, dst) == ([0, 3], [3, 4]):              # 3 is the second pair's source: only (3, 4), an empty copy, is one
            p.fork([3], [4])
        d.check(p)
    d.status.zero_()
    assert d.do("fork", [0, 2, 0], [5, 5, 6]) == kvq.KVQ_ERR_BOUNDS       # 5 twice: the first holds
    p.fork([0, 0], [5, 6])
    d.check(p)
    # no page left for the half-filled one
    d = Device(num_pages=7)
    d.do("reserve", [100] + [0] * 8)
    d.grow(0, 100)
    p = d.plain()
    assert int(d.status.item()) == 0
    assert d.do("fork", [0, 0], [1, 2]) == kvq.KVQ_ERR_BOUNDS
    p.fork([0, 0], [1, 2])
    d.check(p)


def test_free_reports_counts_that_do_not_match():
    kvq = _kvq()
    d = Device()
    d.do("reserve", [100] + [0] * 8)
    d.ref[int(d.c.page_table[0, 1])] = 0
    assert d.do("free", [0]) == kvq.KVQ_ERR_BOUNDS
    assert (d.ref == 0).all() and (d.c.page_table == -1).all()
    d.status.zero_()
    assert d.do("free", [12]) == kvq.KVQ_ERR_BOUNDS


def test_forked_sequences_decode_alike_and_write_apart():
    """A fork's decode equals its source's bit for bit; appends and flushes on one leave the other."""
    import synth
    kvq = _kvq()
    # (n_new sizes the table: the 540 tokens reserved below need ceil((540 - 64) / 16) = 30 of its entries)
    w = synth.WUSH_CHUNK_B16.replace(batch=3, ctx_lo=500, ctx_hi=500, n_new=60, chunk_queries=False, s_flush=1)
    run = harness.DeviceRun(w, do_step=False)
    r, c = run.runner, run.runner.cache
    dev = run.device
    ref = torch.zeros(run.cfg.num_pages, dtype=torch.int32, device=dev)
    held = c.page_table[c.page_table >= 0].long()
    ref.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    kvq.kv_seq_free(run.cfg, c, ref, one(1, 2), r.status)
    kvq.kv_seq_fork(run.cfg, c, ref, one(0, 0), one(1, 2), r.status)
    kvq.kv_pages_reserve(run.cfg, c, ref, one(40, 40, 40), r.status)
    q = run.q.clone()
    q[1:] = q[:1]
    qo = torch.empty_like(q)
    r.append(None, None, None, None, q, qo)
    out = torch.empty_like(r.out)
    r.decode(qo, out)
    torch.cuda.synchronize()
    assert int(r.status.item()) == 0
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    # 30 more tokens for sequence 1 only, flushed: 0 and 2 still read what they did
    rows = torch.randn((30, w.n_kv_heads, 128), device=dev).to(torch.bfloat16)
    pos = torch.arange(500, 530, dtype=torch.int32, device=dev)
    r.append(rows, rows, torch.full((30,), 1, dtype=torch.int32, device=dev), pos)
    r.flush(64)
    again = torch.empty_like(r.out)
    ws = kvq.workspace(run.cfg, 600, dev)
    kvq.kv_attn_decode(run.cfg, c, qo, again, r.sm_scale, 600, ws, r.status)
    torch.cuda.synchronize()
    assert int(r.status.item()) == 0
    a, b = again[0], again[2]
    assert torch.equal(a, b) and not torch.equal(again[1], a)
    assert (a - out[0]).abs().max() <= 2e-3 * out[0].abs().max()           # (another split, the same cache)
