"""kv_rope_qk: norm, rotary positions, transform and append, against float64 with phases in whole numbers."""

import numpy as np
import pytest
import torch

import bit_rotated_kv_gb300 as kvq
import synth
from tests import harness, step_ref

pytestmark = pytest.mark.gpu
D = 128


def _f64(t):
    return t.detach().double().cpu().numpy()


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


class Call:
    """A call's inputs, its cache, and what the formulas say of it."""

    def __init__(self, rows, hq=8, hkv=2, kind="invertible", tv=True, layout=kvq.KVQ_ROPE_HALF, rot=128, norm=True, scale=1.0, seed=1,
                 pos=None, far=None, sink=16, cap=None, ctx=None, theta=1e6, gap=0, size=1.0, tail=0):
        rng = np.random.default_rng(seed)
        self.rows, self.hq, self.hkv, self.kind, self.layout, self.rot = rows, hq, hkv, kind, layout, rot
        w = synth.TINY_GQA4.replace(n_q_heads=hq, n_kv_heads=hkv, transform=kind, value_transform="orthogonal" if tv else "identity", seed=seed)
        self.tr, (tk, tkit, self.tv) = harness.device_transform(w, torch.device("cuda"))
        had = [step_ref.hadamard()] * hkv
        self.tk, self.tkit = (had, had) if tk is None else (tk, tkit)
        # rows of two sequences in turn, from ctx on
        self.seq = np.arange(rows) % 2
        self.ctx = np.array([5, 300]) if ctx is None else np.array(ctx)
        self.pos = self.ctx[self.seq] + np.arange(rows) // 2 if pos is None else np.asarray(pos)
        self.far = None if far is None else np.asarray(far)
        edge = np.maximum(sink, self.ctx - 32)
        need = int((self.pos + 1 - edge[self.seq]).max()) if rows else 16
        self.cap = cap or max(48, harness.round16(need))
        self.cfg = kvq.KVConfig(n_q_heads=hq, n_kv_heads=hkv, batch=2, max_pages_per_seq=1, num_pages=1, ring_cap=self.cap, s_sink=sink,
                                s_keep=24, s_flush=8)
        self.cache = kvq.KVCache(self.cfg)
        self.cache.seq_len.copy_(_i32(self.ctx))
        self.cache.s_quant.copy_(_i32(edge))
        for t in (self.cache.sink_k, self.cache.sink_v, self.cache.ring_k, self.cache.ring_v):
            t.fill_(7.0)                                   # (rows that are not written stay what they were)
        # one fused projection, `gap` channels between its rows
        width = (hq + 2 * hkv) * D
        x = rng.standard_normal((rows + tail, width + gap)) * size
        x.reshape(rows + tail, -1)[:, 3] *= 15
        self.fused = torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16)
        heads = self.fused[:rows, :width].unflatten(1, (hq + 2 * hkv, D))
        self.q, self.k, self.v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
        self.wq, self.wk = (rng.uniform(-1, 2, D).astype(np.float32) for _ in range(2)) if norm else (None, None)
        self.eps = 1e-5
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.rope = kvq.Rope.make(layout, rot, theta, q_norm=dev(self.wq), k_norm=dev(self.wk), norm_eps=self.eps)
        self.rope.scale = scale
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((rows + tail, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.args = [self.seq, self.pos, self.far]

    def run(self, stream=None, rope="own"):
        seq, pos = _i32(self.seq), _i32(self.pos)
        far = None if self.far is None else _i32(self.far)
        kvq.kv_rope_qk(self.cfg, self.tr, self.rope if rope == "own" else rope, self.q, self.q_out, pos if far is None else far, self.k, self.v,
                       seq, pos, far, self.cache, self.status, stream)
        torch.cuda.synchronize()
        return self

    def want(self, rope=True):
        far = self.pos if self.far is None else self.far
        angle = step_ref.phases(self.rope.freq.cpu().tolist(), far) if rope else np.zeros((self.rows, 0))
        out = []
        for x, w, mats, gqa in ((self.q, self.wq, self.tkit, self.hq // self.hkv), (self.k, self.wk, self.tk, 1)):
            y, m = step_ref.placed(_f64(x), angle, self.layout == kvq.KVQ_ROPE_INTERLEAVED, self.rope.scale if rope else 1.0, w if rope else None, self.eps)
            out.append(step_ref.transformed(y, m, mats, gqa))
        v = _f64(self.v)
        out.append((v, 0 * v) if self.tv is None else step_ref.transformed(v, np.abs(v), self.tv, 1))
        return out

    def check(self, rope=True, rows=None, status=0):
        """Every row of the caches and q_out: those written, and that the others were left alone."""
        (q, qb), k, v = self.want(rope)
        assert int(self.status.item()) == status
        rows = np.arange(self.rows) if rows is None else np.asarray(rows)
        got = _f64(self.q_out[:self.rows])
        assert step_ref.near(got, q, qb).all(), np.argwhere(~step_ref.near(got, q, qb))[:4]
        assert bool((self.q_out[self.rows:] == 7.0).all())
        c = self.cache
        for (x, b), sink, ring in ((k, c.sink_k, c.ring_k), (v, c.sink_v, c.ring_v)):
            sink, ring = _f64(sink), _f64(ring)
            for r in rows:
                s, p = self.seq[r], self.pos[r]
                at = (sink, p) if p < self.cfg.s_sink else (ring, p % self.cap)
                g = at[0][s, :, at[1]]
                assert step_ref.near(g, x[r], b[r]).all(), (r, np.argwhere(~step_ref.near(g, x[r], b[r]))[:4])
                at[0][s, :, at[1]] = 7.0
            assert (sink == 7.0).all() and (ring == 7.0).all()
        want = self.ctx.copy()
        for r in rows:
            want[self.seq[r]] = max(want[self.seq[r]], self.pos[r] + 1)
        assert c.seq_len.tolist() == want.tolist()


@pytest.mark.parametrize("kind,tv", [("invertible", True), ("orthogonal", False), ("hadamard", True), ("hadamard", False), ("identity", False)])
@pytest.mark.parametrize("layout", [kvq.KVQ_ROPE_HALF, kvq.KVQ_ROPE_INTERLEAVED], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 64, 96, 6, 2, 126])
def test_layouts(kind, tv, layout, rot):
    Call(9, kind=kind, tv=tv, layout=layout, rot=rot, norm=rot != 64, scale=1.25 if rot == 96 else 1.0).run().check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 1), (16, 8), (64, 8)])
@pytest.mark.parametrize("rows", [1, 2, 7, 33])
def test_head_layouts(hq, hkv, rows):
    Call(rows, hq, hkv, tv=rows != 7, gap=8 * (rows % 3)).run().check()


# (prefill sizes: more (row, head) pairs than fill the SMs' first tiles, odd ones among them)
@pytest.mark.parametrize("rows,hq,hkv,kind,tv,layout,rot,norm", [
    (1201, 16, 4, "invertible", False, 0, 128, True), (2051, 8, 8, "orthogonal", True, 1, 128, True), (5003, 4, 1, "hadamard", False, 0, 128, False),
    (700, 64, 8, "hadamard", True, 1, 64, True), (1203, 8, 4, "invertible", True, 0, 96, True), (2500, 8, 2, "identity", False, 0, 6, False),
    (3001, 8, 1, "invertible", True, 1, 0, True), (1300, 32, 8, "orthogonal", False, 0, 126, False)])
def test_prefill_sizes(rows, hq, hkv, kind, tv, layout, rot, norm):
    Call(rows, hq, hkv, kind, tv, layout, rot, norm, gap=8).run().check()


# (the sizes at which calls go to the tensor cores: 12 pairs a row, with Hadamard matrices 10)
@pytest.mark.parametrize("kind,rows", [("orthogonal", 74), ("invertible", 75), ("hadamard", 127), ("hadamard", 128), ("orthogonal", 160)])
def test_sizes_about_the_choice(kind, rows):
    Call(rows, kind=kind, tv=kind != "hadamard", rot=96, layout=rows % 2).run().check()


# (the sizes from which on runs of work differ in length: no pair left out at either end)
@pytest.mark.parametrize("rows,hq,hkv,tv", [(7801, 32, 8, False), (7800, 32, 8, False), (155_701, 1, 1, True), (20_011, 8, 8, False)])
def test_long_prefill(rows, hq, hkv, tv):
    Call(rows, hq, hkv, tv=tv).run().check()


@pytest.mark.parametrize("rows", [3, 3001])
def test_positions(rows):
    """Positions in the text that are not the tokens' numbers: far, negative, at the ends of the type."""
    far = np.random.default_rng(3).integers(-2**31, 2**31, rows)
    far[:3] = [2**31 - 1, -2**31, 1 << 20]
    Call(rows, far=far, rot=64).run().check()


@pytest.mark.parametrize("rows", [4, 3001])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 3e4, 1e30])
def test_magnitudes(rows, size):
    """Rows of any magnitude.  (With a norm, squares beyond float32 are reported: test_not_finite.)"""
    Call(rows, size=size, norm=size in (1e-4, 3e4)).run().check()


def test_wide_rows():
    """Channels that lie up to 30 binades apart within a row, and rows of zeros."""
    for rows in (6, 3001):
        c = Call(rows, norm=False, rot=64)
        rng = np.random.default_rng(5)
        c.fused.mul_(torch.from_numpy(2.0 ** -rng.integers(0, 30, c.fused.shape)).cuda().to(torch.bfloat16))
        c.fused[rows // 2] = 0
        c.run().check()


@pytest.mark.parametrize("rows", [5, 3001])
def test_without_rope(rows):
    c = Call(rows)
    c.run(rope=None)
    c.check(rope=False)


@pytest.mark.parametrize("rows", [3, 2600])
def test_queries_or_keys_alone(rows):
    a, b = Call(rows, tv=False), Call(rows, tv=False)
    pos, seq = _i32(a.pos), _i32(a.seq)
    kvq.kv_rope_qk(a.cfg, a.tr, a.rope, a.q, a.q_out, pos, None, None, None, None, None, a.cache, a.status)
    kvq.kv_rope_qk(a.cfg, a.tr, a.rope, None, None, None, a.k, a.v, seq, pos, None, a.cache, a.status)
    kvq.kv_rope_qk(a.cfg, a.tr, a.rope, None, None, None, None, None, None, None, None, a.cache, a.status)
    torch.cuda.synchronize()
    a.check()
    b.run()
    if rows == 3:                                          # (the same kernel either way)
        assert torch.equal(a.q_out, b.q_out) and torch.equal(a.cache.ring_k, b.cache.ring_k)


@pytest.mark.parametrize("rows", [6, 3001])
def test_rows_out_of_bounds_are_skipped(rows):
    c = Call(rows)
    bad = {0: (-1, 40), 1: (2, 40), 2: (0, -1), 3: (1, 200), 4: (0, 16 + c.cap)}
    for r, (s, p) in bad.items():
        c.seq[r], c.pos[r] = s, p
    c.far = c.pos                                          # (the queries' positions as they are)
    c.run()
    c.check(rows=range(5, rows), status=kvq.KVQ_ERR_BOUNDS)


@pytest.mark.parametrize("rows", [6, 3001])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_not_finite(rows, norm):
    """A row that holds an infinity or NaN: its own results are not finite, the others are what they were."""
    c = Call(rows, norm=norm, rot=64)
    c.q[1, 0, 100] = float("inf")
    c.k[2, 1, 5] = float("nan")
    c.v[3, 0, 77] = float("-inf")
    if norm:
        c.q[4, 2, :] = 1e25
    c.run()
    assert int(c.status.item()) == kvq.KVQ_ERR_NONFINITE
    got = c.q_out[:rows].float()
    bad = torch.zeros(rows, c.hq, dtype=torch.bool, device="cuda")
    bad[1, 0] = True
    bad[4, 2] = norm
    assert bool((~torch.isfinite(got)).any(-1)[bad].all()) and bool(torch.isfinite(got[~bad]).all())
    for r, h, t in ((2, 1, "k"), (3, 0, "v")):
        s, p = c.seq[r], c.pos[r]
        sink, ring = getattr(c.cache, f"sink_{t}"), getattr(c.cache, f"ring_{t}")
        row = sink[s, h, p] if p < c.cfg.s_sink else ring[s, h, p % c.cap]
        assert not bool(torch.isfinite(row).any())
    # the same call with those rows at zero: every other row bit for bit
    d = Call(rows, norm=norm, rot=64)
    d.fused.copy_(c.fused)
    d.q[1, 0] = d.k[2, 1] = d.v[3, 0] = d.q[4, 2] = 0
    d.run()
    assert int(d.status.item()) == 0
    same = (c.q_out[:rows] == d.q_out[:rows]).all(-1)
    same[4, 2] = True
    assert bool(same[~bad].all())


def test_captured_and_on_another_stream():
    for rows in (4, 3001):
        c, d = Call(rows), Call(rows).run()
        seq, pos = _i32(c.seq), _i32(c.pos)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            kvq.kv_rope_qk(c.cfg, c.tr, c.rope, c.q, c.q_out, pos, c.k, c.v, seq, pos, None, c.cache, c.status)
        torch.cuda.synchronize()
        c.check()
        keep = c.q_out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kvq.kv_rope_qk(c.cfg, c.tr, c.rope, c.q, c.q_out, pos, c.k, c.v, seq, pos, None, c.cache, c.status)
        for _ in range(2):
            c.q_out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.q_out, keep) and torch.equal(c.q_out, d.q_out)
        c.fused.mul_(0.5)                                  # (other numbers in the same places)
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_the_same_every_time():
    for rows in (5, 3001):
        a, b = Call(rows).run(), Call(rows).run()
        assert torch.equal(a.q_out, b.q_out) and torch.equal(a.cache.ring_k, b.cache.ring_k) and torch.equal(a.cache.ring_v, b.cache.ring_v)


def test_against_the_exact_transform():
    """Rows that bf16 holds after the rotation (none at position 0): kv_rotate_qk's exact product, or its neighbour."""
    c = Call(12, norm=False, far=np.zeros(12, np.int64)).run()
    d = Call(12, norm=False)
    kvq.kv_rotate_qk(d.cfg, d.tr, d.q.contiguous(), d.q_out, d.k.contiguous(), d.v.contiguous(), _i32(d.seq), _i32(d.pos), d.cache, d.status)
    torch.cuda.synchronize()
    for x, y in ((c.q_out, d.q_out), (c.cache.ring_k, d.cache.ring_k), (c.cache.sink_v, d.cache.sink_v)):
        step = (x.view(torch.int16).int() - y.view(torch.int16).int()).abs()
        assert int(step.max()) <= 1 and float((step > 0).float().mean()) < 0.01


def test_offsets_beyond_32_bits():
    """Rows whose stride takes them past 2^31 elements of the projection."""
    stride = (1 << 30) + 8
    big = torch.empty(2 * stride + 2048, dtype=torch.bfloat16, device="cuda")
    c = Call(3, 8, 2)
    wide = big.as_strided((3, 12, D), (stride, D, 1))
    wide.copy_(c.fused[:3, :12 * D].unflatten(1, (12, D)))
    c.q, c.k, c.v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    c.run().check()


def test_calls_at_once():
    """Three streams at once: two calls on the tensor cores and kv_rotate_qk's, which take tensor memory of the same SMs."""
    a, b, c = Call(4003, 8, 8, kind="orthogonal"), Call(3001, 16, 4, layout=1, seed=2), Call(3001, 8, 8, seed=3)
    d, x = Call(3001, 8, 8, seed=3), [_i32(v) for v in (a.seq, a.pos, b.seq, b.pos, c.seq, c.pos)]
    rot = lambda z, s: kvq.kv_rotate_qk(z.cfg, z.tr, z.q.contiguous(), z.q_out, z.k.contiguous(), z.v.contiguous(), x[4], x[5], z.cache, z.status, s)  # noqa: E731
    rot(d, None)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    rows = [t.contiguous() for t in (c.q, c.k, c.v)]
    torch.cuda.synchronize()
    for _ in range(8):
        for z, s, i in ((a, streams[0], 0), (b, streams[1], 2)):
            kvq.kv_rope_qk(z.cfg, z.tr, z.rope, z.q, z.q_out, x[i + 1], z.k, z.v, x[i], x[i + 1], None, z.cache, z.status, s)
        kvq.kv_rotate_qk(c.cfg, c.tr, rows[0], c.q_out, rows[1], rows[2], x[4], x[5], c.cache, c.status, streams[2])
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert torch.equal(c.q_out, d.q_out) and torch.equal(c.cache.ring_k, d.cache.ring_k) and int(c.status.item()) == 0


def test_a_call_behind_it():
    """The next call in the stream begins while this one's last blocks run: what it reads is whole."""
    a = Call(3001)
    seq, pos = _i32(a.seq), _i32(a.pos)
    again = torch.full_like(a.q_out, 7.0)
    for _ in range(6):
        a.q_out.fill_(7.0)
        kvq.kv_rope_qk(a.cfg, a.tr, a.rope, a.q, a.q_out, pos, a.k, a.v, seq, pos, None, a.cache, a.status)
        kvq.kv_rope_qk(a.cfg, a.tr, None, a.q_out, again, None, None, None, None, None, None, a.cache, a.status)
    torch.cuda.synchronize()
    a.check()
    first = again.clone()
    kvq.kv_rope_qk(a.cfg, a.tr, None, a.q_out, again, None, None, None, None, None, None, a.cache, a.status)
    torch.cuda.synchronize()
    assert torch.equal(first, again)


@pytest.mark.parametrize("rows", [4, 100, 3001])
def test_matrices_written_just_before(rows):
    """A call sees what the stream wrote into the matrices just before it."""
    a, b = Call(rows, kind="invertible", tv=True, seed=1), Call(rows, kind="invertible", tv=True, seed=2)
    b.fused.copy_(a.fused)
    own = [[t.clone() for t in (z.tr.t_k, z.tr.t_k_inv_t, z.tr.t_v)] for z in (a, b)]
    a.run()
    b.rope = a.rope
    b.run()
    want = [(z.q_out.clone(), z.cache.ring_k.clone(), z.cache.ring_v.clone()) for z in (a, b)]
    assert not torch.equal(want[0][0], want[1][0])
    seq, pos = _i32(a.seq), _i32(a.pos)
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        for t, w in zip((a.tr.t_k, a.tr.t_k_inv_t, a.tr.t_v), own[i % 2], strict=True):
            t.copy_(w)
        kvq.kv_rope_qk(a.cfg, a.tr, a.rope, a.q, a.q_out, pos, a.k, a.v, seq, pos, None, a.cache, a.status)
        got.append((a.q_out.clone(), a.cache.ring_k.clone(), a.cache.ring_v.clone()))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2], strict=True)), i
