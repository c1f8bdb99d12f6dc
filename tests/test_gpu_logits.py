"""kv_logits_probs and kv_token_counts against float64 and plain counting."""

import numpy as np
import pytest
import torch

import bit_rotated_kv_gb300 as kvq
from tests import spec_ref, step_ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _dev(a, dtype=None):
    return None if a is None else torch.tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


def _cfg(batch):
    return kvq.KVConfig(n_q_heads=1, n_kv_heads=1, batch=batch, max_pages_per_seq=1, num_pages=1, ring_cap=272)


class Call:
    def __init__(self, counts_of_rows, vocab, dtype="f32", seed=1, held=True, bias=0, mask=None, tree=None, heat=(0.7, 1.0, 1.3), rules=True,
                 pad=0):
        rng = self.rng = np.random.default_rng(seed)
        n, batch = list(counts_of_rows), len(counts_of_rows)
        self.n, self.vocab, self.batch, self.rows = n, vocab, batch, sum(n)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        x = rng.normal(0, 3, (self.rows, vocab + pad)).astype(np.float32)
        self.logits = torch.from_numpy(x).cuda().to(TYPES[dtype])[:, :vocab]
        stride = vocab + vocab % 2
        self.counts = None
        if held:
            c = rng.integers(0, 4, (batch, stride)) * (rng.random((batch, stride)) < 0.3) | (rng.random((batch, stride)) < 0.1) * 0x8000
            self.counts = c.astype(np.uint16)
        self.rules = {"temperature": rng.choice(heat, batch).astype(np.float32)}
        if rules:
            self.rules |= {"repetition": rng.choice([1.0, 1.2, 0.8], batch).astype(np.float32), "frequency": rng.uniform(-0.2, 0.5, batch).astype(np.float32),
                           "presence": rng.uniform(-0.2, 1, batch).astype(np.float32)}
        self.bias = {}
        if bias:
            for b in range(batch):
                k = min(vocab, int(rng.integers(0, bias + 1)))
                t = np.sort(rng.choice(vocab, k, replace=False))
                self.bias[b] = {int(v): (float("-inf") if rng.random() < 0.1 else float(np.float32(rng.normal(0, 4)))) for v in t}
        self.allowed = self.mask_row = None
        if mask is not None:
            words = (vocab + 31) // 32 + 1
            self.allowed = rng.random((self.rows, words * 32)) < mask
            self.allowed[np.arange(self.rows), rng.integers(0, vocab, self.rows)] = True
            self.mask_row = rng.permutation(self.rows).astype(np.int32)
            self.mask_row[rng.random(self.rows) < 0.2] = -1
        self.parent = self.token = None
        if tree:
            self.parent = np.concatenate([spec_ref.random_tree(rng, k, tree) for k in n if k]).astype(np.int32)
            self.token = rng.integers(0, min(vocab, 12), self.rows).astype(np.int32)     # (the same ones again and again)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.p = torch.full((self.rows, vocab + pad), 7.0, device="cuda")[:, :vocab]

    def device_rules(self):
        f = lambda n: _dev(self.rules.get(n))  # noqa: E731
        r = kvq.LogitRules(temperature=f("temperature"), repetition=f("repetition"), frequency=f("frequency"), presence=f("presence"))
        if self.counts is not None:
            r.counts = _dev(self.counts.view(np.int16))
        if self.bias:
            k = [len(self.bias[b]) for b in range(self.batch)]
            r.bias_cu = _dev(np.concatenate([[0], np.cumsum(k)]).astype(np.int32))
            r.bias_token = _dev(np.array([t for b in range(self.batch) for t in self.bias[b]], np.int32))
            r.bias = _dev(np.array([v for b in range(self.batch) for v in self.bias[b].values()], np.float32))
        if self.allowed is not None:
            r.mask = _dev(np.packbits(self.allowed, axis=1, bitorder="little").view(np.int32))
            r.mask_row = _dev(self.mask_row)
        return r

    def run(self, stream=None):
        kvq.kv_logits_probs(_cfg(self.batch), self.device_rules(), self.logits, _dev(self.cu), _dev(self.parent), _dev(self.token), self.p, self.status,
                            stream)
        torch.cuda.synchronize()
        return self

    def above(self, b, i):
        """Tokens of node i of sequence b and its ancestors, roots left out."""
        out, at = [], i
        if self.parent is not None:
            first = self.cu[b]
            while self.parent[first + at] >= 0:
                out.append(int(self.token[first + at]))
                at = self.parent[first + at]
        return out

    def check(self, zeros=(), status=0, only=None):
        assert int(self.status.item()) == status
        logits, p = self.logits.double().cpu().numpy(), self.p.double().cpu().numpy()
        for b in range(self.batch):
            for r in range(self.cu[b], self.cu[b + 1]) if only is None else [r for r in only if self.cu[b] <= r < self.cu[b + 1]]:
                if r in zeros:
                    assert (p[r] == 0).all(), r
                    continue
                m = None if self.allowed is None or self.mask_row[r] < 0 else self.allowed[self.mask_row[r], :self.vocab]
                c = None if self.counts is None else self.counts[b, :self.vocab]
                x, size = step_ref.values(logits[r], c, self.above(b, r - self.cu[b]), self.rules | ({"bias": self.bias} if self.bias else {}), b, m)
                want, tol = step_ref.probabilities(x, size, float(self.rules["temperature"][b]))
                assert (np.abs(p[r] - want) <= tol).all(), (r, np.argwhere(np.abs(p[r] - want) > tol)[:4])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1, 3, 31, 33, 1000, 32000, 100003])
def test_types_and_vocabularies(dtype, vocab):
    Call([1, 1, 1], vocab, dtype).run().check()
    Call([2, 0, 3], vocab, dtype, bias=20, mask=0.3, tree="random", heat=(0.5, 0.0)).run().check()


def test_largest_vocabulary():
    Call([1, 2], kvq.KVQ_LOGITS_MAX_VOCAB, "bf16", bias=500, mask=0.5).run().check()
    Call([1], kvq.KVQ_LOGITS_MAX_VOCAB - 1, "f32").run().check()


@pytest.mark.parametrize("rows", [1, 5, 40, 200, 700])
@pytest.mark.parametrize("vocab", [151, 5000, 50021])
def test_many_rows(rows, vocab):
    """Every split of a row over CTAs."""
    c = Call([1] * rows, vocab, "bf16", bias=9, mask=0.9, seed=rows).run()
    c.check(only=range(0, rows, 1 + rows // 25))


@pytest.mark.parametrize("kind", ["chain", "star", "roots", "random"])
def test_paths(kind):
    Call([1, 128, 0, 37], 2003, "f32", tree=kind, bias=12).run().check()
    Call([1, 128, 0, 37], 2003, "f16", tree=kind, held=False, rules=True).run().check()


@pytest.mark.parametrize("what", ["temperature", "repetition", "frequency", "presence", "counts", "bias", "mask", "nothing"])
def test_each_rule_alone(what):
    c = Call([2, 1], 777, held=what not in ("temperature", "bias", "mask", "nothing"), bias=30 if what == "bias" else 0, mask=0.4 if what == "mask" else None)
    for name in list(c.rules):
        if name != what:
            c.rules[name] = np.zeros(2, np.float32) if name in ("frequency", "presence") else np.ones(2, np.float32)
    rules = c.device_rules()
    for name in ("temperature", "repetition", "frequency", "presence"):
        if name != what:
            setattr(rules, name, None)
    c.device_rules = lambda: None if what == "nothing" else rules
    c.run().check()


def test_greedy_takes_the_lowest_of_equals():
    for vocab in (40, 70000):
        c = Call([1, 1, 2], vocab, "bf16", held=False, rules=False, heat=(0.0,))
        c.logits[:] = -1.0
        c.logits[0, [vocab - 1, 33, 34]] = 2.0
        c.logits[1, [vocab - 2]] = 2.0
        c.logits[3, vocab // 2:] = 0.0
        c.run().check()
        assert c.p.argmax(-1).tolist() == [33, vocab - 2, 0, vocab // 2] and bool((c.p.sum(-1) == 1).all())


def test_temperatures():
    """From next to nothing (the best token's neighbours vanish) to the largest (all tokens alike)."""
    c = Call([1] * 6, 500, held=False, rules=False)
    c.rules["temperature"] = np.array([1e-38, 1e-30, 1e-3, 10.0, 1e30, 3e38], np.float32)
    c.logits[0, 7] = 50.0
    c.logits[1, 9] = 50.0
    c.run().check()


@pytest.mark.parametrize("vocab", [100, 40000])
def test_masked_places_hold_anything(vocab):
    """Infinities and NaN under the mask; the lowest values of the type as somebody else's mask."""
    c = Call([1, 1, 1, 1], vocab, held=True, mask=0.5, bias=0)
    c.mask_row = np.arange(4, dtype=np.int32)
    c.allowed[3, :10] = True
    off = torch.from_numpy(~c.allowed[:, :vocab]).cuda()
    junk = torch.tensor([float("nan"), float("inf"), float("-inf"), 3.4e38], device="cuda")[torch.arange(vocab, device="cuda") % 4]
    c.logits.copy_(torch.where(off, junk, c.logits))
    c.logits[2] = torch.where(off[2], c.logits[2], torch.full_like(c.logits[2], torch.finfo(torch.float32).min))
    c.rules["repetition"][2], c.rules["frequency"][2], c.rules["presence"][2] = 1.0, 0.0, 0.0
    c.logits[3, 10:] = float("-inf")
    c.run()
    assert int(c.status.item()) == 0
    p = c.p.cpu().numpy()
    n = int(c.allowed[2, :vocab].sum())
    assert np.allclose(p[2], c.allowed[2, :vocab] / n, rtol=2**-16) and (p[3, 10:] == 0).all()
    c.check(only=[0, 1])


@pytest.mark.parametrize("vocab", [100, 40000])
def test_nothing_left_and_not_finite(vocab):
    c = Call([1] * 9, vocab, held=True, mask=0.5)
    c.mask_row = np.array([0, 1, -1, -1, -1, -1, -1, -1, -1], np.int32)
    c.allowed[0] = False                                   # a mask that leaves nothing
    c.logits[2] = float("-inf")
    c.logits[3, vocab - 1] = float("nan")
    c.logits[4, 0] = float("inf")
    c.rules["temperature"][5] = float("nan")
    c.rules["repetition"][6] = 0.0
    c.rules["frequency"][7] = float("inf")
    c.run()
    c.check(zeros=(0, 2, 3, 4, 5, 6, 7), status=kvq.KVQ_ERR_NONFINITE)
    for name, bad in (("temperature", -1.0), ("temperature", float("inf")), ("repetition", -2.0), ("presence", float("nan"))):
        c = Call([1, 1], vocab, held=True)
        c.rules[name][0] = bad
        c.run().check(zeros=(0,), status=kvq.KVQ_ERR_NONFINITE)


def test_faults_on_the_device():
    bounds = kvq.KVQ_ERR_BOUNDS
    c = Call([1, 1, 1], 300, mask=0.5)
    c.mask_row = np.array([3, 0, -2], np.int32)            # masks that do not exist
    c.run().check(zeros=(0, 2), status=bounds)
    c = Call([5, 130], 300, tree="chain")                  # more nodes than a tree may have
    c.run().check(zeros=range(5, 135), status=bounds)
    c = Call([6], 300, tree="chain")
    c.token[2] = 300                                       # not in the vocabulary: left out
    c.run()
    c.token[2] = 5
    c.check(only=[0, 1], status=bounds)
    assert bool((c.p.sum(-1) - 1).abs().max() < 1e-5)
    c = Call([6], 300, tree="chain")
    c.parent[3] = 4                                        # not a lower node: the path ends there
    c.run().check(only=[0, 1, 2], status=bounds)
    c = Call([2, 2], 300)
    rows = c.p.clone()
    c.cu[2] = 3                                            # the last row is no sequence's
    c.run().check(only=[0, 1, 2], status=bounds)
    assert torch.equal(c.p[3], rows[3])
    c = Call([1, 1], 300, bias=20)
    r = c.device_rules()
    r.bias_token, r.bias = torch.tensor([5, 5, -1, 300, 7], dtype=torch.int32, device="cuda"), torch.full((5,), 2.0, device="cuda")
    r.bias_cu = torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda")
    c.device_rules = lambda: r
    c.run()
    assert int(c.status.item()) == bounds and bool((c.p.sum(-1) - 1).abs().max() < 1e-5)
    c.bias = {0: {}, 1: {}}
    c.check(only=[1], status=bounds)


def test_in_place_and_rows_apart():
    for vocab, pad in ((1000, 24), (1001, 3), (30000, 0)):
        c = Call([2, 3], vocab, pad=pad, bias=8, mask=0.5, tree="random").run()
        c.check()
        d = Call([2, 3], vocab, pad=pad, bias=8, mask=0.5, tree="random")
        around = d.logits.as_strided((5, vocab + pad), (vocab + pad, 1))[:, vocab:].clone()
        d.p = d.logits
        d.run()
        assert torch.equal(c.p, d.p) and int(d.status.item()) == 0
        assert torch.equal(d.logits.as_strided((5, vocab + pad), (vocab + pad, 1))[:, vocab:], around)


def test_offsets_beyond_32_bits():
    stride = (1 << 30) + 4
    c, d = Call([1, 2], 5000), Call([1, 2], 5000).run()
    big = torch.empty(2 * stride + 5000, device="cuda")
    c.p = big.as_strided((3, 5000), (stride, 1))
    logits = torch.empty(2 * stride + 5000, device="cuda").as_strided((3, 5000), (stride, 1))
    logits.copy_(c.logits)
    c.logits = logits
    c.run()
    assert torch.equal(c.p, d.p)


def test_captured_and_on_another_stream():
    c, d = Call([3, 2], 20000, bias=8, tree="random"), Call([3, 2], 20000, bias=8, tree="random").run()
    args = (_cfg(2), c.device_rules(), c.logits, _dev(c.cu), _dev(c.parent), _dev(c.token), c.p, c.status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kvq.kv_logits_probs(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c.p, d.p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kv_logits_probs(*args)
    for _ in range(3):
        c.p.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.p, d.p)


# ---- counts ------------------------------------------------------------------------------------
def _tally(counts, b, tokens, prompt):
    for t in tokens:
        c = int(counts[b, t])
        counts[b, t] = c | 0x8000 if prompt else (c & 0x8000) | min(step_ref.MOST, (c & step_ref.MOST) + 1)


@pytest.mark.parametrize("vocab", [1, 5, 1001, 50000])
@pytest.mark.parametrize("n", [[1], [700, 0, 3000], [40000]])
def test_counts(vocab, n):
    rng, batch = np.random.default_rng(4), len(n)
    stride = vocab + vocab % 2 + 2
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    token = np.minimum(vocab - 1, vocab * rng.random(int(cu[-1])) ** 3).astype(np.int32)
    want = np.zeros((batch, stride), np.uint16)
    got = torch.zeros((batch, stride), dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kind in (kvq.KVQ_COUNT_PROMPT, kvq.KVQ_COUNT_OUTPUT, kvq.KVQ_COUNT_OUTPUT):
        nxt = _dev(rng.integers(0, vocab, batch).astype(np.int32)) if kind == kvq.KVQ_COUNT_OUTPUT else None
        kvq.kv_token_counts(_cfg(batch), got, vocab, kind, _dev(cu), _dev(token), None, None, nxt, status)
        for b in range(batch):
            _tally(want, b, token[cu[b]:cu[b + 1]], kind == kvq.KVQ_COUNT_PROMPT)
            if nxt is not None:
                _tally(want, b, [int(nxt[b])], False)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and np.array_equal(got.cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("vocab,n", [(1001, [200000, 0, 300001, 100003]), (70001, [524288 + 5]), (16384, [3, 400000, 200000]), (524288, [100003]), (600001, [120000]),
                                     (33, [70000, 6]), (131072, [65536 + 3, 0, 1])])
def test_long_prompts(vocab, n):
    """Enough rows for the sweep: slices' ends, tokens outside the vocabulary, rows of no sequence, counts that are there already."""
    rng, batch = np.random.default_rng(6), len(n)
    stride = vocab + vocab % 2
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    token = np.minimum(vocab - 1, vocab * rng.random(int(cu[-1])) ** 3).astype(np.int32)
    token[rng.integers(0, len(token), 100)] = vocab - 1
    have = rng.integers(0, 9, (batch, stride)).astype(np.uint16)
    for cut, outside in ((0, False), (7, False), (0, True)):
        tok = token.copy()
        if outside:
            tok[rng.integers(0, len(tok), 50)] = rng.choice([-1, vocab, 1 << 30], 50)
        at = cu.copy()
        at[0], at[-1] = cut, cu[-1] - cut
        got, status = torch.tensor(have.view(np.int16), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        kvq.kv_token_counts(_cfg(batch), got, vocab, kvq.KVQ_COUNT_PROMPT, _dev(at), _dev(tok), None, None, None, status)
        want = have.copy()
        for b in range(batch):
            t = tok[at[b]:at[b + 1]]
            want[b, t[(t >= 0) & (t < vocab)]] |= 0x8000
        torch.cuda.synchronize()
        assert int(status.item()) == (kvq.KVQ_ERR_BOUNDS if cut or outside else 0)
        assert np.array_equal(got.cpu().numpy().view(np.uint16), want)


def test_counts_of_kept_paths():
    rng = np.random.default_rng(5)
    n, vocab = [1, 9, 0, 128], 77
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    token = rng.integers(0, vocab, int(cu[-1])).astype(np.int32)
    path, kept, want = np.full(int(cu[-1]), -1, np.int32), np.zeros(4, np.int32), np.zeros((4, 78), np.uint16)
    nxt = np.array([3, 3, -1, 70], np.int32)
    for b in (0, 1, 3):
        kept[b] = rng.integers(1, n[b] + 1)
        nodes = np.concatenate([[0], np.sort(rng.choice(np.arange(1, n[b]), kept[b] - 1, replace=False))]).astype(int)
        path[cu[b]:cu[b] + kept[b]] = nodes
        _tally(want, b, [*token[cu[b] + nodes[1:]], nxt[b]], False)
    got, status = torch.zeros((4, 78), dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_cfg(4), got, vocab, kvq.KVQ_COUNT_OUTPUT, _dev(cu), _dev(token), _dev(path), _dev(kept), _dev(nxt), status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kv_token_counts(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and np.array_equal(got.cpu().numpy().view(np.uint16), want)
    # a step without drafts: the next tokens alone
    kvq.kv_token_counts(_cfg(4), got, vocab, kvq.KVQ_COUNT_OUTPUT, None, None, None, None, _dev(nxt), status)
    for b in (0, 1, 3):
        _tally(want, b, [nxt[b]], False)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy().view(np.uint16), want)


def test_counts_leave_out_what_is_out_of_bounds():
    got, status = torch.zeros((2, 10), dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, token = np.array([0, 4, 6], np.int32), np.array([1, -1, 9, 2, 4, 4, 5, 5], np.int32)
    kvq.kv_token_counts(_cfg(2), got, 9, kvq.KVQ_COUNT_OUTPUT, _dev(cu), _dev(token), None, None, _dev(np.array([9, 8], np.int32)), status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS
    assert got.tolist() == [[0, 1, 1, 0, 0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 2, 0, 0, 0, 1, 0]]
    got.zero_()
    status.zero_()
    path, kept = np.array([0, 3, 4, 2, 0, 1, 0, 0], np.int32), np.array([9, 2], np.int32)
    kvq.kv_token_counts(_cfg(2), got, 9, kvq.KVQ_COUNT_OUTPUT, _dev(cu), _dev(np.array([1, 0, 3, 2, 4, 6, 5, 5], np.int32)), _dev(path), _dev(kept), None,
                        status)
    torch.cuda.synchronize()
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS
    assert got.tolist() == [[0, 0, 1, 1, 0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0, 1, 0, 0, 0]]


def test_counts_stop_at_the_most():
    got, status = torch.zeros((1, 4), dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    got[0, :] = torch.tensor([32766, -2, 32767, 5])        # (-2: the prompt's, 32766 times)
    token = np.concatenate([np.zeros(5), np.ones(1), np.full(3, 2), np.full(70000, 3)]).astype(np.int32)
    kvq.kv_token_counts(_cfg(1), got, 4, kvq.KVQ_COUNT_OUTPUT, _dev(np.array([0, len(token)], np.int32)), _dev(token), None, None, None, status)
    torch.cuda.synchronize()
    assert got.tolist() == [[32767, -1, 32767, 32767]] and int(status.item()) == 0
