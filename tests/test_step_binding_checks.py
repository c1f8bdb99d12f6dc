"""The binding and the C entry points of a step's two ends refuse what the kernels would misread or write past.  (No GPU: every call
here is refused, the sound ones because their tensors are not on one.)"""

import ctypes
import os

import pytest
import torch

import bit_rotated_kv_gb300 as kvq

B, N, V, HQ, HKV = 2, 5, 90, 4, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(kvq.LIB_PATH):
        from bit_rotated_kv_gb300 import build_lib
        build_lib.build()


CFG = kvq.KVConfig(n_q_heads=HQ, n_kv_heads=HKV, batch=B, max_pages_per_seq=8, num_pages=24, ring_cap=272)


class _Cache:
    pages = torch.zeros((24, 1, 1152), dtype=torch.uint8)

    @staticmethod
    def c():
        return kvq.CCache()


def _i(n):
    return torch.zeros(n, dtype=torch.int32)


def _m():
    return torch.zeros(HKV, 128, 128)


def _args():
    x = torch.zeros((N, HQ + 2 * HKV, 128), dtype=torch.bfloat16)
    tr = kvq.Transform(kvq.KVQ_TRANSFORM_DENSE, _m(), _m(), _m())
    rope = kvq.Rope(kvq.KVQ_ROPE_HALF, 128, torch.zeros(64, dtype=torch.int64), 1.0, torch.ones(128), torch.ones(128))
    rules = kvq.LogitRules(torch.ones(B), torch.ones(B), torch.ones(B), torch.ones(B), torch.zeros(B, V, dtype=torch.int16), _i(B + 1), _i(3), torch.ones(3),
                           torch.zeros(2, 3, dtype=torch.int32), _i(N))
    return {
        "kv_rope_qk": (kvq.kv_rope_qk, dict(cfg=CFG, tr=tr, rope=rope, q=x[:, :HQ], q_out=torch.zeros((N, HQ, 128), dtype=torch.bfloat16), q_pos=_i(N),
                                            k=x[:, HQ:HQ + 1], v=x[:, HQ + 1:], seq_idx=_i(N), pos=_i(N), rope_pos=_i(N), cache=_Cache, status=_i(1))),
        "kv_logits_probs": (kvq.kv_logits_probs, dict(cfg=CFG, rules=rules, logits=torch.zeros(N, V), cu_rows=_i(B + 1), parent=_i(N), token=_i(N),
                                                      p=torch.zeros(N, V), status=_i(1))),
        "kv_token_counts": (kvq.kv_token_counts, dict(cfg=CFG, counts=torch.zeros(B, V, dtype=torch.int16), vocab=V, kind=kvq.KVQ_COUNT_OUTPUT, cu_rows=_i(B + 1),
                                                      token=_i(N), path=_i(N), n_accept=_i(B), next_token=_i(B), status=_i(1))),
    }


@pytest.fixture
def here(monkeypatch):
    monkeypatch.setattr(kvq, "_current_device", lambda: -1)


def _refusal(call, code=kvq.KVQ_ERR_INVALID_ARG, **other):
    fn, kw = _args()[call]
    with pytest.raises(kvq.KVQError) as e:
        fn(**{**kw, **other})
    assert e.value.code == code
    return str(e.value)


TENSORS = [(call, name) for call, (_, kw) in _args().items() for name, t in kw.items() if torch.is_tensor(t)]


@pytest.mark.parametrize("call", sorted(_args()))
def test_tensors_off_the_device_are_refused(call):
    assert "device" in _refusal(call)


@pytest.mark.parametrize("call,name", TENSORS)
def test_another_type_is_refused(here, call, name):
    t = _args()[call][1][name]
    assert call in _refusal(call, **{name: t.to(torch.int64 if t.dtype in (torch.int32, torch.int16) else torch.float64)})


@pytest.mark.parametrize("call,name", [c for c in TENSORS if c[1] != "status" and c not in (("kv_token_counts", "token"), ("kv_rope_qk", "q"))])
def test_too_few_elements_are_refused(here, call, name):
    t = _args()[call][1][name]
    assert call in _refusal(call, **{name: t[:-1]})


@pytest.mark.parametrize("call,name", [c for c in TENSORS if c[1] != "status"])
def test_gaps_are_refused(here, call, name):
    t = _args()[call][1][name]
    assert call in _refusal(call, **{name: torch.stack([t, t], -1)[..., 0]})


@pytest.mark.parametrize("call,name", [("kv_rope_qk", x) for x in ("q_out", "q_pos", "v", "seq_idx", "pos")] + [("kv_logits_probs", x) for x in ("cu_rows", "p")]
                         + [("kv_token_counts", x) for x in ("counts", "cu_rows")])
def test_missing_tensors_are_refused(here, call, name):
    assert call in _refusal(call, **{name: None})


def test_heads_and_rows(here):
    x = torch.zeros((N, 8, 128), dtype=torch.bfloat16)
    for bad in (x, x[:, :HQ, :64], x[:, 0:8:2], x[:, :HQ].transpose(0, 1), x[0, :HQ].expand(N, HQ, 128), x[:, :HQ].flatten(1)):
        assert ": q" in _refusal("kv_rope_qk", q=bad)
    assert ": k" in _refusal("kv_rope_qk", k=x[:N - 1, :1].expand(N - 1, 2, 128))
    for bad in (torch.zeros(V, N).t(), torch.zeros(1, V).expand(N, V), torch.zeros(N * V), torch.zeros(N, V, dtype=torch.int32)):
        assert "logits" in _refusal("kv_logits_probs", logits=bad) or bad.dtype == torch.float32
    assert "counts" in _refusal("kv_token_counts", counts=torch.zeros(B, V + 1, dtype=torch.int16))        # (an odd stride)


def test_rules_and_rope(here):
    good = _args()["kv_logits_probs"][1]["rules"]
    for name, bad in (("temperature", torch.ones(B - 1)), ("repetition", torch.ones(B).double()), ("frequency", torch.ones(2 * B)[::2]),
                      ("presence", torch.ones(B - 1)), ("counts", torch.zeros(B, V - 2, dtype=torch.int16)), ("counts", torch.zeros(B - 1, V, dtype=torch.int16)),
                      ("bias_cu", _i(B)), ("bias", torch.ones(2)), ("bias_token", torch.ones(3)), ("mask", torch.zeros(2, 2, dtype=torch.int32)),
                      ("mask", torch.zeros(2, 3)), ("mask_row", _i(N - 1))):
        kw = {f: getattr(good, f) for f in good.__dataclass_fields__}
        assert name in _refusal("kv_logits_probs", rules=kvq.LogitRules(**{**kw, name: bad}))
    r = _args()["kv_rope_qk"][1]["rope"]
    for name, bad in (("freq", torch.zeros(63, dtype=torch.int64)), ("freq", torch.zeros(64)), ("q_norm", torch.ones(127)), ("k_norm", torch.ones(128).double()),
                      ("freq", None)):
        kw = {f: getattr(r, f) for f in r.__dataclass_fields__}
        assert name in _refusal("kv_rope_qk", rope=kvq.Rope(**{**kw, name: bad}))
    for name in ("t_k", "t_v"):
        tr = kvq.Transform(kvq.KVQ_TRANSFORM_DENSE, _m(), _m(), _m())
        setattr(tr, name, _m().transpose(1, 2))
        assert name in _refusal("kv_rope_qk", tr=tr)


# ---- the C entry points: addresses that are never read ---------------------------------------------------
X = 1 << 20


def _rope(**kw):
    c, t = CFG.c(), kvq.CTransform(kw.pop("kind", 0), 0, *kw.pop("mats", (X, X, X)))
    cache = kvq.CCache(*([X] * 9))
    base = dict(layout=0, rot_dim=128, scale=1.0, norm_eps=1e-6, freq=X, q_norm=X, k_norm=X)
    r = kvq.CRope(*{**base, **{k: kw.pop(k) for k in list(kw) if k in base}}.values())
    args = dict(q=X, qs=512, out=1 << 30, qpos=X, nq=N, k=X, ks=128, v=X, vs=128, seq=X, pos=X, far=0, nkv=N) | kw
    return kvq.lib().kv_rope_qk(ctypes.byref(c), ctypes.byref(t), ctypes.byref(r), *args.values(), ctypes.byref(cache), None, None)


def test_rope_refusals():
    inval = kvq.KVQ_ERR_INVALID_ARG
    for bad in (dict(layout=2), dict(rot_dim=130), dict(rot_dim=3), dict(rot_dim=-2), dict(freq=0), dict(freq=X + 4), dict(scale=float("nan")),
                dict(norm_eps=0.0), dict(norm_eps=float("inf")), dict(q_norm=X + 8), dict(kind=7), dict(mats=(0, X, X)), dict(mats=(X, 0, X)), dict(mats=(X, X, X + 8)),
                dict(q=0), dict(q=X + 8), dict(qs=504), dict(qs=516), dict(out=0), dict(out=(1 << 30) + 8), dict(qpos=0), dict(nq=-1), dict(nkv=-1), dict(k=0),
                dict(k=X + 2), dict(ks=120), dict(v=0), dict(vs=132), dict(seq=0), dict(pos=0), dict(far=X + 2), dict(out=X + 512), dict(out=X - 4096)):
        assert _rope(**bad) == inval, bad
    assert _rope(nq=0, nkv=0) == 0


def _probs(**kw):
    names = [f[0] for f in kvq.CLogitRules._fields_]
    base = dict.fromkeys(names, X) | dict(count_stride=V, mask_stride=3, n_bias=3, n_masks=2)
    u = kvq.CLogitRules(*{**base, **{k: kw.pop(k) for k in list(kw) if k in base}}.values())
    args = dict(logits=X, kind=1, ls=V, vocab=V, cu=X, parent=X, token=X, n=N, p=1 << 30, ps=V) | kw
    return kvq.lib().kv_logits_probs(ctypes.byref(CFG.c()), ctypes.byref(u), *args.values(), None, None)


def test_probs_refusals():
    inval = kvq.KVQ_ERR_INVALID_ARG
    for bad in (dict(kind=3), dict(kind=-1), dict(n=-1), dict(vocab=0), dict(cu=0), dict(cu=X + 2), dict(parent=0), dict(token=0), dict(logits=0), dict(logits=X + 1),
                dict(p=0), dict(p=X + 2), dict(ls=V - 1), dict(ps=V - 1), dict(count_stride=V - 1), dict(count_stride=V + 1), dict(counts=X + 2), dict(bias=0), dict(bias_token=0),
                dict(n_bias=-1), dict(mask_stride=2), dict(n_masks=-1), dict(mask_row=X + 1), dict(temperature=X + 1), dict(p=X), dict(p=X + 4 * V), dict(kind=0, p=X, ps=V + 1),
                dict(kind=0, p=X + 4)):
        assert _probs(**bad) == inval, bad
    assert _probs(vocab=kvq.KVQ_LOGITS_MAX_VOCAB + 1) == kvq.KVQ_ERR_UNSUPPORTED
    assert _probs(n=0, logits=0, p=0) == 0


def _counts(**kw):
    args = dict(counts=X, stride=V, vocab=V, kind=1, cu=X, token=X, n=N, path=X, acc=X, nxt=X) | kw
    return kvq.lib().kv_token_counts(ctypes.byref(CFG.c()), *args.values(), None, None)


def test_counts_refusals():
    inval = kvq.KVQ_ERR_INVALID_ARG
    for bad in (dict(counts=0), dict(counts=X + 2), dict(stride=V - 1), dict(stride=V + 1), dict(vocab=0), dict(kind=2), dict(n=-1), dict(cu=0), dict(token=0), dict(path=0),
                dict(acc=0), dict(kind=0), dict(kind=0, path=0, acc=0), dict(nxt=X + 1), dict(token=X + 3)):
        assert _counts(**bad) == inval, bad
    assert _counts(n=(1 << 30) + 1) == kvq.KVQ_ERR_UNSUPPORTED
    assert _counts(n=0, nxt=0, path=0, acc=0) == 0


def test_rope_rows_under_the_output():
    """q_out anywhere on the rows of q, of k or of v: refused (a fused projection's rows reach from its first q to its last v)."""
    far = dict(q=1 << 32, k=1 << 33, v=1 << 34)
    for name, size in (("q", 4 * 1024 + 1024), ("k", 4 * 256 + 256), ("v", 4 * 256 + 256)):
        for out in (X - 5 * 1024 + 16, X, X + size - 16):
            assert _rope(**{**far, name: X}, out=out) == kvq.KVQ_ERR_INVALID_ARG, (name, out)


@pytest.mark.parametrize("part,kept", [("bias_cu", ("bias_token", "bias")), ("bias_cu", ("bias",)), ("bias_cu", ("bias_token",)), ("mask", ("mask_row",))])
def test_halves_of_a_rule_are_refused(here, part, kept):
    """Tensors of a rule without the one that turns it on: the rule would not be applied, a forgotten bias_cu unban what is banned."""
    good = _args()["kv_logits_probs"][1]["rules"]
    rules = kvq.LogitRules(**{f: None if f[:4] == part[:4] and f not in kept else getattr(good, f) for f in good.__dataclass_fields__})
    assert f"without {part}" in _refusal("kv_logits_probs", rules=rules)
    for f in kept:
        setattr(rules, f, None)
    assert "parent" in _refusal("kv_logits_probs", rules=rules, parent=_i(1))      # (nothing of it: that rule is not applied)
