"""The binding of the drafted-tree and page-pool calls refuses tensors that the kernels would misread or
write past: other types, too few elements, gaps, other devices.  (No GPU: every call here is refused, the
sound ones because their tensors are not on one.)"""

import os

import pytest
import torch

import bit_rotated_kv_gb300 as kvq

B, N, PAGES = 2, 5, 24


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(kvq.LIB_PATH):
        from bit_rotated_kv_gb300 import build_lib
        build_lib.build()


CFG = kvq.KVConfig(n_q_heads=4, n_kv_heads=1, batch=B, max_pages_per_seq=8, num_pages=PAGES, ring_cap=272)


class _Cache:
    pages = torch.zeros((PAGES, 1, 1152), dtype=torch.uint8)

    @staticmethod
    def c():
        return kvq.CCache()


def _i(n):
    return torch.zeros(n, dtype=torch.int32)


def _args():
    q = torch.zeros((N, 4, 128), dtype=torch.bfloat16)
    return {
        "kv_attn_tree": (kvq.kv_attn_tree, dict(cfg=CFG, cache=_Cache, q_rot=q, cu_rows=_i(B + 1), parent=_i(N), out=q.clone(), sm_scale=1.0,
                                                max_ctx=64, workspace=torch.zeros(4096, dtype=torch.uint8), status=_i(1))),
        "kv_verify_tree": (kvq.kv_verify_tree, dict(cfg=CFG, cu_rows=_i(B + 1), parent=_i(N), token=_i(N), p=torch.zeros(N, 9), q=None,
                                                    u=torch.zeros(N), path=_i(N), n_accept=_i(B), next_token=_i(B), status=_i(1))),
        "kv_tree_commit": (kvq.kv_tree_commit, dict(cfg=CFG, cache=_Cache, cu_rows=_i(B + 1), path=_i(N), n_accept=_i(B), status=_i(1))),
        "kv_pages_reserve": (kvq.kv_pages_reserve, dict(cfg=CFG, cache=_Cache, page_ref=_i(PAGES), n_tokens=_i(B), status=_i(1))),
        "kv_seq_fork": (kvq.kv_seq_fork, dict(cfg=CFG, cache=_Cache, page_ref=_i(PAGES), src=_i(1), dst=_i(1), status=_i(1))),
        "kv_seq_free": (kvq.kv_seq_free, dict(cfg=CFG, cache=_Cache, page_ref=_i(PAGES), seqs=_i(2), status=_i(1))),
        "kv_pages_compact": (kvq.kv_pages_compact, dict(cfg=CFG, cache=_Cache, page_ref=_i(PAGES), n_live=_i(1),
                                                        workspace=torch.zeros(4096, dtype=torch.uint8), status=_i(1))),
    }


TENSORS = [(call, name) for call, (_, kw) in _args().items() for name, t in kw.items() if torch.is_tensor(t) and name != "p"]


@pytest.fixture
def here(monkeypatch):
    """The host's tensors pass for those of the current device (every call below is refused for something else)."""
    monkeypatch.setattr(kvq, "_current_device", lambda: -1)


def _refusal(call, **other):
    fn, kw = _args()[call]
    with pytest.raises(kvq.KVQError) as e:
        fn(**{**kw, **other})
    assert e.value.code == kvq.KVQ_ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("call", sorted(_args()))
def test_tensors_off_the_device_are_refused(call):
    assert "device" in _refusal(call)


@pytest.mark.parametrize("call,name", TENSORS)
def test_another_type_is_refused(here, call, name):
    t = _args()[call][1][name]
    if name == "workspace":
        return                                        # (bytes, whatever they are called)
    assert name in _refusal(call, **{name: t.to(torch.int64 if t.dtype == torch.int32 else torch.float64)})


@pytest.mark.parametrize("call,name", [c for c in TENSORS if c[1] not in ("seqs", "src", "dst", "status", "q_rot", "token", "workspace")
                                       and c != ("kv_tree_commit", "path")])
def test_too_few_elements_are_refused(here, call, name):
    t = _args()[call][1][name]
    assert name in _refusal(call, **{name: t.flatten()[:-1].clone()})


@pytest.mark.parametrize("call,name", [c for c in TENSORS if c[1] not in ("status", "n_live", "src", "dst")])
def test_gaps_are_refused(here, call, name):
    t = _args()[call][1][name]
    assert name in _refusal(call, **{name: torch.stack([t, t], -1)[..., 0]})


@pytest.mark.parametrize("call", sorted(_args()))
def test_missing_tensors_are_refused(here, call):
    for c, name in TENSORS:
        if c == call and name not in ("status", "q_rot", "token", "path", "src", "dst", "seqs", "workspace"):
            assert name in _refusal(call, **{name: None})


def test_rows_of_probabilities(here):
    for bad in (None, torch.zeros(N, 9).double(), torch.zeros(N - 1, 9), torch.zeros(9, N).t(), torch.zeros(1, 9).expand(N, 9), torch.zeros(N)):
        assert ": p" in _refusal("kv_verify_tree", p=bad)
    for bad in (torch.zeros(N, 8), torch.zeros(N, 9).half()):
        assert ": q" in _refusal("kv_verify_tree", q=bad)
