"""Python binding of the rotated INT2 paged KV-cache library (libkvq.so, sm_103a).

Argument marshalling only: every step of the hot path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  The shared library is built
in-tree (``bit_rotated_kv_gb300/_build/libkvq.so``, see ``build_lib.py``); importing
this module fails loudly when it is missing -- there is no CPU fallback.

Entry points (same names as the C ABI in include/kvq.h):
  kv_rotate_qk, kv_quant_flush, kv_attn_decode, kv_attn_decode_bf16, kv_attn_workspace_bytes,
  kv_attn_tree, kv_verify_tree, kv_tree_commit (a tree of drafted tokens: attention, check, rows kept),
  kv_pages_reserve, kv_seq_fork, kv_seq_free, kv_pages_compact (the page pool),
  kv_rope_qk, kvq_rope_frequencies (norm, rotary positions, transform and append of a step's rows),
  kv_logits_probs, kv_token_counts (logits to probabilities, and what the penalties go by),
  kvq_page_head_bytes, kvq_page_bytes, kvq_status_string
plus ``KVConfig`` / ``KVCache`` / ``Rope`` helpers that allocate the caller-owned buffers.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = -1
KVQ_ERR_UNSUPPORTED = -2
KVQ_ERR_CUDA = -3
KVQ_ERR_BOUNDS = -4
KVQ_ERR_NONFINITE = -5
KVQ_ERR_TIMEOUT = -6
KVQ_ERR_WORKSPACE = -7

KVQ_QUANT_AFFINE_KAPPA = 0
KVQ_QUANT_QUEST_RMS = 1
KVQ_TRANSFORM_DENSE = 0
KVQ_TRANSFORM_HADAMARD = 1
KVQ_KEY_PER_TOKEN = 0
KVQ_KEY_PER_CHANNEL = 1
KVQ_TREE_MAX_NODES = 128
KVQ_POOL_MAX_SEQS = 16384
KVQ_ROPE_HALF = 0
KVQ_ROPE_INTERLEAVED = 1
KVQ_ROPE_PLAIN = 0
KVQ_ROPE_LINEAR = 1
KVQ_ROPE_NTK = 2
KVQ_ROPE_BANDS = 3
KVQ_ROPE_YARN = 4
KVQ_COUNT_MOST = 32767
KVQ_COUNT_PROMPT = 0
KVQ_COUNT_OUTPUT = 1
KVQ_LOGITS_F32 = 0
KVQ_LOGITS_BF16 = 1
KVQ_LOGITS_F16 = 2
KVQ_LOGITS_MAX_VOCAB = 524288

EXPORTED = ("kv_rotate_qk", "kv_quant_flush", "kv_append_chunk", "kv_attn_chunk", "kv_attn_chunk_workspace_bytes", "kv_attn_decode", "kv_attn_decode_bf16", "kv_attn_decode_noalloc",
            "kv_attn_workspace_bytes",
            "kv_attn_tree", "kv_attn_tree_workspace_bytes", "kv_verify_tree", "kv_tree_commit",
            "kv_pages_reserve", "kv_seq_fork", "kv_seq_free", "kv_pages_compact", "kv_pages_compact_workspace_bytes",
            "kv_rope_qk", "kvq_rope_frequencies", "kv_logits_probs", "kv_token_counts",
            "kvq_page_head_bytes", "kvq_page_bytes", "kvq_status_string", "kvq_version",
            "kvq_selftest_scale_division", "kvq_selftest_tc_integer_sums")


class CConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "head_dim", "n_q_heads", "n_kv_heads", "page_size", "group_size", "quantizer", "key_l2norm",
        "s_sink", "s_keep", "s_flush", "ring_cap", "batch", "max_pages_per_seq", "num_pages",
        "attn_splits", "key_axis")] + [("kappa_k", ctypes.c_double), ("kappa_v", ctypes.c_double),
                                       ("quest_alpha", ctypes.c_double)]


class CCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "pages", "page_table", "seq_len", "s_quant", "sink_k", "sink_v", "ring_k", "ring_v", "counters")]


class CTransform(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("t_k", ctypes.c_void_p),
                ("t_k_inv_t", ctypes.c_void_p), ("t_v", ctypes.c_void_p)]


class CRope(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("scale", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("freq", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p)]


class CLogitRules(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("counts", ctypes.c_void_p), ("count_stride", ctypes.c_int64),
                ("bias_cu", ctypes.c_void_p), ("bias_token", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_int64), ("mask_row", ctypes.c_void_p), ("n_bias", ctypes.c_int32),
                ("n_masks", ctypes.c_int32)]


class KVQError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {kvq_status_string(code)} ({code})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        l = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER
        l.kv_rotate_qk.argtypes = [P(CConfig), P(CTransform), vp, vp, i32, vp, vp, vp, vp, i32, P(CCache), vp, vp]
        l.kv_rotate_qk.restype = ctypes.c_int
        l.kv_quant_flush.argtypes = [P(CConfig), P(CCache), i32, vp, vp]
        l.kv_append_chunk.restype = ctypes.c_int
        l.kv_attn_chunk.argtypes = [P(CConfig), P(CCache), vp, vp, i32, vp, ctypes.c_float, i32, vp, sz, vp, vp]
        l.kv_attn_chunk.restype = ctypes.c_int
        l.kv_attn_chunk_workspace_bytes.argtypes = [P(CConfig), i32, i32]
        l.kv_attn_chunk_workspace_bytes.restype = sz
        l.kv_append_chunk.argtypes = [P(CConfig), P(CTransform), vp, vp, vp, i32, P(CCache), vp, vp]
        l.kv_quant_flush.restype = ctypes.c_int
        i64 = ctypes.c_int64
        l.kv_attn_tree.argtypes = [P(CConfig), P(CCache), vp, vp, vp, i32, vp, ctypes.c_float, i32, vp, sz, vp, vp]
        l.kv_attn_tree.restype = ctypes.c_int
        l.kv_attn_tree_workspace_bytes.argtypes = [P(CConfig), i32, i32]
        l.kv_attn_tree_workspace_bytes.restype = sz
        l.kv_verify_tree.argtypes = [P(CConfig), vp, vp, vp, i32, vp, i64, vp, i64, i32, vp, vp, vp, vp, vp, vp]
        l.kv_verify_tree.restype = ctypes.c_int
        l.kv_tree_commit.argtypes = [P(CConfig), P(CCache), vp, i32, vp, vp, vp, vp]
        l.kv_tree_commit.restype = ctypes.c_int
        l.kv_pages_reserve.argtypes = [P(CConfig), P(CCache), vp, vp, vp, vp]
        l.kv_pages_reserve.restype = ctypes.c_int
        l.kv_seq_fork.argtypes = [P(CConfig), P(CCache), vp, vp, vp, i32, vp, vp]
        l.kv_seq_fork.restype = ctypes.c_int
        l.kv_seq_free.argtypes = [P(CConfig), P(CCache), vp, vp, i32, vp, vp]
        l.kv_seq_free.restype = ctypes.c_int
        l.kv_pages_compact.argtypes = [P(CConfig), P(CCache), vp, vp, vp, sz, vp, vp]
        l.kv_pages_compact.restype = ctypes.c_int
        l.kv_pages_compact_workspace_bytes.argtypes = [P(CConfig)]
        l.kv_pages_compact_workspace_bytes.restype = sz
        dbl = ctypes.c_double
        l.kvq_rope_frequencies.argtypes = [i32, dbl, i32, dbl, dbl, dbl, dbl, vp, vp]
        l.kvq_rope_frequencies.restype = ctypes.c_int
        l.kv_rope_qk.argtypes = [P(CConfig), P(CTransform), P(CRope), vp, i64, vp, vp, i32, vp, i64, vp, i64, vp, vp, vp, i32,
                                 P(CCache), vp, vp]
        l.kv_rope_qk.restype = ctypes.c_int
        l.kv_logits_probs.argtypes = [P(CConfig), P(CLogitRules), vp, i32, i64, i32, vp, vp, vp, i32, vp, i64, vp, vp]
        l.kv_logits_probs.restype = ctypes.c_int
        l.kv_token_counts.argtypes = [P(CConfig), vp, i64, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp]
        l.kv_token_counts.restype = ctypes.c_int
        l.kv_attn_decode.argtypes = [P(CConfig), P(CCache), vp, vp, ctypes.c_float, i32, vp, sz, vp, vp]
        l.kv_attn_decode.restype = ctypes.c_int
        l.kv_attn_decode_bf16.argtypes = [P(CConfig), P(CCache), vp, vp, ctypes.c_float, i32, vp, sz, vp, vp]
        l.kv_attn_decode_bf16.restype = ctypes.c_int
        l.kv_attn_decode_noalloc.argtypes = [P(CConfig), P(CCache), vp, vp, ctypes.c_float, i32, vp, vp]
        l.kv_attn_decode_noalloc.restype = ctypes.c_int
        l.kv_attn_workspace_bytes.argtypes = [P(CConfig), i32]
        l.kv_attn_workspace_bytes.restype = sz
        l.kvq_page_head_bytes.argtypes = [P(CConfig)]
        l.kvq_page_head_bytes.restype = sz
        l.kvq_page_bytes.argtypes = [P(CConfig)]
        l.kvq_page_bytes.restype = sz
        l.kvq_status_string.argtypes = [ctypes.c_int]
        l.kvq_status_string.restype = ctypes.c_char_p
        l.kvq_version.argtypes = []
        l.kvq_version.restype = ctypes.c_int
        l.kvq_selftest_scale_division.argtypes = [vp, vp]
        l.kvq_selftest_scale_division.restype = ctypes.c_int
        l.kvq_selftest_tc_integer_sums.argtypes = [vp, vp]
        l.kvq_selftest_tc_integer_sums.restype = ctypes.c_int
        _lib = l
    return _lib


def kvq_status_string(code: int) -> str:
    return lib().kvq_status_string(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != KVQ_OK:
        raise KVQError(rc, where)


@dataclass
class KVConfig:
    """Python mirror of kvq_config (see include/kvq.h for every field)."""
    n_q_heads: int
    n_kv_heads: int
    batch: int
    max_pages_per_seq: int
    num_pages: int
    ring_cap: int
    head_dim: int = 128
    page_size: int = 16
    group_size: int = 128
    quantizer: int = KVQ_QUANT_AFFINE_KAPPA
    key_l2norm: bool = False
    s_sink: int = 64
    s_keep: int = 256
    s_flush: int = 8
    attn_splits: int = 0
    kappa_k: float = 0.99
    kappa_v: float = 0.99
    quest_alpha: float = 1.4935705
    key_axis: int = 0                    # KVQ_KEY_PER_TOKEN / KVQ_KEY_PER_CHANNEL

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cc":                    # any change rebuilds the C struct on next use
            object.__setattr__(self, "_cc", None)

    def c(self) -> CConfig:
        """The C struct (built once, rebuilt only after a field changes)."""
        cc = self.__dict__.get("_cc")
        if cc is None:
            cc = CConfig(self.head_dim, self.n_q_heads, self.n_kv_heads, self.page_size, self.group_size,
                         self.quantizer, int(bool(self.key_l2norm)), self.s_sink, self.s_keep, self.s_flush,
                         self.ring_cap, self.batch, self.max_pages_per_seq, self.num_pages, self.attn_splits,
                         int(self.key_axis), float(self.kappa_k), float(self.kappa_v), float(self.quest_alpha))
            object.__setattr__(self, "_cc", cc)
        return cc

    @property
    def gqa(self) -> int:
        return self.n_q_heads // self.n_kv_heads


def kvq_page_head_bytes(cfg: KVConfig) -> int:
    c = cfg.c()
    return int(lib().kvq_page_head_bytes(ctypes.byref(c)))


def kvq_page_bytes(cfg: KVConfig) -> int:
    c = cfg.c()
    return int(lib().kvq_page_bytes(ctypes.byref(c)))


def kv_attn_workspace_bytes(cfg: KVConfig, max_ctx: int) -> int:
    c = cfg.c()
    return int(lib().kv_attn_workspace_bytes(ctypes.byref(c), int(max_ctx)))


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        # (the raw handle: torch.cuda.current_stream() makes an object of it, ten times as slow)
        return int(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return int(getattr(stream, "cuda_stream", stream))


class KVCache:
    """Caller-owned device buffers of one cache (all zero-initialised; s_quant = s_sink)."""

    def __init__(self, cfg: KVConfig, device="cuda"):
        self.cfg = cfg
        dev = torch.device(device)
        B, H, d = cfg.batch, cfg.n_kv_heads, cfg.head_dim
        phb = kvq_page_head_bytes(cfg)
        if phb == 0:
            raise KVQError(KVQ_ERR_UNSUPPORTED, "KVCache")
        self.page_head_bytes = phb
        self.pages = torch.zeros((cfg.num_pages, H, phb), dtype=torch.uint8, device=dev)
        self.page_table = torch.full((B, cfg.max_pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.seq_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.s_quant = torch.full((B,), cfg.s_sink, dtype=torch.int32, device=dev)
        ns = max(cfg.s_sink, 1)
        self.sink_k = torch.zeros((B, H, ns, d), dtype=torch.bfloat16, device=dev)
        self.sink_v = torch.zeros((B, H, ns, d), dtype=torch.bfloat16, device=dev)
        self.ring_k = torch.zeros((B, H, cfg.ring_cap, d), dtype=torch.bfloat16, device=dev)
        self.ring_v = torch.zeros((B, H, cfg.ring_cap, d), dtype=torch.bfloat16, device=dev)
        self.counters = torch.zeros(B, dtype=torch.int32, device=dev)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cc":                    # a replaced buffer rebuilds the C struct on next use
            object.__setattr__(self, "_cc", None)

    def c(self) -> CCache:
        """The C struct of device pointers (built once, rebuilt only after a buffer is replaced)."""
        cc = self.__dict__.get("_cc")
        if cc is None:
            cc = CCache(_ptr(self.pages), _ptr(self.page_table), _ptr(self.seq_len), _ptr(self.s_quant),
                        _ptr(self.sink_k), _ptr(self.sink_v), _ptr(self.ring_k), _ptr(self.ring_v),
                        _ptr(self.counters))
            object.__setattr__(self, "_cc", cc)
        return cc


@dataclass
class Transform:
    """Per-head transforms as device float32 tensors [Hkv, d, d] (or Hadamard)."""
    kind: int = KVQ_TRANSFORM_DENSE
    t_k: torch.Tensor | None = None
    t_k_inv_t: torch.Tensor | None = None
    t_v: torch.Tensor | None = None

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cc":
            object.__setattr__(self, "_cc", None)

    def c(self) -> CTransform:
        """The C struct (built once, rebuilt only after a field changes)."""
        cc = self.__dict__.get("_cc")
        if cc is None:
            cc = CTransform(self.kind, 0, _ptr(self.t_k), _ptr(self.t_k_inv_t), _ptr(self.t_v))
            object.__setattr__(self, "_cc", cc)
        return cc


def kv_rotate_qk(cfg: KVConfig, tr: Transform, q, q_out, k, v, seq_idx, pos, cache: KVCache,
                 status, stream=None) -> None:
    """q [n, Hq, d] -> q_out; k, v [m, Hkv, d] into the cache at (seq_idx[r], pos[r])."""
    c, t = cfg.c(), tr.c()
    n_q = 0 if q is None else int(q.shape[0])
    n_kv = 0 if k is None else int(k.shape[0])
    cc = cache.c()
    rc = lib().kv_rotate_qk(ctypes.byref(c), ctypes.byref(t), _ptr(q), _ptr(q_out), n_q, _ptr(k), _ptr(v),
                            _ptr(seq_idx), _ptr(pos), n_kv, ctypes.byref(cc), _ptr(status), _stream(stream))
    _check(rc, "kv_rotate_qk")


def kv_append_chunk(cfg: KVConfig, tr: Transform, k, v, cu_rows, cache: KVCache, status, stream=None) -> None:
    """k, v [n, Hkv, d]: rows cu_rows[b] .. cu_rows[b+1]-1 appended to sequence b, transformed
    and quantized on write in one pass (the effect of kv_rotate_qk + kv_quant_flush)."""
    c, t = cfg.c(), tr.c()
    n = 0 if k is None else int(k.shape[0])
    cc = cache.c()
    rc = lib().kv_append_chunk(ctypes.byref(c), ctypes.byref(t), _ptr(k), _ptr(v), _ptr(cu_rows), n,
                               ctypes.byref(cc), _ptr(status), _stream(stream))
    _check(rc, "kv_append_chunk")


def kv_attn_chunk_workspace_bytes(cfg: KVConfig, n_rows: int, max_ctx: int) -> int:
    return int(lib().kv_attn_chunk_workspace_bytes(ctypes.byref(cfg.c()), int(n_rows), int(max_ctx)))


def kv_attn_chunk(cfg: KVConfig, cache: KVCache, q_rot, cu_rows, out, sm_scale: float, max_ctx: int, workspace,
                  status, stream=None) -> None:
    """q_rot [n, Hq, d] (rows cu_rows[b] .. cu_rows[b+1]-1 the last tokens of sequence b) ->
    out [n, Hq, d] float32: causal attention over the cache after the append."""
    n = int(q_rot.shape[0])
    c, cc = cfg.c(), cache.c()
    rc = lib().kv_attn_chunk(ctypes.byref(c), ctypes.byref(cc), _ptr(q_rot), _ptr(cu_rows), n, _ptr(out),
                             float(sm_scale), int(max_ctx), _ptr(workspace), int(workspace.numel()), _ptr(status),
                             _stream(stream))
    _check(rc, "kv_attn_chunk")


def kv_quant_flush(cfg: KVConfig, cache: KVCache, max_tokens_per_seq: int, status, stream=None) -> None:
    c, cc = cfg.c(), cache.c()
    rc = lib().kv_quant_flush(ctypes.byref(c), ctypes.byref(cc), int(max_tokens_per_seq), _ptr(status),
                              _stream(stream))
    _check(rc, "kv_quant_flush")


def kv_attn_decode(cfg: KVConfig, cache: KVCache, q_rot, out, sm_scale: float, max_ctx: int, workspace,
                   status, stream=None) -> None:
    c, cc = cfg.c(), cache.c()
    nbytes = int(workspace.numel() * workspace.element_size())
    rc = lib().kv_attn_decode(ctypes.byref(c), ctypes.byref(cc), _ptr(q_rot), _ptr(out), float(sm_scale),
                              int(max_ctx), _ptr(workspace), nbytes, _ptr(status), _stream(stream))
    _check(rc, "kv_attn_decode")


def kv_attn_decode_bf16(cfg: KVConfig, cache: KVCache, q_rot, out, sm_scale: float, max_ctx: int, workspace,
                        status, stream=None) -> None:
    """kv_attn_decode with a bf16 output tensor [B, Hq, d] (the float32 result rounded once)."""
    c, cc = cfg.c(), cache.c()
    nbytes = int(workspace.numel() * workspace.element_size())
    rc = lib().kv_attn_decode_bf16(ctypes.byref(c), ctypes.byref(cc), _ptr(q_rot), _ptr(out), float(sm_scale),
                                   int(max_ctx), _ptr(workspace), nbytes, _ptr(status), _stream(stream))
    _check(rc, "kv_attn_decode_bf16")


NOALLOC_WORKSPACE_BYTES = 8 << 20


def kv_attn_decode_noalloc(cfg: KVConfig, cache: KVCache, q_rot, out, sm_scale: float, max_ctx: int, status,
                           stream=None) -> None:
    """kv_attn_decode with the library's fixed internal scratch (no workspace argument)."""
    c, cc = cfg.c(), cache.c()
    rc = lib().kv_attn_decode_noalloc(ctypes.byref(c), ctypes.byref(cc), _ptr(q_rot), _ptr(out), float(sm_scale),
                                      int(max_ctx), _ptr(status), _stream(stream))
    _check(rc, "kv_attn_decode_noalloc")


def _current_device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _addr(dev: int, t, dtype, least: int, what: str) -> int:
    """Address of a tensor of this type with at least so many elements, one after another, on the current device.
    Anything else is refused: the kernels take addresses, and would read other numbers or write past the end.
    None stands for no elements."""
    if t is None:
        if least > 0:
            raise KVQError(KVQ_ERR_INVALID_ARG, what)
        return 0
    if t.dtype is not dtype or t.numel() < least or not t.is_contiguous():
        raise KVQError(KVQ_ERR_INVALID_ARG, what)
    if t.get_device() != dev:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{what} (another device)")
    return t.data_ptr()


def _status(dev: int, status, where: str) -> int:
    return 0 if status is None else _addr(dev, status, torch.int32, 1, f"{where}: status")


def _cache(dev: int, cache: KVCache, where: str):
    if cache.pages.get_device() != dev:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{where}: cache (another device)")
    return ctypes.byref(cache.c())


def _stream_of(dev: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(getattr(stream, "cuda_stream", stream))


def _nbytes(t) -> int:
    return int(t.numel() * t.element_size())


def kv_attn_tree_workspace_bytes(cfg: KVConfig, n_rows: int, max_ctx: int) -> int:
    return int(lib().kv_attn_tree_workspace_bytes(ctypes.byref(cfg.c()), int(n_rows), int(max_ctx)))


def kv_attn_tree(cfg: KVConfig, cache: KVCache, q_rot, cu_rows, parent, out, sm_scale: float, max_ctx: int,
                 workspace, status, stream=None) -> None:
    """q_rot [n, Hq, d] (rows cu_rows[b] .. cu_rows[b+1]-1 the drafted nodes of sequence b, its last
    tokens; parent [n] int32 local to the sequence, -1 for a root) -> out [n, Hq, d] bf16: every node
    attends to the tokens before the drafts, its ancestors and itself."""
    n, dev, i32, bf16 = q_rot.shape[0], _current_device(), torch.int32, torch.bfloat16
    size = n * cfg.n_q_heads * cfg.head_dim
    q = _addr(dev, q_rot, bf16, size, "kv_attn_tree: q_rot")
    cu = _addr(dev, cu_rows, i32, cfg.batch + 1, "kv_attn_tree: cu_rows")
    par = _addr(dev, parent, i32, n, "kv_attn_tree: parent")
    o = _addr(dev, out, bf16, size, "kv_attn_tree: out")
    ws = _addr(dev, workspace, workspace.dtype, 0, "kv_attn_tree: workspace")
    rc = lib().kv_attn_tree(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_attn_tree"), q, cu, par, n, o, float(sm_scale),
                            int(max_ctx), ws, _nbytes(workspace), _status(dev, status, "kv_attn_tree"), _stream_of(dev, stream))
    _check(rc, "kv_attn_tree")


def _prob_rows(dev: int, t, n: int, vocab: int, what: str):
    """Address and row stride of n rows of float32 probabilities, each row's one after another."""
    if t is None:
        return 0, 0
    if (t.dim() != 2 or t.dtype is not torch.float32 or t.shape[0] != n or t.shape[1] != vocab or (vocab > 1 and t.stride(1) != 1)
            or (n > 1 and t.stride(0) < vocab)):
        raise KVQError(KVQ_ERR_INVALID_ARG, what)
    if t.get_device() != dev:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{what} (another device)")
    return t.data_ptr(), max(t.stride(0), vocab)


def kv_verify_tree(cfg: KVConfig, cu_rows, parent, token, p, q, u, path, n_accept, next_token, status,
                   stream=None) -> None:
    """p (and q, or None for chosen drafts) [n, vocab] float32 with contiguous rows; token, parent, path [n]
    int32; u [n] float32; n_accept, next_token [batch] int32."""
    n, dev, i32, batch = token.shape[0], _current_device(), torch.int32, cfg.batch
    if p is None:
        raise KVQError(KVQ_ERR_INVALID_ARG, "kv_verify_tree: p")
    vocab = p.shape[-1]
    pa, ps = _prob_rows(dev, p, n, vocab, "kv_verify_tree: p")
    qa, qs = _prob_rows(dev, q, n, vocab, "kv_verify_tree: q")
    cu = _addr(dev, cu_rows, i32, batch + 1, "kv_verify_tree: cu_rows")
    par = _addr(dev, parent, i32, n, "kv_verify_tree: parent")
    tok = _addr(dev, token, i32, n, "kv_verify_tree: token")
    uu = _addr(dev, u, torch.float32, n, "kv_verify_tree: u")
    out = _addr(dev, path, i32, n, "kv_verify_tree: path")
    acc = _addr(dev, n_accept, i32, batch, "kv_verify_tree: n_accept")
    nxt = _addr(dev, next_token, i32, batch, "kv_verify_tree: next_token")
    rc = lib().kv_verify_tree(ctypes.byref(cfg.c()), cu, par, tok, n, pa, ps, qa, qs, vocab, uu, out, acc, nxt,
                              _status(dev, status, "kv_verify_tree"), _stream_of(dev, stream))
    _check(rc, "kv_verify_tree")


def kv_tree_commit(cfg: KVConfig, cache: KVCache, cu_rows, path, n_accept, status, stream=None) -> None:
    """Keep the rows of the accepted paths (kv_verify_tree's path and n_accept); seq_len drops the others."""
    dev, i32 = _current_device(), torch.int32
    cu = _addr(dev, cu_rows, i32, cfg.batch + 1, "kv_tree_commit: cu_rows")
    at = _addr(dev, path, i32, 0, "kv_tree_commit: path")
    acc = _addr(dev, n_accept, i32, cfg.batch, "kv_tree_commit: n_accept")
    rc = lib().kv_tree_commit(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_tree_commit"), cu, path.numel(), at, acc,
                              _status(dev, status, "kv_tree_commit"), _stream_of(dev, stream))
    _check(rc, "kv_tree_commit")


def kv_pages_reserve(cfg: KVConfig, cache: KVCache, page_ref, n_tokens, status, stream=None) -> None:
    """Pages for n_tokens[b] (int32 [batch]) more tokens of every sequence, lowest free ids first."""
    dev, i32 = _current_device(), torch.int32
    ref = _addr(dev, page_ref, i32, cfg.num_pages, "kv_pages_reserve: page_ref")
    tokens = _addr(dev, n_tokens, i32, cfg.batch, "kv_pages_reserve: n_tokens")
    rc = lib().kv_pages_reserve(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_pages_reserve"), ref, tokens,
                                _status(dev, status, "kv_pages_reserve"), _stream_of(dev, stream))
    _check(rc, "kv_pages_reserve")


def kv_seq_fork(cfg: KVConfig, cache: KVCache, page_ref, src, dst, status, stream=None) -> None:
    """Sequence dst[i] becomes a copy of sequence src[i] (int32 [n] each), sharing its whole INT2 pages."""
    dev, i32 = _current_device(), torch.int32
    n = src.numel()
    ref = _addr(dev, page_ref, i32, cfg.num_pages, "kv_seq_fork: page_ref")
    a = _addr(dev, src, i32, 0, "kv_seq_fork: src")
    b = _addr(dev, dst, i32, 0, "kv_seq_fork: dst")
    if dst.numel() != n:
        raise KVQError(KVQ_ERR_INVALID_ARG, "kv_seq_fork: src and dst")
    rc = lib().kv_seq_fork(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_seq_fork"), ref, a, b, n,
                           _status(dev, status, "kv_seq_fork"), _stream_of(dev, stream))
    _check(rc, "kv_seq_fork")


def kv_seq_free(cfg: KVConfig, cache: KVCache, page_ref, seqs, status, stream=None) -> None:
    """Sequences seqs (int32 [n]) give up their pages and become empty."""
    dev, i32 = _current_device(), torch.int32
    ref = _addr(dev, page_ref, i32, cfg.num_pages, "kv_seq_free: page_ref")
    at = _addr(dev, seqs, i32, 0, "kv_seq_free: seqs")
    rc = lib().kv_seq_free(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_seq_free"), ref, at, seqs.numel(),
                           _status(dev, status, "kv_seq_free"), _stream_of(dev, stream))
    _check(rc, "kv_seq_free")


def kv_pages_compact_workspace_bytes(cfg: KVConfig) -> int:
    return int(lib().kv_pages_compact_workspace_bytes(ctypes.byref(cfg.c())))


def kv_pages_compact(cfg: KVConfig, cache: KVCache, page_ref, n_live, workspace, status, stream=None) -> None:
    """Held pages move to ids 0 .. n_live - 1 (n_live int32 [1], out) and the tables follow them."""
    dev, i32 = _current_device(), torch.int32
    ref = _addr(dev, page_ref, i32, cfg.num_pages, "kv_pages_compact: page_ref")
    live = _addr(dev, n_live, i32, 1, "kv_pages_compact: n_live")
    ws = _addr(dev, workspace, workspace.dtype, 0, "kv_pages_compact: workspace")
    rc = lib().kv_pages_compact(ctypes.byref(cfg.c()), _cache(dev, cache, "kv_pages_compact"), ref, live, ws, _nbytes(workspace),
                                _status(dev, status, "kv_pages_compact"), _stream_of(dev, stream))
    _check(rc, "kv_pages_compact")


def kvq_rope_frequencies(rot_dim: int, theta: float, scaling: int = KVQ_ROPE_PLAIN, factor: float = 1.0, context: float = 0.0,
                         a: float = 0.0, b: float = 0.0):
    """(freq, scale): turns per token of every pair in units of 2^-64, as an int64 host tensor of the same bits,
    and the factor of the rotated channels."""
    freq = torch.zeros(max(0, int(rot_dim) // 2), dtype=torch.int64)
    scale = ctypes.c_float(1.0)
    rc = lib().kvq_rope_frequencies(int(rot_dim), float(theta), int(scaling), float(factor), float(context), float(a), float(b),
                                    freq.data_ptr() if len(freq) else None, ctypes.byref(scale))
    _check(rc, "kvq_rope_frequencies")
    return freq, float(scale.value)


@dataclass
class Rope:
    """Rotary positions and the norms of query and key heads (see kvq_rope in include/kvq.h)."""
    layout: int
    rot_dim: int
    freq: torch.Tensor | None            # [rot_dim / 2] int64 (the bits of uint64) on the device
    scale: float = 1.0
    q_norm: torch.Tensor | None = None   # [d] float32 on the device
    k_norm: torch.Tensor | None = None
    norm_eps: float = 1e-6

    @classmethod
    def make(cls, layout: int, rot_dim: int, theta: float, scaling: int = KVQ_ROPE_PLAIN, factor: float = 1.0, context: float = 0.0,
             a: float = 0.0, b: float = 0.0, q_norm=None, k_norm=None, norm_eps: float = 1e-6, device="cuda") -> "Rope":
        """With the frequencies of kvq_rope_frequencies."""
        freq, scale = kvq_rope_frequencies(rot_dim, theta, scaling, factor, context, a, b)
        return cls(layout, int(rot_dim), freq.to(device), scale, q_norm, k_norm, norm_eps)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cc":
            object.__setattr__(self, "_cc", None)

    def c(self, dev: int) -> CRope:
        """The C struct (built once for a device, again after a field changes)."""
        cc = self.__dict__.get("_cc")
        if cc is None or cc[0] != dev:
            f32 = torch.float32
            norm = [0 if w is None else _addr(dev, w, f32, 128, f"kv_rope_qk: {n}") for n, w in (("q_norm", self.q_norm), ("k_norm", self.k_norm))]
            cc = (dev, CRope(int(self.layout), int(self.rot_dim), float(self.scale), float(self.norm_eps),
                             _addr(dev, self.freq, torch.int64, max(0, int(self.rot_dim) // 2), "kv_rope_qk: freq"), *norm))
            object.__setattr__(self, "_cc", cc)
        return cc[1]


def _head_rows(dev: int, t, n: int, heads: int, what: str):
    """Address and row stride of [n, heads, 128] bf16, each row's heads one after another."""
    if t is None:
        if n > 0:
            raise KVQError(KVQ_ERR_INVALID_ARG, what)
        return 0, heads * 128
    if t.dtype is not torch.bfloat16 or t.shape != (n, heads, 128):
        raise KVQError(KVQ_ERR_INVALID_ARG, what)
    row, head, channel = t.stride()
    if channel != 1 or (heads > 1 and head != 128) or (n > 1 and row < heads * 128):
        raise KVQError(KVQ_ERR_INVALID_ARG, what)
    if t.get_device() != dev:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{what} (another device)")
    return t.data_ptr(), row if n > 1 else heads * 128


def _transform(dev: int, tr: Transform, cfg: KVConfig):
    """The C struct of a transform whose matrices have been looked at (once for a device and a number of heads, again after a
    field changes)."""
    cc, key = tr.c(), (dev, cfg.n_kv_heads)
    seen = tr.__dict__.get("_seen")
    if seen is None or seen[0] is not cc or seen[1] != key:
        for name in ("t_k", "t_k_inv_t", "t_v"):
            t = getattr(tr, name)
            if t is not None:
                _addr(dev, t, torch.float32, cfg.n_kv_heads * 128 * 128, f"kv_rope_qk: {name}")
        seen = (cc, key, ctypes.byref(cc))
        object.__setattr__(tr, "_seen", seen)
    return seen[2]


def kv_rope_qk(cfg: KVConfig, tr: Transform, rope: Rope | None, q, q_out, q_pos, k, v, seq_idx, pos, rope_pos, cache: KVCache,
               status, stream=None) -> None:
    """q [n, Hq, d] -> q_out (contiguous); k, v [m, Hkv, d] into the cache at (seq_idx[r], pos[r]): norm of the heads, rotation
    by q_pos [n] and rope_pos [m] (None: pos), transform.  q, k, v may be views of one fused projection [n, Hq + 2 Hkv, d]."""
    dev, i32 = _current_device(), torch.int32
    n_q = 0 if q is None else q.shape[0]
    n_kv = 0 if k is None else k.shape[0]
    hq, hkv = cfg.n_q_heads, cfg.n_kv_heads
    qa, qs = _head_rows(dev, q, n_q, hq, "kv_rope_qk: q")
    ka, ks = _head_rows(dev, k, n_kv, hkv, "kv_rope_qk: k")
    va, vs = _head_rows(dev, v, n_kv, hkv, "kv_rope_qk: v")
    out = _addr(dev, q_out, torch.bfloat16, n_q * hq * 128, "kv_rope_qk: q_out")
    qp = _addr(dev, q_pos, i32, n_q, "kv_rope_qk: q_pos") if q_pos is not None or (rope is not None and rope.rot_dim > 0) else 0
    seq = _addr(dev, seq_idx, i32, n_kv, "kv_rope_qk: seq_idx")
    at = _addr(dev, pos, i32, n_kv, "kv_rope_qk: pos")
    far = 0 if rope_pos is None else _addr(dev, rope_pos, i32, n_kv, "kv_rope_qk: rope_pos")
    rc = lib().kv_rope_qk(cfg.c(), _transform(dev, tr, cfg), None if rope is None else rope.c(dev), qa, qs, out, qp, n_q, ka, ks, va, vs,
                          seq, at, far, n_kv, _cache(dev, cache, "kv_rope_qk"), _status(dev, status, "kv_rope_qk"), _stream_of(dev, stream))
    if rc:
        _check(rc, "kv_rope_qk")


@dataclass
class LogitRules:
    """What kv_logits_probs applies (see kvq_logit_rules in include/kvq.h); None: not that rule.  Biases need bias_cu, a mask_row
    its mask: the other tensors without them are refused."""
    temperature: torch.Tensor | None = None   # [batch] float32; so the next three
    repetition: torch.Tensor | None = None
    frequency: torch.Tensor | None = None
    presence: torch.Tensor | None = None
    counts: torch.Tensor | None = None        # [batch, >= vocab] int16 (the bits of uint16), as kv_token_counts keeps it
    bias_cu: torch.Tensor | None = None       # [batch + 1] int32
    bias_token: torch.Tensor | None = None    # [n] int32
    bias: torch.Tensor | None = None          # [n] float32
    mask: torch.Tensor | None = None          # [masks, >= vocab / 32] int32
    mask_row: torch.Tensor | None = None      # [rows] int32

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_cc":
            object.__setattr__(self, "_cc", None)

    def c(self, dev: int, batch: int, rows: int, vocab: int) -> CLogitRules:
        """The C struct (built once for these sizes, again after a field changes)."""
        key = (dev, batch, rows, vocab)
        cc = self.__dict__.get("_cc")
        if cc is None or cc[0] != key:
            w, i32, f32 = "kv_logits_probs", torch.int32, torch.float32
            for part, rest in (("bias_cu", ("bias_token", "bias")), ("mask", ("mask_row",))):
                for n in rest:                             # (a rule that its other half is missing for would not be applied)
                    if getattr(self, part) is None and getattr(self, n) is not None:
                        raise KVQError(KVQ_ERR_INVALID_ARG, f"{w}: {n} without {part}")
            per_seq = [0 if t is None else _addr(dev, t, f32, batch, f"{w}: {n}")
                       for n, t in (("temperature", self.temperature), ("repetition", self.repetition), ("frequency", self.frequency),
                                    ("presence", self.presence))]
            counts, stride = (0, 0) if self.counts is None else _count_rows(dev, self.counts, batch, vocab, w)
            n_bias = 0 if self.bias_token is None else self.bias_token.numel()
            biases = [0, 0, 0]
            if self.bias_cu is not None:
                biases = [_addr(dev, self.bias_cu, i32, batch + 1, f"{w}: bias_cu"), _addr(dev, self.bias_token, i32, 0, f"{w}: bias_token"),
                          _addr(dev, self.bias, f32, n_bias, f"{w}: bias")]
            mask, mask_stride, masks, mask_row = 0, 0, 0, 0
            if self.mask is not None:
                m = self.mask
                if m.dim() != 2 or m.dtype is not i32 or m.shape[1] < (vocab + 31) // 32 or not m.is_contiguous():
                    raise KVQError(KVQ_ERR_INVALID_ARG, f"{w}: mask")
                mask, mask_stride, masks = _addr(dev, m, i32, 0, f"{w}: mask"), m.shape[1], m.shape[0]
                mask_row = 0 if self.mask_row is None else _addr(dev, self.mask_row, i32, rows, f"{w}: mask_row")
            cc = (key, CLogitRules(*per_seq, counts, stride, *biases, mask, mask_stride, mask_row, n_bias, masks))
            object.__setattr__(self, "_cc", cc)
        return cc[1]


def _count_rows(dev: int, t, batch: int, vocab: int, where: str):
    """Address and row stride of [batch, >= vocab] counts."""
    if t is None or t.dim() != 2:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{where}: counts")
    n, width = t.shape
    if n != batch or width < vocab or width % 2:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{where}: counts")
    return _addr(dev, t, torch.int16, 0, f"{where}: counts"), width


_LOGIT_TYPES = {torch.float32: KVQ_LOGITS_F32, torch.bfloat16: KVQ_LOGITS_BF16, torch.float16: KVQ_LOGITS_F16}


def kv_logits_probs(cfg: KVConfig, rules: LogitRules | None, logits, cu_rows, parent, token, p, status, stream=None) -> None:
    """logits [n, vocab] (float32, bfloat16 or float16; rows contiguous) -> p [n, vocab] float32 (for float32 logits it may be
    the same tensor): rows cu_rows[b] .. cu_rows[b+1]-1 are sequence b's.  parent, token [n] int32: a tree of drafts, or None."""
    dev, i32, w = _current_device(), torch.int32, "kv_logits_probs"
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None or logits.dim() != 2 or p is None or p.dtype is not torch.float32 or p.shape != logits.shape:
        raise KVQError(KVQ_ERR_INVALID_ARG, f"{w}: p" if kind is not None and logits.dim() == 2 else f"{w}: logits")
    n, vocab = logits.shape
    rows = []
    for t, name in ((logits, "logits"), (p, "p")):
        row, token_step = t.stride()
        if (vocab > 1 and token_step != 1) or (n > 1 and row < vocab):
            raise KVQError(KVQ_ERR_INVALID_ARG, f"{w}: {name}")
        if t.get_device() != dev:
            raise KVQError(KVQ_ERR_INVALID_ARG, f"{w}: {name} (another device)")
        rows += t.data_ptr(), row if n > 1 else vocab
    cu = _addr(dev, cu_rows, i32, cfg.batch + 1, "kv_logits_probs: cu_rows")
    par = 0 if parent is None else _addr(dev, parent, i32, n, "kv_logits_probs: parent")
    tok = 0 if token is None else _addr(dev, token, i32, n, "kv_logits_probs: token")
    rc = lib().kv_logits_probs(cfg.c(), None if rules is None else rules.c(dev, cfg.batch, n, vocab), rows[0], kind, rows[1], vocab, cu, par,
                               tok, n, rows[2], rows[3], _status(dev, status, w), _stream_of(dev, stream))
    if rc:
        _check(rc, w)


def kv_token_counts(cfg: KVConfig, counts, vocab: int, kind: int, cu_rows, token, path, n_accept, next_token, status,
                    stream=None) -> None:
    """counts [batch, >= vocab, even] int16 (the bits of uint16; zero for a new sequence): rows cu_rows[b] .. cu_rows[b+1]-1 of
    token [n] marked as sequence b's prompt or counted as generated; with path [n] and n_accept [batch] the kept nodes' only, and
    with next_token [batch] the token behind them."""
    dev, i32, w = _current_device(), torch.int32, "kv_token_counts"
    n = 0 if token is None else token.numel()
    at, stride = _count_rows(dev, counts, cfg.batch, vocab, w)
    cu = _addr(dev, cu_rows, i32, cfg.batch + 1 if n else 0, f"{w}: cu_rows")
    tok = _addr(dev, token, i32, n, f"{w}: token")
    kept = 0 if path is None else _addr(dev, path, i32, n, f"{w}: path")
    acc = 0 if n_accept is None else _addr(dev, n_accept, i32, cfg.batch, f"{w}: n_accept")
    nxt = 0 if next_token is None else _addr(dev, next_token, i32, cfg.batch, f"{w}: next_token")
    rc = lib().kv_token_counts(cfg.c(), at, stride, int(vocab), int(kind), cu, tok, n, kept, acc, nxt, _status(dev, status, w),
                               _stream_of(dev, stream))
    if rc:
        _check(rc, w)


def kvq_selftest_scale_division(mismatches, stream=None) -> None:
    """Device self-check of the quantizer's scale division against IEEE division; adds the
    number of differing results to `mismatches` (a zeroed int64 device tensor of one element)."""
    rc = lib().kvq_selftest_scale_division(_ptr(mismatches), _stream(stream))
    _check(rc, "kvq_selftest_scale_division")


def kvq_selftest_tc_integer_sums(mismatches, stream=None) -> None:
    """Device self-check that the tensor cores add the rotation's integer digit products exactly;
    adds the number of differing sums to `mismatches` (a zeroed int64 device tensor of one
    element)."""
    rc = lib().kvq_selftest_tc_integer_sums(_ptr(mismatches), _stream(stream))
    _check(rc, "kvq_selftest_tc_integer_sums")


def workspace(cfg: KVConfig, max_ctx: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace tensor for kv_attn_decode."""
    n = kv_attn_workspace_bytes(cfg, max_ctx)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)
