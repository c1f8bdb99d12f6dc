"""Plain references of the drafted-tree and page-pool calls, written from include/kvq.h: float64
attention over the cache as read back, verification in Python integers, and the pool as lists."""

from __future__ import annotations

import numpy as np

from tests import layout

ONE = 1 << 60


def bf16(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ---- attention -----------------------------------------------------------------------------------
def unit_kv(cfg, snap: dict, table: np.ndarray, b: int, h: int):
    """(K, V) float64 [L, 128] of one (sequence, kv head), INT2 tokens dequantized."""
    L, sq, sink, cap = int(snap["seq_len"][b]), int(snap["s_quant"][b]), cfg.s_sink, cfg.ring_cap
    a, e = min(sink, L), max(min(sink, L), min(sq, L))
    axis = int(cfg.key_axis)
    u = layout.decode_unit(snap["pages"], table[b], h, sink, e, cfg.group_size, bool(cfg.key_l2norm), axis)
    f = lambda x: np.asarray(x, np.float64)  # noqa: E731
    if axis:
        page = np.arange(e - a) // 16
        k = f(u["delta_k"])[page] * (f(u["codes_k"]) - f(u["zero_k"])[page]) if e > a else np.zeros((0, 128))
    else:
        k = np.repeat(f(u["delta_k"]), cfg.group_size, 1) * (f(u["codes_k"]) - np.repeat(f(u["zero_k"]), cfg.group_size, 1))
    if cfg.key_l2norm and e > a:
        k = k * f(u["norm_k"])[:, None]
    v = np.repeat(f(u["delta_v"]), cfg.group_size, 1) * (f(u["codes_v"]) - np.repeat(f(u["zero_v"]), cfg.group_size, 1))
    slots = np.arange(e, L) % cap
    K = np.concatenate([bf16(snap["sink_k"][b, h, :a]), k, bf16(snap["ring_k"][b, h, slots])])
    V = np.concatenate([bf16(snap["sink_v"][b, h, :a]), v, bf16(snap["ring_v"][b, h, slots])])
    return K, V


def tree_attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, parent, scale: float) -> np.ndarray:
    """q [n, g, 128] float64, the nodes being the last n tokens -> [n, g, 128]."""
    n, L = len(parent), len(K)
    out = np.zeros_like(q)
    for i in range(n):
        seen = list(range(L - n))
        at = i
        while at >= 0:
            seen.append(L - n + at)
            at = int(parent[at])
        s = (q[i] @ K[seen].T) * scale
        p = np.exp(s - s.max(-1, keepdims=True))
        out[i] = (p / p.sum(-1, keepdims=True)) @ V[seen]
    return out


def random_tree(rng, n: int, kind: str) -> np.ndarray:
    if kind == "chain":
        return np.arange(-1, n - 1).astype(np.int32)
    if kind == "roots":
        return np.full(n, -1, np.int32)
    if kind == "star":
        return np.where(np.arange(n) == 0, -1, 0).astype(np.int32)
    i = np.arange(n)
    return np.where(i == 0, -1, np.maximum(0, i - rng.integers(1, 6, n))).astype(np.int32)


# ---- verification ---------------------------------------------------------------------------------
def _units(row):
    return [int(min(max(float(x), 0.0), 1.0) * ONE) for x in np.asarray(row, np.float64)]


def _mul(a: int, b: int) -> int:
    return (a * b) >> 60


def verify(parent, token, p, q, u):
    """One sequence: (path, next token) by the definition, in exact integers."""
    n, cur, path = len(parent), 0, [0]
    r, z, gone = _units(p[0]), ONE, False
    for c in range(1, n):
        if parent[c] != cur or gone:
            continue
        x = int(token[c])
        want = z if q is None else _mul(z, _units(q[cur][x:x + 1])[0])
        if _mul(_units([u[c]])[0], want) < r[x]:
            cur, r, z = c, _units(p[c]), ONE
            path.append(c)
            continue
        if q is None:
            z = max(0, z - r[x])
            r = list(r)
            r[x] = 0
        else:
            Q = _units(q[cur])
            r = [max(0, a - _mul(z, b)) for a, b in zip(r, Q)]
            z = sum(r)
        if z == 0:
            r, gone = _units(p[cur]), True
    if sum(r) == 0:
        r = _units(p[cur])
    goal, upto = _mul(_units([u[0]])[0], sum(r)), 0
    for x, w in enumerate(r):
        upto += w
        if upto > goal:
            return path, x
    return path, -1


# ---- the page pool ---------------------------------------------------------------------------------
class Pool:
    """Tables, counts, lengths and page contents as plain lists and arrays."""

    def __init__(self, cfg, snap, table, ref):
        self.cfg = cfg
        self.s = {k: np.array(v) for k, v in snap.items() if isinstance(v, np.ndarray)}
        self.table, self.ref = np.array(table), np.array(ref)

    def _free(self):
        return [i for i in range(self.cfg.num_pages) if self.ref[i] == 0]

    def free(self, seqs):
        for b in seqs:
            for c, t in enumerate(self.table[b]):
                if t >= 0:
                    self.ref[t] -= 1
                self.table[b, c] = -1
            self.s["seq_len"][b], self.s["s_quant"][b] = 0, self.cfg.s_sink

    def reserve(self, tokens):
        for b, t in enumerate(tokens):
            if t <= 0:
                continue
            want = -(-(int(self.s["seq_len"][b]) + int(t) - self.cfg.s_sink) // 16)
            have = int((self.table[b] >= 0).sum())
            free = self._free()
            if want > self.cfg.max_pages_per_seq:
                continue
            if want - have > len(free):
                return
            for c in range(have, want):
                self.table[b, c] = free[c - have]
                self.ref[free[c - have]] = 1

    def fork(self, src, dst):
        cfg, s = self.cfg, self.s
        for i, (a, b) in enumerate(zip(src, dst)):
            tokens = max(0, int(s["s_quant"][a]) - cfg.s_sink)
            full, part = tokens // 16, tokens % 16 > 0
            if part:
                free = self._free()
                if not free:
                    return
                self.table[b, full] = free[0]
                self.ref[free[0]] = 1
                s["pages"][free[0]] = s["pages"][self.table[a, full]]
            for c in range(full):
                self.table[b, c] = self.table[a, c]
                self.ref[self.table[a, c]] += 1
            L, e = int(s["seq_len"][a]), int(s["s_quant"][a])
            for t in range(min(L, cfg.s_sink)):
                for k in ("sink_k", "sink_v"):
                    s[k][b, :, t] = s[k][a, :, t]
            for t in range(max(e, cfg.s_sink), L):
                for k in ("ring_k", "ring_v"):
                    s[k][b, :, t % cfg.ring_cap] = s[k][a, :, t % cfg.ring_cap]
            s["seq_len"][b], s["s_quant"][b] = L, e

    def compact(self):
        live = [i for i in range(self.cfg.num_pages) if self.ref[i] > 0]
        n = len(live)
        holes = [i for i in range(n) if self.ref[i] == 0]
        for a, b in zip([i for i in live if i >= n], holes):
            self.s["pages"][b] = self.s["pages"][a]
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.table[self.table == a] = b
        return n
