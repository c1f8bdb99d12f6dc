"""kv_rope_qk over the number range: rows, norm weights and matrices of any size, on both kernels, against float64.

Row counts: 4 to 9 run on the CUDA cores, 403 and 3001 on the tensor cores."""

import numpy as np
import pytest
import torch

import bit_rotated_kv_gb300 as kvq
from tests import step_ref
from tests.test_gpu_rope import D, Call, _f64

pytestmark = pytest.mark.gpu


def _sized(c, exponents):
    """Row r of the projection times 2^exponents[r] (exact: bfloat16 keeps its digits)."""
    c.fused.mul_(torch.from_numpy(2.0 ** np.asarray(exponents, np.float64))[:, None].cuda())
    return c


def _weights(c, wq, wk):
    c.wq, c.wk = (np.asarray(w, np.float32) for w in (wq, wk))
    c.rope.q_norm, c.rope.k_norm = (torch.from_numpy(w).cuda() for w in (c.wq, c.wk))
    return c


# ---- rows far below the norm's epsilon -----------------------------------------------------------
@pytest.mark.parametrize("rows", [4, 3001])
@pytest.mark.parametrize("size", [1e-3, 1e-8, 1e-10, 1e-12, 1e-30])
def test_small_rows_with_a_norm(rows, size):
    Call(rows, size=size).run().check()


@pytest.mark.parametrize("rows", [7, 403])
@pytest.mark.parametrize("kind,layout,rot,hq,hkv", [("orthogonal", 0, 128, 16, 4), ("invertible", 1, 128, 16, 4), ("hadamard", 0, 96, 64, 8),
                                                    ("orthogonal", 1, 64, 16, 4), ("invertible", 0, 6, 8, 8), ("orthogonal", 0, 0, 8, 8)])
def test_rows_of_all_sizes_with_a_norm(rows, kind, layout, rot, hq, hkv):
    """Ordinary rows, rows about epsilon and rows down to the smallest numbers side by side, and one of zeros."""
    c = Call(rows, hq, hkv, kind, layout=layout, rot=rot)
    _sized(c, -(np.arange(rows) * 7 % 130.0))
    c.fused[rows // 2] = 0
    c.run().check()


@pytest.mark.parametrize("rows", [6, 403])
@pytest.mark.parametrize("eps", [1e-30, 1e-6, 1e3, 1e30])
def test_epsilons(rows, eps):
    c = Call(rows, 16, 4)
    c.eps = c.rope.norm_eps = eps
    _sized(c, -(np.arange(rows) % 5 * 25.0))
    c.run().check()


# ---- norm weights ----------------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [5, 403])
@pytest.mark.parametrize("rot", [128, 64])
def test_norm_weights_of_zero(rows, rot):
    """Weights that are all zero (rows of zeros, not NaN), beside ordinary ones."""
    c = _weights(Call(rows, 16, 4, rot=rot, size=0.01), np.zeros(D), np.linspace(-1, 1, D))
    c.run().check()
    assert not bool(c.q_out[:rows].any())


@pytest.mark.parametrize("rows", [5, 403])
@pytest.mark.parametrize("layout,rot", [(0, 128), (1, 128), (0, 64), (1, 64), (0, 6), (0, 0)])
@pytest.mark.parametrize("low,high", [(-12, 0), (-40, 20), (20, 60), (-90, -80), (-125, -120)])
@pytest.mark.parametrize("size", [0, -20])
def test_norm_weights_of_any_size(rows, layout, rot, low, high, size):
    """Weights that lie far apart, far above 1 or far below: the largest ones at channels where some rows have nothing."""
    c = Call(rows, 16, 4, layout=layout, rot=rot)
    rng = np.random.default_rng(2)
    w = [rng.choice([-1.0, 1.0], D) * 2.0 ** rng.uniform(low, high, D) for _ in range(2)]
    big = np.zeros((rows, 24, D), bool)
    for heads, x in ((slice(0, 16), w[0]), (slice(16, 20), w[1])):
        big[:, heads] = np.abs(x) > 2.0 ** (low + 2)
    big[::2] = False
    c.fused.masked_fill_(torch.from_numpy(big.reshape(rows, -1)).cuda(), 0.0)
    _sized(_weights(c, *w), np.full(rows, float(size)))
    c.run().check()


@pytest.mark.parametrize("rows", [5, 403])
@pytest.mark.parametrize("layout,rot", [(0, 64), (1, 64), (0, 126), (1, 30)])
@pytest.mark.parametrize("scale", [2.0**-40, 0.0, 2.0**40])
@pytest.mark.parametrize("size", [-90, 0, 60])
def test_factors_far_from_the_other_channels(rows, layout, rot, scale, size):
    """The rotated channels' factor takes them far from the others; rows that hold the one kind alone, or the other, or both."""
    c = Call(rows, 16, 4, "orthogonal", layout=layout, rot=rot, norm=False, scale=scale, seed=4)
    heads = c.fused.unflatten(1, (24, D))
    heads[0::3, :20, rot:] = 0
    heads[1::3, :20, :rot] = 0
    _sized(c, np.full(rows, float(size)))
    c.run().check()


# ---- rows and matrices at the ends of the range ----------------------------------------------------
@pytest.mark.parametrize("rows", [5, 403])
@pytest.mark.parametrize("x,t", [(-64, -60), (-100, -20), (-20, -96), (40, -100), (-100, 40), (90, -110)])
def test_small_products(rows, x, t):
    """Rows and matrices whose products come near the smallest numbers, or whose sizes make up for each other."""
    c = _sized(Call(rows, 16, 4, norm=False, rot=64), np.full(rows, float(x)))
    for m in (c.tr.t_k, c.tr.t_k_inv_t, c.tr.t_v):
        m.mul_(2.0**t)
    c.tk, c.tkit, c.tv = (_f64(m) for m in (c.tr.t_k, c.tr.t_k_inv_t, c.tr.t_v))
    c.run().check()
    assert bool(c.q_out[:rows].any(-1).all())


@pytest.mark.parametrize("rows", [5, 403])
@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_norm_weights_that_are_not_finite(rows, which, value):
    c = Call(rows, 16, 4)
    getattr(c.rope, which)[77] = value
    c.run()
    assert int(c.status.item()) == kvq.KVQ_ERR_NONFINITE
    if which == "k_norm":                                  # (the queries are what they were)
        c.status.zero_()
        d = Call(rows, 16, 4).run()
        assert torch.equal(c.q_out, d.q_out)


# ---- channels far apart under matrices that do not mix them ---------------------------------------
def _within(got, want, m, mats, gqa):
    """The header's bound: half a step of bf16, 2^-17 sum |T_ij| m_j, and 2^-22 of (max m_j) sum |T_ij| + (max |T_ij|) sum m_j.

    (Placed entries and the matrix's are two fp16 under powers of two that put a row's largest pair, and each matrix row's largest entry, at 2^-2 or
    above and below 2^15.  hi takes 11 bits exactly down to 2^-14, lo the next 11 of them to nearest, both in steps of 2^-24 at the finest: an entry
    is off by 2^-21 of itself and 2 * 2^-25, that is 2^-22 of its row's largest.)"""
    for h in range(got.shape[1]):
        t = np.abs(np.asarray(mats[h // gqa], np.float64))
        bound = 2.0**-17 * (m[:, h] @ t.T) + 2.0**-22 * (m[:, h].max(-1, keepdims=True) * t.sum(-1) + m[:, h].sum(-1, keepdims=True) * t.max(-1))
        off = np.abs(got[:, h] - want[:, h])
        assert (off <= 2.0**-8 * np.abs(want[:, h]) * (1 + 2.0**-8) + bound + 2.0**-133).all(), h


@pytest.mark.parametrize("rows", [6, 403])
@pytest.mark.parametrize("kind", ["identity", "diagonal", "invertible"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_channels_far_apart(rows, kind, norm):
    """Channels up to 60 binades apart within a row, under matrices that leave them apart."""
    c = Call(rows, 16, 4, "identity" if kind == "diagonal" else kind, norm=norm, rot=64, tv=kind != "identity")
    rng = np.random.default_rng(5)
    c.fused.mul_(torch.from_numpy(2.0 ** -rng.integers(0, 60, c.fused.shape)).cuda().to(torch.bfloat16))
    if kind == "diagonal":
        d = [torch.from_numpy(2.0 ** rng.integers(-30, 1, D)).float().cuda() for _ in range(2)]
        for t, x in zip((c.tr.t_k, c.tr.t_k_inv_t), d, strict=True):
            t.mul_(x)                                      # (each column by its own: rows of different sizes)
        c.tk, c.tkit = _f64(c.tr.t_k), _f64(c.tr.t_k_inv_t)
    c.run()
    assert int(c.status.item()) == 0
    angle = step_ref.phases(c.rope.freq.cpu().tolist(), c.pos)
    y, m = step_ref.placed(_f64(c.q), angle, False, 1.0, c.wq, c.eps)
    _within(_f64(c.q_out[:rows]), step_ref.transformed(y, m, c.tkit, 4)[0], m, c.tkit, 4)
    y, m = step_ref.placed(_f64(c.k), angle, False, 1.0, c.wk, c.eps)
    want = step_ref.transformed(y, m, c.tk, 1)[0]
    sink, ring = _f64(c.cache.sink_k), _f64(c.cache.ring_k)
    got = np.stack([sink[s, :, p] if p < c.cfg.s_sink else ring[s, :, p % c.cap] for s, p in zip(c.seq, c.pos, strict=True)])
    _within(got, want, m, c.tk, 1)


# ---- forms of the tensor-core kernel that need a call of their own --------------------------------
@pytest.mark.parametrize("rows", [7, 403])
@pytest.mark.parametrize("layout,rot", [(0, 128), (1, 128), (0, 96), (1, 64), (0, 6), (0, 126)])
@pytest.mark.parametrize("scale", [1.25, 0.0, 2.0**-20, 2.0**30])
def test_scales_without_a_norm(rows, layout, rot, scale):
    """YaRN's factor on heads that have no norm; factors that take the rotated channels far from the others."""
    for kind in ("orthogonal", "hadamard"):
        Call(rows, 16, 4, kind, layout=layout, rot=rot, norm=False, scale=scale, seed=4).run().check()


@pytest.mark.parametrize("rows", [7, 403])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_matrices_whose_rows_differ_in_size(rows, norm):
    """Rows of one matrix up to 2^40 apart, rows of zeros among them."""
    c = Call(rows, 16, 4, norm=norm, rot=64)
    rng = np.random.default_rng(8)
    for t in (c.tr.t_k, c.tr.t_k_inv_t, c.tr.t_v):
        f = 2.0 ** rng.integers(-20, 21, (t.shape[0], D))
        f[:, 5] = 0
        f[1] = np.where(np.arange(D) == 9, 2.0**9, 1.0)    # (one matrix: a row alone)
        t.mul_(torch.from_numpy(f).float().cuda()[:, :, None])
    c.tk, c.tkit, c.tv = (_f64(m) for m in (c.tr.t_k, c.tr.t_k_inv_t, c.tr.t_v))
    c.run().check()
