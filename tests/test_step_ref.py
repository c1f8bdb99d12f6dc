"""The frequencies that the library computes on the host, against the formulas, and the plain references of a
step's ends against special cases.  (No GPU.)"""

import math
import os

import numpy as np
import pytest

import bit_rotated_kv_gb300 as kvq
from tests import step_ref


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(kvq.LIB_PATH):
        from bit_rotated_kv_gb300 import build_lib
        build_lib.build()


CASES = [("plain", kvq.KVQ_ROPE_PLAIN, 1.0, 0, 0, 0), ("linear", kvq.KVQ_ROPE_LINEAR, 8.0, 0, 0, 0), ("ntk", kvq.KVQ_ROPE_NTK, 4.0, 0, 0, 0),
         ("bands", kvq.KVQ_ROPE_BANDS, 8.0, 8192, 1, 4), ("yarn", kvq.KVQ_ROPE_YARN, 4.0, 32768, 32, 1), ("yarn", kvq.KVQ_ROPE_YARN, 0.5, 4096, 32, 1)]


@pytest.mark.parametrize("kind,code,factor,context,a,b", CASES)
@pytest.mark.parametrize("rot,theta", [(128, 1e6), (64, 1e4), (4, 5e5), (126, 1e4)])
def test_frequencies(kind, code, factor, context, a, b, rot, theta):
    freq, scale = kvq.kvq_rope_frequencies(rot, theta, code, factor, context, a, b)
    want, want_scale = step_ref.frequencies(rot, theta, kind, factor, context, a, b)
    got = np.array([(int(f) & (2**64 - 1)) / 2**64 for f in freq.tolist()]) * 2 * math.pi
    # (pow, the division and the mix: a few roundings of float64 each, and one unit of 2^-64 turns)
    assert np.all(np.abs(got - want) <= 16 * 2.0**-53 * want + 2 * math.pi * 2.0**-63)
    assert scale == np.float32(want_scale)


def test_frequencies_refused():
    bad = [dict(rot_dim=130), dict(rot_dim=5), dict(rot_dim=-2), dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")),
           dict(factor=0.0), dict(factor=float("inf")), dict(scaling=5), dict(scaling=-1), dict(scaling=kvq.KVQ_ROPE_NTK, rot_dim=2),
           dict(scaling=kvq.KVQ_ROPE_BANDS), dict(scaling=kvq.KVQ_ROPE_BANDS, context=8192, a=4, b=1),
           dict(scaling=kvq.KVQ_ROPE_YARN, context=8192, a=1, b=32), dict(scaling=kvq.KVQ_ROPE_YARN, context=-1, a=32, b=1)]
    for kw in bad:
        with pytest.raises(kvq.KVQError) as e:
            kvq.kvq_rope_frequencies(**{"rot_dim": 64, "theta": 1e4, **kw})
        assert e.value.code == kvq.KVQ_ERR_INVALID_ARG, kw
    freq, scale = kvq.kvq_rope_frequencies(0, 1e4)
    assert len(freq) == 0 and scale == 1.0


def test_phases_are_exact_at_far_positions():
    freq = [1 << 62, (1 << 63) + 1, 3]
    got = step_ref.phases(freq, [2**31 - 1, -1])
    assert got[0, 0] == pytest.approx(0.75 * 2 * math.pi) and got[1, 0] == pytest.approx(0.75 * 2 * math.pi)
    assert got[1, 2] == pytest.approx(2 * math.pi)


def test_rotation_keeps_lengths_and_depends_on_differences():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 1, 128))
    freq = [int(2**64 / (2 * math.pi) * 1e4 ** (-2 * i / 128)) for i in range(64)]
    for inter in (False, True):
        dots = []
        for shift in (0, 12345):
            y, _ = step_ref.placed(x, step_ref.phases(freq, [7 + shift, 3 + shift]), inter)
            assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
            dots.append(float(y[0, 0] @ y[1, 0]))
        assert dots[0] == pytest.approx(dots[1])
    h = step_ref.hadamard()
    assert np.allclose(h @ h.T, np.eye(128))


def test_values_by_hand():
    rules = {"bias": {0: {1: 2.0, 3: -np.inf}}, "repetition": [2.0], "frequency": [0.5], "presence": [0.25]}
    counts = np.array([0x8000, 3, 0, 0, 0x8001], np.uint16)
    x, _ = step_ref.values([4.0, 2.0, 1.0, 5.0, -6.0], counts, [2, 2], rules, 0, np.array([1, 1, 1, 1, 0], bool))
    assert x.tolist() == [2.0, 2.0 - 1.5 - 0.25, 0.5 - 1.0 - 0.25, -np.inf, -np.inf]
    p, _ = step_ref.probabilities(np.array([1.0, 3.0, 3.0]), np.ones(3), 0)
    assert p.tolist() == [0.0, 1.0, 0.0]
    p, _ = step_ref.probabilities(np.array([0.0, math.log(3.0), -np.inf]), np.ones(3), 1.0)
    assert np.allclose(p, [0.25, 0.75, 0.0])
