"""kv_rope_qk over the number range: rows, norm weights and matrices of any size, on both kernels, against float64.

Row counts: 4 to 9 run on the CUDA cores, 403 and 3001 on the tensor cores."""

import numpy as np
import pytest
import torch

from tests.test_gpu_rope import Call

pytestmark = pytest.mark.gpu


def _sized(c, exponents):
    """Row r of the projection times 2^exponents[r] (exact: bfloat16 keeps its digits)."""
    c.fused.mul_(torch.from_numpy(2.0 ** np.asarray(exponents, np.float64))[:, None].cuda())
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
