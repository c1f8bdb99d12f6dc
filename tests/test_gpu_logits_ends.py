"""kv_logits_probs at the smallest temperatures."""

import numpy as np
import pytest
import torch

from tests.test_gpu_logits import Call

pytestmark = pytest.mark.gpu
HEATS = np.array([1e-45, 1e-38, 2.0**-121, 2.0**-120, 2.0**-119, 1e-30, 1e-6], np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [500, 40000])
def test_the_best_token_has_it_all(dtype, vocab):
    c = Call([1] * len(HEATS), vocab, dtype, held=False, rules=False)
    c.rules["temperature"] = HEATS
    c.logits[:, vocab // 3] = 50.0
    c.run()
    assert int(c.status.item()) == 0
    want = torch.zeros_like(c.p)
    want[:, vocab // 3] = 1.0
    assert torch.equal(c.p, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [500, 40000])
def test_equal_maxima_share(dtype, vocab):
    """Two tokens with the largest logit: half each at every temperature above 0, the lower id alone at 0."""
    heats = np.concatenate([HEATS, [0.0]]).astype(np.float32)
    c = Call([1] * len(heats), vocab, dtype, held=False, rules=False)
    c.rules["temperature"] = heats
    c.logits[:, [7, vocab - 2]] = 50.0
    c.run()
    assert int(c.status.item()) == 0
    want = torch.zeros_like(c.p)
    want[:, [7, vocab - 2]] = 0.5
    want[-1, [7, vocab - 2]] = torch.tensor([1.0, 0.0], device="cuda")
    assert torch.equal(c.p, want)
