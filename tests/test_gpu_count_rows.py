"""kv_token_counts: ends of sequences behind the last row, on both sides of the choice of kernel."""

import numpy as np
import pytest
import torch

import bit_rotated_kv_gb300 as kvq
from tests import step_ref
from tests.test_gpu_logits import _cfg, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [[300, 40], [300, 0], [90000, 70001], [70003]])
@pytest.mark.parametrize("more", [1, 5, 1 << 30])
@pytest.mark.parametrize("kind", [kvq.KVQ_COUNT_PROMPT, kvq.KVQ_COUNT_OUTPUT])
def test_an_end_behind_the_last_row(n, more, kind):
    """The rows that there are belong to their sequence all the same, and the call reports the end."""
    rng, batch, vocab = np.random.default_rng(3), len(n), 1001
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    token = rng.integers(0, vocab, int(cu[-1])).astype(np.int32)
    at = cu.copy()
    at[-1] += more
    want = np.zeros((batch, vocab + 1), np.uint16)
    for b in range(batch):
        t = token[cu[b]:cu[b + 1]]
        if kind == kvq.KVQ_COUNT_PROMPT:
            want[b, t] = 0x8000
        else:
            want[b] = np.minimum(np.bincount(t, minlength=vocab + 1), step_ref.MOST)
    got, status = torch.zeros((batch, vocab + 1), dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kv_token_counts(_cfg(batch), got, vocab, kind, _dev(at), _dev(token), None, None, None, status)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy().view(np.uint16), want)
    assert int(status.item()) == kvq.KVQ_ERR_BOUNDS
