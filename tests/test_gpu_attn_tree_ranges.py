"""kv_attn_tree over caches whose numbers or shapes lie at the ends of what the cache can hold, against
float64 attention over the cache read back.

Tolerance per (node, head): as in test_gpu_attn_tree -- half a bf16 step of the value (2^-8 relative, the one
rounding of the output) plus the attention parity tolerance of 2e-3 of the row's largest value."""

import pytest
import torch

from tests.test_gpu_attn_tree import BASE, _call, _compare, _drafted

pytestmark = pytest.mark.gpu

# 64 nodes of 4 heads on 2 kv heads, 19 sequences: 152 row tiles, so that a CTA has all of a sequence's tiles
ONE_SPLIT = BASE.replace(batch=19, n_q_heads=8, n_kv_heads=2)


@pytest.mark.parametrize("keep", [256, 1500])
def test_window_tiles_and_page_tiles_of_one_cta(keep):
    """Four (fourteen) tiles of window rows and the pages share a CTA's memory in turn; again and again, with
    the same bits each time."""
    w = ONE_SPLIT.replace(ctx_lo=1900, ctx_hi=2300, s_keep=keep)
    run, q, cu, parent = _drafted(w, [64] * 19, "random")
    first = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    _compare(run, q, cu, parent, first, [(0, 0), (7, 1), (18, 1)])
    for _ in range(20):
        assert torch.equal(_call(run, q, cu, parent).view(torch.int16), first.view(torch.int16))
    assert int(run.runner.status.item()) == 0
