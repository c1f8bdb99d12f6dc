"""kv_attn_tree_workspace_bytes bounds every smaller call (host arithmetic, no GPU)."""

import random

import pytest

import bit_rotated_kv_gb300 as kvq


def _configs():
    rng = random.Random(4)
    for _ in range(60):
        hkv = rng.choice([1, 2, 4, 8, 40])
        axis = rng.random() < 0.2
        yield kvq.KVConfig(n_q_heads=hkv * rng.choice([1, 2, 4, 8]), n_kv_heads=hkv, batch=rng.choice([1, 2, 3, 16, 19, 64, 300]),
                           max_pages_per_seq=rng.choice([4, 700, 70000]), num_pages=1000, ring_cap=4096, s_sink=rng.choice([0, 64]),
                           s_keep=rng.choice([0, 256, 3000]), s_flush=16, key_axis=int(axis), group_size=rng.choice([32, 128]),
                           attn_splits=rng.choice([0, 0, 0, 5, 200]))


@pytest.mark.parametrize("cfg", list(_configs()), ids=lambda c: f"b{c.batch}-h{c.n_q_heads}-{c.n_kv_heads}-s{c.attn_splits}-a{c.key_axis}")
def test_workspace_grows_with_both_sizes(cfg):
    rng = random.Random(cfg.batch)
    most = min(65535, cfg.batch * kvq.KVQ_TREE_MAX_NODES)
    rows = sorted({1, 2, 3, 4, 8, 31, 32, 33, most} | {rng.randint(1, most) for _ in range(60)})
    rows = [r for r in rows if r <= most]
    ctxs = sorted({0, 1, 100, 2047, 2048, 5000, 32768, 131072, 1 << 20} | {rng.randint(1, 200000) for _ in range(6)})
    size = {(r, c): kvq.kv_attn_tree_workspace_bytes(cfg, r, c) for r in rows for c in ctxs}
    for i, r in enumerate(rows):
        for j, c in enumerate(ctxs):
            assert size[r, c] > 0
            assert i == 0 or size[r, c] >= size[rows[i - 1], c], (r, c)
            assert j == 0 or size[r, c] >= size[r, ctxs[j - 1]], (r, c)


def test_sixteen_sequences_of_32k():
    cfg = kvq.KVConfig(n_q_heads=32, n_kv_heads=8, batch=16, max_pages_per_seq=2048, num_pages=32768, ring_cap=512)
    at = lambda n: kvq.kv_attn_tree_workspace_bytes(cfg, n, 32768)  # noqa: E731
    assert at(512) <= at(1024) <= at(2048)
    assert at(2048) < 256 << 20                       # (and stays a small part of what the cache takes)
