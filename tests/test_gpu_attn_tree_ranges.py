"""kv_attn_tree over caches whose numbers or shapes lie at the ends of what the cache can hold, against
float64 attention over the cache read back.

Tolerance per (node, head): as in test_gpu_attn_tree -- half a bf16 step of the value (2^-8 relative, the one
rounding of the output) plus the attention parity tolerance of 2e-3 of the row's largest value."""

import pytest
import torch

from tests import spec_ref
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


def _heads(w, h):
    return slice(h * w.gqa, (h + 1) * w.gqa)


def _rows(cu, b):
    return slice(int(cu[b]), int(cu[b + 1]))


WEIGHT_SHAPES = {
    "one_split": (ONE_SPLIT.replace(ctx_lo=7900, ctx_hi=8000), [64] * 19),
    "one_split_g32": (ONE_SPLIT.replace(ctx_lo=7900, ctx_hi=8000, group_size=32), [64] * 19),
    "splits": (BASE.replace(batch=1, n_q_heads=8, n_kv_heads=2, ctx_lo=32000, ctx_hi=32000), [64]),
    "narrow": (BASE.replace(batch=1, n_q_heads=8, n_kv_heads=2, ctx_lo=8000, ctx_hi=8000), [6]),
}


@pytest.mark.parametrize("lead", [13.3, 15.7, 18.0, 20.0, 24.0])
@pytest.mark.parametrize("shape", sorted(WEIGHT_SHAPES))
def test_a_sink_takes_the_weight_and_gives_nothing(shape, lead):
    """Token 0's key agrees with every query by `lead` nats, and its value row is zero: the output is what the
    other tokens leave (at 13.3 nats a tenth of the weight on 32 K tokens, at 24 nats 2 in 10^6)."""
    w, counts = WEIGHT_SHAPES[shape]
    run, q, cu, parent = _drafted(w, counts, "random")
    c, scale, gen = run.runner.cache, run.runner.sm_scale, torch.Generator("cuda").manual_seed(9)
    for b in range(w.batch):
        for h in range(w.n_kv_heads):
            u = torch.randn(128, generator=gen, device="cuda")
            u /= u.norm()
            q[_rows(cu, b), _heads(w, h)] += (8 * u).to(torch.bfloat16)
            c.sink_k[b, h, 0] = (u * (lead / (8 * scale))).to(torch.bfloat16)
    c.sink_v[:, :, 0] = 0
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    _compare(run, q, cu, parent, out, [(0, 0), (w.batch - 1, 1)])


def _key_scales(run):
    """(Delta16, z16) of every key token and group, [pages, heads, 16, G, 2], a view of the pool."""
    ng = 128 // run.cfg.group_size
    p = run.runner.cache.pages
    return p[:, :, 1024:1024 + 64 * ng].view(torch.float16).unflatten(-1, (16, ng, 2))


def _value_deltas(run):
    """Value Delta16, [pages, heads, 8 token pairs, G, 2], a view of the pool."""
    ng = 128 // run.cfg.group_size
    p = run.runner.cache.pages
    return p[:, :, 1024 + 64 * ng:1024 + 96 * ng].view(torch.float16).unflatten(-1, (8, ng, 2))


@pytest.mark.parametrize("where", ["first_page", "middle"])
@pytest.mark.parametrize("lead", [13.3, 20.0])
@pytest.mark.parametrize("shape", ["one_split", "one_split_g32", "splits"])
def test_a_token_of_the_pages_takes_the_weight_and_gives_nothing(shape, lead, where):
    """The same with a quantized token: every query agrees with it, its key is stretched, its values are zero."""
    w, counts = WEIGHT_SHAPES[shape]
    w = w.replace(s_sink=0)
    run, q, cu, parent = _drafted(w, counts, "random")
    scale, snap = run.runner.sm_scale, run.snapshot()
    keys, dv = _key_scales(run), _value_deltas(run)
    for b in range(w.batch):
        t = 0 if where == "first_page" else int(snap["s_quant"][b]) // 2
        pid = int(run.table[b, t // 16])
        for h in range(w.n_kv_heads):
            k = torch.from_numpy(spec_ref.unit_kv(run.cfg, snap, run.table, b, h)[0][t]).cuda()
            norm = float(k.norm())
            q[_rows(cu, b), _heads(w, h)] += (8 * k / norm).to(torch.bfloat16)
            keys[pid, h, t % 16, :, 0] *= lead / (8 * norm * scale)
            dv[pid, h, t % 16 // 2, :, t % 2] = 0
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    _compare(run, q, cu, parent, out, [(0, 0), (w.batch - 1, 1)])


OFFSET_COUNTS = {"wide": [64, 40], "narrow": [6, 3]}


@pytest.mark.parametrize("zero", [600.0, 5000.0, 60000.0])
@pytest.mark.parametrize("trees", sorted(OFFSET_COUNTS))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("l2", [False, True])
def test_keys_far_from_zero(group, trees, zero, l2):
    """Every group of every key lies about one away from 0, its codes a z-th of that apart."""
    base = BASE.replace(transform="hadamard", key_l2norm=True) if l2 else BASE
    w = base.replace(batch=2, n_q_heads=8, n_kv_heads=2, ctx_lo=900, ctx_hi=1500, group_size=group)
    run, q, cu, parent = _drafted(w, OFFSET_COUNTS[trees], "random")
    keys = _key_scales(run)
    gen = torch.Generator("cuda").manual_seed(11)
    off = torch.randn(keys.shape[:-1], generator=gen, device="cuda")
    keys[..., 1] = (-torch.sign(off) * zero * (1 + 0.08 * torch.rand(off.shape, generator=gen, device="cuda"))).half()
    keys[..., 0] = (off.abs() / (zero * (128 ** 0.5 if l2 else 1))).half()
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    _compare(run, q, cu, parent, out, [(0, 0), (1, 1)])


@pytest.mark.parametrize("apart", [6, 10, 14])
@pytest.mark.parametrize("trees", sorted(OFFSET_COUNTS))
@pytest.mark.parametrize("group", [32, 64])
def test_a_group_of_small_keys_under_large_queries(group, trees, apart):
    """One group's keys 2^-apart of the others', its queries 2^apart times theirs: all groups weigh alike."""
    w = BASE.replace(batch=2, n_q_heads=8, n_kv_heads=2, ctx_lo=900, ctx_hi=1500, group_size=group)
    run, q, cu, parent = _drafted(w, OFFSET_COUNTS[trees], "random")
    keys, c = _key_scales(run), run.runner.cache
    for g in range(128 // group):
        small = slice(g * group, (g + 1) * group)
        pages, rows = keys.clone(), [t.clone() for t in (c.sink_k, c.ring_k)]
        keys[..., g, 0] = (keys[..., g, 0].float() * 2.0 ** -apart).half()
        for t in (c.sink_k, c.ring_k):
            t[..., small] *= 2.0 ** -apart
        qg = q.clone()
        qg[..., small] *= 2.0 ** apart
        out = _call(run, qg, cu, parent)
        assert int(run.runner.status.item()) == 0
        _compare(run, qg, cu, parent, out, [(0, 0), (1, 1)])
        keys.copy_(pages)
        c.sink_k.copy_(rows[0])
        c.ring_k.copy_(rows[1])


def _value_zeros(run):
    """Value z16, as _value_deltas."""
    ng = 128 // run.cfg.group_size
    p = run.runner.cache.pages
    return p[:, :, 1024 + 96 * ng:1024 + 128 * ng].view(torch.float16).unflatten(-1, (8, ng, 2))


@pytest.mark.parametrize("zero", [1.5, 600.0, 60000.0])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_values_up_to_the_end_of_fp16(group, zero):
    """Values of up to 65504 in magnitude are held; one beyond that is reported.

    The values' signs are drawn, so that a row may cancel far below them, and its error is that of the terms:
    p is rounded to fp16 (at most 2^-11 p), Delta z likewise (2^-11 |Delta z|, and |Delta z| <= |v| + 3 Delta), and
    Delta c - Delta z once more (2^-11 |v|).  So sum p v is off by at most 2^-11 (3 sum p |v| + 3 Delta sum p), and the
    output's rounding to bf16 adds 2^-8 of it.  (The scores' errors, some 2^-20, are far below that bound's slack:
    it adds up the roundings of all tokens in one direction.)"""
    import bit_rotated_kv_gb300 as kvq
    w = BASE.replace(batch=2, n_q_heads=8, n_kv_heads=2, ctx_lo=900, ctx_hi=1500, group_size=group)
    run, q, cu, parent = _drafted(w, [64, 40], "random")
    d, z = _value_deltas(run), _value_zeros(run)
    gen = torch.Generator("cuda").manual_seed(12)
    sign = torch.randint(0, 2, z.shape, generator=gen, device="cuda") * 2 - 1
    z[...] = (sign * zero).half()
    delta = 60000.0 / (zero + 3)
    d[...] = delta
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    qf, of, snap = q.double().cpu().numpy(), out.double().cpu().numpy(), run.snapshot()
    for b, h in ((0, 0), (1, 1)):
        rows, heads = _rows(cu, b), _heads(w, h)
        K, V = spec_ref.unit_kv(run.cfg, snap, run.table, b, h)
        at = lambda v: spec_ref.tree_attention(qf[rows, heads], K, v, parent[rows], run.runner.sm_scale)  # noqa: E731
        ref, size = at(V), at(abs(V))
        assert (abs(of[rows, heads] - ref) <= 2.0 ** -8 * abs(ref) + 2.0 ** -11 * 3 * (size + delta)).all(), (b, h)
    d[...] = 30000.0                                  # (1.5 + 3) x 30000, and more
    z[...] = (-zero * sign.abs()).half()
    _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == kvq.KVQ_ERR_NONFINITE


def test_a_workspace_of_the_largest_size_serves_smaller_calls():
    """Calls of fewer rows and shorter contexts than the workspace was sized for, through both kernels; the bytes
    behind it are left."""
    import bit_rotated_kv_gb300 as kvq
    runs = [_drafted(BASE.replace(batch=4, ctx_lo=ctx, ctx_hi=ctx + 300), counts, "random")
            for ctx, counts in ((500, [128, 30, 90, 128]), (9000, [128, 128, 128, 128]), (9000, [20, 30, 10, 20]), (9000, [5, 1, 2, 1]),
                                (2000, [1, 1, 1, 1]), (9000, [0, 0, 60, 0]), (700, [0, 2, 0, 0]))]
    big = max(runs, key=lambda r: r[0].runner.cfg.max_pages_per_seq)[0]
    n = kvq.kv_attn_tree_workspace_bytes(big.cfg, 512, int(big.runner.cache.seq_len.max()))
    room = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    room[n:] = 77
    ws = room[:n]
    for _ in range(2):
        for run, q, cu, parent in runs:
            run.cfg.max_pages_per_seq, was = big.cfg.max_pages_per_seq, run.cfg.max_pages_per_seq
            table = run.runner.cache.page_table
            wide = torch.full((4, big.cfg.max_pages_per_seq), -1, dtype=torch.int32, device="cuda")
            wide[:, :was] = table
            run.runner.cache.page_table = wide
            out = _call(run, q, cu, parent, ws)
            assert int(run.runner.status.item()) == 0
            _compare(run, q, cu, parent, out, [(2, 3)])
            run.cfg.max_pages_per_seq, run.runner.cache.page_table = was, table
    assert bool((room[n:] == 77).all())


@pytest.mark.parametrize("splits", [0, 40])
def test_tickets_are_zero_after_every_call(splits):
    """The row kernel's joins of one and of two levels (40 splits of 8 columns): same bits each time, and the
    tickets at the head of the workspace, three or more a grid row, as they were."""
    import bit_rotated_kv_gb300 as kvq
    w = BASE.replace(batch=3, n_q_heads=8, n_kv_heads=2, ctx_lo=3000, ctx_hi=5000)
    run, q, cu, parent = _drafted(w, [5, 0, 7], "random")
    run.cfg.attn_splits = splits
    n = kvq.kv_attn_tree_workspace_bytes(run.cfg, q.shape[0], int(run.runner.cache.seq_len.max()))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    tickets = ws[:4 * 3 * w.batch * kvq.KVQ_TREE_MAX_NODES * w.n_kv_heads]
    first = _call(run, q, cu, parent, ws)
    _compare(run, q, cu, parent, first, [(0, 0), (2, 1)])
    assert bool((ws != 0).any())                      # (partials were joined through it)
    for _ in range(3):
        assert int(run.runner.status.item()) == 0 and not bool(tickets.any())
        assert torch.equal(_call(run, q, cu, parent, ws).view(torch.int16), first.view(torch.int16))
