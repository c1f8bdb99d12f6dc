"""kv_attn_tree: every node of a drafted tree attends to the tokens before the drafts, its
ancestors and itself -- against float64 attention over the cache read back.

Tolerance per (node, head): half a bf16 step of the value (2^-8 relative, the one rounding of the
output) plus the attention parity tolerance of 2e-3 of the row's largest value."""

import numpy as np
import pytest
import torch

import synth
from tests import harness, spec_ref

pytestmark = pytest.mark.gpu
ATTN_TOL = 2e-3


def _drafted(w, counts, kind, seed=0, poison=True, ctx=None):
    """A prefilled cache with the drafts of counts[b] nodes appended (no flush), q' and the tree."""
    from bit_rotated_kv_gb300.runner import _rows_for
    counts = np.asarray(counts)
    run = harness.DeviceRun(w.replace(n_new=max(1, int(counts.max()))), do_step=False,
                            pool_fill=0xFF if poison else None)
    r, dev = run.runner, run.device
    ib, it = _rows_for(run.k_all, run.lengths, run.lengths + counts)
    if ib is not None:
        r.append(run.k_all[ib, it].contiguous(), run.v_all[ib, it].contiguous(), ib.to(torch.int32), it.to(torch.int32))
    torch.cuda.synchronize()
    if poison:                                       # whatever no token lives in holds NaN
        c = r.cache
        for b in range(w.batch):
            L, e = int(c.seq_len[b]), int(c.s_quant[b])
            dead = np.ones(run.cfg.ring_cap, bool)
            dead[np.arange(max(e, w.s_sink), max(L, w.s_sink)) % run.cfg.ring_cap] = False
            at = torch.from_numpy(np.nonzero(dead)[0]).to(dev)
            for t in (c.ring_k, c.ring_v):
                t[b, :, at] = float("nan")
            for t in (c.sink_k, c.sink_v):
                t[b, :, min(L, w.s_sink):] = float("nan")
    rng = np.random.default_rng(seed)
    parent = np.concatenate([spec_ref.random_tree(rng, int(n), kind) for n in counts]).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(counts.sum()), w.n_q_heads, 128)).astype(np.float32)).to(dev).to(torch.bfloat16)
    return run, q, cu, parent


def _call(run, q, cu, parent, ws=None, stream=None):
    import bit_rotated_kv_gb300 as kvq
    r = run.runner
    max_ctx = int(r.cache.seq_len.max())
    if ws is None:
        n = kvq.kv_attn_tree_workspace_bytes(r.cfg, q.shape[0], max_ctx)
        ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=run.device)
    out = torch.full_like(q, float("nan"))
    dev = lambda a: torch.from_numpy(a).to(run.device)  # noqa: E731
    kvq.kv_attn_tree(r.cfg, r.cache, q, dev(cu), dev(parent), out, r.sm_scale, max_ctx, ws, r.status, stream)
    torch.cuda.synchronize()
    return out


def _compare(run, q, cu, parent, out, units):
    g, snap = run.w.gqa, run.snapshot()
    qf, of = q.double().cpu().numpy(), out.double().cpu().numpy()
    for b, h in units:
        rows = slice(int(cu[b]), int(cu[b + 1]))
        if rows.start == rows.stop:
            continue
        K, V = spec_ref.unit_kv(run.cfg, snap, run.table, b, h)
        ref = spec_ref.tree_attention(qf[rows, h * g:(h + 1) * g], K, V, parent[rows], run.runner.sm_scale)
        got = of[rows, h * g:(h + 1) * g]
        tol = np.abs(ref) * 2.0 ** -8 + ATTN_TOL * np.abs(ref).max(-1, keepdims=True)
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (b, h, np.argwhere(bad)[:4], float(np.nanmax(np.abs(got - ref) / np.maximum(np.abs(ref).max(-1, keepdims=True), 1e-30))))


BASE = synth.WUSH_CHUNK_B16.replace(chunk_queries=False, transform="orthogonal")
CASES = {
    # name: workload, nodes per sequence, kind of tree
    "g128_gqa4": (BASE.replace(batch=2, ctx_lo=700, ctx_hi=900), [13, 64], "random"),
    "g64_ragged_zero": (BASE.replace(batch=3, ctx_lo=400, ctx_hi=1500, group_size=64), [5, 0, 33], "random"),
    "g32_l2_hadamard_gqa8": (synth.QWEN3_32B_128K.replace(batch=2, ctx_lo=1500, ctx_hi=2500), [16, 3], "random"),
    "g64_l2": (synth.QWEN3_32B_128K.replace(batch=1, ctx_lo=1030, ctx_hi=1030, group_size=64), [9], "random"),
    "g128_l2": (synth.QWEN3_32B_128K.replace(batch=1, ctx_lo=1030, ctx_hi=1030, group_size=128), [9], "random"),
    "g32_plain_gqa1": (BASE.replace(batch=2, n_q_heads=8, ctx_lo=600, ctx_hi=700, group_size=32), [7, 20], "random"),
    "gqa2": (BASE.replace(batch=1, n_q_heads=16, ctx_lo=900, ctx_hi=900), [31], "random"),
    "one_node": (BASE.replace(batch=2, ctx_lo=500, ctx_hi=800), [1, 1], "random"),
    "most_nodes": (BASE.replace(batch=2, ctx_lo=500, ctx_hi=800), [128, 127], "random"),
    "most_nodes_gqa8": (synth.QWEN3_32B_128K.replace(batch=1, ctx_lo=777, ctx_hi=777), [128], "random"),
    "deep_chain": (BASE.replace(batch=1, ctx_lo=600, ctx_hi=600), [100], "chain"),
    "only_roots": (BASE.replace(batch=1, ctx_lo=600, ctx_hi=600), [40], "roots"),
    "star": (BASE.replace(batch=1, ctx_lo=600, ctx_hi=600), [40], "star"),
    "empty_context": (BASE.replace(batch=1, ctx_lo=0, ctx_hi=0), [10], "random"),
    "inside_sink": (BASE.replace(batch=2, ctx_lo=3, ctx_hi=40), [10, 30], "random"),
    "across_the_sink_edge": (BASE.replace(batch=1, ctx_lo=60, ctx_hi=60), [20], "random"),
    "windows_only": (BASE.replace(batch=1, ctx_lo=200, ctx_hi=200), [24], "random"),
    "partial_pages_flush1": (BASE.replace(batch=3, ctx_lo=340, ctx_hi=420, s_flush=1), [4, 9, 17], "random"),
    "odd_sink": (BASE.replace(batch=2, ctx_lo=500, ctx_hi=600, s_sink=5, s_keep=48), [11, 6], "random"),
    "quest": (BASE.replace(batch=1, ctx_lo=900, ctx_hi=900, quantizer="quest"), [12], "random"),
    "per_channel_keys": (synth.QWEN3_32B_128K.replace(batch=2, ctx_lo=500, ctx_hi=900, key_axis="channel"), [6, 14], "random"),
    "per_channel_plain": (BASE.replace(batch=1, ctx_lo=600, ctx_hi=600, key_axis="channel", s_flush=16, kappa_k=1.0), [21], "random"),
    # the same edges with trees wide enough for the tensor-core kernel
    "wide_short_contexts": (BASE.replace(batch=4, ctx_lo=0, ctx_hi=70), [40, 90, 128, 33], "random"),
    "wide_empty_contexts": (BASE.replace(batch=4, ctx_lo=0, ctx_hi=0), [17, 64, 128, 1], "random"),
    "wide_g32_l2": (synth.QWEN3_32B_128K.replace(batch=2, ctx_lo=500, ctx_hi=1500), [64, 100], "random"),
    "wide_g32_gqa1": (BASE.replace(batch=2, n_q_heads=8, ctx_lo=600, ctx_hi=700, group_size=32), [128, 101], "random"),
    "wide_g64_l2": (synth.QWEN3_32B_128K.replace(batch=2, ctx_lo=1030, ctx_hi=1030, group_size=64), [70, 40], "random"),
    "wide_g128_l2": (synth.QWEN3_32B_128K.replace(batch=2, ctx_lo=1030, ctx_hi=1030, group_size=128), [70, 40], "random"),
    "wide_flush1": (BASE.replace(batch=3, ctx_lo=340, ctx_hi=420, s_flush=1), [50, 40, 17], "random"),
    "wide_odd_sink": (BASE.replace(batch=2, ctx_lo=500, ctx_hi=600, s_sink=5, s_keep=48), [50, 31], "random"),
    "wide_quest": (BASE.replace(batch=2, ctx_lo=900, ctx_hi=900, quantizer="quest"), [42, 43], "random"),
    "wide_gqa2": (BASE.replace(batch=3, n_q_heads=16, ctx_lo=900, ctx_hi=1200), [60, 70, 80], "random"),
    "no_sink": (BASE.replace(batch=1, ctx_lo=333, ctx_hi=333, s_sink=0, s_keep=32), [7], "random"),
    "wide_no_sink": (BASE.replace(batch=2, ctx_lo=333, ctx_hi=420, s_sink=0, s_keep=32), [66, 40], "random"),
    "drafts_are_the_window": (BASE.replace(batch=1, ctx_lo=333, ctx_hi=333, s_sink=0, s_keep=0, s_flush=1), [7], "random"),
    "wide_drafts_are_the_window": (BASE.replace(batch=2, ctx_lo=333, ctx_hi=420, s_sink=0, s_keep=0, s_flush=1), [66, 40], "random"),
    "mid_context": (BASE.replace(batch=1, n_q_heads=8, n_kv_heads=2, ctx_lo=9000, ctx_hi=9000), [48], "random"),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_attn_tree(name):
    w, counts, kind = CASES[name]
    run, q, cu, parent = _drafted(w, counts, kind)
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    _compare(run, q, cu, parent, out, harness.units_sample(w, 6, seed=3))


def test_chain_equals_chunk_attention():
    w = BASE.replace(batch=2, ctx_lo=500, ctx_hi=900)
    run, q, cu, parent = _drafted(w, [30, 17], "chain")
    out = _call(run, q, cu, parent)
    r = run.runner
    ref = torch.empty(q.shape, dtype=torch.float32, device=run.device)
    r.attn_chunk(q, torch.from_numpy(cu).to(run.device), ref, r.chunk_workspace(q.shape[0]))
    torch.cuda.synchronize()
    assert int(r.status.item()) == 0
    err = (out.float() - ref).abs()
    # both within the parity tolerance of the same float64 result, and one bf16 rounding
    assert (err <= ref.abs() * 2.0 ** -8 + 2 * ATTN_TOL * ref.abs().amax(-1, keepdim=True)).all()


def test_same_call_twice_gives_the_same_bits_and_clean_counters():
    w = BASE.replace(batch=2, ctx_lo=1500, ctx_hi=3000, group_size=64)
    run, q, cu, parent = _drafted(w, [40, 23], "random")
    import bit_rotated_kv_gb300 as kvq
    n = kvq.kv_attn_tree_workspace_bytes(run.cfg, q.shape[0], int(run.runner.cache.seq_len.max()))
    ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=run.device)
    a = _call(run, q, cu, parent, ws)
    b = _call(run, q, cu, parent, ws)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_captured_and_replayed_on_another_stream():
    import bit_rotated_kv_gb300 as kvq
    w = BASE.replace(batch=1, ctx_lo=800, ctx_hi=800)
    run, q, cu, parent = _drafted(w, [20], "random")
    r, dev = run.runner, run.device
    first = _call(run, q, cu, parent)
    max_ctx = int(r.cache.seq_len.max())
    ws = torch.zeros(max(256, kvq.kv_attn_tree_workspace_bytes(r.cfg, 20, max_ctx)), dtype=torch.uint8, device=dev)
    cu_d, par_d, out = torch.from_numpy(cu).to(dev), torch.from_numpy(parent).to(dev), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.kv_attn_tree(r.cfg, r.cache, q, cu_d, par_d, out, r.sm_scale, max_ctx, ws, r.status, side)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    assert int(r.status.item()) == 0


@pytest.mark.parametrize("counts", [[6], [16, 20, 16, 30]], ids=["narrow", "wide"])
@pytest.mark.parametrize("side", ["k", "v"])
def test_a_draft_that_is_not_finite_reaches_the_nodes_that_see_it_only(counts, side):
    w = BASE.replace(batch=len(counts), ctx_lo=500, ctx_hi=700)
    run, q, cu, parent = _drafted(w, counts, "random", seed=5)
    r, cap = run.runner, run.cfg.ring_cap
    bad = 3                                          # node 3 of every sequence: one channel of one kv head
    ring = r.cache.ring_k if side == "k" else r.cache.ring_v
    before = ring.clone()
    for b, n in enumerate(counts):
        slot = (int(r.cache.seq_len[b]) - n + bad) % cap
        ring[b, 0, slot, 77] = float("inf") if b % 2 else float("nan")
    out = _call(run, q, cu, parent)
    assert int(r.status.item()) == 0
    ring.copy_(before)
    clean = _call(run, q, cu, parent)
    g = run.w.gqa
    for b, n in enumerate(counts):
        par = parent[int(cu[b]):int(cu[b + 1])]
        for i in range(n):
            at, sees = i, False
            while at >= 0:
                sees |= at == bad
                at = int(par[at])
            o, c = out[int(cu[b]) + i], clean[int(cu[b]) + i]
            assert torch.equal(o[g:], c[g:])         # the other kv heads
            if sees:
                # (an infinite key against a negative query is a score of -inf: the token has no weight)
                none = (q[int(cu[b]) + i, :g, 77] < 0) if side == "k" and b % 2 else torch.zeros(g, dtype=torch.bool, device="cuda")
                assert torch.equal(torch.isfinite(o[:g]), none[:, None].expand(g, 128))
            else:                                    # within both results' error
                tol = c[:g].float().abs() * 2.0 ** -7 + 2 * ATTN_TOL * c[:g].float().abs().amax(-1, keepdim=True)
                assert ((o[:g].float() - c[:g].float()).abs() <= tol).all()


@pytest.mark.parametrize("counts", [[6], [16, 20, 16, 30]], ids=["narrow", "wide"])
@pytest.mark.parametrize("factor", [1e20, 1e-20, float("inf"), float("nan")])
def test_queries_of_one_node_do_not_reach_the_others(counts, factor):
    w = BASE.replace(batch=len(counts), ctx_lo=500, ctx_hi=700)
    run, q, cu, parent = _drafted(w, counts, "random", seed=6)
    odd = [int(cu[b]) + 4 for b in range(len(counts))]   # node 4 of every sequence, two of its heads
    q[odd, 1::2] *= factor
    out = _call(run, q, cu, parent)
    assert int(run.runner.status.item()) == 0
    # the others against float64, and the odd rows where they are finite and small
    clean = q.clone()
    if factor != 1e-20:
        clean[odd] = 0
        out[odd] = _call(run, clean, cu, parent)[odd]
    _compare(run, clean, cu, parent, out, [(b, h) for b in range(len(counts)) for h in (0, 7)])


@pytest.mark.parametrize("counts", [[6], [40, 33]], ids=["narrow", "wide"])
def test_pages_beyond_4_gib(counts):
    w = BASE.replace(batch=len(counts), ctx_lo=900, ctx_hi=1100)
    run, q, cu, parent = _drafted(w, counts, "random")
    want = _call(run, q, cu, parent)
    c = run.runner.cache
    few = run.cfg.num_pages
    many = (5 << 30) // c.pages[0].numel() + few     # the same pages, at the far end of a pool of more than 5 GiB
    pool = torch.zeros((many, *c.pages.shape[1:]), dtype=torch.uint8, device=run.device)
    pool[many - few:] = c.pages
    run.cfg.num_pages, c.pages = many, pool
    c.page_table += torch.where(c.page_table >= 0, many - few, 0).to(torch.int32)
    assert torch.equal(_call(run, q, cu, parent).view(torch.int16), want.view(torch.int16))
    assert int(run.runner.status.item()) == 0


def test_one_workspace_serves_trees_of_any_size():
    """Calls of both kernels and of many sizes in turn: the tickets of each are as it needs them."""
    import bit_rotated_kv_gb300 as kvq
    runs = [_drafted(BASE.replace(batch=2, ctx_lo=ctx, ctx_hi=ctx + 300), counts, "random")
            for ctx, counts in ((500, [64, 30]), (500, [3, 2]), (3000, [1, 1]), (500, [40, 128]), (3000, [9, 9]), (900, [2, 5]))]
    sizes = [kvq.kv_attn_tree_workspace_bytes(r[0].cfg, r[1].shape[0], int(r[0].runner.cache.seq_len.max())) for r in runs]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    own = [_call(*r) for r in runs]
    for _ in range(2):
        for r, want in zip(runs, own):
            assert torch.equal(_call(*r, ws=ws).view(torch.int16), want.view(torch.int16))
            assert int(r[0].runner.status.item()) == 0


def test_rows_behind_the_last_sequence_are_left():
    w = BASE.replace(batch=1, ctx_lo=600, ctx_hi=600)
    run, q, cu, parent = _drafted(w, [9], "random")
    more = torch.cat([q, q[:3]])                     # rows that no sequence has
    par = np.concatenate([parent, np.full(3, -1, np.int32)])
    import bit_rotated_kv_gb300 as kvq
    out = _call(run, more, cu, par)
    assert int(run.runner.status.item()) == kvq.KVQ_ERR_BOUNDS
    _compare(run, q, cu, parent, out[:9], [(0, 0)])


def test_faults_are_reported():
    import bit_rotated_kv_gb300 as kvq
    w = BASE.replace(batch=2, ctx_lo=600, ctx_hi=700)
    run, q, cu, parent = _drafted(w, [9, 8], "random")
    r = run.runner
    # a node whose parent comes after it
    bad = parent.copy()
    bad[4] = 6
    _call(run, q, cu, bad)
    assert int(r.status.item()) == kvq.KVQ_ERR_BOUNDS
    r.status.zero_()
    # nodes that a flush has quantized: that sequence gets zeros, the other its result
    keep = r.cache.s_quant.clone()
    r.cache.s_quant[0] = r.cache.seq_len[0] - 4
    out = _call(run, q, cu, parent)
    assert int(r.status.item()) == kvq.KVQ_ERR_BOUNDS
    assert (out[:9] == 0).all()
    r.cache.s_quant.copy_(keep)
    _compare(run, q, cu, parent, out, [(1, 0), (1, 5)])
