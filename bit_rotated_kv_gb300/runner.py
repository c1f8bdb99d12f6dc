"""Drive the C-ABI calls for a batch of sequences: chunked prefill of the cache, one serving
step (append n_new tokens, flush, decode -- or the fused append, then decode), one speculative step
(a tree of drafts appended and attended to, checked, the kept path's rows left in the cache), the two
ends of a step (from the projections' rows, and from logits to tokens), and the page pool behind
them (reserve, fork, free, compact).  Argument marshalling only --
torch is used for device buffers, gathers of input rows and streams; every step of the
method runs in the library's kernels."""

from __future__ import annotations

import math

import numpy as np
import torch

from . import (KVQ_COUNT_OUTPUT, KVQ_COUNT_PROMPT, KVQ_TREE_MAX_NODES, KVCache, KVConfig, Transform, kv_append_chunk, kv_attn_chunk, kv_attn_chunk_workspace_bytes,
               kv_attn_decode, kv_attn_tree, kv_attn_tree_workspace_bytes, kv_logits_probs, kv_pages_compact,
               kv_pages_compact_workspace_bytes, kv_pages_reserve, kv_quant_flush, kv_rope_qk, kv_rotate_qk, kv_seq_fork, kv_seq_free,
               kv_token_counts, kv_tree_commit, kv_verify_tree, workspace)


def _rows_for(k_all: torch.Tensor, lengths_lo, lengths_hi):
    """Gather rows [lo_b, hi_b) of every sequence from k_all [B, T, H, d] into [rows, H, d]
    plus int32 seq_idx / pos on the same device."""
    idx_b, idx_t = [], []
    for b, (lo, hi) in enumerate(zip(lengths_lo, lengths_hi)):
        if hi > lo:
            idx_b.append(np.full(hi - lo, b, np.int64))
            idx_t.append(np.arange(lo, hi, dtype=np.int64))
    if not idx_b:
        return None, None
    ib = torch.from_numpy(np.concatenate(idx_b)).to(k_all.device)
    it = torch.from_numpy(np.concatenate(idx_t)).to(k_all.device)
    return ib, it


class DecodeRunner:
    """Owns one cache plus the scratch of a decode step.

    Calls go to ``stream`` (default: the current stream of ``device`` when the runner is
    made, resolved once); a method's own ``stream`` argument overrides it for that call."""

    def __init__(self, cfg: KVConfig, transform: Transform, max_ctx: int, device="cuda", stream=None):
        self.cfg = cfg
        self.tr = transform
        self.device = torch.device(device)
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        self.stream = int(getattr(stream, "cuda_stream", stream))
        self.cache = KVCache(cfg, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.max_ctx = int(max_ctx)
        self.ws = workspace(cfg, self.max_ctx, device)
        self.q_out = torch.empty((cfg.batch, cfg.n_q_heads, cfg.head_dim), dtype=torch.bfloat16,
                                 device=self.device)
        self.out = torch.empty((cfg.batch, cfg.n_q_heads, cfg.head_dim), dtype=torch.float32,
                               device=self.device)
        self.sm_scale = 1.0 / math.sqrt(cfg.head_dim)
        # the page pool: how many table entries hold each page (set_page_table counts them)
        self.page_ref = torch.zeros(cfg.num_pages, dtype=torch.int32, device=self.device)
        self.n_live = torch.zeros(1, dtype=torch.int32, device=self.device)
        # next_tokens: trees of one node, a sequence to a row (cu_rows, token and parent, path, n_accept)
        i32 = dict(dtype=torch.int32, device=self.device)
        self._ones = (torch.arange(cfg.batch + 1, **i32), torch.full((cfg.batch,), -1, **i32), torch.zeros(cfg.batch, **i32),
                      torch.zeros(cfg.batch, **i32))

    def set_page_table(self, table: np.ndarray) -> None:
        table = np.ascontiguousarray(table, np.int32)
        self.cache.page_table.copy_(torch.from_numpy(table))
        held = table[(table >= 0) & (table < self.cfg.num_pages)]
        self.page_ref.copy_(torch.from_numpy(np.bincount(held, minlength=self.cfg.num_pages).astype(np.int32)))

    def append(self, k_rows, v_rows, seq_idx, pos, q=None, q_out=None, stream=None) -> None:
        kv_rotate_qk(self.cfg, self.tr, q, q_out, k_rows, v_rows, seq_idx, pos, self.cache, self.status,
                     self.stream if stream is None else stream)

    def append_chunk(self, k_rows, v_rows, cu_rows, stream=None) -> None:
        """Rows cu_rows[b] .. cu_rows[b+1]-1 of k_rows / v_rows appended to sequence b, transformed
        and quantized on write in one pass (seq_len and s_quant advance)."""
        kv_append_chunk(self.cfg, self.tr, k_rows, v_rows, cu_rows, self.cache, self.status,
                        self.stream if stream is None else stream)

    def flush(self, max_tokens: int, stream=None) -> None:
        kv_quant_flush(self.cfg, self.cache, max_tokens, self.status, self.stream if stream is None else stream)

    def decode(self, q_rot, out, stream=None) -> None:
        kv_attn_decode(self.cfg, self.cache, q_rot, out, self.sm_scale, self.max_ctx, self.ws, self.status,
                       self.stream if stream is None else stream)

    def chunk_workspace(self, n_rows: int) -> torch.Tensor:
        """A zeroed workspace for kv_attn_chunk over n_rows query rows."""
        n = kv_attn_chunk_workspace_bytes(self.cfg, n_rows, self.max_ctx)
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=self.device)

    def attn_chunk(self, q_rot, cu_rows, out, ws, stream=None) -> None:
        """Causal attention of chunk query rows q_rot [n, Hq, d] over the cache (after their
        tokens were appended) into out [n, Hq, d] float32."""
        kv_attn_chunk(self.cfg, self.cache, q_rot, cu_rows, out, self.sm_scale, self.max_ctx, ws, self.status,
                      self.stream if stream is None else stream)

    def prefill(self, k_all: torch.Tensor, v_all: torch.Tensor, lengths, chunk: int) -> None:
        """Append tokens [0, lengths[b]) of k_all / v_all [B, T, Hkv, d] (bf16, device) in chunks,
        flushing after each chunk."""
        lengths = [int(x) for x in lengths]
        T = max(lengths) if lengths else 0
        for c0 in range(0, T, chunk):
            lo = [min(c0, L) for L in lengths]
            hi = [min(c0 + chunk, L) for L in lengths]
            ib, it = _rows_for(k_all, lo, hi)
            if ib is None:
                continue
            k = k_all[ib, it].contiguous()
            v = v_all[ib, it].contiguous()
            self.append(k, v, ib.to(torch.int32), it.to(torch.int32))
            self.flush(chunk + self.cfg.s_flush)

    def step_inputs(self, k_all, v_all, ctx, n_new: int):
        """(k_rows, v_rows, seq_idx, pos) of the n_new tokens after ctx[b] of every sequence."""
        ctx = [int(x) for x in ctx]
        ib, it = _rows_for(k_all, ctx, [c + n_new for c in ctx])
        return (k_all[ib, it].contiguous(), v_all[ib, it].contiguous(), ib.to(torch.int32),
                it.to(torch.int32))

    def step_fused(self, q, k_rows, v_rows, cu_rows, stream=None) -> None:
        """The same serving step with the appended chunk transformed and quantized in one pass:
        append, rotate the queries, decode."""
        self.append_chunk(k_rows, v_rows, cu_rows, stream)
        kv_rotate_qk(self.cfg, self.tr, q, self.q_out, None, None, None, None, self.cache, self.status,
                     self.stream if stream is None else stream)
        self.decode(self.q_out, self.out, stream)

    def step(self, q, k_rows, v_rows, seq_idx, pos, n_new: int, stream=None) -> None:
        """One serving step: rotate the new rows and the queries, flush, decode."""
        self.append(k_rows, v_rows, seq_idx, pos, q, self.q_out, stream)
        self.flush(n_new + self.cfg.s_flush, stream)
        self.decode(self.q_out, self.out, stream)

    # ---- from the projections' rows ----------------------------------------------------------------
    def rope_append(self, rope, k_rows, v_rows, seq_idx, pos, q=None, q_out=None, q_pos=None, rope_pos=None, stream=None) -> None:
        """append for rows as the projections leave them (views of one fused tensor do): norm of the heads, rotation by
        position, transform, write.  q_pos, rope_pos: positions in the text (rope_pos None: pos)."""
        kv_rope_qk(self.cfg, self.tr, rope, q, q_out, q_pos, k_rows, v_rows, seq_idx, pos, rope_pos, self.cache, self.status,
                   self.stream if stream is None else stream)

    def rope_step(self, rope, q, k_rows, v_rows, seq_idx, pos, q_pos, n_new: int, stream=None) -> None:
        """step for such rows: q_pos [batch] is each sequence's newest position."""
        self.rope_append(rope, k_rows, v_rows, seq_idx, pos, q, self.q_out, q_pos, None, stream)
        self.flush(n_new + self.cfg.s_flush, stream)
        self.decode(self.q_out, self.out, stream)

    # ---- from logits to tokens -----------------------------------------------------------------------
    def next_tokens(self, rules, logits, p, u, next_token, stream=None) -> None:
        """A token for every sequence (next_token [batch]) from its row of logits [batch, vocab] under `rules` and a uniform
        number u [batch]; p [batch, vocab] holds the probabilities, and rules.counts, where given, counts the tokens."""
        stream = self.stream if stream is None else stream
        cu, root, path, n_accept = self._ones
        kv_logits_probs(self.cfg, rules, logits, cu, None, None, p, self.status, stream)
        kv_verify_tree(self.cfg, cu, root, path, p, None, u, path, n_accept, next_token, self.status, stream)
        if rules is not None and rules.counts is not None:
            kv_token_counts(self.cfg, rules.counts, logits.shape[1], KVQ_COUNT_OUTPUT, None, None, None, None, next_token, self.status, stream)

    def accept_logits(self, rules, cu_rows, parent, token, logits, p, q, u, path, n_accept, next_token, max_nodes: int,
                      stream=None) -> None:
        """accept from the target's logits [n, vocab] under `rules`, every node's by the penalties of its own path; p [n, vocab]
        holds the probabilities (for float32 logits it may be the logits), and rules.counts, where given, counts the tokens kept."""
        stream = self.stream if stream is None else stream
        kv_logits_probs(self.cfg, rules, logits, cu_rows, parent, token, p, self.status, stream)
        self.accept(cu_rows, parent, token, p, q, u, path, n_accept, next_token, max_nodes, stream)
        if rules is not None and rules.counts is not None:
            kv_token_counts(self.cfg, rules.counts, logits.shape[1], KVQ_COUNT_OUTPUT, cu_rows, token, path, n_accept, next_token,
                            self.status, stream)

    def count_prompts(self, counts, vocab: int, cu_rows, token, stream=None) -> None:
        """Rows cu_rows[b] .. cu_rows[b+1]-1 of token are sequence b's prompt (its row of counts zeroed by the caller)."""
        kv_token_counts(self.cfg, counts, vocab, KVQ_COUNT_PROMPT, cu_rows, token, None, None, None, self.status,
                        self.stream if stream is None else stream)

    # ---- speculative decoding: tree_step, then accept --------------------------------------------
    def tree_workspace(self, n_rows: int) -> torch.Tensor:
        """A zeroed workspace for trees of up to n_rows nodes in all."""
        n_rows = max(1, min(n_rows, self.cfg.batch * KVQ_TREE_MAX_NODES, 65535))
        n = kv_attn_tree_workspace_bytes(self.cfg, n_rows, self.max_ctx)
        return torch.zeros(max(n, 256), dtype=torch.uint8, device=self.device)

    def tree_step(self, q, k_rows, v_rows, seq_idx, pos, cu_rows, parent, q_out, out, ws, stream=None, rope=None,
                  rope_pos=None) -> None:
        """Append the drafted nodes (row cu_rows[b] + i is node i of sequence b, at position length + i)
        and attend from each to the tokens before the drafts, its ancestors and itself: out [n, Hq, d] bf16.
        With rope the rows are the projections': rope_pos [n] is each node's position in the text, length + depth."""
        if rope is None:
            self.append(k_rows, v_rows, seq_idx, pos, q, q_out, stream)
        else:
            self.rope_append(rope, k_rows, v_rows, seq_idx, pos, q, q_out, rope_pos, rope_pos, stream)
        kv_attn_tree(self.cfg, self.cache, q_out, cu_rows, parent, out, self.sm_scale, self.max_ctx, ws, self.status,
                     self.stream if stream is None else stream)

    def accept(self, cu_rows, parent, token, p, q, u, path, n_accept, next_token, max_nodes: int, stream=None) -> None:
        """Check the drafts against the target's probabilities p (q: the draft's, or None), keep the rows of
        the path that holds, drop the others, and flush."""
        stream = self.stream if stream is None else stream
        kv_verify_tree(self.cfg, cu_rows, parent, token, p, q, u, path, n_accept, next_token, self.status, stream)
        self.commit(cu_rows, path, n_accept, max_nodes, stream)

    def commit(self, cu_rows, path, n_accept, max_nodes: int, stream=None) -> None:
        """Keep the rows of the given paths only (every layer's cache takes the same ones), and flush."""
        kv_tree_commit(self.cfg, self.cache, cu_rows, path, n_accept, self.status, self.stream if stream is None else stream)
        self.flush(max_nodes + self.cfg.s_flush, stream)

    # ---- the page pool -----------------------------------------------------------------------------
    def reserve(self, n_tokens, stream=None) -> None:
        """Pages for n_tokens[b] (device int32 [batch]) more tokens of every sequence."""
        kv_pages_reserve(self.cfg, self.cache, self.page_ref, n_tokens, self.status, self.stream if stream is None else stream)

    def fork(self, src, dst, stream=None) -> None:
        """Sequence dst[i] becomes a copy of src[i] (device int32 [n]); whole INT2 pages are shared."""
        kv_seq_fork(self.cfg, self.cache, self.page_ref, src, dst, self.status, self.stream if stream is None else stream)

    def free(self, seqs, stream=None) -> None:
        """Sequences seqs (device int32 [n]) give up their pages and become empty."""
        kv_seq_free(self.cfg, self.cache, self.page_ref, seqs, self.status, self.stream if stream is None else stream)

    def compact_workspace(self) -> torch.Tensor:
        return torch.zeros(max(256, kv_pages_compact_workspace_bytes(self.cfg)), dtype=torch.uint8, device=self.device)

    def compact(self, ws, stream=None) -> torch.Tensor:
        """Move the held pages to the front of the pool; their number is in the device tensor returned."""
        kv_pages_compact(self.cfg, self.cache, self.page_ref, self.n_live, ws, self.status,
                         self.stream if stream is None else stream)
        return self.n_live
