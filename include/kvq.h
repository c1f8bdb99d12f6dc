/*
 * kvq.h -- C ABI of the rotated INT2 paged KV cache for GB300 (sm_103a).
 *
 * Three calls make up the serving hot path shared by the methods on these pages:
 *   [OSCAR] "OSCAR: Offline Spectral Covariance-Aware Rotation for 2-bit KV Cache
 *           Quantization" (paperlayer summary)
 *   [OScaR] "OScaR: The Occam's Razor for Extreme KV Cache Quantization in LLMs and
 *           Beyond" (reading note, in Chinese)
 *   [WUSH]  "WUSH-KV: KV Cache Quantization with Data-Adaptive Transforms" (digest)
 *
 *   kv_rotate_qk    fixed per-head transform of new keys/values on write and the
 *                   matching compensation of queries ([WUSH] core method and
 *                   inference algorithm; [OScaR] step 1 "Canalized Rotation";
 *                   [OSCAR] section 3 "Online Deployment").
 *   kv_quant_flush  quantize-on-write of the BF16 tokens that left the recent
 *                   window into INT2 pages ([WUSH] inference algorithm, S_flush
 *                   spans; [OSCAR] section 4 "KV Cache Update"; [OScaR] step 2
 *                   "Omni-Token Scaling" and the integer-quantization basics).
 *   kv_attn_decode  GQA decode attention reading the mixed BF16 / INT2 cache
 *                   directly ([OSCAR] section 4 "Decoding Attention Kernel";
 *                   [OScaR] "系统设计与 CUDA 实现"; [WUSH] GQA background).
 *   kv_attn_chunk   causal attention of a chunk's queries over the same cache
 *                   (the prefill path; [WUSH] inference algorithm).
 *   kv_append_chunk the first two fused for a prefill chunk: transform on write
 *                   and quantize-on-write in one pass, rows bound for INT2 never
 *                   written as BF16 ([OScaR] "系统设计与 CUDA 实现", key-quant
 *                   kernel; [OSCAR] section 4 "KV Cache Update").
 *
 * and, for speculative decoding and a shared page pool next to them,
 *
 *   kv_attn_tree, kv_verify_tree, kv_tree_commit
 *                   attention of a tree of drafted tokens over the cache, the check of
 *                   the drafts against the target's probabilities, and the rows kept.
 *   kv_pages_reserve, kv_seq_fork, kv_seq_free, kv_pages_compact
 *                   pages handed out, shared by sequences, given back and made dense.
 *
 * and, for the two ends of a step, from the projections' rows and to the tokens,
 *
 *   kv_rope_qk      head norm, rotary positions, transform and append in one call.
 *   kv_logits_probs penalties, biases, a grammar's mask and the temperature on logits: the
 *                   probabilities that kv_verify_tree takes.
 *   kv_token_counts what the penalties go by: the tokens each sequence holds.
 *
 * Conventions shared by every call
 *   - Every pointer inside a struct or argument is a DEVICE pointer unless said
 *     otherwise; the structs themselves live in host memory and are read during
 *     the call only.  The caller allocates, owns and frees every buffer; the
 *     library never allocates, frees, synchronizes, or keeps a pointer after it
 *     returns.
 *   - bf16 values are passed as uint16_t bit patterns; float16 scale data as
 *     uint16_t bit patterns.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).
 *   - Return value: KVQ_OK, or a negative KVQ_ERR_* code for a fault found on
 *     the host before anything is launched (bad argument, unsupported shape,
 *     CUDA launch error).
 *   - Faults found on the device (a page id or position out of range, a
 *     non-finite scale, a bounded wait that ran out) never trap: the offending
 *     unit of work is skipped and the first such code is stored into
 *     *d_status (a device int32 the caller zeroes and reads when it likes).
 *   - Overlap between consecutive calls: every kernel lets the next kernel of the
 *     stream begin early (programmatic dependent launch) and waits for the kernel
 *     before it -- the caller's or this library's -- to complete before it reads a
 *     per-call input (q, k, v, seq_idx, pos, cu_rows) or touches the cache state.
 *     Configuration is read before that wait: the transform matrices (kv_rotate_qk,
 *     kv_append_chunk, kv_rope_qk) and the page table (kv_attn_decode, kv_attn_chunk).  These
 *     must not be written by the kernel launched immediately before the call on
 *     the same stream; a copy, or any earlier kernel, may write them.
 *
 * Supported shapes: head_dim 128; page_size 16; group_size 32, 64 or 128;
 * GQA ratio Hq/Hkv in {1, 2, 4, 8}; 2-bit codes.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------- */
#define KVQ_OK                 0
#define KVQ_ERR_INVALID_ARG   (-1)  /* null pointer, inconsistent sizes, bad enum          */
#define KVQ_ERR_UNSUPPORTED   (-2)  /* valid but not implemented (head_dim, G, GQA ratio)  */
#define KVQ_ERR_CUDA          (-3)  /* a CUDA runtime call or launch failed                */
#define KVQ_ERR_BOUNDS        (-4)  /* device: page id / position / ring slot out of range */
#define KVQ_ERR_NONFINITE     (-5)  /* device: a scale, zero point, norm, value, logit or probability is not finite */
#define KVQ_ERR_TIMEOUT       (-6)  /* device: a bounded wait on an async copy ran out     */
#define KVQ_ERR_WORKSPACE     (-7)  /* workspace smaller than kv_attn_workspace_bytes()    */

/* ---- enums ----------------------------------------------------------------- */
#define KVQ_QUANT_AFFINE_KAPPA 0  /* kappa-quantile clipped asymmetric affine (OSCAR / WUSH) */
#define KVQ_QUANT_QUEST_RMS    1  /* QuEST RMS grid: Delta = 2 alpha rms / 3, z = 1.5 (WUSH) */

#define KVQ_KEY_PER_TOKEN      0  /* keys: Delta, z per token and group of G channels (OSCAR / WUSH) */
#define KVQ_KEY_PER_CHANNEL    1  /* keys: Delta, z per channel and 16-token page (KIVI, OScaR)     */

#define KVQ_TRANSFORM_DENSE    0  /* dense per-head float32 matrices T_K, T_K^{-T}, T_V       */
#define KVQ_TRANSFORM_HADAMARD 1  /* normalised Walsh-Hadamard on keys and queries (OScaR)    */

/* ---- configuration ----------------------------------------------------------
 * One POD struct, passed to every call (the pages' hyper-parameters plus shapes).
 * kappa: the quantile level of the clipping range, in [0.5, 1]; the group range
 * is [(1-kappa)-quantile, kappa-quantile] of the group's own values with linear
 * interpolation; kappa = 1 is min/max.  Windows: tokens [0, s_sink) stay BF16,
 * tokens [s_quant, L) are the BF16 recent window, [s_sink, s_quant) is INT2; the
 * flush rule quantizes [s_quant, s_quant + s_flush) while L - s_quant >= s_keep +
 * s_flush.  ring_cap: capacity of the BF16 recent ring in tokens (a multiple of
 * page_size; at least s_keep + s_flush + the most tokens appended between two
 * flushes).  attn_splits: INT2 splits per (sequence, kv head) in kv_attn_decode
 * (0 = automatic).  key_axis: KVQ_KEY_PER_TOKEN quantizes each key like each value,
 * per token and group of G channels; KVQ_KEY_PER_CHANNEL quantizes keys per channel
 * over the 16 tokens of a page -- KIVI's blocks along the token axis, the range of
 * channel j being the kappa-quantile range of its 16 values ([OScaR] "背景：KIVI 与逐通道
 * 量化范式" and algorithm, key processing) -- after the l2 scaling when key_l2norm;
 * it needs the AFFINE_KAPPA quantizer and s_flush a multiple of 16 (every flush then
 * quantizes whole pages; KVQ_ERR_UNSUPPORTED otherwise).  Values are per token either
 * way. */
typedef struct kvq_config {
  int32_t head_dim;          /* d  (128)                               */
  int32_t n_q_heads;         /* Hq                                     */
  int32_t n_kv_heads;        /* Hkv; query head hq reads kv head hq / (Hq/Hkv) */
  int32_t page_size;         /* P  (16 tokens per page)                */
  int32_t group_size;        /* G  (32, 64, 128 channels per group)    */
  int32_t quantizer;         /* KVQ_QUANT_*                            */
  int32_t key_l2norm;        /* 1: keys are l2-scaled after the transform, norm kept as float16 */
  int32_t s_sink;            /* BF16 sink tokens                       */
  int32_t s_keep;            /* BF16 recent tokens kept after a flush  */
  int32_t s_flush;           /* tokens quantized per flush span        */
  int32_t ring_cap;          /* BF16 recent ring capacity (tokens)     */
  int32_t batch;             /* B: sequences                           */
  int32_t max_pages_per_seq; /* columns of the page table              */
  int32_t num_pages;         /* physical pages in the pool             */
  int32_t attn_splits;       /* 0 = automatic                          */
  int32_t key_axis;          /* KVQ_KEY_PER_*                          */
  double  kappa_k;           /* key clipping quantile                  */
  double  kappa_v;           /* value clipping quantile                */
  double  quest_alpha;       /* QuEST clip in RMS units                */
} kvq_config;

/* ---- the cache ----------------------------------------------------------------
 * All device memory, owned by the caller.
 *
 * pages      [num_pages][Hkv][kvq_page_head_bytes(cfg)] bytes.  Logical INT2 page
 *            p of sequence b holds tokens [s_sink + 16p, s_sink + 16p + 16) and
 *            lives in physical page page_table[b * max_pages_per_seq + p].  One
 *            (page, kv head) chunk, tokens t = 0..15 of the page:
 *              [0, 512)      key codes in MMA-fragment order: u32 word 4*l + r
 *                            (l = 0..31, r = 0..3) holds token (l/4) + 8*(r%2);
 *                            its bits 2s and 16+2s (s = 0..7) hold the codes of
 *                            channels 16s + 2*(l%4) + 8*(r/2) + e, e = 0 / 1.
 *              [512, 1024)   value codes in MMA-fragment order: u32 word 4*l + r,
 *                            bits 2m + 16e (m = 0..7) hold the code of channel
 *                            16m + (l/4) + 8*(r%2) of token 2*(l%4) + 8*(r/2) + e.
 *              [1024, ...)   key scales: KVQ_KEY_PER_TOKEN: (Delta16, z16) float16
 *                            pairs [16 tokens][d/G] (64 d/G bytes); KVQ_KEY_PER_CHANNEL:
 *                            Delta16 [256 bytes] then z16 [256 bytes], each 64 u32
 *                            pairs, pair 16 q + 2 s + h holding channels
 *                            16 s + 8 h + 2 q and + 1 (the B-fragment order of the
 *                            decode's MMAs: q = 0..3, s = 0..7, h = 0..1); then
 *                            value Delta16 [8 token pairs][d/G][2] and value z16
 *                            [8 token pairs][d/G][2] (token t at pair t/2, slot t%2);
 *                            then (only when key_l2norm) key norms s16 float16 [16];
 *                            then (KVQ_KEY_PER_CHANNEL only) int32 E: the binary
 *                            exponent of the page's largest key Delta16 (at least -14);
 *                            the chunk is padded to a multiple of 32 bytes.
 *            Token t dequantizes as x_hat_c = s16 * Delta16 * (code_c - z16), with
 *            s16 = 1 without key_l2norm ([OScaR] step 2 dequantisation), Delta16 and
 *            z16 those of its group or, for per-channel keys, of channel c.
 * page_table [B][max_pages_per_seq] int32 physical page ids (-1 = none).
 * seq_len    [B] int32 tokens in each sequence; kv_rotate_qk raises it to
 *            pos + 1 for every row it writes.
 * s_quant    [B] int32 right edge of the INT2 region; must start at s_sink;
 *            kv_quant_flush advances it.
 * sink_k/v   [B][Hkv][s_sink][d] bf16 rows of tokens 0 .. s_sink-1.
 * ring_k/v   [B][Hkv][ring_cap][d] bf16; token t >= s_sink lives in slot t % ring_cap
 *            while it is in the recent window.
 * counters   [B] int32, zero before the first call; every call leaves it zero.
 */
typedef struct kvq_cache {
  void*          pages;
  const int32_t* page_table;
  int32_t*       seq_len;
  int32_t*       s_quant;
  uint16_t*      sink_k;
  uint16_t*      sink_v;
  uint16_t*      ring_k;
  uint16_t*      ring_v;
  int32_t*       counters;
} kvq_cache;

/* ---- the per-head transforms (device pointers, float32, row-major) -----------
 * DENSE:    k' = T_K k, q' = T_K^{-T} q (so q'^T k' = q^T k for any invertible
 *           T_K; for orthogonal T_K pass T_K itself), v' = T_V v (t_v NULL: values
 *           are stored unchanged, T_V folded into the projection weights).
 *           t_k, t_k_inv_t, t_v: [Hkv][d][d], element (i, j) at i*d + j.
 * HADAMARD: k' = H k, q' = H q with the normalised Walsh-Hadamard matrix (entries
 *           +-1/sqrt(d)); t_k and t_k_inv_t are ignored; t_v as for DENSE.
 * Every output row is the exact product rounded once to bf16 (nearest-even). */
typedef struct kvq_transform {
  int32_t      kind;         /* KVQ_TRANSFORM_* */
  int32_t      reserved;
  const float* t_k;
  const float* t_k_inv_t;
  const float* t_v;
} kvq_transform;

/* Bytes of one (page, kv head) chunk, and of one physical page (all kv heads). */
KVQ_API size_t kvq_page_head_bytes(const kvq_config* cfg);
KVQ_API size_t kvq_page_bytes(const kvq_config* cfg);

/* kv_rotate_qk: transform new rows on write, compensate queries on read.
 *   q        [n_q_rows][Hq][d] bf16 queries (may be NULL when n_q_rows == 0)
 *   q_out    [n_q_rows][Hq][d] bf16: q' (query head hq uses kv head hq/(Hq/Hkv))
 *   k, v     [n_kv_rows][Hkv][d] bf16 new keys / values (NULL when n_kv_rows == 0)
 *   seq_idx  [n_kv_rows] int32 sequence of each row; pos [n_kv_rows] int32 token
 *            position.  Row r goes to the sink (pos < s_sink) or to ring slot
 *            pos % ring_cap; pos must satisfy s_quant[b] <= pos < s_quant[b] +
 *            ring_cap for pos >= s_sink, otherwise the row is skipped with
 *            KVQ_ERR_BOUNDS in *d_status.  seq_len[b] is raised to pos + 1.
 * q, k, v and the matrices must be 16-byte aligned, q_out 8-byte aligned
 * (KVQ_ERR_INVALID_ARG otherwise).
 * Execution: one kernel for decode-sized calls.  From 19,456 dense (row, head) pairs on
 * (about one 128-row block per SM) the dense rows run on the tensor cores and the copies /
 * Hadamard rows in a second kernel launched first; the outputs are bit-identical either way
 * (see kvq_selftest_tc_integer_sums for the one hardware property that path relies on).
 * Source: [WUSH] inference algorithm (transform each new key and query, append at
 * full precision); [OScaR] algorithm, key and query processing (online FHT of K and Q). */
KVQ_API int kv_rotate_qk(const kvq_config* cfg, const kvq_transform* tr,
                 const uint16_t* q, uint16_t* q_out, int32_t n_q_rows,
                 const uint16_t* k, const uint16_t* v,
                 const int32_t* seq_idx, const int32_t* pos, int32_t n_kv_rows,
                 const kvq_cache* cache, int32_t* d_status, void* stream);

/* kv_quant_flush: apply the flush rule to every sequence: while seq_len - s_quant
 * >= s_keep + s_flush, quantize tokens [s_quant, s_quant + s_flush) of every kv
 * head from the BF16 ring into their INT2 page and advance s_quant.  At most
 * min(max_tokens_per_seq, ring_cap - s_keep) tokens (rounded down to whole
 * spans) are quantized per sequence by one call; the rest wait for the next call
 * (the ring never holds more than ring_cap - s_keep tokens past S_keep).  Per token (all float
 * operations IEEE round-to-nearest, none fused):
 *   key_l2norm (keys only): s = sqrt(sum x^2) in float64, s16 = fp16(s),
 *     y = x / s16 in float32 (y = 0 when s16 = 0);
 *   per group of G values, AFFINE_KAPPA: sorted a[], pos = (G-1)*kappa in float64,
 *     i = floor(pos), f = fp32(pos - i), hi = a[i] + f*(a[i+1] - a[i]) (a[G-1] when
 *     i = G-1), lo likewise at (G-1)*(1-kappa); Delta = (hi - lo)/3,
 *     Delta16 = fp16(Delta) (1 if it rounds to 0), z16 = fp16(-(lo / Delta16));
 *   QUEST_RMS: rms = sqrt(sum y^2 / G) in float64, Delta16 = fp16(2*alpha*rms/3)
 *     (1 if 0), z16 = 1.5 (not combined with key_l2norm);
 *   code = clamp(round_half_even(y / Delta16 + z16), 0, 3).
 * Source: [WUSH] inference algorithm (S_quant, S_flush-aligned spans, per-group
 * quantizer in place); [OSCAR] section 4 "KV Cache Update"; [OScaR] algorithm,
 * key processing (norm, residual buffer quantized when full) and the
 * integer-quantization formulas. */
KVQ_API int kv_quant_flush(const kvq_config* cfg, const kvq_cache* cache, int32_t max_tokens_per_seq,
                   int32_t* d_status, void* stream);

/* kv_append_chunk: append a chunk of new tokens to every sequence -- the effect of
 * kv_rotate_qk on those rows followed by kv_quant_flush, in one pass.
 *   k, v     [n_rows][Hkv][d] bf16 new keys / values (16-byte aligned; NULL when
 *            n_rows == 0)
 *   cu_rows  [B + 1] int32 (device): the rows of sequence b are cu_rows[b] ..
 *            cu_rows[b+1] - 1, in token order; cu_rows[0] = 0 and cu_rows[B] =
 *            n_rows (rows outside [cu_rows[0], cu_rows[B]) are skipped with
 *            KVQ_ERR_BOUNDS).  A sequence may append no rows.
 * Row r of sequence b gets position p = seq_len[b] + r - cu_rows[b]; seq_len[b]
 * then advances by cu_rows[b+1] - cu_rows[b], and the flush rule of
 * kv_quant_flush runs on the advanced length with no cap (s_quant advances by
 * whole S_flush spans while seq_len - s_quant >= s_keep + s_flush).  Keys are
 * transformed by T_K (DENSE only: KVQ_ERR_UNSUPPORTED for HADAMARD), values by T_V
 * or copied.  A row with p < s_sink goes to the sink, one below the new s_quant is
 * quantized straight into its INT2 page (as kv_quant_flush would), the others go
 * to their ring slot; tokens already in the ring that the new s_quant passes are
 * quantized from the ring.  Every byte written -- pages, sink and ring rows,
 * seq_len, s_quant -- equals what kv_rotate_qk at those positions followed by
 * kv_quant_flush (max_tokens_per_seq large enough) writes; the ring only has to
 * hold the tokens that stay in the window, not the whole chunk.
 * Execution: three kernels (flush of the ring tokens, copied rows, dense rows on
 * the tensor cores); meant for prefill-sized chunks (decode-sized appends are
 * cheaper through kv_rotate_qk + kv_quant_flush).
 * Source: [OScaR] "系统设计与 CUDA 实现" (key-quant kernel: transform, scaling and
 * INT2 packing on chip, input read once, codes written once); [OSCAR] section 4
 * "KV Cache Update" (fused prefill clip + quantize); [WUSH] inference algorithm. */
KVQ_API int kv_append_chunk(const kvq_config* cfg, const kvq_transform* tr,
                    const uint16_t* k, const uint16_t* v, const int32_t* cu_rows, int32_t n_rows,
                    const kvq_cache* cache, int32_t* d_status, void* stream);

/* kv_attn_chunk: attention of the queries of an appended chunk (the prefill path) over the
 * cache as it stands after the append.
 *   q_rot    [n_rows][Hq][d] bf16 compensated queries (kv_rotate_qk output), row r of
 *            sequence b for cu_rows[b] <= r < cu_rows[b+1] (the layout of kv_append_chunk)
 *   cu_rows  [B + 1] int32 (device): rows of sequence b; row r sits at position
 *            p = seq_len[b] - (cu_rows[b+1] - r), i.e. the rows are the last tokens of the
 *            sequence, in order (rows outside [cu_rows[0], cu_rows[B]) get KVQ_ERR_BOUNDS)
 *   out      [n_rows][Hq][d] float32
 * Row r attends causally to tokens [0, p] as the cache holds them: BF16 sink rows, INT2
 * tokens below min(s_quant, p + 1) dequantized, BF16 ring rows from s_quant to p -- the
 * result of kv_attn_decode for a sequence whose length were p + 1.  max_ctx bounds seq_len as
 * for kv_attn_decode; n_rows is at most 65535 (KVQ_ERR_UNSUPPORTED beyond); workspace of
 * kv_attn_chunk_workspace_bytes(cfg, n_rows, max_ctx) bytes, zero-filled before its first use
 * (every call leaves its ticket counters zero).
 * Execution: the decode kernel with one grid row per query row, so each query streams its own
 * prefix of the cache (L2 keeps a sequence's pages between the rows that share them).
 * Source: [WUSH] inference algorithm (mixed-precision attention over the S_sink / S_keep windows
 * and the INT2 middle); [OSCAR] section 4 "Decoding Attention Kernel" (BF16 and INT2 segments
 * of one attention). */
KVQ_API size_t kv_attn_chunk_workspace_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx);
KVQ_API int kv_attn_chunk(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                  const int32_t* cu_rows, int32_t n_rows, float* out, float sm_scale, int32_t max_ctx,
                  void* workspace, size_t ws_bytes, int32_t* d_status, void* stream);

/* ---- speculative decoding ------------------------------------------------------
 * A draft proposes a tree of tokens per sequence; the target model scores all of them in
 * one pass and the longest path that survives its probabilities is kept.  One step:
 *   kv_rotate_qk    the drafts' rows at positions seq_len + i (i = 0 .. n-1 in index order;
 *                   RoPE, which the caller applies, uses a node's depth, the slot does not),
 *                   and their queries
 *   kv_attn_tree    every layer's attention
 *   kv_verify_tree  from the target's probabilities at every node
 *   kv_tree_commit  every layer's cache: the accepted rows stay, the others go
 *   kv_quant_flush  as after any append
 * No flush may run between the append and the commit: the drafts are BF16 rows of the window,
 * so ring_cap must hold them as well.
 *
 * The tree: cu_rows [B + 1] as for kv_append_chunk; row cu_rows[b] + i is node i of sequence b;
 * parent [n_rows] int32 holds each node's parent, local to its sequence and smaller than the
 * node's own index, or -1 for a root.  At most KVQ_TREE_MAX_NODES nodes per sequence. */
#define KVQ_TREE_MAX_NODES 128

/* kv_attn_tree: attention of a tree of drafted tokens.
 *   q_rot    [n_rows][Hq][d] bf16 compensated queries (kv_rotate_qk output)
 *   cu_rows, parent: the tree (above); the nodes are the last n tokens of their sequence
 *   out      [n_rows][Hq][d] bf16 (16-byte aligned): the float32 result rounded once
 * Node i of sequence b, with L0 = seq_len[b] - n, attends to tokens [0, L0), to its ancestors
 * (token L0 + j for node j) and to itself, as the cache holds them.  A chain (parent i - 1) gives
 * kv_attn_chunk's result; several roots are allowed.  max_ctx, sm_scale as for kv_attn_decode
 * (max_ctx counts the nodes); workspace of kv_attn_tree_workspace_bytes(cfg, n_rows, max_ctx)
 * bytes, zero-filled before its first use (every call leaves its counters zero).  That size is enough for every
 * call of up to n_rows rows and max_ctx tokens with the same config, one after another (it does not shrink as they
 * grow; 0 for sizes that are refused); calls that may run at the same time need a workspace each.  n_rows is at most 65535 (KVQ_ERR_UNSUPPORTED beyond)
 * and batch * KVQ_TREE_MAX_NODES (KVQ_ERR_INVALID_ARG).  KVQ_ERR_BOUNDS in *d_status, and zeros for
 * the rows of a sequence whose nodes are more than KVQ_TREE_MAX_NODES or do not all lie in the BF16
 * windows; a node whose ancestors are not in index order is reported and sees those up to the fault.
 * Rows behind the last sequence are not written (KVQ_ERR_BOUNDS when cu_rows does not cover n_rows).  A
 * draft whose K or V is not finite changes the rows of the nodes that see it, and only those.
 * An INT2 value beyond fp16's 65504 is more than the tensor-core kernel (below) can hold: it reports
 * KVQ_ERR_NONFINITE, as for a value before the drafts that is not finite, and the results are not finite.
 * Execution: trees of up to about 32 columns (nodes x query heads per kv head), and small calls, run the
 * decode kernel with eight columns to a grid row; wider ones a tensor-core kernel that reads a
 * sequence's cache once for every 64 columns.  The two round differently (both within the attention's
 * error); which one runs follows from cfg, n_rows and max_ctx alone.
 * Source: [OSCAR] section 4 "Decoding Attention Kernel" (attention over the mixed cache);
 * the tree of drafts has no counterpart on the pages. */
KVQ_API size_t kv_attn_tree_workspace_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx);
KVQ_API int kv_attn_tree(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                 const int32_t* cu_rows, const int32_t* parent, int32_t n_rows, uint16_t* out, float sm_scale,
                 int32_t max_ctx, void* workspace, size_t ws_bytes, int32_t* d_status, void* stream);

/* kv_verify_tree: which drafted tokens the target keeps, and the token after them (speculative
 * sampling over a tree: the tokens kept are distributed as the target's).  Node 0 of every
 * sequence is its only root: the token sampled last, which is kept always.
 *   token    [n_rows] int32: the drafted tokens (node 0's is not read)
 *   p        float32 rows of `vocab` target probabilities, p_stride elements apart: row r is the
 *            distribution of the token after node r
 *   q        float32 rows of the draft's probabilities likewise (row r: what r's children were
 *            drawn from, independently of one another), or NULL when the drafts were not drawn
 *            but chosen (the draft's best tokens): a miss then only rules its token out
 *   u        [n_rows] float32 uniform numbers in [0, 1): node c > 0's decides node c; node 0's
 *            draws the last token
 *   path     [n_rows] int32 out: path[cu_rows[b] + j] for j < n_accept[b] are the kept nodes from
 *            node 0 down (strictly increasing); -1 behind them
 *   n_accept [B] int32 out: kept nodes, node 0 counted; 0 for a sequence without rows
 *   next_token [B] int32 out: the token after the last kept node (-1: none)
 * Walking down from node 0, the children of the current node are tried in index order: child c with
 * token x is kept when u_c Z q(x) < r(x), where r = p and Z = 1 at first; a miss makes r the
 * elementwise max(r - Z q, 0) and Z its sum (with q NULL: r(x) = 0, Z less by what it was).  When
 * nothing is left of r (rounding), r is p again and no further child is tried.  The last token is the
 * smallest x whose cumulative sum of r exceeds u_0 sum r.  Probabilities and numbers are taken in
 * units of 2^-60 and products rounded down to them, so the result is the same on every run.
 * Probabilities above 1 count as 1; negative or non-finite ones as 0, with KVQ_ERR_NONFINITE, as is a
 * distribution whose sum is 0 or at least 4 (next_token -1).  A sequence whose rows are not such a
 * tree, or whose tokens are not below vocab: KVQ_ERR_BOUNDS, n_accept 0, next_token -1.
 * Of cfg only batch is used (at most 65535, and vocab at most 2^30: KVQ_ERR_UNSUPPORTED). */
KVQ_API int kv_verify_tree(const kvq_config* cfg, const int32_t* cu_rows, const int32_t* parent, const int32_t* token,
                   int32_t n_rows, const float* p, int64_t p_stride, const float* q, int64_t q_stride, int32_t vocab,
                   const float* u, int32_t* path, int32_t* n_accept, int32_t* next_token, int32_t* d_status,
                   void* stream);

/* kv_tree_commit: keep the rows of the accepted path.  For every sequence with n rows and
 * L0 = seq_len - n, token L0 + j becomes the row of node path[cu_rows[b] + j] (j < n_accept[b]; path
 * strictly increasing, as kv_verify_tree writes it) and seq_len becomes L0 + n_accept[b].  Rows move
 * within the BF16 sink and ring.  A sequence whose path is not one, or whose nodes are not in the
 * BF16 windows, is left as it is, with KVQ_ERR_BOUNDS.  Once per layer, on that layer's cache. */
KVQ_API int kv_tree_commit(const kvq_config* cfg, const kvq_cache* cache, const int32_t* cu_rows, int32_t n_rows,
                   const int32_t* path, const int32_t* n_accept, int32_t* d_status, void* stream);

/* ---- the page pool ---------------------------------------------------------------
 * page_ref [num_pages] int32: how many page-table entries hold each physical page (0: free).  The
 * caller zeroes it once; tables filled by hand must be counted in it.  A sequence's entries are a
 * prefix of its row of the table, -1 behind them.  Pages are handed out lowest id first, to
 * sequences in order, so the tables do not depend on timing.  These calls write the page table
 * (cache->page_table must be writable memory), and any call may follow them on the stream.  They
 * run on the stream in order like any other, one pool at a time: two of them must not overlap on
 * the same pool.  A pool is one layer's: every layer has its own pages, page table, lengths and page_ref, and takes
 * each call itself (kv_seq_fork copies that layer's rows and half-filled page).  A call of n sequences or pairs
 * looks at every page count of the pool and, kv_seq_fork, at all n pairs for each.  At most KVQ_POOL_MAX_SEQS sequences (pairs) per call (KVQ_ERR_UNSUPPORTED). */
#define KVQ_POOL_MAX_SEQS 16384

/* kv_pages_reserve: pages for n_tokens[b] (device int32 [B]) more tokens of every sequence, as if
 * they were all quantized: its row then covers [s_sink, seq_len[b] + n_tokens[b]).  n_tokens[b] <= 0
 * reserves nothing.  Sequences are served in order; from the first one on that the pool cannot
 * serve, none gets any (KVQ_ERR_BOUNDS, as for one that would need more than max_pages_per_seq). */
KVQ_API int kv_pages_reserve(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref,
                     const int32_t* n_tokens, int32_t* d_status, void* stream);

/* kv_seq_fork: sequence dst[i] becomes a copy of sequence src[i] (device int32 [n]; one source may
 * have many copies).  Whole INT2 pages are shared; the half-filled last one gets a page of its own;
 * the live sink and ring rows are copied; pages that src holds beyond its INT2 region are not.  dst
 * must hold nothing (a new sequence, or after kv_seq_free).  A pair is skipped with KVQ_ERR_BOUNDS when
 * a sequence does not exist, dst holds something, is another pair's source or an earlier pair's
 * destination, or when the pool has no page left for it or an earlier pair. */
KVQ_API int kv_seq_fork(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, const int32_t* src,
                const int32_t* dst, int32_t n, int32_t* d_status, void* stream);

/* kv_seq_free: sequences seqs[0 .. n-1] (device int32) give up their pages (free once no other
 * sequence holds them) and become empty (seq_len 0, s_quant s_sink).  Listing one twice is harmless. */
KVQ_API int kv_seq_free(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, const int32_t* seqs,
                int32_t n, int32_t* d_status, void* stream);

/* kv_pages_compact: move pages so that the held ones are 0 .. n_live - 1 (n_live: device int32, out),
 * and rename them in every table.  The k-th held page at or above n_live moves to the k-th free page
 * below it, so nothing moves that need not.  The table must cover every sequence that uses the
 * pool.  Workspace of kv_pages_compact_workspace_bytes(cfg) bytes. */
KVQ_API size_t kv_pages_compact_workspace_bytes(const kvq_config* cfg);
KVQ_API int kv_pages_compact(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, int32_t* n_live,
                     void* workspace, size_t ws_bytes, int32_t* d_status, void* stream);

/* ---- from the projections' rows ----------------------------------------------------
 * Rotary positions: channels (a, b) of a head turn by position * f_i, f_i falling with i = 0 ..
 * rot_dim/2 - 1.  Phases are kept as whole numbers, position * freq[i] mod 2^64 in units of 2^-64
 * turns, so that they are exact at any position. */
#define KVQ_ROPE_HALF        0   /* pair i: channels i and i + rot_dim/2 */
#define KVQ_ROPE_INTERLEAVED 1   /* pair i: channels 2i and 2i + 1       */

typedef struct kvq_rope {
  int32_t         layout;    /* KVQ_ROPE_*                                                        */
  int32_t         rot_dim;   /* rotated channels, a head's first: even, 0 .. d; the others pass   */
  float           scale;     /* multiplies the rotated channels (1, or a scaling's factor)        */
  float           norm_eps;  /* of the norms below (1e-30 or more)                                */
  const uint64_t* freq;      /* [rot_dim/2] device: turns per token in units of 2^-64             */
  const float*    q_norm;    /* [d] device: weights of the RMS norm of every query head before    */
  const float*    k_norm;    /*     the rotation; of every key head (NULL: no norm)               */
} kvq_rope;

/* kvq_rope_frequencies: freq and scale of the usual choices (freq is HOST memory, [rot_dim/2]; computed in
 * float64).  w_i = theta^(-2 i / rot_dim) radians a token, and by `scaling`:
 *   KVQ_ROPE_PLAIN   w_i
 *   KVQ_ROPE_LINEAR  w_i / factor (position interpolation)
 *   KVQ_ROPE_NTK     w_i with theta * factor^(rot_dim / (rot_dim - 2)) for theta (rot_dim > 2)
 *   KVQ_ROPE_BANDS   by wavelength, context / lambda_i = context w_i / 2 pi: below a: w_i / factor; above b:
 *                    w_i; between them the two mixed, b's share (context / lambda_i - a) / (b - a)
 *   KVQ_ROPE_YARN    YaRN (Peng et al., 2023): by index, w_i mixed with w_i / factor along a ramp from pair
 *                    floor(at(a)) to ceil(at(b)), at(t) = rot_dim ln(context / (2 pi t)) / (2 ln theta), clipped to
 *                    0 .. rot_dim - 1; scale = 0.1 ln(factor) + 1 (1 for factor <= 1)
 * scale (HOST, may be NULL) is 1 for the others.  context, a, b are read by the last two only (a < b and a > b >
 * 0 there).  theta > 1, factor > 0: KVQ_ERR_INVALID_ARG otherwise. */
#define KVQ_ROPE_PLAIN  0
#define KVQ_ROPE_LINEAR 1
#define KVQ_ROPE_NTK    2
#define KVQ_ROPE_BANDS  3
#define KVQ_ROPE_YARN   4
KVQ_API int kvq_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, double context, double a,
                         double b, uint64_t* freq, float* scale);

/* kv_rope_qk: the rows of the query, key and value projections as they come: norm of the heads, rotation by
 * position, transform, and the append.
 *   q        [n_q_rows][Hq][d] bf16, rows q_stride elements apart (so for k and v: three parts of one fused
 *            projection do; strides are multiples of 8 and at least H d, bases 16-byte aligned)
 *   q_out    [n_q_rows][Hq][d] bf16 (16-byte aligned): T_K^{-T} rope(norm(q)); must not overlap the rows of q, k or v
 *            (each from its first row's beginning to its last one's end)
 *   q_pos    [n_q_rows] int32: each query's position in the text (any value; NULL when n_q_rows == 0)
 *   k, v     [n_kv_rows][Hkv][d] bf16 likewise; seq_idx, pos [n_kv_rows] int32 as for kv_rotate_qk
 *   rope_pos [n_kv_rows] int32: each key's position in the text where it is not its token's number (the nodes
 *            of a drafted tree: the number of tokens before the drafts plus the node's depth); NULL: pos
 * Keys become T_K rope(norm(k)), values T_V v or copies of v, written to sink and ring as kv_rotate_qk does:
 * the same bounds, status and seq_len.  n_kv_rows and n_q_rows may differ, and either may be 0.
 * Arithmetic is float32 (the norm's mean, the rotation, the transform's sums) with one rounding to bf16 at the end; on the
 * tensor cores (Execution) sines and cosines have 20 bits, and the transform's operands 21, as pairs of fp16.  With m_j the
 * length of channel j's pair after the norm, and besides that rounding, output i is off by at most 2^-17 sum_j |T_ij| m_j, and on
 * the tensor cores by 2^-22 (max_j m_j sum_j |T_ij| + max_j |T_ij| sum_j m_j) more: that counts where T_i is next to nothing at the
 * row's large channels (identity, diagonal), below which 22 bits are kept.  It is not kv_rotate_qk's exact product, whose
 * input rows are rounded after the rotation.  Copied values are exact.  A head whose row holds an infinity or NaN, or (with a norm)
 * whose squares sum to more than float32 holds, gets a row that is not finite, and KVQ_ERR_NONFINITE (copied values aside); so
 * do all heads of a norm with a weight that is not finite.
 * rope NULL: no norm and no rotation (q_pos may then be NULL).
 * Of cfg the heads, batch, s_sink and ring_cap are used.
 * Execution: fewer than 896 (row, head) pairs that have a matrix (Hadamard: 1280) run on the CUDA cores, a slice of a matrix to a CTA;
 * larger calls on the tensor cores, both operands as pairs of fp16 under powers of two, values that are copied in a
 * launch before.  The two round differently.
 * Source: [WUSH] inference algorithm and [OScaR] algorithm, key and query processing (the transform follows RoPE);
 * norm and rotation are the models' own (Qwen3's heads). */
KVQ_API int kv_rope_qk(const kvq_config* cfg, const kvq_transform* tr, const kvq_rope* rope, const uint16_t* q,
               int64_t q_stride, uint16_t* q_out, const int32_t* q_pos, int32_t n_q_rows, const uint16_t* k,
               int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* seq_idx, const int32_t* pos,
               const int32_t* rope_pos, int32_t n_kv_rows, const kvq_cache* cache, int32_t* d_status, void* stream);

/* ---- from logits to tokens ------------------------------------------------------------
 * counts [B][count_stride] uint16 (device, 4-byte aligned, count_stride even and at least vocab): what sequence b holds
 * of each token: the highest bit for one that its prompt holds, below it how often it has been generated (no more
 * than KVQ_COUNT_MOST is kept).  The caller zeroes a row when a sequence takes its place (and copies it when one is
 * forked); kv_token_counts writes it, kv_logits_probs reads it. */
#define KVQ_COUNT_MOST   32767
#define KVQ_COUNT_PROMPT 0
#define KVQ_COUNT_OUTPUT 1

#define KVQ_LOGITS_F32  0
#define KVQ_LOGITS_BF16 1
#define KVQ_LOGITS_F16  2
#define KVQ_LOGITS_MAX_VOCAB 524288

typedef struct kvq_logit_rules {         /* device pointers; NULL: that rule is not applied */
  const float*    temperature; /* [B] >= 0; 0: the best token alone, the lowest id among equals (NULL: 1)        */
  const float*    repetition;  /* [B] 2^-60 .. 2^60: logits of tokens held, prompt or generated: l > 0: l / r, else l * r */
  const float*    frequency;   /* [B]: less by this for every time the token has been generated                 */
  const float*    presence;    /* [B]: less by this once the token has been generated                           */
  const uint16_t* counts;      /* as above (NULL: nothing is held yet)                                          */
  int64_t         count_stride;
  const int32_t*  bias_cu;     /* [B + 1]: sequence b's biases are entries bias_cu[b] .. bias_cu[b+1] - 1 of    */
  const int32_t*  bias_token;  /* [n_bias]: token ids, strictly increasing within a sequence, and               */
  const float*    bias;        /* [n_bias]: what is added to their logits (-infinity bans a token)              */
  const uint32_t* mask;        /* [n_masks][mask_stride]: bit v % 32 of word v / 32 set: token v is allowed     */
  int64_t         mask_stride; /* words, at least vocab / 32 rounded up                                         */
  const int32_t*  mask_row;    /* [n_rows]: the mask of each row, -1: none (NULL: mask r for row r)             */
  int32_t         n_bias;
  int32_t         n_masks;
} kvq_logit_rules;

/* kv_logits_probs: the rows of probabilities that kv_verify_tree takes (with one row a sequence: the next token's).
 *   logits   n_rows rows of `vocab` numbers, l_stride elements apart, of type KVQ_LOGITS_* (aligned to their size)
 *   cu_rows  [B + 1] as for kv_append_chunk: rows of sequence b
 *   parent, token [n_rows] int32: the tree as for kv_verify_tree, or NULL: the rows are no drafts.  The tokens of a
 *            node and its ancestors count as generated in its row, roots left out: theirs has been counted
 *   p        n_rows rows of `vocab` float32, p_stride elements apart; may be the logits themselves (float32, equal
 *            strides), and must not overlap them otherwise (from the first row's beginning to the last one's end)
 * In this order, in float32, one rounding an operation: l + bias; repetition; less frequency * times; less presence;
 * masked tokens to -infinity, whatever stood there; softmax of l / temperature (one between 0 and 2^-120 counts as 2^-120, which only
 * logits within 2^-113 of the largest can tell from it).  The softmax takes the special function units' exponential: besides the
 * roundings before it, p is off by at most 2^-17 + 2^-22 (max l - l) / temperature of itself.
 * KVQ_ERR_NONFINITE and a row of zeros: where nothing is left (every token masked or at -infinity), where a logit that
 * is not masked becomes NaN or +infinity, or where a number of the sequence's rules is not finite, the temperature
 * negative or the repetition not within 2^-60 .. 2^60.  Probabilities below 2^-126 are 0.  KVQ_ERR_BOUNDS and a row
 * of zeros: a mask that does not exist, more than KVQ_TREE_MAX_NODES nodes in a sequence.  KVQ_ERR_BOUNDS: a parent that
 * is not a lower node (the row goes by the path up to there), a token of the path or of a bias outside the vocabulary
 * (left out), biases out of order (an entry that is not above the one before it may be left out), and cu_rows that do
 * not cover n_rows: rows behind the last sequence are not written.  Sums are taken in one order: the same bits on every
 * run.
 * vocab is at most KVQ_LOGITS_MAX_VOCAB.  Of cfg only batch is used.
 * Execution: a cluster of CTAs holds a row in shared memory: one read of the logits, one write of p.  Logits of
 * four masked neighbours are not read. */
KVQ_API int kv_logits_probs(const kvq_config* cfg, const kvq_logit_rules* rules, const void* logits, int32_t logits_type,
                    int64_t l_stride, int32_t vocab, const int32_t* cu_rows, const int32_t* parent, const int32_t* token,
                    int32_t n_rows, float* p, int64_t p_stride, int32_t* d_status, void* stream);

/* kv_token_counts: tokens into counts.  Rows cu_rows[b] .. cu_rows[b+1] - 1 of token [n_rows] are sequence b's:
 *   KVQ_COUNT_PROMPT  they are marked as its prompt's (path, n_accept, next_token NULL);
 *   KVQ_COUNT_OUTPUT  they are counted as generated: all of them (path and n_accept NULL), or, after
 *                     kv_verify_tree, those of the kept nodes path[cu_rows[b] + j], 0 < j < n_accept[b] (node 0
 *                     was counted when it was drawn), and with next_token [B] the token behind them (-1: none).
 * Equal tokens may come any number of times.  Tokens outside the vocabulary, nodes outside the tree and rows of no
 * sequence are left out, with KVQ_ERR_BOUNDS; KVQ_ERR_BOUNDS also where cu_rows ends behind n_rows (the rows that there are
 * are taken).  cu_rows does not fall: which rows are taken where it does is not said.  Of cfg only batch is used; n_rows is at most 2^30 (KVQ_ERR_UNSUPPORTED).
 * Execution: an atomic for each of a warp's different tokens; prompts of 2^16 rows or more, and on average 2^14 and a sixth of
 * the vocabulary a sequence, in one sweep over the counts, without atomics.  No other call may write the same rows of counts at
 * the same time. */
KVQ_API int kv_token_counts(const kvq_config* cfg, uint16_t* counts, int64_t count_stride, int32_t vocab, int32_t kind,
                    const int32_t* cu_rows, const int32_t* token, int32_t n_rows, const int32_t* path,
                    const int32_t* n_accept, const int32_t* next_token, int32_t* d_status, void* stream);

/* kv_attn_decode: one decode step of GQA attention for every sequence.
 *   q_rot   [B][Hq][d] bf16 compensated queries (kv_rotate_qk output)
 *   out     [B][Hq][d] float32 attention output (in the T_V space)
 *   sm_scale logit scale (1/sqrt(d) for standard attention)
 *   max_ctx  an upper bound of seq_len over the batch (sizes the split grid)
 *   workspace, ws_bytes: device scratch of at least kv_attn_workspace_bytes(cfg,
 *            max_ctx) bytes, zero-filled before its first use; every call leaves the
 *            ticket counters at its head zero again (the rest is overwritten).
 * Softmax over sink | INT2 | recent tokens with online (max, sum) merging across
 * splits in one launch; all g = Hq/Hkv query heads of a kv head share one read.
 * batch <= 65535 (KVQ_ERR_UNSUPPORTED otherwise: it is a grid dimension).
 * Source: [OSCAR] section 4 "Decoding Attention Kernel"; [OScaR] attention fused
 * kernel (in-register dequantisation, split attention); [WUSH] GQA. */
KVQ_API int kv_attn_decode(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                   float* out, float sm_scale, int32_t max_ctx,
                   void* workspace, size_t ws_bytes, int32_t* d_status, void* stream);

/* kv_attn_decode_bf16: kv_attn_decode with a bf16 output.
 *   out     [B][Hq][d] bf16 (8-byte aligned): the float32 result of kv_attn_decode rounded
 *           once to bf16 (nearest-even) -- the same kernel, only the final store differs.
 * Arguments, workspace and errors as kv_attn_decode.  For callers whose next GEMM (the
 * output projection, in the T_V space) takes bf16 activations; the rounding adds up to
 * 2^-8 relative per element on top of the float32 result.
 * Source: [OSCAR] section 4 "Decoding Attention Kernel" (decode attention over the mixed
 * cache); the output precision is not fixed by the pages. */
KVQ_API int kv_attn_decode_bf16(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                                uint16_t* out, float sm_scale, int32_t max_ctx,
                                void* workspace, size_t ws_bytes, int32_t* d_status, void* stream);

/* kv_attn_decode_noalloc: kv_attn_decode without a caller-supplied workspace, for callers
 * that cannot allocate device memory on this path -- for example a plugin running inside a
 * serving framework whose memory pool owns the whole device and forbids direct cudaMalloc,
 * or code that must not call cudaMalloc because it can synchronize the device.  This call
 * allocates nothing: its scratch is a fixed array of KVQ_NOALLOC_WORKSPACE_BYTES (8 MiB) of
 * device memory inside the library, held by every GPU that loads the library until the
 * process exits.  Arguments, results and errors are those of kv_attn_decode, except:
 *   - KVQ_ERR_WORKSPACE when kv_attn_workspace_bytes(cfg, max_ctx) exceeds the fixed size;
 *   - the first call on a device does a set-up, once per device, while that device is
 *     current: it looks up the array's device address and zero-fills the array (an async
 *     memset on `stream`), so make that first call before any stream capture; later calls
 *     add nothing to the stream but the decode kernel (each completed call leaves the ticket
 *     counters at the array's head zero again, as kv_attn_decode does for its workspace);
 *   - the address is kept for the life of the process: do not use this entry point after a
 *     cudaDeviceReset (or any other teardown of the device's primary context) in the same
 *     process, because the kept address no longer names device memory then;
 *   - every call shares the one array, which keeps the last call's contents; calls whose
 *     work overlaps on the GPU (other streams, other threads) race on it and give wrong
 *     results -- serialize them.
 * This entry point has no counterpart on the pages; it only changes where the scratch of
 * kv_attn_decode lives. */
#define KVQ_NOALLOC_WORKSPACE_BYTES (8u << 20)
KVQ_API int kv_attn_decode_noalloc(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                                   float* out, float sm_scale, int32_t max_ctx, int32_t* d_status, void* stream);

/* Workspace bytes kv_attn_decode needs for contexts up to max_ctx (host only). */
KVQ_API size_t kv_attn_workspace_bytes(const kvq_config* cfg, int32_t max_ctx);

/* Static description of a status code. */
KVQ_API const char* kvq_status_string(int code);

/* kvq_selftest_scale_division: the quantizer divides by a float16 scale with a
 * correctly rounded reciprocal and one exact-remainder correction instead of an IEEE
 * division.  This launches a check of that path against IEEE division on the device:
 * every finite bf16 dividend with every positive finite float16 scale, plus 2^29 hashed
 * float32 dividends (the l2-scaled keys); the number of bitwise differences is ADDED to
 * *d_mismatches (a device uint64 the caller zeroes).  Not part of the method on the pages:
 * a self-test of this implementation.  Returns KVQ_ERR_INVALID_ARG for a NULL pointer. */
KVQ_API int kvq_selftest_scale_division(unsigned long long* d_mismatches, void* stream);

/* kvq_selftest_tc_integer_sums: for prefill-sized calls kv_rotate_qk runs its dense rows on
 * the tensor cores with both operands written as integer digits in [-128, 128] (exact
 * bf16 values), so every accumulated sum is an integer below 2^23; the outputs are exact
 * as long as the tensor cores add such integers exactly, which the hardware documentation
 * does not state.  This launches a check of that on the device: hashed and extreme digit
 * matrices through the rotation's own sequence of MMAs, every accumulator compared with
 * the integer sum formed on the CUDA cores; the number of differences is ADDED to
 * *d_mismatches (a device uint64 the caller zeroes).  Not part of the method on the pages:
 * a self-test of this implementation.  Returns KVQ_ERR_INVALID_ARG for a NULL pointer. */
KVQ_API int kvq_selftest_tc_integer_sums(unsigned long long* d_mismatches, void* stream);

/* Library ABI version (major * 100 + minor). */
KVQ_API int kvq_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
