// Internal launchers shared between the translation units of the library (not exported).
#pragma once

#include <cuda_runtime.h>
#include "../../include/kvq.h"

extern "C" {
int kvq_launch_rotate(const kvq_config* cfg, const kvq_transform* tr, const uint16_t* q, uint16_t* q_out,
                      int32_t n_q_rows, const uint16_t* k, const uint16_t* v, const int32_t* seq_idx,
                      const int32_t* pos, int32_t n_kv_rows, const kvq_cache* cache, int32_t* d_status,
                      cudaStream_t stream);
int kvq_launch_flush(const kvq_config* cfg, const kvq_cache* cache, int32_t max_tokens, int32_t* d_status,
                     cudaStream_t stream);
int kvq_launch_flush_append(const kvq_config* cfg, const kvq_cache* cache, const int32_t* cu_rows,
                            int32_t* d_status, cudaStream_t stream);
int kvq_launch_append(const kvq_config* cfg, const kvq_transform* tr, const uint16_t* k, const uint16_t* v,
                      const int32_t* cu_rows, int32_t n_rows, const kvq_cache* cache, int32_t* d_status,
                      cudaStream_t stream);
int kvq_launch_attn(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot, void* out, int out_bf16,
                    float sm_scale, int32_t max_ctx, void* ws, int32_t* d_status, cudaStream_t stream);
int kvq_launch_attn_chunk(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot, const int32_t* cu_rows,
                          int32_t n_rows, float* out, float sm_scale, int32_t max_ctx, void* ws, int32_t* d_status,
                          cudaStream_t stream);
size_t kvq_attn_chunk_ws_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx);
size_t kvq_attn_tree_head_bytes(const kvq_config* cfg);
size_t kvq_attn_tree_rows_part_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx);
int kvq_launch_attn_tree_rows(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                              const int32_t* cu_rows, const int32_t* parent, int32_t n_rows, uint16_t* out,
                              float sm_scale, int32_t max_ctx, void* ws, int32_t* d_status, cudaStream_t stream);
size_t kvq_attn_tree_ws_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx);
int kvq_launch_attn_tree(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot, const int32_t* cu_rows,
                         const int32_t* parent, int32_t n_rows, uint16_t* out, float sm_scale, int32_t max_ctx,
                         void* ws, int32_t* d_status, cudaStream_t stream);
int kvq_launch_verify_tree(const kvq_config* cfg, const int32_t* cu_rows, const int32_t* parent, const int32_t* token,
                           int32_t n_rows, const float* p, int64_t p_stride, const float* q, int64_t q_stride,
                           int32_t vocab, const float* u, int32_t* path, int32_t* n_accept, int32_t* next_token,
                           int32_t* d_status, cudaStream_t stream);
int kvq_launch_tree_commit(const kvq_config* cfg, const kvq_cache* cache, const int32_t* cu_rows, int32_t n_rows,
                           const int32_t* path, const int32_t* n_accept, int32_t* d_status, cudaStream_t stream);
int kvq_launch_pages_reserve(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, const int32_t* n_tokens,
                             int32_t* d_status, cudaStream_t stream);
int kvq_launch_seq_fork(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, const int32_t* src,
                        const int32_t* dst, int32_t n, int32_t* d_status, cudaStream_t stream);
int kvq_launch_seq_free(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, const int32_t* seqs,
                        int32_t n, int32_t* d_status, cudaStream_t stream);
size_t kvq_compact_ws_bytes(const kvq_config* cfg);
int kvq_launch_pages_compact(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, int32_t* n_live,
                             void* ws, int32_t* d_status, cudaStream_t stream);
int kvq_launch_attn_noalloc(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot, float* out,
                            float sm_scale, int32_t max_ctx, int32_t* d_status, cudaStream_t stream);
int kvq_launch_rope(const kvq_config* cfg, const kvq_transform* tr, const kvq_rope* rope, const uint16_t* q,
                    int64_t q_stride, uint16_t* q_out, const int32_t* q_pos, int32_t n_q_rows, const uint16_t* k,
                    int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* seq_idx, const int32_t* pos,
                    const int32_t* rope_pos, int32_t n_kv_rows, const kvq_cache* cache, int32_t* d_status,
                    cudaStream_t stream);
int kvq_launch_logits_probs(const kvq_config* cfg, const kvq_logit_rules* rules, const void* logits, int32_t logits_type,
                            int64_t l_stride, int32_t vocab, const int32_t* cu_rows, const int32_t* parent,
                            const int32_t* token, int32_t n_rows, float* p, int64_t p_stride, int32_t* d_status,
                            cudaStream_t stream);
int kvq_launch_token_counts(const kvq_config* cfg, uint16_t* counts, int64_t count_stride, int32_t vocab, int32_t kind,
                            const int32_t* cu_rows, const int32_t* token, int32_t n_rows, const int32_t* path,
                            const int32_t* n_accept, const int32_t* next_token, int32_t* d_status, cudaStream_t stream);
int kvq_launch_div_selftest(unsigned long long* d_mismatches, cudaStream_t stream);
int kvq_launch_tc_selftest(unsigned long long* d_mismatches, cudaStream_t stream);
size_t kvq_attn_counter_bytes(const kvq_config* cfg, int32_t max_ctx);
size_t kvq_attn_ws_bytes(const kvq_config* cfg, int32_t max_ctx);
void kvq_attn_splits(const kvq_config* cfg, int32_t max_ctx, int* n_int2, int* n_win);
}
