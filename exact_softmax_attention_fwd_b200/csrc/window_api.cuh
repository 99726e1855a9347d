// window_api.cuh -- the C entry points of attention with a sliding window and
// visible first tokens (declared in attn.h): argument checks on the host, before
// any CUDA call, and the launches.  Included by attn_api.cu, whose helpers it
// uses; the kernels are the masked instantiations of the prefill and backward
// kernels.
#pragma once

extern "C" {

int attn_fwd_window_sinks(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                          int Hq, int Hkv, int Sq, int Sk, int d, float scale,
                          const int32_t* k_lens, int window, int sinks, attn_stream_t stream) {
  const int st = check_prefill_args(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, d, 1, scale, k_lens);
  if (st != ATTN_OK) return st;
  if (window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return prefill_dense(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, d, 1, scale, k_lens, window, 0,
                       nullptr, 1, reinterpret_cast<cudaStream_t>(stream), sinks);
}

size_t attn_bwd_window_sinks_workspace_size(int B, int Hq, int Hkv, int Sq, int Sk, int d,
                                            int window, int sinks) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || Sk < 0 || (d != 64 && d != 128) ||
      window < 0 || sinks < 0)
    return 0;
  return bwd_workspace_bytes(B, Hq, Sq) + bwd_far(B, Hq, Hkv, Sq, Sk, d, window, sinks).bytes;
}

int attn_bwd_window_sinks(const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* d_o, void* dq, void* dk, void* dv, int B,
                          int Hq, int Hkv, int Sq, int Sk, int d, float scale,
                          const int32_t* k_lens, int window, int sinks, void* workspace,
                          size_t workspace_bytes, attn_stream_t stream) {
  if (window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return bwd_dense(q, k, v, o, lse, d_o, dq, dk, dv, B, Hq, Hkv, Sq, Sk, d, 1, scale, k_lens,
                   window, 0, nullptr, 1, workspace, workspace_bytes, stream, sinks);
}

int attn_fwd_paged_window(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* cu_seqlens_q,
                          const int32_t* seq_lens_k, int page_size, int B, int Hq, int Hkv,
                          long long total_q, int max_seqlen_q, int max_pages_per_seq,
                          int num_pages, int d, float scale, int window, int sinks, void* o,
                          float* lse, void* workspace, size_t workspace_bytes,
                          attn_stream_t stream) {
  const int st = check_paged_prefill_args(q, k_cache, v_cache, block_table, cu_seqlens_q,
                                          seq_lens_k, page_size, B, Hq, Hkv, total_q, max_seqlen_q,
                                          max_pages_per_seq, num_pages, d, 1, scale, o, lse);
  if (st != ATTN_OK) return st;
  if (window < 0 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_fwd_varlen_workspace_size(B, total_q, max_seqlen_q);
  if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_ALIGNMENT;
  if (total_q == 0) return ATTN_OK;
  // no window: one that reaches every key (the masked kernel is also the one
  // that leaves the rows behind a sequence's end unread)
  return paged_prefill_run(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, page_size,
                           B, Hq, Hkv, total_q, max_seqlen_q, max_pages_per_seq, num_pages, d, 1,
                           scale, o, lse, workspace, reinterpret_cast<cudaStream_t>(stream),
                           window > 0 ? window : INT_MAX, window > 0 ? sinks : 0);
}

}  // extern "C"
