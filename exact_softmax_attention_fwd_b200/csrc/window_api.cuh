// window_api.cuh -- the C entry points of attention with a sliding window and
// visible first tokens (declared in attn.h): argument checks on the host, before
// any CUDA call, and the launches.  Included by attn_api.cu, whose helpers it
// uses; prefill and backward are the masked instantiations of their kernels,
// decode has a kernel of its own.
#pragma once

#include "decode_window_sm100.cuh"

namespace attn_b200 {
namespace {

// Query heads of a KV head that share a tile of the paged kernel, as a power of
// two (0: each head has tiles of its own): all of a group's, when they are 2, 4,
// 8 or 16.  It pays where chunks are short and costs a little where one is long:
// 32 / 8 heads, window 1024, with and without it, 16 chunks of 64 tokens take 41
// and 109 us, 32 of 8 tokens 59 and 177, 8 of 5 to 1024 tokens 47 and 59, and one
// of 8192 tokens 240 and 224.
int window_pack(int Hq, int Hkv) {
  const int group = Hq / Hkv;
  for (int s = 1; s <= 4; ++s)
    if (group == 1 << s) return s;
  return 0;
}

template <int D, bool FP8>
int launch_decode_window(const CUtensorMap& mk, const CUtensorMap& mv, DecodeWindowParams& p,
                         int max_chunks, cudaStream_t stream) {
  using W = DecodeWinCfg<D, FP8>;
  auto kern = attn_decode_window_kernel<D, FP8>;
  static std::atomic<unsigned long long> smem_set{0};
  if (!set_smem_once(kern, W::smem(kWinWarps), smem_set)) return ATTN_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  const long long pairs = (long long)p.f.d.B * p.f.d.Hkv;
  const WinShape shape = win_shape<D, FP8>(pairs, max_chunks, sms);
  const int cs = shape.cluster;
  p.cluster = cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * cs));
  cfg.blockDim = dim3(shape.warps * 32);
  cfg.dynamicSmemBytes = W::smem(shape.warps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, mk, mv, p) != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int decode_window_run(bool fp8, const void* q, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, const int32_t* block_table,
                      const int32_t* seq_lens, int page_size, int B, int Hq, int Hkv, int d,
                      int max_pages_per_seq, int num_pages, float scale, int window, int sinks,
                      void* o, float* lse, attn_stream_t stream) {
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_table == nullptr ||
      seq_lens == nullptr || o == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (fp8 && (k_scale == nullptr || v_scale == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages_per_seq < 1 || num_pages < 1 ||
      page_size < 1)
    return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > (1ll << 27) || (long long)max_pages_per_seq * page_size > (1ll << 30) ||
      (long long)num_pages * page_size > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size % 16 != 0 || page_size > 256) return ATTN_ERR_UNSUPPORTED;
  if (Hq / Hkv > 8) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned4(block_table) || !aligned4(seq_lens) || (lse != nullptr && !aligned4(lse)))
    return ATTN_ERR_ALIGNMENT;
  if (fp8 && (!aligned4(k_scale) || !aligned4(v_scale))) return ATTN_ERR_ALIGNMENT;
  DecodeWindowParams p;
  std::memset(&p, 0, sizeof(p));
  DecodeParams& prm = p.f.d;
  prm.q = static_cast<const uint16_t*>(q);
  prm.block_table = block_table;
  prm.seq_lens = seq_lens;
  prm.o = static_cast<uint16_t*>(o);
  prm.lse = lse;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.group = Hq / Hkv;
  prm.page_size = page_size;
  prm.max_pages = max_pages_per_seq;
  prm.num_pages = num_pages;
  prm.scale_log2 = scale * 1.4426950408889634f;
  p.f.k_scale = k_scale;
  p.f.v_scale = v_scale;
  p.window = window > 0 ? window : INT_MAX;
  p.sinks = window > 0 ? sinks : 0;
  // the most chunks a sequence can have visible
  const long long cap = (long long)max_pages_per_seq * page_size / 16;
  const int max_chunks =
      (int)std::min(cap, ((long long)p.window + 15) / 16 + 1 + ((long long)p.sinks + 15) / 16);
  CUtensorMap mk, mv;
  const long long pool_tokens = (long long)num_pages * page_size;
  const bool maps_ok =
      fp8 ? make_token_map_u8(&mk, k_cache, d, Hkv, pool_tokens) &&
                make_token_map_u8(&mv, v_cache, d, Hkv, pool_tokens)
          : make_token_map(&mk, k_cache, d, Hkv, pool_tokens, 16) &&
                make_token_map(&mv, v_cache, d, Hkv, pool_tokens, 16);
  if (!maps_ok) return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d == 128)
    return fp8 ? launch_decode_window<128, true>(mk, mv, p, max_chunks, st)
               : launch_decode_window<128, false>(mk, mv, p, max_chunks, st);
  return fp8 ? launch_decode_window<64, true>(mk, mv, p, max_chunks, st)
             : launch_decode_window<64, false>(mk, mv, p, max_chunks, st);
}

}  // namespace
}  // namespace attn_b200

extern "C" {

int attn_decode_paged_window(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* seq_lens, int page_size,
                             int B, int Hq, int Hkv, int d, int max_pages_per_seq, int num_pages,
                             float scale, int window, int sinks, void* o, float* lse,
                             attn_stream_t stream) {
  return decode_window_run(false, q, k_cache, v_cache, nullptr, nullptr, block_table, seq_lens,
                           page_size, B, Hq, Hkv, d, max_pages_per_seq, num_pages, scale, window,
                           sinks, o, lse, stream);
}

int attn_decode_paged_window_fp8(const void* q, const void* k_cache, const void* v_cache,
                                 const float* k_scale, const float* v_scale,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 int page_size, int B, int Hq, int Hkv, int d,
                                 int max_pages_per_seq, int num_pages, float scale, int window,
                                 int sinks, void* o, float* lse, attn_stream_t stream) {
  return decode_window_run(true, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                           page_size, B, Hq, Hkv, d, max_pages_per_seq, num_pages, scale, window,
                           sinks, o, lse, stream);
}

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

size_t attn_fwd_paged_window_workspace_size(int B, int Hq, int Hkv, long long total_q,
                                            int max_seqlen_q) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || total_q < 0 || total_q > 0x7fffffffLL ||
      max_seqlen_q < 1 || max_seqlen_q > kVarlenMaxLevels * 256)
    return 0;
  return 16 + 8 * (size_t)varlen_max_units(B, total_q << window_pack(Hq, Hkv));
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
  const size_t need = attn_fwd_paged_window_workspace_size(B, Hq, Hkv, total_q, max_seqlen_q);
  if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_ALIGNMENT;
  if (total_q == 0) return ATTN_OK;
  // no window: one that reaches every key (the masked kernel is also the one
  // that leaves the rows behind a sequence's end unread)
  return paged_prefill_run(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, page_size,
                           B, Hq, Hkv, total_q, max_seqlen_q, max_pages_per_seq, num_pages, d, 1,
                           scale, o, lse, workspace, reinterpret_cast<cudaStream_t>(stream),
                           window > 0 ? window : INT_MAX, window > 0 ? sinks : 0,
                           window_pack(Hq, Hkv));
}

}  // extern "C"
