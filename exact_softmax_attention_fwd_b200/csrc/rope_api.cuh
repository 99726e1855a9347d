// rope_api.cuh -- the C entry points of rope_sm100.cuh (declared in attn.h):
// argument checks on the host, before any CUDA call, and the launches.
// Included by attn_api.cu, whose helpers it uses.
#pragma once

#include "rope_sm100.cuh"

namespace attn_b200 {
namespace {

// Heads that one block turns: as many as leave about `blocks` blocks of 256
// threads for every SM (the angles of a token are computed once per block, so
// long runs of heads are cheapest when there are tokens enough), and one head
// when there are few tokens.  Measured: the rotation of 8192 tokens x 40 heads
// takes 29.4 us with 8 blocks an SM, 30.5 with 16, 31.0 with 32; the append of
// 10341 tokens x 48 heads, whose blocks begin with a chain of look-ups, 48.8,
// 48.6 and 47.6, and 46.9 us with 24.
constexpr int kRopeBlocks = 8, kAppendBlocks = 24;

int rope_heads_per_block(long long token_blocks, int heads, int sms, int blocks) {
  const long long slots = (long long)blocks * sms;
  const long long want = (token_blocks * heads + slots - 1) / slots;
  return (int)(want < 1 ? 1 : want > heads ? heads : want);
}

// Whether a [B, H, S] tensor of d-element rows with these strides (elements)
// writes every element once: extents over 1 nest inside one another.
bool rope_rows_apart(const long long s[3], const long long ext[3], int d) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[order[j]] > s[order[j + 1]]) std::swap(order[j], order[j + 1]);
  long long reach = d;
  for (int i = 0; i < 3; ++i) {
    if (ext[order[i]] <= 1) continue;
    if (s[order[i]] < reach) return false;
    reach = s[order[i]] * (ext[order[i]] - 1) + reach;
  }
  return true;
}

// Strides (elements) of n nested extents: not negative, reaching at most 2^42
// elements, and (for the 16-byte pieces) multiples of 8.  A stride of an
// extent of one is never used: it is set to 0, whatever it was.
int rope_check_strides(long long* s, const long long* ext, int n) {
  for (int i = 0; i < n; ++i) {
    if (ext[i] <= 1) s[i] = 0;
    if (s[i] < 0 || (ext[i] > 1 && s[i] > (1ll << 42) / (ext[i] - 1))) return ATTN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i)
    if (s[i] % 8 != 0) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

template <int D>
int launch_rope(const RopeParams& p, int interleaved, cudaStream_t stream) {
  constexpr int tokens = kRopeThreads / (D / 16);
  const dim3 grid((unsigned)((p.n_tokens + tokens - 1) / tokens),
                  (unsigned)((p.H + p.heads_per_block - 1) / p.heads_per_block));
  if (interleaved)
    attn_rope_kernel<D, true><<<grid, kRopeThreads, 0, stream>>>(p);
  else
    attn_rope_kernel<D, false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int rope_run(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
             const int32_t* positions, long long pos_stride, int B, int Hq, int Hkv, int S, int d,
             int rotary_dim, int interleaved, float mscale, const long long* strides,
             float sin_sign, attn_stream_t stream) {
  if (B < 1 || Hq < 1 || Hkv < 0 || S < 0 || inv_freq == nullptr) return ATTN_ERR_INVALID_ARG;
  if (S > 0 && (q == nullptr || q_out == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (S > 0 && Hkv > 0 && (k == nullptr || k_out == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (B > (1 << 24) || S > (1 << 30) || (long long)B * S > 0x7fffffffLL || Hq > 32767 ||
      Hkv > 32767)
    return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(mscale) || pos_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(q_out) || (Hkv > 0 && (!aligned16(k) || !aligned16(k_out))))
    return ATTN_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0 ||
      (positions != nullptr && !aligned4(positions)))
    return ATTN_ERR_ALIGNMENT;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  long long* to[4] = {p.qs, p.ks, p.qos, p.kos};
  for (int t = 0; t < 4; ++t) {
    const int H = (t & 1) ? Hkv : Hq;
    const long long dense[3] = {(long long)H * S * d, (long long)S * d, d};
    for (int i = 0; i < 3; ++i) to[t][i] = strides != nullptr ? strides[3 * t + i] : dense[i];
    if ((t & 1) && Hkv == 0) continue;
    const long long ext[3] = {B, H, S};
    const int bad = rope_check_strides(to[t], ext, 3);
    if (bad != ATTN_OK) return bad;
    if (t >= 2 && S > 0 && !rope_rows_apart(to[t], ext, d)) return ATTN_ERR_INVALID_ARG;
  }
  // in place only row by row
  if (S > 0 && ((q_out == q && !std::equal(p.qs, p.qs + 3, p.qos)) ||
                (Hkv > 0 && k_out == k && !std::equal(p.ks, p.ks + 3, p.kos))))
    return ATTN_ERR_INVALID_ARG;
  if (S == 0) return ATTN_OK;
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.S = S;
  p.Hq = Hq;
  p.H = Hq + Hkv;
  p.n_tokens = (long long)B * S;
  p.rot_chunks = rotary_dim / 16;
  p.mscale = mscale;
  p.sin_sign = sin_sign;
  const int per_block = kRopeThreads / (d / 16);
  p.heads_per_block = rope_heads_per_block((p.n_tokens + per_block - 1) / per_block, p.H, sms,
                                           kRopeBlocks);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return d == 128 ? launch_rope<128>(p, interleaved, st) : launch_rope<64>(p, interleaved, st);
}

template <int D, bool FP8>
int launch_append(const AppendParams& p, int interleaved, cudaStream_t stream) {
  constexpr int tokens = kRopeThreads / (D / 16);
  const dim3 grid((unsigned)((p.total + tokens - 1) / tokens),
                  (unsigned)((p.H + p.heads_per_block - 1) / p.heads_per_block));
  if (interleaved)
    attn_append_kernel<D, true, FP8><<<grid, kRopeThreads, 0, stream>>>(p);
  else
    attn_append_kernel<D, false, FP8><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int append_run(bool fp8, const void* q, const void* k, const void* v, void* q_out, void* k_cache,
               void* v_cache, const float* k_scale, const float* v_scale,
               const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* seq_lens,
               const int32_t* positions, const double* inv_freq, int page_size, int B, int Hq,
               int Hkv, long long total, int max_pages_per_seq, int num_pages, int d,
               int rotary_dim, int interleaved, float mscale, const long long* strides,
               attn_stream_t stream) {
  if (k_cache == nullptr || v_cache == nullptr || block_table == nullptr || seq_lens == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (fp8 && (k_scale == nullptr || v_scale == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (total > 0 && (k == nullptr || v == nullptr || (q == nullptr) != (Hq == 0) ||
                    (q != nullptr && q_out == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 0 || Hkv < 1 || Hq > 32767 || Hkv > 16383 || max_pages_per_seq < 1 ||
      num_pages < 1 || page_size < 1)
    return ATTN_ERR_INVALID_ARG;
  if (total < 0 || total > 0x7fffffffLL || (cu_seqlens == nullptr && total != B))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)max_pages_per_seq * page_size > 0x7fffffffLL ||
      (long long)num_pages * page_size > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (page_size % 16 != 0 || page_size > 256) return ATTN_ERR_UNSUPPORTED;
  if (inv_freq != nullptr && (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16 != 0))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (q != nullptr && (!aligned16(q) || !aligned16(q_out))))
    return ATTN_ERR_ALIGNMENT;
  if (!aligned4(block_table) || !aligned4(seq_lens) ||
      (cu_seqlens != nullptr && !aligned4(cu_seqlens)) ||
      (positions != nullptr && !aligned4(positions)) ||
      (inv_freq != nullptr && (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0) ||
      (fp8 && (!aligned4(k_scale) || !aligned4(v_scale))))
    return ATTN_ERR_ALIGNMENT;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  long long* to[3] = {p.qs, p.ks, p.vs};
  for (int t = 0; t < 3; ++t) {
    to[t][0] = strides != nullptr ? strides[2 * t] : (long long)(t == 0 ? Hq : Hkv) * d;
    to[t][1] = strides != nullptr ? strides[2 * t + 1] : d;
    if (t == 0 && q == nullptr) continue;
    const long long ext[2] = {total, t == 0 ? Hq : Hkv};
    const int bad = rope_check_strides(to[t], ext, 2);
    if (bad != ATTN_OK) return bad;
  }
  // in place only when q is contiguous, as q_out is (strides of extents of one are 0)
  if (total > 0 && q != nullptr && q_out == q &&
      ((total > 1 && p.qs[0] != (long long)Hq * d) || (Hq > 1 && p.qs[1] != d)))
    return ATTN_ERR_INVALID_ARG;
  if (total == 0) return ATTN_OK;
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_CUDA;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.cu = cu_seqlens;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.B = B;
  p.total = (int)total;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.H = Hq + 2 * Hkv;
  p.page_size = page_size;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.rot_chunks = inv_freq != nullptr ? rotary_dim / 16 : 0;
  p.mscale = mscale;
  const int per_block = kRopeThreads / (d / 16);
  p.heads_per_block = rope_heads_per_block((total + per_block - 1) / per_block, p.H, sms,
                                           kAppendBlocks);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (fp8)
    return d == 128 ? launch_append<128, true>(p, interleaved, st)
                    : launch_append<64, true>(p, interleaved, st);
  return d == 128 ? launch_append<128, false>(p, interleaved, st)
                  : launch_append<64, false>(p, interleaved, st);
}

}  // namespace
}  // namespace attn_b200

extern "C" {

int attn_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
              const int32_t* positions, long long pos_stride, int B, int Hq, int Hkv, int S, int d,
              int rotary_dim, int interleaved, float mscale, const long long* strides,
              attn_stream_t stream) {
  return rope_run(q, k, q_out, k_out, inv_freq, positions, pos_stride, B, Hq, Hkv, S, d,
                  rotary_dim, interleaved, mscale, strides, 1.f, stream);
}

int attn_rope_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out,
                  const double* inv_freq, const int32_t* positions, long long pos_stride, int B,
                  int Hq, int Hkv, int S, int d, int rotary_dim, int interleaved, float mscale,
                  const long long* strides, attn_stream_t stream) {
  return rope_run(dq, dk, dq_out, dk_out, inv_freq, positions, pos_stride, B, Hq, Hkv, S, d,
                  rotary_dim, interleaved, mscale, strides, -1.f, stream);
}

int attn_append_paged(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                      void* v_cache, const int32_t* block_table, const int32_t* cu_seqlens,
                      const int32_t* seq_lens, const int32_t* positions, const double* inv_freq,
                      int page_size, int B, int Hq, int Hkv, long long total,
                      int max_pages_per_seq, int num_pages, int d, int rotary_dim,
                      int interleaved, float mscale, const long long* strides,
                      attn_stream_t stream) {
  return append_run(false, q, k, v, q_out, k_cache, v_cache, nullptr, nullptr, block_table,
                    cu_seqlens, seq_lens, positions, inv_freq, page_size, B, Hq, Hkv, total,
                    max_pages_per_seq, num_pages, d, rotary_dim, interleaved, mscale, strides,
                    stream);
}

int attn_append_paged_fp8(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                          void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* block_table, const int32_t* cu_seqlens,
                          const int32_t* seq_lens, const int32_t* positions,
                          const double* inv_freq, int page_size, int B, int Hq, int Hkv,
                          long long total, int max_pages_per_seq, int num_pages, int d,
                          int rotary_dim, int interleaved, float mscale, const long long* strides,
                          attn_stream_t stream) {
  return append_run(true, q, k, v, q_out, k_cache, v_cache, k_scale, v_scale, block_table,
                    cu_seqlens, seq_lens, positions, inv_freq, page_size, B, Hq, Hkv, total,
                    max_pages_per_seq, num_pages, d, rotary_dim, interleaved, mscale, strides,
                    stream);
}

}  // extern "C"
