// rope_sm100.cuh -- rotary positions, and the append of rotated keys and values
// to a paged cache.
//
// Mathematics.  A head row x of d elements has R = 2 n rotated elements, read
// as n pairs (a_i, b_i): elements (i, i + n) in the half layout, (2i, 2i + 1)
// in the interleaved one; elements R .. d-1 pass unchanged.  At position p the
// pair turns by t_i = p * inv_freq[i] and is scaled by m:
//     a' = m (a cos t - b sin t),   b' = m (a sin t + b cos t).
// The map is linear and, up to m, orthogonal, so its gradient is the same map
// with -t: the backward kernel is this one with the sine's sign turned.
//
// Angles.  t reaches millions of radians at far positions, where an fp32
// product p * inv_freq is off by whole radians' fractions.  The number of
// turns, p * inv_freq / (2 pi), is formed and reduced to [-1/2, 1/2] in
// fp64; the sine and cosine of the remainder are taken in fp32, good to about
// 5e-7, far below the bf16 (2^-8 of the value) rounding of the result.  The
// rotation itself is fp32, rounded once on the way out.
//
// Organisation.  A thread owns 8 pairs of one token (16 elements, two 16-byte
// pieces), computes their cosines and sines once, and applies them to a run of
// heads: the angles are shared by all heads of a token, so that what the run
// costs is its loads and stores, and these bound the kernel: 29.4 us for 8192
// tokens x 40 heads of 128 (168 MB, 5.7 TB/s; an elementwise kernel over as many
// contiguous bytes takes 26.4 us).  Without the angles it takes 27.9 us.  Tried
// and slower: fewer or more rows in flight, loads issued before the angles
// (fewer blocks fit an SM), angles shared through shared memory.  Nothing is
// shared between threads; no shared memory and no barrier is used.  A thread
// reads both of its pieces of a row before it writes either, which is what
// makes a rotation in place safe.
#pragma once

#include "sm100_primitives.cuh"

namespace attn_b200 {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads whose rows a thread has in flight

struct RopeParams {
  const uint16_t* q;      // element (b, h, s, :) at b * qs[0] + h * qs[1] + s * qs[2]
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  long long qs[3], ks[3], qos[3], kos[3];
  const double* inv_freq;  // [R / 2] radians per position
  const int* positions;    // row b at b * pos_stride, or nullptr: s
  long long pos_stride;
  int S, Hq, H;            // H = Hq + Hkv heads in all
  long long n_tokens;      // B * S
  int rot_chunks;          // R / 16: chunks of 8 pairs that turn
  int heads_per_block;
  float mscale, sin_sign;
};

// A 16-byte load of data that is read once (no L1 line is kept; the line may be
// written by this kernel, when it works in place, so it is not a read-only load).
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// Element offsets of the two 8-element pieces of chunk c of a head row.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_pieces(int c, int rot_chunks, int& e0, int& e1) {
  if (INTERLEAVED || c >= rot_chunks) {  // 16 neighbours (the unrotated tail is copied so)
    e0 = 16 * c;
    e1 = e0 + 8;
  } else {
    e0 = 8 * c;
    e1 = 8 * rot_chunks + 8 * c;
  }
}

// The fraction of a turn that t turns leave, in [-1/2, 1/2] to 2^-33, for |t| <
// 2^51.  Additions do the roundings (1.5 * 2^52 leaves whole turns, 1.5 * 2^20
// leaves 32 bits of fraction in the low word): the fp64 rounding and conversion
// instructions run at a small part of their rate.
__device__ __forceinline__ float rope_fraction(double t) {
  const double whole = __dadd_rn(__dadd_rn(t, 6755399441055744.0), -6755399441055744.0);
  const double r = __dadd_rn(t, -whole);
  return (float)__double2loint(__dadd_rn(r, 1572864.0)) * 2.3283064365386963e-10f;  // 2^-32
}

// cos and sin (times m, and the sine's sign) of chunk c's 8 pairs at position
// pos.  The angle is reduced already, so that the fast sine and cosine are
// good to 2^-21 of the pair's size, 2^12 below the result's rounding.
__device__ __forceinline__ void rope_angles(const double* inv_freq, int c, int pos, float mscale,
                                            float sin_sign, float (&cs)[8], float (&sn)[8]) {
  const double p = (double)pos * 0.15915494309189533576888;  // 1 / (2 pi): turns per radian
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = 6.2831853071795865f * rope_fraction(p * __ldg(inv_freq + 8 * c + i));
    cs[i] = __cosf(t) * mscale;
    sn[i] = __sinf(t) * (mscale * sin_sign);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The 16 elements of a chunk as fp32, turned: y[0..7] goes to piece 0, y[8..15] to piece 1.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_turn(uint4 x0, uint4 x1, const float (&cs)[8],
                                          const float (&sn)[8], float (&y)[16]) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = INTERLEAVED ? bf16_lo(w[i]) : (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    const float b = INTERLEAVED  ? bf16_hi(w[i])
                    : (i & 1) ? bf16_hi(w[4 + i / 2])
                              : bf16_lo(w[4 + i / 2]);
    y[INTERLEAVED ? 2 * i : i] = a * cs[i] - b * sn[i];
    y[INTERLEAVED ? 2 * i + 1 : 8 + i] = a * sn[i] + b * cs[i];
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// Grid: x over tiles of 256 / (d / 16) tokens, y over runs of heads_per_block heads.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) attn_rope_kernel(const RopeParams p) {
  constexpr int TPT = D / 16;  // threads (chunks) per token
  const int c = threadIdx.x % TPT;
  const long long token = (long long)blockIdx.x * (kRopeThreads / TPT) + threadIdx.x / TPT;
  if (token >= p.n_tokens) return;
  const long long b = token / p.S;
  const int s = (int)(token - b * p.S);
  const bool turns = c < p.rot_chunks;
  int e0, e1;
  rope_pieces<INTERLEAVED>(c, p.rot_chunks, e0, e1);
  const int h_begin = blockIdx.y * p.heads_per_block;
  const int h_end = min(h_begin + p.heads_per_block, p.H);
  const uint16_t* q_src = p.q + b * p.qs[0] + s * p.qs[2];
  const uint16_t* k_src = p.k + b * p.ks[0] + s * p.ks[2];
  uint16_t* q_dst = p.q_out + b * p.qos[0] + s * p.qos[2];
  uint16_t* k_dst = p.k_out + b * p.kos[0] + s * p.kos[2];
  // A few heads' pieces are in flight together: the kernel is bound by its loads
  // and stores.
  uint4 x0[kRopeBatch], x1[kRopeBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (h + i < h_end) {
        const uint16_t* src =
            h + i < p.Hq ? q_src + (h + i) * p.qs[1] : k_src + (h + i - p.Hq) * p.ks[1];
        x0[i] = ld_once_v4(src + e0);
        x1[i] = ld_once_v4(src + e1);
      }
    }
  };
  float cs[8], sn[8];
  if (turns) {
    const int pos = p.positions == nullptr ? s : __ldg(p.positions + b * p.pos_stride + s);
    rope_angles(p.inv_freq, c, pos, p.mscale, p.sin_sign, cs, sn);
  }
  for (int h = h_begin; h < h_end; h += kRopeBatch) {
    load(h);
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (h + i < h_end) {
        uint16_t* dst =
            h + i < p.Hq ? q_dst + (h + i) * p.qos[1] : k_dst + (h + i - p.Hq) * p.kos[1];
        if (turns) {
          float y[16];
          rope_turn<INTERLEAVED>(x0[i], x1[i], cs, sn, y);
          x0[i] = pack_bf16x8(y);
          x1[i] = pack_bf16x8(y + 8);
        }
        *reinterpret_cast<uint4*>(dst + e0) = x0[i];
        *reinterpret_cast<uint4*>(dst + e1) = x1[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append: token t of the packed batch belongs to sequence b, cu[b] <= t <
// cu[b+1], and is key number seq_lens[b] - (cu[b+1] - t) of it; its K and V go
// to row (key % page_size) of page block_table[b][key / page_size].  Without
// cu there is one token per sequence (decode), key number seq_lens[b] - 1.
// K (and Q, when it is given) are rotated on the way; V is copied.  For an
// E4M3 cache the values are divided by the page's scale and rounded once.
// Measured: 10341 tokens x 48 heads of 128 in 8 chunks, 46.9 us (254 MB, 5.4 TB/s; an
// elementwise kernel over as many contiguous bytes takes 38.9 us); 64 single
// tokens 2.75 us, little more than a launch; as many tokens into an E4M3 cache, whose 16
// values of a thread and head are divided one by one, 66.7 us (233 MB).  Its blocks begin with a chain of
// dependent loads (offsets, length, block table); looking places up and sharing
// angles through shared memory, for blocks that take whole tokens, measured 49 us
// and 3.3 us.
// ---------------------------------------------------------------------------
struct AppendParams {
  const uint16_t* q;   // nullptr: no queries
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;     // [total, Hq, d]
  void* k_cache;       // [num_pages, page_size, Hkv, d] bf16 or E4M3 codes
  void* v_cache;
  const float* k_scale;  // [num_pages, Hkv] (E4M3 caches)
  const float* v_scale;
  const int* block_table;
  const int* cu;         // [B + 1] or nullptr
  const int* seq_lens;   // [B]
  const int* positions;  // [total] or nullptr: the key's number
  const double* inv_freq;
  long long qs[2], ks[2], vs[2];  // token and head strides
  int B, total, Hq, Hkv, H, page_size, max_pages, num_pages;  // H = Hq + 2 Hkv
  int rot_chunks, heads_per_block;
  float mscale;
};

// The sequence of packed token t: the last b with cu[b] <= t (or -1), found by halving.
__device__ __forceinline__ int append_sequence(const int* cu, int B, int t) {
  int lo = -1, hi = B;  // cu[lo] <= t < cu[hi] while the offsets do not decrease
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Where token t goes: its sequence and key number, or false when it goes
// nowhere (a token of no sequence, an idle sequence, or offsets and lengths
// that do not fit each other, which are flagged).
__device__ __forceinline__ bool append_place(const AppendParams& p, int t, int& b, int& key) {
  const long long cap = (long long)p.max_pages * p.page_size;
  if (p.cu == nullptr) {
    b = t;
    const int len = __ldg(p.seq_lens + b);
    if (len == 0) return false;  // an idle row of the batch
    if (len < 0 || len > cap) {
      flag_device_error(kDevErrBadLength);
      return false;
    }
    key = len - 1;
    return true;
  }
  b = append_sequence(p.cu, p.B, t);
  if (b < 0) return false;
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  if (t >= c1) return false;  // behind the last sequence, or (offsets that decrease) in none
  const int len = __ldg(p.seq_lens + b);
  if (c0 < 0 || c1 > p.total || len < c1 - c0 || len > cap) {
    flag_device_error(kDevErrBadLength);
    return false;
  }
  key = len - (c1 - t);
  return true;
}

// Two floats -> two E4M3 codes (nearest, saturating at +-448); `lo` in bits 0-7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values over a scale as E4M3 codes; a zero scale stands for a page of zeros.
__device__ __forceinline__ uint2 pack_e4m3x8(const float* y, float scale) {
  if (scale == 0.f) return make_uint2(0u, 0u);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = y[i] / scale;
  return make_uint2(pack_e4m3x2(z[0], z[1]) | (pack_e4m3x2(z[2], z[3]) << 16),
                    pack_e4m3x2(z[4], z[5]) | (pack_e4m3x2(z[6], z[7]) << 16));
}

template <int D, bool INTERLEAVED, bool FP8>
__global__ void __launch_bounds__(kRopeThreads) attn_append_kernel(const AppendParams p) {
  constexpr int TPT = D / 16;
  if (p.cu != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.B; i += kRopeThreads)
      if (__ldg(p.cu + i) > __ldg(p.cu + i + 1)) flag_device_error(kDevErrBadLength);
  const int c = threadIdx.x % TPT;
  const long long token_ll = (long long)blockIdx.x * (kRopeThreads / TPT) + threadIdx.x / TPT;
  if (token_ll >= p.total) return;
  const int t = (int)token_ll;
  int b, key;
  if (!append_place(p, t, b, key)) return;
  const int h_begin = blockIdx.y * p.heads_per_block;
  const int h_end = min(h_begin + p.heads_per_block, p.H);
  const int h_k = p.Hq, h_v = p.Hq + p.Hkv;  // first K and V head of the head index
  int page = -1;
  if (h_end > h_k) {
    page = __ldg(p.block_table + (size_t)b * p.max_pages + key / p.page_size);
    if (page < 0 || page >= p.num_pages) {
      flag_device_error(kDevErrBadPage);
      page = -1;
    }
  }
  const bool turns = c < p.rot_chunks;
  float cs[8], sn[8];
  if (turns && h_begin < h_v) {
    const int pos = p.positions == nullptr ? key : __ldg(p.positions + t);
    rope_angles(p.inv_freq, c, pos, p.mscale, 1.f, cs, sn);
  }
  int e0, e1;
  rope_pieces<INTERLEAVED>(c, p.rot_chunks, e0, e1);
  for (int h = h_begin; h < h_end; ++h) {
    const bool is_q = h < h_k, is_v = h >= h_v;
    if (!is_q && page < 0) continue;
    const int hh = is_q ? h : is_v ? h - h_v : h - h_k;
    const long long* si = is_q ? p.qs : is_v ? p.vs : p.ks;
    const uint16_t* src = (is_q ? p.q : is_v ? p.v : p.k) + (long long)t * si[0] + hh * si[1];
    const uint4 x0 = *reinterpret_cast<const uint4*>(src + e0);
    const uint4 x1 = *reinterpret_cast<const uint4*>(src + e1);
    const size_t row = is_q ? (size_t)t * p.Hq + hh
                            : ((size_t)page * p.page_size + key % p.page_size) * p.Hkv + hh;
    const bool turn = turns && !is_v;
    if (FP8 && !is_q) {
      float y[16];
      if (turn) {
        rope_turn<INTERLEAVED>(x0, x1, cs, sn, y);
      } else {
        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[2 * i] = bf16_lo(w[i]);
          y[2 * i + 1] = bf16_hi(w[i]);
        }
      }
      const float scale = __ldg((is_v ? p.v_scale : p.k_scale) + (size_t)page * p.Hkv + hh);
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + row * D;
      *reinterpret_cast<uint2*>(dst + e0) = pack_e4m3x8(y, scale);
      *reinterpret_cast<uint2*>(dst + e1) = pack_e4m3x8(y + 8, scale);
    } else {
      uint16_t* dst =
          (is_q ? p.q_out : static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache)) + row * D;
      if (turn) {
        float y[16];
        rope_turn<INTERLEAVED>(x0, x1, cs, sn, y);
        *reinterpret_cast<uint4*>(dst + e0) = pack_bf16x8(y);
        *reinterpret_cast<uint4*>(dst + e1) = pack_bf16x8(y + 8);
      } else {
        *reinterpret_cast<uint4*>(dst + e0) = x0;
        *reinterpret_cast<uint4*>(dst + e1) = x1;
      }
    }
  }
}

}  // namespace attn_b200
