// decode_window_sm100.cuh -- single-query attention over a paged KV cache with a
// sliding window and visible first tokens.
//
// Mathematics: the query of a sequence of n keys sits at position n - 1 and sees
// keys [max(0, n - window), n) and [0, min(sinks, max(0, n - window))): softmax
// attention over those, by the online recurrence of the decode kernel
// (decode_sm100.cuh), whose warp this kernel uses.
//
// What bounds it: the visible keys' bytes, or, for few sequences, the latency of
// one pass.  A window bounds the keys of a sequence whatever its length, so that
// they fit one cluster of CTAs at most: a CTA of 1 to 4 warps, or a cluster of 2
// to 8 CTAs of 4 warps, takes one (sequence, KV head) (which of these: see
// win_shape), each warp an equal run of its 16-token chunks, and the warps'
// partial results (running maximum, sums and accumulator) are merged in shared
// memory, first within each CTA, then across the cluster's CTAs through
// distributed shared memory.  So there is one launch, no
// workspace, and no partial result in memory; the merge's order is fixed, so
// the result is the same on every run.
//
// Measured (64 sequences, 32 query and 8 KV heads of 128, window 1024, 4 first
// tokens): 48 us for 251 MB of visible bf16 keys and values, 5.2 TB/s, 0.80 of the
// measured copy rate; one sequence 6.2 us, with a window of 128 4.8 us, about 2 us of
// them the launch and the rest dependent loads (length, block table, rows); over an
// E4M3 cache the 64 sequences take 31 us (125 MB).  At most 8 CTAs share a (sequence,
// KV head), so that few sequences with windows of tens of thousands of tokens leave
// SMs idle, which the split kernel fills: 131072 keys, no window, one sequence of 8 KV
// heads 173 us against its 103, of one KV head 177 against 34; 8192 keys 16 against 21.
//
// Chunks: the list of the first tokens' chunks, then the window's (a chunk that
// both touch is listed once).  A 16-bit mask per chunk says which of its tokens
// count; the others, slots behind the sequence's end and pages outside the
// pool among them, may hold anything.
#pragma once

#include "decode_sm100.cuh"

namespace attn_b200 {

constexpr int kWinWarps = 4;  // per CTA, at most

struct DecodeWindowParams {
  DecodeFp8Params f;   // o_part, lse_part, n_split unused
  int window, sinks;   // window >= 1 (INT_MAX: none)
  int cluster;         // CTAs per (sequence, KV head)
};

template <int D, bool FP8>
struct DecodeWinCfg {
  using C = DecodeTmaCfg<D, FP8>;
  static constexpr int RING = C::STAGES * C::STAGE;  // of one warp
  static constexpr int BARS = 128;                   // all warps' mbarriers
  // a merged part: O [8][D] (sums of weights times values), then m, l, lr [8] each
  static constexpr int PART = 8 * D * 4 + 3 * 8 * 4;
  // a CTA of n warps: their rings, barriers, its part; + runtime 1024-byte alignment
  __host__ __device__ static constexpr int smem(int n) { return n * RING + BARS + PART + 1024; }
  // CTAs of n warps that fit an SM: 227 KB, and 64 K registers at MAX_REGS a thread
  static constexpr int CTAS4 = 232448 / (smem(4) + 1024) < 4 ? 232448 / (smem(4) + 1024) : 4;
  static constexpr int MAX_REGS = 65536 / (CTAS4 * 4 * 32);
  __host__ __device__ static constexpr int ctas(int n) {
    return min2(232448 / (smem(n) + 1024), 65536 / (MAX_REGS * 32 * n));
  }
  __host__ __device__ static constexpr int min2(int a, int b) { return a < b ? a : b; }
  static_assert(RING >= PART, "a warp's partial result reuses its ring");
  static_assert(kWinWarps * C::STAGES * 8 <= BARS, "barriers");
};

// Warps per CTA and CTAs per (sequence, KV head).  A CTA's time is about that of
// its prologue (length, block table, first rows: dependent loads, worth four
// steps) and its warps' steps; a grid's is that times its waves of resident
// CTAs, and a second wave is often nearly empty.  So the shape with the least
// waves * (4 + steps) is taken.  Measured on 64 sequences x 8 KV heads, window 1024
// (512 pairs), CTAs of 4 warps were 1.15 waves over an E4M3 cache, 43 us, and
// clusters of 2, 4 and 8 at 8 sequences took 10.4 us (4 CTAs, one wave) and
// 16.4 us (8 CTAs, 1.7 waves).
struct WinShape {
  int warps, cluster;
};

template <int D, bool FP8>
inline WinShape win_shape(long long pairs, int max_chunks, int sms) {
  using W = DecodeWinCfg<D, FP8>;
  constexpr int NH = DecodeTmaCfg<D, FP8>::NH;
  const WinShape shapes[] = {{4, 8}, {4, 4}, {4, 2}, {4, 1}, {3, 1}, {2, 1}, {1, 1}};
  WinShape best = {4, 1};
  long long least = 0;
  for (const WinShape& s : shapes) {
    const long long resident = (long long)W::ctas(s.warps) * sms;
    const long long waves = (pairs * s.cluster + resident - 1) / resident;
    const int warps = s.warps * s.cluster;
    const long long steps = ((max_chunks + warps - 1) / warps + NH - 1) / NH;
    const long long cost = waves * (4 + steps);
    if (least == 0 || cost < least || (cost == least && warps < best.warps * best.cluster)) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// The tokens of chunk `t0 .. t0 + 15` that count, as a bit mask.
__device__ __forceinline__ uint32_t win_chunk_mask(int t0, int lo, int len, int s_end) {
  auto ones = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u; };
  return (ones(len - t0) & ~ones(lo - t0)) | ones(s_end - t0);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;"
               ::: "memory");
}

// An address of this CTA's shared memory, in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kWinWarps * 32, DecodeWinCfg<D, FP8>::CTAS4)
    attn_decode_window_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const DecodeWindowParams wp) {
  using C = DecodeTmaCfg<D, FP8>;
  using W = DecodeWinCfg<D, FP8>;
  constexpr int NH = C::NH;
  const DecodeParams& p = wp.f.d;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_warps = blockDim.x >> 5;
  const int off_bars = n_warps * W::RING, off_part = off_bars + W::BARS;
  const int cs = wp.cluster;
  const int rank = (int)(blockIdx.x % (unsigned)cs);
  const int pair = (int)(blockIdx.x / (unsigned)cs);
  const int kvh = pair % p.Hkv, b = pair / p.Hkv;
  const int hq0 = kvh * p.group;
  const uint32_t ring = sbase + warp * W::RING;
  const uint32_t bars = sbase + off_bars + warp * C::STAGES * 8;

  DecodeWarp<D, FP8> w;
  uint32_t qraw[D / 8];
  w.load_q(qraw, p.q, (size_t)b * p.Hq + hq0, p.group);
  const int len = decode_clamped_len(p, b, threadIdx.x == 0 && rank == 0 && kvh == 0);

  // the chunk list: ns chunks of first tokens, then chunk index + gap
  const int lo = len > wp.window ? len - wp.window : 0;
  const int s_end = min(wp.sinks, lo);
  const int ns = (s_end + 15) / 16;
  const int gap = max(lo / 16, ns) - ns;
  const int n_all = max((len + 15) / 16 - gap, 0);
  // this warp's run of it, whole steps
  const int share = ((n_all + cs * n_warps - 1) / (cs * n_warps) + NH - 1) / NH * NH;
  const int c_begin = min((rank * n_warps + warp) * share, n_all);
  const int c_end = min(c_begin + share, n_all);
  auto chunk_token = [&](int c) { return 16 * (c < ns ? c : c + gap); };

  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) mbar_init(bars + 8u * s, 1);
    mbar_init_fence();
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  __syncwarp();
  w.begin(qraw, p.scale_log2);
  float vmax = FP8 ? 0.f : 1.f;  // E4M3: the unit of the accumulator (0: only zeros so far)
  float vtop = 0.f;              // and the largest V scale met
  int it = 0;        // steps done: ring slot and phase
  bool ok = true;
  // 32 chunks at a time: each lane holds one chunk's page and scales
  for (int c0 = c_begin; ok && c0 < c_end; c0 += 32) {
    const int n_chunks = min(32, c_end - c0);
    const int n_steps = (n_chunks + NH - 1) / NH;
    int my_tok = -1;  // the chunk's first token in the pool
    uint32_t my_vis = 0;
    float my_ks = 0.f, my_vs = 0.f;
    if (lane < n_chunks) {
      const int t = chunk_token(c0 + lane);
      const int pg = p.block_table[(size_t)b * p.max_pages + t / p.page_size];
      if (pg >= 0 && pg < p.num_pages) {
        my_tok = pg * p.page_size + t % p.page_size;
        my_vis = win_chunk_mask(t, lo, len, s_end);
        if (FP8) {
          my_ks = __ldg(wp.f.k_scale + (size_t)pg * p.Hkv + kvh);
          my_vs = __ldg(wp.f.v_scale + (size_t)pg * p.Hkv + kvh);
        }
      } else {
        flag_device_error(kDevErrBadPage);
      }
    }
    auto issue = [&](int i) {  // step i of these chunks
      int tok[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) tok[h] = __shfl_sync(0xffffffffu, my_tok, NH * i + h);
      if (lane == 0) {
        const int slot = (it + i) % C::STAGES;
        decode_issue<D, FP8>(&tm_k, &tm_v, ring + slot * C::STAGE, bars + 8u * slot, kvh, tok);
      }
    };
    int n_issued = 0;
    for (; n_issued < C::STAGES && n_issued < n_steps; ++n_issued) issue(n_issued);
    if (FP8) {
      // The accumulator's unit is the round's own largest V scale, as the split
      // kernel's is for its 512 tokens, so that the round's weights P * vs / unit
      // keep their f16 precision whatever came before.  A round of zero scales keeps
      // the unit, and none is below 2^-64 of the largest (the sums stay finite).
      float m = fabsf(my_vs);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (m > 0.f && m != vmax) {
        vtop = fmaxf(vtop, m);
        m = fmaxf(m, vtop * 0x1p-64f);
        if (vmax > 0.f) {
          const float r = vmax / m;
#pragma unroll
          for (int mc = 0; mc < D / 16; ++mc)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.acc[mc][e] *= r;
        }
        vmax = m;
      }
    }
    const float my_rel = decode_v_rel(my_tok >= 0, my_vs, vmax);
    const float my_kq = my_ks * w.qscale;
    int i = 0;
#pragma unroll 1
    for (; i < n_steps; ++i) {
      const int slot = (it + i) % C::STAGES;
      uint32_t vis[NH];
      float kqc[NH], rel[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int c = NH * i + h;
        vis[h] = __shfl_sync(0xffffffffu, my_vis, c);
        kqc[h] = FP8 ? __shfl_sync(0xffffffffu, my_kq, c) : 1.f;
        rel[h] = FP8 ? __shfl_sync(0xffffffffu, my_rel, c) : 1.f;
      }
      const bool landed =
          mbar_wait(bars + 8u * slot, (uint32_t)((it + i) / C::STAGES) & 1u, nullptr);
      if (!__all_sync(0xffffffffu, landed)) {  // timed out: flagged, wind down
        ok = false;
        break;
      }
      w.step(ring + slot * C::STAGE, p.scale_log2, vis, kqc, rel, [&] {
        if (n_issued < n_steps) issue(n_issued++);
      });
    }
    // after a timed-out wait: no copy may still be landing when the ring is
    // written over below (bounded waits)
    if (lane == 0)
      for (int j = i; j < n_issued; ++j)
        mbar_wait(bars + 8u * ((it + j) % C::STAGES), (uint32_t)((it + j) / C::STAGES) & 1u,
                  nullptr);
    __syncwarp();
    it += i;
  }

  // ---- this warp's part, into its ring: sums [8][D], then m, l, lr [8]
  w.finish_sums();
  {
    float* part = reinterpret_cast<float*>(sptr + warp * W::RING);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float* dst = part + (2 * w.tq + hh) * D + w.g;
#pragma unroll
      for (int mc = 0; mc < D / 16; ++mc) {
        dst[16 * mc] = w.acc[mc][hh] * vmax;
        dst[16 * mc + 8] = w.acc[mc][2 + hh] * vmax;
      }
    }
    if (w.tq == 0) {
      part[8 * D + w.g] = w.m_run;
      part[8 * D + 8 + w.g] = w.l_run;
      part[8 * D + 16 + w.g] = w.lr_run;
    }
  }
  __syncthreads();
  // ---- the CTA's part
  {
    float* out = reinterpret_cast<float*>(sptr + off_part);
    auto part = [&](int i) { return reinterpret_cast<const float*>(sptr + i * W::RING); };
    for (int e = threadIdx.x * 4; e < p.group * D; e += blockDim.x * 4) {
      const int h = e / D;
      float m[kWinWarps], ls[kWinWarps], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWinWarps; ++i) {
        m[i] = i < n_warps ? part(i)[8 * D + h] : -INFINITY;
        ls[i] = i < n_warps ? part(i)[8 * D + 8 + h] : 0.f;
        mx = fmaxf(mx, m[i]);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f, lr = 0.f;
#pragma unroll
      for (int i = 0; i < kWinWarps; ++i) {
        if (ls[i] == 0.f) continue;  // saw nothing (scores of NaN leave m at -inf, but l NaN)
        const float f = ex2(m[i] - mx);
        const float4 x = *reinterpret_cast<const float4*>(part(i) + e);
        sum.x = fmaf(f, x.x, sum.x);
        sum.y = fmaf(f, x.y, sum.y);
        sum.z = fmaf(f, x.z, sum.z);
        sum.w = fmaf(f, x.w, sum.w);
        l = fmaf(f, ls[i], l);
        lr = fmaf(f, part(i)[8 * D + 16 + h], lr);
      }
      *reinterpret_cast<float4*>(out + e) = sum;
      if (e % D == 0) {
        out[8 * D + h] = mx;
        out[8 * D + 8 + h] = l;
        out[8 * D + 16 + h] = lr;
      }
    }
  }
  cluster_sync();
  // ---- the result: the cluster's CTAs share its elements
  {
    const uint32_t local = sbase + off_part;
    const int n_threads = cs * blockDim.x;
    for (int e = (rank * (int)blockDim.x + (int)threadIdx.x) * 4; e < p.group * D;
         e += n_threads * 4) {
      const int h = e / D;
      float m[8], ls[8], mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = i < cs ? cluster_ld(cluster_map(local + (8 * D + h) * 4, i)) : -INFINITY;
        ls[i] = i < cs ? cluster_ld(cluster_map(local + (8 * D + 8 + h) * 4, i)) : 0.f;
        mx = fmaxf(mx, m[i]);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f, lr = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (ls[i] == 0.f) continue;
        const float f = ex2(m[i] - mx);
        const float4 x = cluster_ld4(cluster_map(local + e * 4, i));
        sum.x = fmaf(f, x.x, sum.x);
        sum.y = fmaf(f, x.y, sum.y);
        sum.z = fmaf(f, x.z, sum.z);
        sum.w = fmaf(f, x.w, sum.w);
        l = fmaf(f, ls[i], l);
        lr = fmaf(f, cluster_ld(cluster_map(local + (8 * D + 16 + h) * 4, i)), lr);
      }
      const float inv = lr == 0.f ? 0.f : 1.f / lr;
      const size_t row = (size_t)b * p.Hq + hq0 + h;
      uint2 o;
      o.x = pack_bf16x2(sum.x * inv, sum.y * inv);
      o.y = pack_bf16x2(sum.z * inv, sum.w * inv);
      *reinterpret_cast<uint2*>(p.o + row * D + e % D) = o;
      if (p.lse != nullptr && e % D == 0)
        p.lse[row] = l == 0.f ? -INFINITY : (mx + lg2(l)) * 0.69314718055994531f;
    }
  }
  cluster_sync();  // no CTA leaves while another may read its part
}

}  // namespace attn_b200
