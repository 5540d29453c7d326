// Rotary positions, and the write of new keys and values into a bf16 cache with
// the keys rotated on the way, sm_103a.
//
// A token at position p turns the pair (x1, x2) number i of a head by the angle
// a = p * inv_freq[i]:  y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
// (m: magnitude; the gradient of this map is the same with -a).  Pairs are the
// columns (i, i + r/2) or (2i, 2i + 1) of the first r; the others are copied.
//
// The angle.  p * inv_freq in fp32 is off by 2^-24 of itself: 0.06 rad at a
// million.  Here a frequency is a whole number of 2^-64 turns, made once a block
// from 128 bits of 1 / (2 pi) (an fp64 product would be off by 2^-53 of the frequency's
// turns: 0.2 rad at position 2^31 for a million radians a position); the product with the
// position modulo 2^64 is the fraction of a turn to a unit for each position (integers
// wrap as turns do), and its upper 32 bits, as a signed number of half turns in [-1, 1),
// go to sincospif: the angle is good to 2^-24 half turns at any position, for frequencies
// up to 2^53.
//
// Work split: a lane owns 2 x 8 values of a token's rows, the pieces that hold
// eight pairs, and keeps their 8 sines and cosines in registers while it walks
// over the heads (queries, keys, values) of its group; a warp takes 32 / (D / 16)
// neighbouring tokens, so heads-first tensors are read in runs of 1 KB / 2, and
// tokens-first ones row by row.  Heads are split over warps only as far as the GPU
// needs warps.  Bound by HBM: 4 bytes a value; the arithmetic takes half of the issue slots.
// Measured: 28 + 4 heads of 128 over 8192 tokens, 134 MB, 24.8 us (5.4 TB/s, the reads from
// HBM, the writes still partly in L2); gradients of 710 MB 108 us (6.6 TB/s); an append of
// 16 prompts, 855 MB, 142 us (6.0 TB/s); of one token to each of 16 sequences 2.8 us.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // heads in flight in a lane (8 loads of 16 bytes)

struct RopeKParams {
  RopeArgs a;
  int head_groups, heads_per_group;
  long long token_groups;
  uint32_t* err_word;
};

// Turns a position, without whole ones, in units of 2^-64: the 53 bits of f times those of
// 1 / (2 pi) at f's exponent, in whole numbers (a few multiplications; fp64 takes longer here).
__device__ __forceinline__ unsigned long long turns64(double f) {
  // 2^128 / (2 pi), rounded down.
  constexpr unsigned __int128 kTurn = ((unsigned __int128)0x28be60db9391054aull << 64) | 0x7f09d5f47d4d3770ull;
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const unsigned long long m = (bits & ((1ull << 52) - 1)) | (1ull << 52);
  const int down = 1075 - (int)((bits >> 52) & 0x7ff);  // f = m 2^-down
  unsigned __int128 w = 0;
  if (down >= 0 && down < 128) w = kTurn >> down;
  if (down < 0 && down > -128) w = kTurn << -down;
  const unsigned long long t = (unsigned long long)((w * m) >> 64);
  return bits >> 63 ? 0ull - t : t;
}

// Turns eight pairs: pieces a and b of 8 bf16 each.  Half layout: pair j is
// (a[j], b[j]); neighbouring pairs: (a[2j], a[2j + 1]) for j < 4, b's behind them.
template <bool INTER>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float (&cs)[8],
                                     const float (&sn)[8]) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
  auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a1 = lo(pa[j]), a2 = hi(pa[j]), b1 = lo(pb[j]), b2 = hi(pb[j]);
      pa[j] = pack_bf16x2(a1 * cs[j] - a2 * sn[j], a2 * cs[j] + a1 * sn[j]);
      pb[j] = pack_bf16x2(b1 * cs[j + 4] - b2 * sn[j + 4], b2 * cs[j + 4] + b1 * sn[j + 4]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a1 = lo(pa[j]), a2 = hi(pa[j]), b1 = lo(pb[j]), b2 = hi(pb[j]);
      const float c0 = cs[2 * j], s0 = sn[2 * j], c1 = cs[2 * j + 1], s1 = sn[2 * j + 1];
      pa[j] = pack_bf16x2(a1 * c0 - b1 * s0, a2 * c1 - b2 * s1);
      pb[j] = pack_bf16x2(b1 * c0 + a1 * s0, b2 * c1 + a2 * s1);
    }
  }
}

// The sequence of packed row t: the last one that starts at or before it, found
// by the warp with 32 probes at a time.  Entries are clamped to [0, total].
__device__ __forceinline__ int find_seq(const int32_t* cu, int num_seqs, int total, int t,
                                        int lane) {
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int probe = lo + lane * step;
    const bool before = probe < hi && (lane == 0 || min(max(cu[probe], 0), total) <= t);
    const int top = 31 - __clz(__ballot_sync(0xffffffffu, before));
    lo += top * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// APPEND: keys and values go to the cache (RopeArgs' cache part); otherwise q and
// k are (batch, heads, tokens) with strides of their own.
template <int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeKParams p) {
  constexpr int kLanes = D / 16;         // lanes of a token's row
  constexpr int kTokens = 32 / kLanes;   // tokens of a warp
  __shared__ unsigned long long s_step[D / 2];
  const RopeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lc = lane % kLanes, lt = lane / kLanes;
  grid_dep_wait();
  const int half = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < half; i += kThreads) s_step[i] = turns64(a.inv_freq[i]);
  if (APPEND && a.cu_seqlens != nullptr && blockIdx.x == 0) {
    bool bad = false;
    for (int i = threadIdx.x; i < a.batch; i += kThreads) {
      const int x = a.cu_seqlens[i], y = a.cu_seqlens[i + 1];
      bad |= x > y || x < 0 || y > a.tokens || (i == 0 && x != 0);
    }
    if (bad) atomicOr(p.err_word, kErrSeqLens);
  }
  __syncthreads();
  const bool rot = lc < a.rotary_dim / 16;
  // Columns of this lane's two pieces.
  const int rest = (D - a.rotary_dim) / 2, c2 = lc - a.rotary_dim / 16;
  const int col_a = rot ? 8 * lc : a.rotary_dim + 8 * c2;
  const int off_b = rot ? half : rest;
  const long long items = p.token_groups * p.head_groups;
  for (long long it = (long long)blockIdx.x * kWarps + warp; it < items;
       it += (long long)gridDim.x * kWarps) {
    const long long tg = it % p.token_groups;
    const int h0 = (int)(it / p.token_groups) * p.heads_per_group;
    const int h1 = min(h0 + p.heads_per_group, a.n_q_heads + (APPEND ? 2 : 1) * a.n_kv_heads);
    const long long t = tg * kTokens + lt;  // token (rope: of all sequences)
    bool live;
    int pos = 0;
    const uint16_t *q_in, *k_in, *v_in = nullptr;
    uint16_t *q_out, *k_out, *v_out = nullptr;
    bool kv_live;
    long long k_out_hs;
    if constexpr (APPEND) {
      int s = -1, c0 = 0, c1 = 0;
      if (a.cu_seqlens == nullptr) {
        s = (int)t, c0 = (int)t, c1 = (int)t + 1;
      } else {
        int ws = 0, w0 = 0, w1 = 0;  // the sequence found last
#pragma unroll 1
        for (int i = 0; i < kTokens; ++i) {
          const int ti = (int)(tg * kTokens) + i;
          if (ti >= a.tokens) break;
          if (ti < w0 || ti >= w1) {
            ws = find_seq(a.cu_seqlens, a.batch, a.tokens, ti, lane);
            w0 = min(max(a.cu_seqlens[ws], 0), a.tokens);
            w1 = min(max(a.cu_seqlens[ws + 1], 0), a.tokens);
          }
          if (i == lt) s = ws, c0 = w0, c1 = w1;
        }
      }
      live = t < a.tokens && t >= c0 && t < c1;
      long long row = 0;
      kv_live = false;
      if (live) {
        const int start = a.kv_lens[s], slot = start + (int)(t - c0);
        pos = a.positions ? a.positions[t] : slot;
        if (start < 0 || (long long)start + (c1 - c0) > a.capacity()) {
          if (lc == 0) atomicOr(p.err_word, kErrKvLen);
        } else if (a.block_table == nullptr) {
          row = (long long)s * a.max_kv_len + slot;
          kv_live = true;
        } else {
          const int blk = a.block_table[(size_t)s * a.max_blocks_per_seq + slot / a.block_size];
          if (blk < 0 || blk >= a.num_blocks) {
            if (lc == 0) atomicOr(p.err_word, kErrBlockIndex);
          } else {
            row = (long long)blk * a.block_size + slot % a.block_size;
            kv_live = true;
          }
        }
      }
      const long long tt = live ? t : 0;
      q_in = a.q + tt * a.q_s.token + col_a;
      q_out = a.q_out + tt * a.qo_s.token + col_a;
      k_in = a.k + tt * a.k_s.token + col_a;
      v_in = a.v + tt * a.v_s.token + col_a;
      k_out = a.k_out + row * a.n_kv_heads * D + col_a;
      v_out = a.v_out + row * a.n_kv_heads * D + col_a;
      k_out_hs = D;
    } else {
      live = kv_live = t < (long long)a.batch * a.tokens;
      const long long tt = live ? t : 0;
      const int b = (int)(tt / a.tokens), n = (int)(tt - (long long)b * a.tokens);
      pos = a.positions ? a.positions[b * a.pos_batch_stride + n] : n;
      q_in = a.q + b * a.q_s.batch + n * a.q_s.token + col_a;
      q_out = a.q_out + b * a.qo_s.batch + n * a.qo_s.token + col_a;
      k_in = a.k + b * a.k_s.batch + n * a.k_s.token + col_a;
      k_out = a.k_out + b * a.ko_s.batch + n * a.ko_s.token + col_a;
      k_out_hs = a.ko_s.head;
    }
    if (!live) continue;
    float cs[8], sn[8];
    if (rot) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // Pair numbers: 8 lc + j, or 4 lc + j in piece a and r/4 + 4 lc + j in b.
        const int i = INTER ? 4 * lc + (j & 3) + (j >= 4 ? half / 2 : 0) : 8 * lc + j;
        const unsigned long long turns = s_step[i] * (unsigned long long)(long long)pos;
        sincospif((float)(int)(turns >> 32) * 4.656612873077393e-10f, &sn[j], &cs[j]);  // 2^-31
        cs[j] *= a.magnitude;
        sn[j] *= a.sin_factor;
      }
    }
    const bool skip_copy = !APPEND && !rot;  // in place, columns that are not turned stay
    for (int hb = h0; hb < h1; hb += kUnroll) {
      uint4 xa[kUnroll], xb[kUnroll];
      uint16_t* dst[kUnroll];
      bool turned[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = hb + u;
        const uint16_t* src = nullptr;
        dst[u] = nullptr;
        turned[u] = rot;
        if (h < h1) {
          if (h < a.n_q_heads) {
            src = q_in + h * a.q_s.head;
            dst[u] = q_out + h * a.qo_s.head;
          } else if (h < a.n_q_heads + a.n_kv_heads) {
            src = k_in + (h - a.n_q_heads) * a.k_s.head;
            if (kv_live) dst[u] = k_out + (h - a.n_q_heads) * k_out_hs;
          } else if constexpr (APPEND) {
            src = v_in + (h - a.n_q_heads - a.n_kv_heads) * a.v_s.head;
            if (kv_live) dst[u] = v_out + (h - a.n_q_heads - a.n_kv_heads) * (long long)D;
            turned[u] = false;
          }
          if (skip_copy && src == dst[u]) dst[u] = nullptr;
        }
        if (dst[u] != nullptr) {
          xa[u] = *reinterpret_cast<const uint4*>(src);
          xb[u] = *reinterpret_cast<const uint4*>(src + off_b);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (dst[u] == nullptr) continue;
        if (turned[u]) turn<INTER>(xa[u], xb[u], cs, sn);
        *reinterpret_cast<uint4*>(dst[u]) = xa[u];
        *reinterpret_cast<uint4*>(dst[u] + off_b) = xb[u];
      }
    }
  }
}

template <int D, bool APPEND>
cudaError_t launch_t(const RopeArgs& a, const LaunchCtx& ctx) {
  constexpr int kTokens = 32 / (D / 16);
  RopeKParams p;
  p.a = a;
  p.err_word = ctx.err_word;
  const long long tokens = APPEND ? a.tokens : (long long)a.batch * a.tokens;
  p.token_groups = (tokens + kTokens - 1) / kTokens;
  const int heads = a.n_q_heads + (APPEND ? 2 : 1) * a.n_kv_heads;
  // Heads of a warp, which share its sines and cosines: as many as leave the GPU 8 warps an SM,
  // up to 8.  With 16 warps, and so fewer heads each: a prompt of 512 with 28 + 4 heads 5.4 us
  // (3.9), of 2048 9.6 (8.5), 16 trees of 64 nodes into the cache 10.3 (8.9); from 4096 rows on
  // and up to 256 the same.  With 4 warps: 3.6, 8.7, 8.8.  Up to 4 heads: 8192 rows 26.0 (24.7),
  // 16 prompts into the cache 163 (142); up to 16: 26.2, 134.
  const long long want = 8LL * std::max(ctx.num_sms, 1);
  int hpg = 8;
  while (hpg > 1 && p.token_groups * ((heads + hpg - 1) / hpg) < want) hpg /= 2;
  p.heads_per_group = hpg;
  p.head_groups = (heads + hpg - 1) / hpg;
  const long long blocks = (p.token_groups * p.head_groups + kWarps - 1) / kWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(blocks, 64LL * std::max(ctx.num_sms, 1)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.interleaved ? cudaLaunchKernelEx(&cfg, rope_kernel<D, true, APPEND>, p)
                       : cudaLaunchKernelEx(&cfg, rope_kernel<D, false, APPEND>, p);
}

template <bool APPEND>
cudaError_t launch_d(const RopeArgs& a, const LaunchCtx& ctx) {
  if (a.head_dim == 256) return launch_t<256, APPEND>(a, ctx);
  if (a.head_dim == 128) return launch_t<128, APPEND>(a, ctx);
  return launch_t<64, APPEND>(a, ctx);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, const LaunchCtx& ctx) { return launch_d<false>(a, ctx); }
cudaError_t launch_cache_append(const RopeArgs& a, const LaunchCtx& ctx) {
  return launch_d<true>(a, ctx);
}

}  // namespace attn
