// Split-KV single-token decode over a key/value cache held in 8 bits, sm_103a.
//
// The bf16 decode's plan (one block per (split, kv head, sequence), the cache
// streamed once through a shared-memory ring and used for all g query heads of
// the kv head, partials merged by their LSE weights) with half the bytes to
// stream, so twice the arithmetic a byte: what a row costs between its arrival
// and its products has to be half of the bf16 kernel's.  The mathematics is
// arranged for that:
//
//   * codes go from shared memory into the tensor core's fragments as fp16
//     (exact: e4m3 is a subset of fp16) with one conversion for two values and
//     no multiplication.  K's scale is a factor of the score and V's of the
//     weight, one number a token each.  For q k the 32-bit register that
//     ldmatrix delivers (4 codes of one token) becomes a B fragment's two
//     registers when the head dimension is taken in the order 4q, 4q+1 | 4q+2,
//     4q+3, which q's fragments follow.  For p v a transposed ldmatrix delivers
//     2 tokens x 2 columns; one byte permutation separates the columns, and the
//     even and odd columns of 16 form one n tile each, so a thread ends up with
//     4 neighbouring columns.
//   * q is scaled by a power of two per row into fp16's range (exact: 8
//     significant bits) and the power is taken back in the score's factor.
//   * weights are split into two fp16 parts, hi + lo (22 bits), so that the
//     fp32 output is not limited by an operand's rounding.  With up to 8 query
//     heads per kv head the parts fill the 16 rows of one product (rows 0-7 hi,
//     8-15 lo), which would be half empty otherwise: no extra product.  With
//     more heads a second product adds the lo parts.
//   * a product's sums over 16 tokens start from zero and are added to O by the
//     FP32 pipe, hi and lo rows together (the tensor core truncates its sums:
//     over 100000 tokens in one split O came out 3e-5 too small).  That also
//     halves the accumulators of the form with up to 8 heads.
//   * the exponentials' reference m bounds score + log2(V's scale), the size of
//     a weight times its scale: weights lie below 2^(kShift + kGrow) = 2^14 and
//     those down to 2^-24 of the largest keep full fp16 precision in hi.  The
//     sum l is taken over the unscaled weights in fp32.  The row maximum is
//     only reduced over the quad when some score exceeds m by 2^kGrow.
//   * masked tokens are cut off in the score and, for V, in the fragment, so
//     nothing that lies in masked places (NaN codes or scales) is used.
#include <cstdint>
#include <cstring>
#include <mutex>
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kStageTokens = 64;   // tokens of a ring stage
constexpr int kConsumerWarps = 4;  // 16 tokens of a stage each
constexpr int kThreads = 32 * (1 + kConsumerWarps);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 4.f;       // log2 units a score may exceed the reference by
constexpr float kShift = 10.f;     // log2 of the weight at the reference

// Where q's fragments live during the stream: registers, or shared memory
// where the accumulators leave no room for them.
__host__ __device__ constexpr bool q_in_smem(int D, bool wide) { return wide || D == 256; }
__host__ __device__ constexpr int q_smem_bytes(int D, bool wide, int groups) {
  return q_in_smem(D, wide) ? groups * (D / 16) * 32 * (wide ? 16 : 8) : 0;
}

// How the producer fills a stage.
enum LoadMode : int { kLoadBox64 = 0, kLoadBox16 = 1, kLoadRows = 2 };

template <int D>
struct Smem {
  static constexpr int kSpan = D < 128 ? D : 128;          // bytes of a swizzled row
  static constexpr int kSpans = D / kSpan;
  static constexpr int kSpanBytes = kStageTokens * kSpan;  // one span of a stage's rows
  static constexpr int kTileBytes = kSpans * kSpanBytes;   // K or V
  static constexpr int kScaleBytes = 2 * kStageTokens * 4;
  static constexpr int kPitch = D + 16;                    // floats of a merged row
  static constexpr int kMaxStages = 16;
  static constexpr int kBar = 0;                           // full, empty
  static constexpr int kFlag = 16 * kMaxStages;
  static constexpr int kMerge = kFlag + 16;                // m, l, weight: [3][4][16]
  static constexpr int kScale = kMerge + 3 * kConsumerWarps * 16 * 4;
  // then the stages' scales, q's fragments, and the ring
  __host__ __device__ static int q_off(int stages) { return kScale + stages * kScaleBytes; }
  __host__ __device__ static int ring_off(int stages, int q_bytes) {
    return (q_off(stages) + q_bytes + 1023) / 1024 * 1024;
  }
  __host__ __device__ static int total(int stages, int q_bytes) {
    return ring_off(stages, q_bytes) + stages * 2 * kTileBytes + 1024;
  }
};

// Byte offset of 16-byte chunk c of a row inside one span: the copies' 128-byte
// swizzle (rows of 128 bytes) or 64-byte swizzle (rows of 64).
template <int kSpan>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  if constexpr (kSpan == 128) return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4));
  return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// c += a b, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 codes to two fp16 pairs (bytes 0, 1 and bytes 2, 3).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(x));
  return f;
}
// x, y as hi + lo, each a pair of fp16.
__device__ __forceinline__ void split_f16x2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x, y);
  const float2 h = unpack_f16x2(hi);
  lo = pack_f16x2(x - h.x, y - h.y);
}
// floor(log2 x) of a positive normal float, as a float (2^23 + e - (2^23 + 127)).
__device__ __forceinline__ float exponent_of(float x) {
  return __uint_as_float(0x4b000000u | (__float_as_uint(x) >> 23)) - 8388735.f;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// 4 bytes to shared memory, or zero without a read where !ok.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}
// One arrival at the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumerWarps) : "memory");
}

struct DecodeFp8KParams {
  DecodeFp8Args a;
  int mode;    // LoadMode
  int stages;
  int q_bytes;  // shared memory for q's fragments
  uint32_t* err_word;
  uint64_t timeout_ns;
};

// kWide: more than 8 query heads per kv head (up to 64).  The warps then form
// G teams of 16 heads that share the stage's sub-blocks, as in the bf16 decode.
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, D == 256 ? (kWide ? 1 : 2) : (kWide ? 2 : 3))
decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const DecodeFp8KParams kp) {
  using L = Smem<D>;
  constexpr int kSpan = L::kSpan;
  const DecodeFp8Args& a = kp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int S = a.num_splits, n_kv = a.c.n_kv_heads, bs = a.c.block_size;
  const int g = a.n_q_heads / n_kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = kp.stages;

  grid_dep_wait();
  grid_dep_launch();

  // ---- this split's tokens (split rule: see the C header) ----
  const long long capacity = a.c.capacity();
  int len = a.kv_lens[b];
  if (len < 0 || (long long)len + a.append > capacity) {
    if (threadIdx.x == 0 && split == 0) atomicOr(kp.err_word, kErrKvLen);
    len = len < 0 ? 0 : (int)capacity - a.append;
  }
  len += a.append;
  const int lo_tok = a.window_left >= 0 ? max(0, len - 1 - a.window_left) : 0;
  const int lo16 = lo_tok / kSplitGranule * kSplitGranule;
  const int n_att = len - lo16;
  const int per = (n_att + S - 1) / S;
  const int chunk = (per + kSplitGranule - 1) / kSplitGranule * kSplitGranule;
  const int t0 = lo16 + (int)min((long long)split * chunk, (long long)n_att);
  const int t1 = min(t0 + chunk, len);
  const int n_tok = t1 - t0;

  float* o_out = a.o_partial + (((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g) * D;
  float* lse_out = a.lse_partial + ((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g;
  if (n_tok <= 0) {  // empty split: o = 0, lse = -inf
    for (int i = threadIdx.x; i < g * D; i += kThreads) o_out[i] = 0.f;
    for (int i = threadIdx.x; i < g; i += kThreads) lse_out[i] = -INFINITY;
    return;
  }
  const int n_iters = (n_tok + kStageTokens - 1) / kStageTokens;

  const uint32_t full0 = smem_u32(smem + L::kBar);
  const uint32_t empty0 = full0 + 8 * stages;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kFlag);
  uint8_t* ring = smem + L::ring_off(stages, kp.q_bytes);
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < stages; ++i) {
      mbar_init(full0 + 8 * i, 1 + 32);  // the copies' bytes, and each lane's scales
      mbar_init(empty0 + 8 * i, kConsumerWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl ctl{abort_flag, kp.err_word, kp.timeout_ns};

  if (warp == 0) {
    // ================= producer =================
    const int32_t* table =
        a.c.block_table ? a.c.block_table + (size_t)b * a.c.max_blocks_per_seq : nullptr;
    const int per_seq = (a.c.max_kv_len + bs - 1) / bs;  // contiguous: scales of a sequence
    // Lane l looks after tokens l and 32 + l of a stage: their blocks' scales,
    // and (box16) the copy of the 16-token groups that they begin.
    auto block_of = [&](int t) -> int {
      if (t < lo_tok || t >= t1) return 0;
      if (table == nullptr) return t / bs;
      const int blk = table[t / bs];
      if (blk < 0 || blk >= a.c.num_blocks) {
        atomicOr(kp.err_word, kErrBlockIndex);
        return 0;  // keep the copy in bounds; the result is flagged invalid
      }
      return blk;
    };
    int blk[2] = {block_of(t0 + lane), block_of(t0 + 32 + lane)};
    int st = 0, wrap = 0;
    for (int it = 0; it < n_iters; ++it) {
      if (wrap > 0 && !mbar_wait_warp(empty0 + 8 * st, (wrap - 1) & 1, ctl)) break;
      const int base = t0 + it * kStageTokens;
      const int cnt = min(kStageTokens, t1 - base);
      uint8_t* sk = ring + (size_t)st * 2 * L::kTileBytes;
      uint8_t* sv = sk + L::kTileBytes;
      const uint32_t full = full0 + 8 * st;
      if (kp.mode == kLoadBox64) {
        // Contiguous cache as (D, n_kv, L, B): one 64-token box for a span.
        if (lane == 0) {
          mbar_arrive_expect_tx(full, 2u * L::kTileBytes);
#pragma unroll
          for (int h = 0; h < L::kSpans; ++h) {
            tma_load_4d(smem_u32(sk + h * L::kSpanBytes), &tm_k, full, h * kSpan, kvh, base, b);
            tma_load_4d(smem_u32(sv + h * L::kSpanBytes), &tm_v, full, h * kSpan, kvh, base, b);
          }
        }
      } else if (kp.mode == kLoadBox16) {
        // Paged cache as (D, n_kv, block_size, num_blocks): one 16-token box for
        // a group (both start at multiples of 16, so a group has one block).  A
        // group's first token may lie left of the window, its last may not.
        const int groups = (cnt + 15) >> 4;
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)groups * 16u * 2u * (uint32_t)D);
        __syncwarp();
        const int last = min(16 * (lane & 3) + 15, cnt - 1);  // of group lane & 3
        const int b0 = __shfl_sync(0xffffffffu, blk[0], last & 31);
        const int b1 = __shfl_sync(0xffffffffu, blk[1], last & 31);
        if (lane < groups) {
          const int phys = last < 32 ? b0 : b1;
          const int slot = (base + 16 * lane) % bs;
#pragma unroll
          for (int h = 0; h < L::kSpans; ++h) {
            tma_load_4d(smem_u32(sk + h * L::kSpanBytes + lane * 16 * kSpan), &tm_k, full,
                        h * kSpan, kvh, slot, phys);
            tma_load_4d(smem_u32(sv + h * L::kSpanBytes + lane * 16 * kSpan), &tm_v, full,
                        h * kSpan, kvh, slot, phys);
          }
        }
      } else {
        // Any other block size: 16-byte asynchronous copies into the swizzled layout.
        constexpr int kChunks = D / 16;
#pragma unroll 4
        for (int i = lane; i < kStageTokens * kChunks; i += 32) {
          const int r = i / kChunks, c = i % kChunks;
          const int b0 = __shfl_sync(0xffffffffu, blk[0], r & 31);
          const int b1 = __shfl_sync(0xffffffffu, blk[1], r & 31);
          const int t = base + r;
          if (r >= cnt || t < lo_tok) continue;
          const size_t row = (size_t)(r < 32 ? b0 : b1) * bs + t % bs;
          const size_t off = (row * n_kv + kvh) * D + (size_t)c * 16;
          const uint32_t to = (c / (kSpan / 16)) * L::kSpanBytes + swz<kSpan>(r, c % (kSpan / 16));
          cp_async16(smem_u32(sk + to), a.c.k + off);
          cp_async16(smem_u32(sv + to), a.c.v + off);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      // The tokens' scales; 0 for those that are masked.
      const uint32_t sc = smem_u32(smem + L::kScale + st * L::kScaleBytes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 32 * h + lane, t = base + r;
        const bool ok = t >= lo_tok && t < t1;
        const size_t idx =
            ((table ? (size_t)0 : (size_t)b * per_seq) + (size_t)blk[h]) * n_kv + kvh;
        cp_async4(sc + 4 * r, a.c.k_scales + idx, ok);
        cp_async4(sc + 4 * (kStageTokens + r), a.c.v_scales + idx, ok);
      }
      cp_async_arrive(full);
      blk[0] = block_of(base + kStageTokens + lane);  // the next stage's, while this one flies
      blk[1] = block_of(base + kStageTokens + 32 + lane);
      if (++st == stages) st = 0, ++wrap;
    }
    // Wait for copies still in flight before the block may leave (abort path
    // only: on the normal path the consumers have waited on every stage).
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*abort_flag && lane == 0) {
      volatile uint32_t no_abort = 0u;
      WaitCtl drain{&no_abort, kp.err_word, kp.timeout_ns};
      for (int it = max(0, n_iters - stages); it < n_iters; ++it)
        mbar_wait(full0 + 8 * (it % stages), (it / stages) & 1, drain);
    }
    return;
  }

  // ================= consumers =================
  const int cw = warp - 1, ctid = threadIdx.x - 32;
  const int G = !kWide ? 1 : (g <= 16 ? 1 : (g <= 32 ? 2 : 4));
  const int team = kConsumerWarps / G;  // warps of a row group
  const int row0 = kWide ? (cw / team) * 16 : 0;
  const int gid = lane >> 2, quad = lane & 3;
  constexpr int kRows = kWide ? 2 : 1;  // query rows a thread looks after
  constexpr int kSteps = D / 16;
  constexpr bool kQSmem = q_in_smem(D, kWide);

  // q as A fragments: thread (gid, quad) takes columns 16 i + 4 quad .. + 3 of
  // step i, rows gid (and gid + 8).  Each row times 2^(13 - exponent of its
  // largest value).
  uint32_t qf[kQSmem ? 1 : kSteps][2];
  uint4* qs = reinterpret_cast<uint4*>(smem + L::q_off(stages)) + (cw / team) * kSteps * 32;
  float sl2[kRows], cap_in[kRows];
  {
    const uint16_t* qsrc = a.q + ((size_t)b * a.n_q_heads + (size_t)kvh * g) * D;
    float up[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row0 + gid + 8 * r;
      uint32_t top = 0u;
      if (row < g) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint2 x = *reinterpret_cast<const uint2*>(qsrc + (size_t)row * D + i * 16 + quad * 4);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = e ? x.y : x.x;
            const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
            if (lo < 0x7f80u) top = max(top, lo);
            if (hi < 0x7f80u) top = max(top, hi);
          }
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(top >> 7) - 127, -110), 127);
      up[r] = __int_as_float((13 - e + 127) << 23);           // 2^(13 - e), e >= -110
      const float down = __int_as_float((max(e - 13, -126) + 127) << 23);
      sl2[r] = a.softcap > 0.f ? a.softcap * kLog2e : a.scale * kLog2e * down;
      cap_in[r] = a.softcap > 0.f ? a.scale * down / a.softcap : 0.f;
    }
    auto frag = [&](int row, int i, float f) -> uint2 {
      if (row >= g) return make_uint2(0u, 0u);
      const uint2 x = *reinterpret_cast<const uint2*>(qsrc + (size_t)row * D + i * 16 + quad * 4);
      return make_uint2(
          pack_f16x2(__uint_as_float(x.x << 16) * f, __uint_as_float(x.x & 0xffff0000u) * f),
          pack_f16x2(__uint_as_float(x.y << 16) * f, __uint_as_float(x.y & 0xffff0000u) * f));
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint2 f0 = frag(row0 + gid, i, up[0]);
      if constexpr (kWide) {
        const uint2 f1 = frag(row0 + gid + 8, i, up[kRows - 1]);
        if (cw % team == 0) qs[i * 32 + lane] = make_uint4(f0.x, f1.x, f0.y, f1.y);
      } else if constexpr (kQSmem) {
        if (cw == 0) reinterpret_cast<uint2*>(qs)[i * 32 + lane] = f0;
      } else {
        qf[i][0] = f0.x;
        qf[i][1] = f0.y;
      }
    }
    if constexpr (kQSmem) consumer_sync();
  }
  const bool capped = a.softcap > 0.f, alibi = a.alibi_slopes != nullptr;
  float al2[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = row0 + gid + 8 * r;
    al2[r] = alibi && row < g ? a.alibi_slopes[kvh * g + row] * kLog2e : 0.f;
  }

  float m[kRows], mr[kRows], l[kRows];  // reference, reference - kShift (0 at first), sum
  float2 acc[D / 8][kRows];  // n tile j: columns 2 quad, 2 quad + 1 of each row
#pragma unroll
  for (int r = 0; r < kRows; ++r) m[r] = -INFINITY, mr[r] = 0.f, l[r] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[j][r] = make_float2(0.f, 0.f);

  int st = 0, wrap = 0;
  for (int it = 0; it < n_iters; ++it) {
    if (!mbar_wait_warp(full0 + 8 * st, wrap & 1, ctl)) break;
    const int base = t0 + it * kStageTokens;
    const uint8_t* tile = ring + (size_t)st * 2 * L::kTileBytes;
    const float* sc = reinterpret_cast<const float*>(smem + L::kScale + st * L::kScaleBytes);
#pragma unroll 1
    for (int sb = cw % team; sb < kStageTokens / 16; sb += team) {
      const int r0 = sb * 16, first = base + r0;
      if (first >= t1) break;
      const bool ragged = first + 16 > t1 || first < lo_tok;
      const uint32_t sk = smem_u32(tile), sv = sk + L::kTileBytes;
      // ---- scores of 16 tokens, two n tiles of 8 ----
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // matrices: tokens 0-7 and 8-15, each at 16-byte chunks 2 i and 2 i + 1
        const int row = r0 + (lane & 7) + ((lane >> 4) << 3);
        const int c = 2 * i + ((lane >> 3) & 1);
        uint32_t x[4];
        ldsm_x4(sk + (c / (kSpan / 16)) * L::kSpanBytes + swz<kSpan>(row, c % (kSpan / 16)), x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1 = 0u, a2, a3 = 0u;
          if constexpr (kWide) {
            const uint4 q = qs[(2 * i + h) * 32 + lane];
            a0 = q.x, a1 = q.y, a2 = q.z, a3 = q.w;
          } else if constexpr (kQSmem) {
            const uint2 q = reinterpret_cast<const uint2*>(qs)[(2 * i + h) * 32 + lane];
            a0 = q.x, a2 = q.y;
          } else {
            a0 = qf[2 * i + h][0], a2 = qf[2 * i + h][1];
          }
          uint32_t b0, b1;
          e4m3x4_to_f16(x[h], b0, b1);
          mma16816(s[0], a0, a1, a2, a3, b0, b1);
          e4m3x4_to_f16(x[2 + h], b0, b1);
          mma16816(s[1], a0, a1, a2, a3, b0, b1);
        }
      }
      // ---- in log2 units, with K's scales; V's scales ----
      float vs[2][2], kv[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 ks = *reinterpret_cast<const float2*>(sc + r0 + n * 8 + quad * 2);
        const float2 v2 =
            *reinterpret_cast<const float2*>(sc + kStageTokens + r0 + n * 8 + quad * 2);
        vs[n][0] = v2.x, vs[n][1] = v2.y;
        kv[n][0] = exponent_of(v2.x), kv[n][1] = exponent_of(v2.y);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[n][2 * r + e];
            const float k1 = e ? ks.y : ks.x;
            if (capped)
              x = tanhf(x * (cap_in[r] * k1)) * sl2[r];
            else
              x *= sl2[r] * k1;
          }
      }
      if (alibi) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[n][2 * r + e] = fmaf(-al2[r], (float)(len - 1 - (first + n * 8 + quad * 2 + e)),
                                     s[n][2 * r + e]);
      }
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of V's tokens 2 quad, 2 quad + 1
      if (ragged) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          keep[n] = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = first + n * 8 + quad * 2 + e;
            const bool in = t >= lo_tok && t < t1;
            if (in) keep[n] |= e ? 0xffff0000u : 0x0000ffffu;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
              if (!in) s[n][2 * r + e] = -INFINITY;
          }
        }
      }
      // ---- online softmax ----
      float mx[kRows];
      bool grow = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        mx[r] = fmaxf(fmaxf(s[0][2 * r] + kv[0][0], s[0][2 * r + 1] + kv[0][1]),
                      fmaxf(s[1][2 * r] + kv[1][0], s[1][2 * r + 1] + kv[1][1]));
        grow |= mx[r] > m[r] + kGrow;
      }
      if (__any_sync(0xffffffffu, grow)) {
        float corr[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          const float now = fmaxf(m[r], mx[r]);
          corr[r] = now == -INFINITY ? 1.f : ex2_approx(m[r] - now);  // 0 at the first token
          m[r] = now;
          mr[r] = now == -INFINITY ? 0.f : now - kShift;
          l[r] *= corr[r];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            acc[j][r].x *= corr[r];
            acc[j][r].y *= corr[r];
          }
      }
      uint32_t hi[kRows][2], lo[kRows][2];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2_approx(s[n][2 * r] - mr[r]);
          const float p1 = ex2_approx(s[n][2 * r + 1] - mr[r]);
          l[r] += p0 + p1;
          split_f16x2(p0 * vs[n][0], p1 * vs[n][1], hi[r][n], lo[r][n]);
        }
      // ---- O += P V ----
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // matrices: tokens 0-7 and 8-15 at chunk 2 i, the same at 2 i + 1
        const int row = r0 + (lane & 7) + (((lane >> 3) & 1) << 3);
        const int c = 2 * i + (lane >> 4);
        uint32_t x[4];
        ldsm_x4_t(sv + (c / (kSpan / 16)) * L::kSpanBytes + swz<kSpan>(row, c % (kSpan / 16)), x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y0 = x[2 * h], y1 = x[2 * h + 1];
          if (ragged) y0 &= keep[0], y1 &= keep[1];
          uint32_t e0, o0, e1, o1;  // even and odd columns
          e4m3x4_to_f16(__byte_perm(y0, 0u, 0x3120), e0, o0);
          e4m3x4_to_f16(__byte_perm(y1, 0u, 0x3120), e1, o1);
          // Each product starts from zero and is added outside: the tensor core
          // truncates its sums, which over hundreds of steps would shrink O.
          float ce[4] = {0.f, 0.f, 0.f, 0.f}, co[4] = {0.f, 0.f, 0.f, 0.f};
          float2(&ae)[kRows] = acc[2 * (2 * i + h)];
          float2(&ao)[kRows] = acc[2 * (2 * i + h) + 1];
          if constexpr (kWide) {
            mma16816(ce, hi[0][0], hi[1][0], hi[0][1], hi[1][1], e0, e1);
            mma16816(co, hi[0][0], hi[1][0], hi[0][1], hi[1][1], o0, o1);
            mma16816(ce, lo[0][0], lo[1][0], lo[0][1], lo[1][1], e0, e1);
            mma16816(co, lo[0][0], lo[1][0], lo[0][1], lo[1][1], o0, o1);
            ae[0] = add2(ae[0], make_float2(ce[0], ce[1]));
            ae[kRows - 1] = add2(ae[kRows - 1], make_float2(ce[2], ce[3]));
            ao[0] = add2(ao[0], make_float2(co[0], co[1]));
            ao[kRows - 1] = add2(ao[kRows - 1], make_float2(co[2], co[3]));
          } else {
            mma16816(ce, hi[0][0], lo[0][0], hi[0][1], lo[0][1], e0, e1);
            mma16816(co, hi[0][0], lo[0][0], hi[0][1], lo[0][1], o0, o1);
            ae[0] = add2(ae[0], add2(make_float2(ce[0], ce[1]), make_float2(ce[2], ce[3])));
            ao[0] = add2(ao[0], add2(make_float2(co[0], co[1]), make_float2(co[2], co[3])));
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * st);
    if (++st == stages) st = 0, ++wrap;
  }

  // ================= merge the warps' states =================
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  consumer_sync();  // every warp is done with the ring
  float* mm = reinterpret_cast<float*>(smem + L::kMerge);  // [warp][16]
  float* ml = mm + kConsumerWarps * 16;
  float* mf = ml + kConsumerWarps * 16;
  constexpr int kWarpRows = kWide ? 16 : 8;
  float* mo = reinterpret_cast<float*>(ring);  // [warp][kWarpRows][kPitch]
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = gid + 8 * r;
    if (quad == 0) {
      mm[cw * 16 + row] = m[r];
      ml[cw * 16 + row] = l[r];
    }
    float* to = mo + (size_t)(cw * kWarpRows + row) * L::kPitch + quad * 4;
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      *reinterpret_cast<float4*>(to + 16 * j) =
          make_float4(acc[2 * j][r].x, acc[2 * j + 1][r].x, acc[2 * j][r].y, acc[2 * j + 1][r].y);
  }
  consumer_sync();
  if (*abort_flag) return;
  // Row r of the kv head belongs to team r / 16: the common reference, each
  // warp's weight 2^(m_w - m) / l, and the LSE.
  if (ctid < g) {
    const int lr = ctid & 15, w0 = kWide ? (ctid >> 4) * team : 0;
    float mt = -INFINITY;
    for (int w = w0; w < w0 + team; ++w) mt = fmaxf(mt, mm[w * 16 + lr]);
    float sum = 0.f;
    for (int w = w0; w < w0 + team; ++w) {
      // A warp that saw no token has m = -inf and l = 0; one whose scores are all
      // NaN has m = -inf and l = NaN, which stays.
      const float f = mm[w * 16 + lr] == -INFINITY ? 1.f : ex2_approx(mm[w * 16 + lr] - mt);
      sum += f * ml[w * 16 + lr];
      mf[w * 16 + lr] = f;
    }
    const float inv = 1.f / sum;
    for (int w = w0; w < w0 + team; ++w) mf[w * 16 + lr] *= inv;
    lse_out[ctid] = (mt - kShift + log2f(sum)) * kLn2;
  }
  consumer_sync();
  for (int e = ctid; e < g * (D / 4); e += 32 * kConsumerWarps) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    const int lr = kWide ? r & 15 : r, w0 = kWide ? (r >> 4) * team : 0;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = w0; w < w0 + team; ++w) {
      const float f = mf[w * 16 + lr];
      const float4 v =
          *reinterpret_cast<const float4*>(mo + (size_t)(w * kWarpRows + lr) * L::kPitch + c);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    *reinterpret_cast<float4*>(o_out + (size_t)r * D + c) = o;
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A (D, n_kv, rows, planes) byte cache with boxes of one span x 1 head x
// box_rows x 1.
template <int D>
bool make_cache_map(CUtensorMap* m, const void* base, int n_kv, long long rows, long long planes,
                    int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  constexpr int kSpan = Smem<D>::kSpan;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n_kv, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)D * (cuuint64_t)n_kv,
                           (cuuint64_t)D * (cuuint64_t)n_kv * (cuuint64_t)rows};
  cuuint32_t box[4] = {(cuuint32_t)kSpan, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             kSpan == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kWide>
cudaError_t launch_t(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  using L = Smem<D>;
  const int g = a.n_q_heads / a.c.n_kv_heads;  // at most 64 (validated)
  const int groups = g <= 16 ? 1 : (g <= 32 ? 2 : 4);
  DecodeFp8KParams kp;
  kp.a = a;
  kp.err_word = ctx.err_word;
  kp.timeout_ns = ctx.timeout_ns;
  kp.q_bytes = q_smem_bytes(D, kWide, groups);
  kp.stages = D == 64 ? 8 : (D == 128 ? 4 : 3);
  const int smem = L::total(kp.stages, kp.q_bytes);
  static bool configured[64] = {};  // the attribute is per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<D, kWide>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         L::total(kp.stages, q_smem_bytes(D, kWide, kWide ? 4 : 1)));
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  CUtensorMap mk, mv;
  std::memset(&mk, 0, sizeof(mk));
  std::memset(&mv, 0, sizeof(mv));
  if (a.c.block_table == nullptr) {
    kp.mode = kLoadBox64;
    if (!make_cache_map<D>(&mk, a.c.k, a.c.n_kv_heads, a.c.max_kv_len, a.batch, kStageTokens) ||
        !make_cache_map<D>(&mv, a.c.v, a.c.n_kv_heads, a.c.max_kv_len, a.batch, kStageTokens))
      return cudaErrorInvalidValue;
  } else if (a.c.block_size % 16 == 0) {
    kp.mode = kLoadBox16;
    if (!make_cache_map<D>(&mk, a.c.k, a.c.n_kv_heads, a.c.block_size, a.c.num_blocks, 16) ||
        !make_cache_map<D>(&mv, a.c.v, a.c.n_kv_heads, a.c.block_size, a.c.num_blocks, 16))
      return cudaErrorInvalidValue;
  } else {
    kp.mode = kLoadRows;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_splits, a.c.n_kv_heads, a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<D, kWide>, mk, mv, kp);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  return a.n_q_heads / a.c.n_kv_heads <= 8 ? launch_t<D, false>(a, ctx) : launch_t<D, true>(a, ctx);
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  if (a.c.head_dim == 256) return launch_d<256>(a, ctx);
  return a.c.head_dim == 128 ? launch_d<128>(a, ctx) : launch_d<64>(a, ctx);
}

}  // namespace attn
