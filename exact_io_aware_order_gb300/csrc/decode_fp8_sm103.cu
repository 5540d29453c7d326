// Split-KV single-token decode over a key/value cache held in 8 bits, sm_103a.
//
// The bf16 decode's plan (one block per (split, kv head, sequence), the cache
// streamed once through a shared-memory ring and used for all g query heads of
// the kv head, partials merged by their LSE weights) with half the bytes to
// stream, so twice the arithmetic a byte: what a row costs between its arrival
// and its products has to be half of the bf16 kernel's.  The mathematics is
// arranged for that:
//
//   * q k runs on the tensor core's e4m3 products, which take K's codes as
//     ldmatrix delivers them.  q, 8 significant bits a value, is split into two
//     e4m3 terms hi + lo / 32, each row scaled by a power of two to a maximum in
//     [2^7, 2^8): exact down to 2^-15 of the row's maximum, off by at most 2^-23
//     of it below.  K's scale is a factor of the score and V's of the weight,
//     one number a token each.
//   * p v runs in fp16: codes are converted (exactly: e4m3 is a subset of
//     fp16).  A transposed ldmatrix delivers 2 tokens x 2 columns; one byte
//     permutation separates the columns, and the even and odd columns of 16 form
//     one n tile each, so a thread ends up with 4 neighbouring columns.  The
//     weights are split into two fp16 parts, hi + lo (22 bits), so that the fp32
//     output is not limited by an operand's rounding.
//   * with up to 8 query heads per kv head the two parts (of q, and of the
//     weights) fill the 16 rows of one product, rows 0-7 hi and 8-15 lo, which
//     would be half empty otherwise.  With more heads a second product adds the
//     lo parts.
//   * p v's sums over 32 tokens start from zero and are added to O by the FP32
//     pipe, hi and lo rows together (the tensor core truncates its sums: over
//     100000 tokens in one split O came out 3e-5 too small).  That also halves
//     the accumulators of the form with up to 8 heads.
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

constexpr int kTile = 32;          // tokens a warp takes at a time
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 4.f;       // log2 units a score may exceed the reference by
constexpr float kShift = 10.f;     // log2 of the weight at the reference
constexpr float kQLo = 32.f;       // q = hi + lo / kQLo

// Where q's fragments live during the stream: registers, or shared memory
// where the accumulators leave no room for them.
__host__ __device__ constexpr bool q_in_smem(int D, bool wide) { return wide || D == 256; }
__host__ __device__ constexpr int q_smem_bytes(int D, bool wide, int groups) {
  return q_in_smem(D, wide) ? groups * (D / 32) * 32 * (wide ? 32 : 16) : 0;
}

// Blocks that share an SM (by their registers; the shared memory is cut to fit).
constexpr int blocks_per_sm(int D, bool wide) { return D == 256 ? 2 : (wide ? 3 : 4); }

// How a half tile is copied.
enum LoadMode : int {
  kLoadBox32 = 0,  // contiguous cache: one box of 32 tokens
  kLoadBox16 = 1,  // paged, block size a multiple of 16: one box for 16 tokens
  kLoadRows = 2    // any other block size: 16-byte copies by the lanes
};

// The boxes write rows of kSpan bytes in the copy's swizzle (head_dim 256: two
// spans after one another), and so do the row copies: ldmatrix's 8 rows of 16
// bytes then lie in distinct banks.
template <int D>
struct Smem {
  static constexpr int kSpan = D < 128 ? D : 128;
  static constexpr int kSpans = D / kSpan;
  static constexpr int kSpanBytes = kTile * kSpan;
  static constexpr int kHalfBytes = kTile * D;             // K or V of a tile
  static constexpr int kScaleBytes = kTile * 4;
  static constexpr int kPitch = D + 16;                    // floats of a merged row
  static constexpr int kMaxSlots = 32;                     // of a block
  static constexpr int kBar = 0;                           // full, empty
  static constexpr int kFlag = 16 * kMaxSlots;
  static constexpr int kMerge = kFlag + 16;                // m, l, weight: [3][4][16]
  static constexpr int kScale = kMerge + 3 * kWarps * 16 * 4;
  // then the slots' scales, q's fragments, and the ring
  __host__ __device__ static constexpr int q_off(int slots) { return kScale + slots * kScaleBytes; }
  __host__ __device__ static constexpr int ring_off(int slots, int q_bytes) {
    return (q_off(slots) + q_bytes + 1023) / 1024 * 1024;
  }
  __host__ __device__ static constexpr int total(int slots, int q_bytes) {
    return ring_off(slots, q_bytes) + slots * kHalfBytes + 1024;
  }
  // The warps' rows are merged in the ring.
  __host__ __device__ static constexpr int merge_bytes(bool wide) {
    return kWarps * (wide ? 16 : 8) * kPitch * 4;
  }
};

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
// c = a b (first) or c += a b: fp16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], bool first, uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (first) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
// The same with e4m3 operands (k = 32).
__device__ __forceinline__ void mma16832_e4m3(float (&c)[4], bool first, const uint4& a,
                                              uint32_t b0, uint32_t b1) {
  if (first) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ uint32_t e4m3x4_pack(float a, float b, float c, float d) {
  return e4m3x2_pack(b, a) | (e4m3x2_pack(d, c) << 16);
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
struct DecodeFp8KParams {
  DecodeFp8Args a;
  int mode;     // LoadMode
  int slots;    // half tiles of the ring, a multiple of kWarps
  int q_bytes;  // shared memory for q's fragments
  uint32_t bs_mul;  // t / block_size = umulhi(t, bs_mul) >> bs_shift for t < 2^31;
  int bs_shift;     // -1: block_size 1
  uint32_t* err_word;
  uint64_t timeout_ns;
};

// Every warp streams its own tiles of 32 tokens: it asks for a half tile (K, or
// V, of 32 tokens and their scales) as soon as it has read the one whose place
// that takes, so no warp stands between the copies and the products, and the
// rings of an SM's 16 warps together hold two thirds of it in flight.
//
// kWide: more than 8 query heads per kv head (up to 64).  The four warps form G
// teams, one for each 16 heads; the warps of one column (the same place in every
// team) share a ring, which its first warp refills once the others have read.
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D, kWide))
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
  const int G = !kWide ? 1 : (g <= 16 ? 1 : (g <= 32 ? 2 : 4));
  const int team = kWarps / G;                       // columns
  const int col = warp % team, rg = warp / team;     // this warp's column and row group

  const uint32_t full0 = smem_u32(smem + L::kBar);
  const uint32_t empty0 = full0 + 8 * kp.slots;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kFlag);
  uint8_t* ring = smem + L::ring_off(kp.slots, kp.q_bytes);
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < kp.slots; ++i) {
      mbar_init(full0 + 8 * i, 1 + 32);  // the copies' bytes, and each lane's scale
      mbar_init(empty0 + 8 * i, G);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  __syncthreads();
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
  const int n_tiles = (n_tok + kTile - 1) / kTile;
  const int my_tiles = col < n_tiles ? (n_tiles - col + team - 1) / team : 0;
  const WaitCtl ctl{abort_flag, kp.err_word, kp.timeout_ns};

  // ================= the column's ring =================
  // Half 2 j is K and half 2 j + 1 is V of the column's tile j (the block's tile
  // col + j team); half h lies in slot h mod slots.
  const int slots = kp.slots / team, slot0 = col * slots;
  const int32_t* table =
      a.c.block_table ? a.c.block_table + (size_t)b * a.c.max_blocks_per_seq : nullptr;
  const int per_seq = (a.c.max_kv_len + bs - 1) / bs;  // contiguous: scales of a sequence
  auto block_index = [&](int t) -> int {
    return kp.bs_shift < 0 ? t : (int)(__umulhi((uint32_t)t, kp.bs_mul) >> kp.bs_shift);
  };
  // Lane l looks after token l of a tile: its block as the table has it (0: masked).
  auto entry = [&](int j) -> int {
    const int t = t0 + (col + j * team) * kTile + lane;
    if (t < lo_tok || t >= t1) return 0;
    const int i = block_index(t);
    return table ? table[i] : i;
  };
  int next_a = 0, next_b = 0;  // entries of the next two tiles to be asked for
  int blk = 0;                 // the current one's
  int put_slot = 0, put_tile = 0;
  bool put_v = false;
  auto put = [&]() {  // asks for the next half; rg 0 only
    const uint32_t full = full0 + 8 * (slot0 + put_slot);
    const int base = t0 + (col + put_tile * team) * kTile, t = base + lane;
    const int cnt = min(kTile, t1 - base);
    const bool ok = t >= lo_tok && t < t1;
    if (!put_v) {
      blk = next_a;
      next_a = next_b;
      next_b = entry(put_tile + 2);
      if (table && (blk < 0 || blk >= a.c.num_blocks)) {
        atomicOr(kp.err_word, kErrBlockIndex);
        blk = 0;  // keep the copy in bounds; the result is flagged invalid
      }
    }
    const uint32_t dst = smem_u32(ring) + (uint32_t)((slot0 + put_slot) * L::kHalfBytes);
    const CUtensorMap* map = put_v ? &tm_v : &tm_k;
    if (kp.mode == kLoadBox32) {
      // Contiguous cache as (D, n_kv, L, B).
      if (lane == 0) {
        mbar_arrive_expect_tx(full, (uint32_t)L::kHalfBytes);
#pragma unroll
        for (int h = 0; h < L::kSpans; ++h)
          tma_load_4d(dst + h * L::kSpanBytes, map, full, h * kSpan, kvh, base, b);
      }
    } else if (kp.mode == kLoadBox16) {
      // Paged cache as (D, n_kv, block_size, num_blocks): tokens and blocks both
      // start at multiples of 16, so 16 tokens have one block, that of the last
      // of them (the first may lie left of the window).
      const int groups = (cnt + 15) >> 4;
      if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)groups * 16u * (uint32_t)D);
      const int phys = __shfl_sync(0xffffffffu, blk, min(16 * (lane & 1) + 15, cnt - 1));
      if (lane < groups) {
        const int at = base + 16 * lane, slot = at - block_index(at) * bs;
#pragma unroll
        for (int h = 0; h < L::kSpans; ++h)
          tma_load_4d(dst + h * L::kSpanBytes + lane * 16 * kSpan, map, full, h * kSpan, kvh, slot,
                      phys);
      }
    } else {
      constexpr int kRowChunks = D / 16, kAtOnce = 32 / kRowChunks;
      const uint8_t* src = put_v ? a.c.v : a.c.k;
      const int in_blk = t - block_index(t) * bs;
      const int c = lane % kRowChunks;
#pragma unroll 4
      for (int r0 = 0; r0 < kTile; r0 += kAtOnce) {
        const int r = r0 + lane / kRowChunks;
        const size_t from =
            (size_t)__shfl_sync(0xffffffffu, blk, r) * bs + __shfl_sync(0xffffffffu, in_blk, r);
        if (base + r < lo_tok || r >= cnt) continue;
        const int cs = c % (kSpan / 16);
        const uint32_t to = (c / (kSpan / 16)) * L::kSpanBytes + r * kSpan +
                            ((cs ^ (kSpan == 128 ? r & 7 : (r >> 1) & 3)) << 4);
        cp_async16(dst + to, src + (from * n_kv + kvh) * D + c * 16);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    // The tokens' scales; 0 for those that are masked.
    const size_t idx = ((table ? (size_t)0 : (size_t)b * per_seq) + (size_t)blk) * n_kv + kvh;
    cp_async4(smem_u32(smem + L::kScale + (slot0 + put_slot) * L::kScaleBytes) + 4 * lane,
              (put_v ? a.c.v_scales : a.c.k_scales) + idx, ok);
    cp_async_arrive(full);
    if (++put_slot == slots) put_slot = 0;
    put_tile += put_v;
    put_v = !put_v;
  };
  const bool putter = !kWide || rg == 0;
  if (putter && my_tiles > 0) {
    next_a = entry(0);
    next_b = entry(1);
    for (int h = 0; h < slots && put_tile < my_tiles; ++h) put();
  }

  // ================= q =================
  const int row0 = kWide ? rg * 16 : 0;
  const int gid = lane >> 2, quad = lane & 3;
  constexpr int kRows = kWide ? 2 : 1;  // query rows a thread looks after
  constexpr int kSteps = D / 32;        // k steps of q k
  constexpr bool kQSmem = q_in_smem(D, kWide);

  // q as A fragments (rows gid and gid + 8, columns 4 quad .. + 3 and 16 + 4
  // quad .. + 3 of each 32): hi and lo parts of 8 rows in one, or of 16 in two.
  uint4 qf[kQSmem ? 1 : kSteps];
  uint4* qs = reinterpret_cast<uint4*>(smem + L::q_off(kp.slots)) +
              rg * kSteps * 32 * (kWide ? 2 : 1);
  float sl2[kRows], cap_in[kRows];
  {
    const uint16_t* qsrc = a.q + ((size_t)b * a.n_q_heads + (size_t)kvh * g) * D + quad * 4;
    float up[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row0 + gid + 8 * r;
      uint32_t top = 0u;
      if (row < g) {
#pragma unroll
        for (int i = 0; i < 2 * kSteps; ++i) {
          const uint2 x = *reinterpret_cast<const uint2*>(qsrc + (size_t)row * D + i * 16);
          top = max(max(top, x.x & 0x7fffu), (x.x >> 16) & 0x7fffu);
          top = max(max(top, x.y & 0x7fffu), (x.y >> 16) & 0x7fffu);
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(top >> 7) - 127, -110), 127);
      up[r] = __int_as_float((7 - e + 127) << 23);            // 2^(7 - e)
      float down = __int_as_float((e - 7 + 127) << 23);
      if (top >= 0x7f80u) down = __int_as_float(0x7fc00000);  // an infinity or NaN: the row is NaN
      sl2[r] = a.scale * kLog2e * down;
      cap_in[r] = 0.f;
      if (a.softcap > 0.f) {
        cap_in[r] = a.scale * down / a.softcap;
        sl2[r] = a.softcap * kLog2e;
      }
    }
    auto part = [&](int row, int i, float f, uint32_t& hi, uint32_t& lo) {
      hi = lo = 0u;
      if (row >= g) return;
      const uint2 x = *reinterpret_cast<const uint2*>(qsrc + (size_t)row * D + i * 16);
      const float v0 = __uint_as_float(x.x << 16) * f, v1 = __uint_as_float(x.x & 0xffff0000u) * f;
      const float v2 = __uint_as_float(x.y << 16) * f, v3 = __uint_as_float(x.y & 0xffff0000u) * f;
      hi = e4m3x4_pack(v0, v1, v2, v3);
      uint32_t h01, h23;
      e4m3x4_to_f16(hi, h01, h23);
      const float2 a01 = unpack_f16x2(h01), a23 = unpack_f16x2(h23);
      lo = e4m3x4_pack((v0 - a01.x) * kQLo, (v1 - a01.y) * kQLo, (v2 - a23.x) * kQLo,
                       (v3 - a23.y) * kQLo);
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint4 f;
      if constexpr (kWide) {
        uint4 fl;
        part(row0 + gid, 2 * i, up[0], f.x, fl.x);
        part(row0 + gid + 8, 2 * i, up[1], f.y, fl.y);
        part(row0 + gid, 2 * i + 1, up[0], f.z, fl.z);
        part(row0 + gid + 8, 2 * i + 1, up[1], f.w, fl.w);
        if (col == 0) {
          qs[(2 * i) * 32 + lane] = f;
          qs[(2 * i + 1) * 32 + lane] = fl;
        }
      } else {
        part(gid, 2 * i, up[0], f.x, f.y);
        part(gid, 2 * i + 1, up[0], f.z, f.w);
        if constexpr (kQSmem) {
          if (col == 0) qs[i * 32 + lane] = f;
        } else {
          qf[i] = f;
        }
      }
    }
    if constexpr (kQSmem) __syncthreads();
  }
  const bool capped = a.softcap > 0.f, alibi = a.alibi_slopes != nullptr;
  float al2[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = row0 + gid + 8 * r;
    al2[r] = alibi && row < g ? a.alibi_slopes[kvh * g + row] * kLog2e : 0.f;
  }

  // Where ldmatrix's lane reads: byte offsets of its row and, before the k
  // step's part is XORed in, of its 16-byte chunk (see Smem).
  constexpr int kChunks = kSpan / 16;
  const int swz = kSpan == 128 ? lane & 7 : (lane >> 1) & 3;
  const int k_row = ((lane & 7) + ((lane >> 4) << 3)) * kSpan;        // tokens 0-7, 8-15 by lane
  const uint32_t k_chunk = (uint32_t)((((lane >> 3) & 1) ^ swz) << 4);
  const int v_row = ((lane & 7) + (((lane >> 3) & 1) << 3)) * kSpan;  // the other way round
  const uint32_t v_chunk = (uint32_t)(((lane >> 4) ^ swz) << 4);

  float m[kRows], mr[kRows], l[kRows];  // reference, reference - kShift (0 at first), sum
  float2 acc[D / 8][kRows];  // n tile j: columns 2 quad, 2 quad + 1 of each row
#pragma unroll
  for (int r = 0; r < kRows; ++r) m[r] = -INFINITY, mr[r] = 0.f, l[r] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[j][r] = make_float2(0.f, 0.f);

  int slot = 0;
  uint32_t parity = 0u;
  int read = 0;  // halves read
  // A half has been read: its place goes to the half `slots` later.
  auto release = [&]() {
    __syncwarp();
    if (kWide && lane == 0) mbar_arrive(empty0 + 8 * (slot0 + slot));
    if (putter && put_tile < my_tiles &&
        (!kWide || mbar_wait_warp(empty0 + 8 * (slot0 + slot), parity, ctl)))
      put();
    ++read;
    if (++slot == slots) slot = 0, parity ^= 1u;
  };
  for (int j = 0; j < my_tiles; ++j) {
    if (!mbar_wait_warp(full0 + 8 * (slot0 + slot), parity, ctl)) break;
    const int first = t0 + (col + j * team) * kTile;
    const uint32_t sk = smem_u32(ring) + (uint32_t)((slot0 + slot) * L::kHalfBytes);
    const float* ksc =
        reinterpret_cast<const float*>(smem + L::kScale + (slot0 + slot) * L::kScaleBytes);
    const bool ragged = first + kTile > t1 || first < lo_tok;

    // ---- scores of 32 tokens: four n tiles of 8 ----
    float s[4][4], sl[kWide ? 4 : 1][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t at = sk + k_row + (2 * i / kChunks) * L::kSpanBytes +
                          (k_chunk ^ (uint32_t)((2 * i % kChunks) << 4));
      uint32_t x[4], y[4];  // tokens 0-7: both halves of the step's 32 columns; tokens 8-15
      ldsm_x4(at, x);
      ldsm_x4(at + 16 * kSpan, y);
      uint4 f;
      if constexpr (kQSmem) f = qs[(kWide ? 2 * i : i) * 32 + lane];
      else f = qf[i];
      mma16832_e4m3(s[0], i == 0, f, x[0], x[1]);
      mma16832_e4m3(s[1], i == 0, f, x[2], x[3]);
      mma16832_e4m3(s[2], i == 0, f, y[0], y[1]);
      mma16832_e4m3(s[3], i == 0, f, y[2], y[3]);
      if constexpr (kWide) {
        f = qs[(2 * i + 1) * 32 + lane];
        mma16832_e4m3(sl[0], i == 0, f, x[0], x[1]);
        mma16832_e4m3(sl[1], i == 0, f, x[2], x[3]);
        mma16832_e4m3(sl[2], i == 0, f, y[0], y[1]);
        mma16832_e4m3(sl[3], i == 0, f, y[2], y[3]);
      }
    }
    // ---- in log2 units, with K's scales ----
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float2 ks = *reinterpret_cast<const float2*>(ksc + n * 8 + quad * 2);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[n][2 * r + e];
          x = fmaf(kWide ? sl[kWide ? n : 0][2 * r + e] : s[n][2 + e], 1.f / kQLo, x);
          const float k1 = e ? ks.y : ks.x;
          if (capped)
            x = tanhf(x * (cap_in[r] * k1)) * sl2[r];
          else
            x *= sl2[r] * k1;
        }
    }
    release();  // K's half
    if (alibi) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            s[n][2 * r + e] = fmaf(-al2[r], (float)(len - 1 - (first + n * 8 + quad * 2 + e)),
                                   s[n][2 * r + e]);
    }
    if (ragged) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = first + n * 8 + quad * 2 + e;
          if (t < lo_tok || t >= t1) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) s[n][2 * r + e] = -INFINITY;
          }
        }
    }
    // ---- V's half: its scales; masked rows are cleared (0 x NaN is NaN) ----
    if (!mbar_wait_warp(full0 + 8 * (slot0 + slot), parity, ctl)) break;
    const uint32_t sv = smem_u32(ring) + (uint32_t)((slot0 + slot) * L::kHalfBytes);
    const float* vsc =
        reinterpret_cast<const float*>(smem + L::kScale + (slot0 + slot) * L::kScaleBytes);
    if (ragged) {
      if (first + lane < lo_tok || first + lane >= t1) {
#pragma unroll
        for (int h = 0; h < L::kSpans; ++h)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            st_shared_v4(sv + h * L::kSpanBytes + lane * kSpan + c * 16,
                         make_float4(0.f, 0.f, 0.f, 0.f));
      }
      __syncwarp();
    }
    float vs[4][2], kv[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float2 v2 = *reinterpret_cast<const float2*>(vsc + n * 8 + quad * 2);
      vs[n][0] = v2.x, vs[n][1] = v2.y;
      kv[n][0] = exponent_of(v2.x), kv[n][1] = exponent_of(v2.y);
    }
    // ---- online softmax ----
    float mx[kRows];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      mx[r] = -INFINITY;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        mx[r] = fmax3(mx[r], s[n][2 * r] + kv[n][0], s[n][2 * r + 1] + kv[n][1]);
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
    uint32_t hi[kRows][4], lo[kRows][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float p0 = ex2_approx(s[n][2 * r] - mr[r]);
        const float p1 = ex2_approx(s[n][2 * r + 1] - mr[r]);
        l[r] += p0 + p1;
        split_f16x2(p0 * vs[n][0], p1 * vs[n][1], hi[r][n], lo[r][n]);
      }
    // ---- O += P V ----
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t at = sv + v_row + (2 * i / kChunks) * L::kSpanBytes +
                          (v_chunk ^ (uint32_t)((2 * i % kChunks) << 4));
      uint32_t x[2][4];  // 16 tokens each: tokens 0-7, 8-15 of chunk 2 i, then of 2 i + 1
      ldsm_x4_t(at, x[0]);
      ldsm_x4_t(at + 16 * kSpan, x[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float ce[4], co[4];  // even and odd columns
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t e0, o0, e1, o1;
          e4m3x4_to_f16(__byte_perm(x[t][2 * h], 0u, 0x3120), e0, o0);
          e4m3x4_to_f16(__byte_perm(x[t][2 * h + 1], 0u, 0x3120), e1, o1);
          const int n = 2 * t;
          if constexpr (kWide) {
            mma16816(ce, t == 0, hi[0][n], hi[1][n], hi[0][n + 1], hi[1][n + 1], e0, e1);
            mma16816(co, t == 0, hi[0][n], hi[1][n], hi[0][n + 1], hi[1][n + 1], o0, o1);
            mma16816(ce, false, lo[0][n], lo[1][n], lo[0][n + 1], lo[1][n + 1], e0, e1);
            mma16816(co, false, lo[0][n], lo[1][n], lo[0][n + 1], lo[1][n + 1], o0, o1);
          } else {
            mma16816(ce, t == 0, hi[0][n], lo[0][n], hi[0][n + 1], lo[0][n + 1], e0, e1);
            mma16816(co, t == 0, hi[0][n], lo[0][n], hi[0][n + 1], lo[0][n + 1], o0, o1);
          }
        }
        float2(&ae)[kRows] = acc[2 * (2 * i + h)];
        float2(&ao)[kRows] = acc[2 * (2 * i + h) + 1];
        if constexpr (kWide) {
          ae[0] = add2(ae[0], make_float2(ce[0], ce[1]));
          ae[1] = add2(ae[1], make_float2(ce[2], ce[3]));
          ao[0] = add2(ao[0], make_float2(co[0], co[1]));
          ao[1] = add2(ao[1], make_float2(co[2], co[3]));
        } else {
          ae[0] = add2(ae[0], add2(make_float2(ce[0], ce[1]), make_float2(ce[2], ce[3])));
          ao[0] = add2(ao[0], add2(make_float2(co[0], co[1]), make_float2(co[2], co[3])));
        }
      }
    }
    if (ragged) fence_proxy_async_smem();  // the cleared rows, before a copy may overwrite them
    release();  // V's half
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (*abort_flag && putter) {
    // Copies still in flight land before the block may leave (on the normal path
    // every half that was asked for has been waited for).
    volatile uint32_t no_abort = 0u;
    WaitCtl drain{&no_abort, kp.err_word, kp.timeout_ns};
    const int asked = 2 * put_tile + (put_v ? 1 : 0);
    for (; read < asked; ++read) {
      mbar_wait_warp(full0 + 8 * (slot0 + slot), parity, drain);
      if (++slot == slots) slot = 0, parity ^= 1u;
    }
  }

  // ================= merge the warps' states =================
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  // Every half has landed and been read once the warps meet: the ring is free.
  __syncthreads();
  float* mm = reinterpret_cast<float*>(smem + L::kMerge);  // [warp][16]
  float* ml = mm + kWarps * 16;
  float* mf = ml + kWarps * 16;
  constexpr int kWarpRows = kWide ? 16 : 8;
  float* mo = reinterpret_cast<float*>(ring);  // [warp][kWarpRows][kPitch]
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = gid + 8 * r;
    if (quad == 0) {
      mm[warp * 16 + row] = m[r];
      ml[warp * 16 + row] = l[r];
    }
    float* to = mo + (size_t)(warp * kWarpRows + row) * L::kPitch + quad * 4;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      *reinterpret_cast<float4*>(to + 16 * j) =
          make_float4(acc[2 * j][r].x, acc[2 * j + 1][r].x, acc[2 * j][r].y, acc[2 * j + 1][r].y);
  }
  __syncthreads();
  if (*abort_flag) return;
  // Row r of the kv head belongs to team r / 16: the common reference, each
  // warp's weight 2^(m_w - m) / l, and the LSE.
  if ((int)threadIdx.x < g) {
    const int lr = threadIdx.x & 15, w0 = kWide ? (threadIdx.x >> 4) * team : 0;
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
    lse_out[threadIdx.x] = (mt - kShift + log2f(sum)) * kLn2;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < g * (D / 4); e += kThreads) {
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

constexpr int kMaxSmem = 227 * 1024;  // of a block; 1 KB of an SM's 228 goes to each block

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
  const uint32_t bs = (uint32_t)a.c.block_size;
  kp.bs_mul = 0u;
  kp.bs_shift = -1;
  if (bs > 1) {
    // With s = ceil(log2 bs), m = ceil(2^(31 + s) / bs) <= 2^32 - 1 (bs > 1) and
    // t < 2^31: t m / 2^(31 + s) exceeds t / bs by less than 1 / bs.
    int s = 0;
    while ((1u << s) < bs) ++s;
    kp.bs_mul = (uint32_t)((((unsigned long long)1 << (31 + s)) + bs - 1) / bs);
    kp.bs_shift = s - 1;
  }
  static bool configured[64] = {};  // the attribute is per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<D, kWide>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  CUtensorMap mk, mv;
  std::memset(&mk, 0, sizeof(mk));
  std::memset(&mv, 0, sizeof(mv));
  if (a.c.block_table == nullptr) {
    kp.mode = kLoadBox32;
    if (!make_cache_map<D>(&mk, a.c.k, a.c.n_kv_heads, a.c.max_kv_len, a.batch, kTile) ||
        !make_cache_map<D>(&mv, a.c.v, a.c.n_kv_heads, a.c.max_kv_len, a.batch, kTile))
      return cudaErrorInvalidValue;
  } else if (a.c.block_size % 16 == 0) {
    kp.mode = kLoadBox16;
    if (!make_cache_map<D>(&mk, a.c.k, a.c.n_kv_heads, a.c.block_size, a.c.num_blocks, 16) ||
        !make_cache_map<D>(&mv, a.c.v, a.c.n_kv_heads, a.c.block_size, a.c.num_blocks, 16))
      return cudaErrorInvalidValue;
  } else {
    kp.mode = kLoadRows;
  }
  // As many slots as the blocks that the registers allow on an SM leave room
  // for, and at least what the merge needs (head_dim 256 with more than 32
  // heads per kv head then has an SM to itself).
  constexpr int kMerge = (L::merge_bytes(kWide) + L::kHalfBytes - 1) / L::kHalfBytes;
  kp.slots = (kMerge > 2 * kWarps ? kMerge + kWarps - 1 : 2 * kWarps) / kWarps * kWarps;
  while (kp.slots + kWarps <= L::kMaxSlots &&
         L::total(kp.slots + kWarps, kp.q_bytes) <= kMaxSmem / blocks_per_sm(D, kWide) - 1024)
    kp.slots += kWarps;
  const int smem = L::total(kp.slots, kp.q_bytes);
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
