// Split-KV single-token decode over a key/value cache held in 8 bits, sm_103a.
//
// The bf16 decode's plan (one block per (split, kv head, sequence), the cache
// streamed once through shared memory and used for all g query heads of the kv
// head, partials merged by their LSE weights) with half the bytes to stream, so
// twice the arithmetic a byte: what a row costs between its arrival and its
// products has to be half of the bf16 kernel's.
//
//   * q k runs on the tensor core's e4m3 products, which take K's codes as
//     ldmatrix delivers them.  q, 8 significant bits a value, is split into e4m3
//     terms, each row scaled by a power of two to a maximum in [2^7, 2^8).  Two of
//     them, hi + lo / 32, hold values down to 2^-14 of the row's maximum exactly
//     and leave at most 2^-22 of it of smaller ones.  Two more, (t3 + t4 / 32) / 2^23,
//     are exact down to 2^-37 of the maximum (at most 2^-45 of it left below) and
//     take a second pass over K's tile.  A tile takes it where n 2^-15 448 (n values
//     below 2^-14 of the maximum, times the largest code) times K's scale, in units
//     of the score, is above 2^-18: otherwise what hi and lo leave cannot change a
//     score's base 2 logarithm by more, whatever the keys.  Normally distributed rows
//     have n = 0 or 1, and ordinary scores stay below that; where a channel of q or of
//     the keys is far larger than the rest most tiles take it (16 sequences of
//     1024-32768 tokens: 104 us, with a channel of 2^5 / 2^12 in every row of q 120 / 129).
//     K's scale is a factor of the score and V's of the weight, one number a token
//     each.
//   * p v runs in fp16: codes are converted (exactly: e4m3 is a subset of
//     fp16).  The byte form of the transposed ldmatrix gives a thread 4
//     neighbouring tokens of one column, which two conversions turn into the two
//     registers of a B fragment; the fragment's token order (4 q, 4 q + 1 | 4 q +
//     2, 4 q + 3) is that of the weights because K's rows are taken in the order
//     that puts them there.  The weights are split into two fp16 parts, hi + lo
//     (22 bits), so that the fp32 output is not limited by an operand's
//     rounding.
//   * with up to 8 query heads per kv head the two parts (of q, and of the
//     weights) fill the 16 rows of one product, rows 0-7 hi and 8-15 lo, which
//     would be half empty otherwise.  With more heads a second product adds the
//     lo parts.
//   * p v's sums over 32 tokens start from zero and are added to O by the FP32
//     pipe, hi and lo rows together (the tensor core truncates its sums: over
//     100000 tokens in one split O came out 3e-5 too small).  That also halves
//     the accumulators of the form with up to 8 heads.
//   * the exponentials' reference m bounds score + log2(V's scale), the size of
//     a weight times its scale: those lie below 2^(kShift + kGrow) = 2^14 (2^15 for
//     scales that are no powers of two) and
//     those down to 2^-24 of the largest keep full fp16 precision in hi.  The
//     sum l is taken over the unscaled weights in fp32.  The row maximum is
//     only reduced over the quad when some score exceeds m by 2^kGrow.
//   * masked rows are not read: their copies fill zeros, and their scores are
//     cut off, so nothing that lies in masked places (NaN codes or scales) is
//     used.
//
// Streaming: every warp copies its own tiles of 32 tokens with 16-byte
// asynchronous copies into a ring of half tiles (K, or V, of 32 tokens) that no
// other warp touches, and asks for the next half as soon as it has read one.
// There is no producer warp and no barrier in the stream, and any block size
// takes the same path (a row's address is one shuffle and one multiply-add).
// Measured on a paged batch of 16 sequences (555 MB, head_dim 128; 83 us at the
// measured copy rate): TMA boxes of 16 tokens by a producer warp 157 us (the
// copies' issue by one warp was the limit), TMA boxes by every warp 114 us, this
// form 104 us with its combine (107 since small values of q are looked after).
#include <cstdint>
#include <type_traits>
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
constexpr float kQLo = 32.f;       // q = hi + lo / kQLo + (t3 + t4 / kQLo) / kQFine: what
constexpr float kQFine = 8388608.f;  // hi and lo leave, 2^-15 at most, becomes 2^8 (kQFine 2^23)
constexpr float kQNoise = 3.8146973e-6f;  // 2^-18, see above
constexpr uint32_t kNoRow = 0xffffffffu;

// Where q's fragments live during the stream: registers, or shared memory
// where the accumulators leave no room for them.
__host__ __device__ constexpr bool q_in_smem(int D, bool wide) { return wide || D == 256; }
// Whether q's finer terms are kept in shared memory; else (where two blocks an SM
// leave no room) they are made again from q in each tile.
__host__ __device__ constexpr bool fine_in_smem(int D, int groups) {
  return D < 256 || groups < 4;
}
__host__ __device__ constexpr int q_smem_bytes(int D, bool wide, int groups) {
  return (q_in_smem(D, wide) + fine_in_smem(D, groups)) * groups * D * (wide ? 32 : 16);
}
// Blocks that share an SM, by their registers.
constexpr int blocks_per_sm(int D) { return D == 64 ? 3 : 2; }

// Half tiles of a warp's ring: what those blocks' shared memory holds.  Two blocks
// with two halves a warp beat one with three (8 sequences of 8000-16000 tokens, 4
// kv heads of 256, 64 heads each: 217 against 307 us; 16 heads each: 64 against 76).
constexpr int ring_slots(int D, bool wide) { return D == 256 ? (wide ? 2 : 3) : 4; }

template <int D, bool kWide>
struct Smem {
  static constexpr int kSlots = ring_slots(D, kWide);
  static constexpr int kHalfBytes = kTile * D;             // K or V of a tile
  static constexpr int kScaleBytes = kTile * 4;
  static constexpr int kPitch = D + 8;                     // floats of a merged row
  static constexpr int kRing = 0;                          // [warp][slot]
  // The warps' rows are merged in the rings.
  static constexpr int kRingBytes = kWarps * kSlots * kHalfBytes;
  static constexpr int kRowsBytes = kWarps * (kWide ? 16 : 8) * kPitch * 4;
  static constexpr int kScale = kRingBytes > kRowsBytes ? kRingBytes : kRowsBytes;
  static constexpr int kMerge = kScale + kWarps * kSlots * kScaleBytes;  // m, l, weight; before: rows' scales
  static constexpr int kQ = kMerge + 3 * kWarps * 16 * 4;  // q's fragments, where kept here
  static constexpr int total(int q_bytes) { return kQ + q_bytes; }
};

// Row r of a half has its 16-byte chunk c at chunk c ^ swizzle(r).  ldmatrix reads
// rows in eights: K's are 0, 1, 4, 5, 8, 9, 12, 13 (or those + 2) of 16, V's are
// consecutive; the chunks of any such eight lie in distinct banks.  Linear over
// XOR, so a step's constant part folds into an immediate.
template <int D>
__host__ __device__ constexpr uint32_t swizzle(uint32_t r) {
  const uint32_t b0 = r & 1u, b1 = (r >> 1) & 1u, b2 = (r >> 2) & 1u, b3 = (r >> 3) & 1u;
  return D == 64 ? (b2 | ((b1 ^ b3) << 1)) : (b0 | (b2 << 1) | ((b1 ^ b3) << 2));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// Two 16 x 16 byte matrices, transposed: thread (gid, quad) gets rows 4 quad ..
// + 3 of columns gid and gid + 8 of the first (row addresses from lanes 0-15),
// then of the second.
__device__ __forceinline__ void ldsm_b8_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
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
// Four neighbouring bf16 values, times f.
__device__ __forceinline__ void scaled4(const uint2& x, float f, float (&v)[4]) {
  v[0] = __uint_as_float(x.x << 16) * f, v[1] = __uint_as_float(x.x & 0xffff0000u) * f;
  v[2] = __uint_as_float(x.y << 16) * f, v[3] = __uint_as_float(x.y & 0xffff0000u) * f;
}
// The e4m3 numbers nearest to four values, which become what those leave of
// them, times kQLo (exactly).
__device__ __forceinline__ uint32_t e4m3_term(float (&v)[4]) {
  const uint32_t t = e4m3x4_pack(v[0], v[1], v[2], v[3]);
  uint32_t t01, t23;
  e4m3x4_to_f16(t, t01, t23);
  const float2 a = unpack_f16x2(t01), b = unpack_f16x2(t23);
  v[0] = (v[0] - a.x) * kQLo, v[1] = (v[1] - a.y) * kQLo;
  v[2] = (v[2] - b.x) * kQLo, v[3] = (v[3] - b.y) * kQLo;
  return t;
}
// hi and lo of four values of q, by way of fp16, which holds the scaled values down
// to 2^-17 exactly (smaller ones are off by 2^-25 at most).
__device__ __forceinline__ void coarse2(uint32_t two, float f, uint32_t& hi, uint32_t& lo) {
  const uint32_t v = pack_f16x2(__uint_as_float(two << 16) * f, __uint_as_float(two & 0xffff0000u) * f);
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 t;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 t, h;\n\t"
      "sub.rn.f16x2 t, %2, t;\n\t"
      "mul.rn.f16x2 t, t, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, t;\n\t"
      "cvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
      : "=r"(hi), "=r"(lo)
      : "r"(v), "r"(0x50005000u));  // 32, 32
}
__device__ __forceinline__ void coarse_terms(const uint2& x, float f, uint32_t& hi, uint32_t& lo) {
  uint32_t h0, l0, h1, l1;
  coarse2(x.x, f, h0, l0);
  coarse2(x.y, f, h1, l1);
  hi = h0 | h1 << 16;
  lo = l0 | l1 << 16;
}
// t3 and t4 of four values of q.
__device__ __forceinline__ void fine_terms(const uint2& x, float f, uint32_t& t3, uint32_t& t4) {
  uint32_t hi, lo, h01, h23, l01, l23;
  coarse_terms(x, f, hi, lo);
  e4m3x4_to_f16(hi, h01, h23);
  e4m3x4_to_f16(lo, l01, l23);
  const float2 a0 = unpack_f16x2(h01), a1 = unpack_f16x2(h23);
  const float2 b0 = unpack_f16x2(l01), b1 = unpack_f16x2(l23);
  float v[4];
  scaled4(x, f, v);
  v[0] = ((v[0] - a0.x) * kQLo - b0.x) * (kQFine / kQLo);
  v[1] = ((v[1] - a0.y) * kQLo - b0.y) * (kQFine / kQLo);
  v[2] = ((v[2] - a1.x) * kQLo - b1.x) * (kQFine / kQLo);
  v[3] = ((v[3] - a1.y) * kQLo - b1.y) * (kQFine / kQLo);
  t3 = e4m3_term(v);
  t4 = e4m3_term(v);
}
// x, y as hi + lo, each a pair of fp16.
__device__ __forceinline__ void split_f16x2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x, y);
  const float2 h = unpack_f16x2(hi);
  lo = pack_f16x2(x - h.x, y - h.y);
}
// floor(log2 x) of a scale, as a float (2^23 + e - (2^23 + 127)); the least one's
// for 0 (a block that is zero as it was allocated), so that the reference stays
// within 60 of the score and a weight within fp32.
__device__ __forceinline__ float exponent_of(float x) {
  const uint32_t e = max(__float_as_uint(x) >> 23, (uint32_t)(127 + kScaleExpMin));
  return __uint_as_float(0x4b000000u | e) - 8388735.f;
}
// l 2^d, d <= 0, where 2^d may be too small for a float and l large: references
// lie up to 120 octaves apart for the same score (V's scales 2^-60 and 2^60), and
// a sum of weights taken against the lower one is that much larger.
__device__ __forceinline__ float scaled_sum(float l, float d, float two_d) {
  if (d > -126.f) return l * two_d;
  const float half = ex2_approx(0.5f * d);
  return l * half * half;
}
// 4 bytes to shared memory, or zero without a read where !ok.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}
// 16 bytes likewise.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}

struct DecodeFp8KParams {
  DecodeFp8Args a;
  uint32_t bs_mul;  // t / block_size = umulhi(t, bs_mul) >> bs_shift for t < 2^31;
  int bs_shift;     // -1: block_size 1
  uint32_t* err_word;
};

// The tokens a sequence's query attends to.
struct Span {
  int len;     // with the appended token
  int lo_tok;  // first token of the window
  int lo16;    // rounded down to the split granule
};
__device__ __forceinline__ Span span_of(const DecodeFp8Args& a, int len, uint32_t* err_word) {
  const long long capacity = a.c.capacity();
  if (len < 0 || (long long)len + a.append > capacity) {
    if (err_word) atomicOr(err_word, kErrKvLen);
    len = len < 0 ? 0 : (int)capacity - a.append;
  }
  Span s;
  s.len = len + a.append;
  s.lo_tok = a.window_left >= 0 ? max(0, s.len - 1 - a.window_left) : 0;
  s.lo16 = s.lo_tok / kSplitGranule * kSplitGranule;
  return s;
}
__device__ __forceinline__ int tiles_of(const Span& s) {
  return (s.len - s.lo16 + kTile - 1) / kTile;
}

// Two ways to divide the work.  With `parts` 0 block (split, kv head, sequence)
// takes one split of the C header's rule.  With parts > 0 the blocks share the
// tiles of all (sequence, kv head) pairs, whatever their lengths:
//   * blocks of their own: each pair gets as many blocks as it takes at `most` tiles a
//     block, the smallest number for which all of them surely fit (or one, where that
//     covers the longest pair), and its tiles evenly over those.  Every block has one
//     segment (a part of one pair).
//   * equal shares: all tiles form one list that the blocks take equal parts of, so
//     that no SM idles; a share may run over several segments.  Going on to the
//     next segment costs a block 4 to 8 us (merge, q, the first tiles' latency), as
//     much as some 16 tiles do.
// So a pair gets blocks of its own where the longest of them has at most kOwnMore
// tiles more than an equal share.  8 kv heads of 128, own / shares: 16 sequences of
// 1500 tokens (14 more) 20.0 / 21.7 us, 8 of 12000 (21 more) 45.7 / 43.5; 36 of 4000
// (one block each, 7 more) 59.7 / 64.2.
// A segment that is a whole pair is the result; of the others a block has at most
// two, its first (which began in an earlier block: partial slot 2 p) and its last
// (slot 2 p + 1).  The combine needs a pair's first and last block: it works them
// out for itself where one load holds all lengths, and else finds them noted by
// the block that has the pair's first tile.
constexpr int kNoteBeyond = 32;  // sequences

// x / y; the 64-bit division is a long sequence, and almost no list needs it.
__device__ __forceinline__ long long div_small(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

constexpr int kOwnMore = 16;
struct Shares {
  int parts;        // blocks that have work: at most one a tile
  bool own;         // blocks of their own for each pair
  int most;         // (own) tiles a block, at most
  long long share;  // (otherwise) the first `more` blocks have share + 1 tiles,
  int more;         // the others share
};
// total: tiles of all pairs; longest: those of the longest pair.
__device__ __forceinline__ Shares shares_of(int parts, long long total, long long pairs,
                                            int longest) {
  Shares s = {};
  s.parts = (int)min((long long)parts, total);
  if (s.parts == 0) return s;
  if (pairs <= s.parts) {
    const int spare = s.parts - (int)pairs;
    s.most = longest;
    if (spare > 0) s.most = (int)min((long long)longest, div_small(total + spare - 1, spare));
    s.own = (long long)(s.most - kOwnMore) * s.parts <= total;
  }
  if (!s.own) {
    s.share = div_small(total, s.parts);
    s.more = (int)(total - s.share * s.parts);
  }
  return s;
}
// (not own) The block that has tile x of the list.
__device__ __forceinline__ int block_of(const Shares& s, long long x) {
  const long long big = (s.share + 1) * s.more;
  return (int)(x < big ? div_small(x, s.share + 1) : s.more + div_small(x - big, s.share));
}

// kWide: more than 8 query heads per kv head (up to 64).  The four warps form G
// teams, one for each 16 heads; team rg's warps take the tiles in turn, and the
// teams copy the same tiles each for itself (they are bound by arithmetic).
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D))
decode_fp8_kernel(const DecodeFp8KParams kp) {
  using L = Smem<D, kWide>;
  const DecodeFp8Args& a = kp.a;
  extern __shared__ __align__(128) uint8_t smem[];
  const int n_kv = a.c.n_kv_heads, bs = a.c.block_size;
  const int g = a.n_q_heads / n_kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = !kWide ? 1 : (g <= 16 ? 1 : (g <= 32 ? 2 : 4));
  const int team = kWarps / G;                       // warps of a team
  const int col = warp % team, rg = warp / team;     // place in the team, row group

  // Behind its step's write, which has waited for the kernels in front of both, the
  // decode finds its place and asks for q while the write runs, and waits before
  // it reads the cache (one sequence of 30719 tokens, steps on 12 caches in one graph:
  // 19.7 -> 17.6 us; called from Python on one cache, 17.6 -> 16.1).
  bool to_wait = a.append != 0;
  if (!to_wait) grid_dep_wait();
  grid_dep_launch();

  int b, kvh;             // the segment's pair
  int raw_len = 0;        // (splits) its length, asked for before q and used after
  Span sp;
  int tile, seg_tiles;    // its first tile in the pair and how many
  int pair_tiles = 0;     // (shares) tiles of the pair
  // (shares) Of the list: where this block is and up to where it goes.
  long long pos = 0, end = 0;
  Shares sh = {};
  int last_block = -1;  // (blocks of their own) the pair's last
  if (a.parts == 0) {
    b = blockIdx.z, kvh = blockIdx.y;
    raw_len = a.kv_lens[b];
    tile = 0, seg_tiles = 0;  // set below, in tokens
  } else {
    // Every warp scans the batch for itself, 32 sequences at a time (twice, where
    // there are more: for all tiles, and for its place).
    int raw = 0, n = 0;  // this lane's length and tiles (of one head)
    auto tiles32 = [&](int i0, bool report) {
      const int i = i0 + lane;
      raw = n = 0;
      if (i < a.batch) {
        raw = a.kv_lens[i];
        n = tiles_of(span_of(a, raw, report ? kp.err_word : nullptr));
        // A sequence without tokens: o = 0, lse = -inf, written by one of the blocks.
        if (n == 0 && report && i % a.parts == (int)blockIdx.x) {
          for (int e = 0; e < a.n_q_heads * D; ++e)
            a.o_final[(size_t)i * a.n_q_heads * D + e] = 0.f;
          for (int e = 0; e < a.n_q_heads; ++e)
            a.lse_final[(size_t)i * a.n_q_heads + e] = -INFINITY;
          if (a.batch > kNoteBeyond)
            for (int e = 0; e < n_kv; ++e) a.pair_blocks[(size_t)i * n_kv + e] = make_int2(0, 0);
        }
      }
    };
    long long all = 0;
    int longest = 0;
    for (int i0 = 0; i0 < a.batch; i0 += 32) {
      tiles32(i0, warp == 0);
      all += __reduce_add_sync(0xffffffffu, n);
      longest = max(longest, __reduce_max_sync(0xffffffffu, n));
    }
    sh = shares_of(a.parts, all * n_kv, (long long)a.batch * n_kv, longest);
    if ((int)blockIdx.x >= sh.parts) return;
    if (sh.own) {
      pos = blockIdx.x;
    } else {
      pos = blockIdx.x * sh.share + min((int)blockIdx.x, sh.more);
      end = pos + sh.share + ((int)blockIdx.x < sh.more ? 1 : 0);
    }
    // Where pos (of the blocks, or of the tiles) lies.
    long long before = 0;  // blocks, or tiles, of one head before the 32 sequences
    int i0 = 0, count, scan;
    unsigned here;
    for (;;) {
      if (a.batch > 32) tiles32(i0, false);
      scan = count = sh.own ? (n + sh.most - 1) / sh.most : n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      here = __ballot_sync(0xffffffffu, pos < (before + scan) * n_kv);
      if (here) break;
      before += __shfl_sync(0xffffffffu, scan, 31);
      i0 += 32;
      if (i0 >= a.batch) return;  // more blocks than the pairs take
    }
    const int at = __ffs(here) - 1;
    b = i0 + at;
    sp = span_of(a, __shfl_sync(0xffffffffu, raw, at), nullptr);
    pair_tiles = __shfl_sync(0xffffffffu, n, at);
    count = __shfl_sync(0xffffffffu, count, at);
    const long long in_seq =
        pos - (before + __shfl_sync(0xffffffffu, scan, at) - count) * n_kv;
    kvh = (int)div_small(in_seq, count);
    const int i = (int)(in_seq - (long long)kvh * count);
    if (sh.own) {
      tile = (int)div_small((long long)i * pair_tiles, count);
      pos = 0;
      end = div_small((i + 1LL) * pair_tiles, count) - tile;
      last_block = blockIdx.x + count - 1;
    } else {
      tile = i;
    }
  }

  // ---- the segment's tokens, and where its result goes ----
  for (;;) {
  // ================= q: asked for first, used while the first tiles fly =================
  const int row0 = kWide ? rg * 16 : 0;
  const int gid = lane >> 2, quad = lane & 3;
  constexpr int kRows = kWide ? 2 : 1;  // query rows a thread looks after
  constexpr int kSteps = D / 32;        // k steps of q k
  constexpr bool kQSmem = q_in_smem(D, kWide);
  // Columns 16 i + 4 quad .. + 3 of rows gid (and gid + 8).
  const uint16_t* qsrc = a.q + ((size_t)b * a.n_q_heads + (size_t)kvh * g) * D + quad * 4;
  auto load_q = [&](int r, int i) -> uint2 {
    const int row = row0 + gid + 8 * r;
    if (row >= g) return make_uint2(0u, 0u);
    return *reinterpret_cast<const uint2*>(qsrc + (size_t)row * D + i * 16);
  };
  uint2 qx[kRows][2 * kSteps];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) qx[r][i] = load_q(r, i);

  if (a.parts == 0)
    sp = span_of(a, raw_len, threadIdx.x == 0 && blockIdx.x == 0 ? kp.err_word : nullptr);
  const int len = sp.len, lo_tok = sp.lo_tok;
  int t0, t1;
  float *o_out, *lse_out;
  if (a.parts == 0) {
    // (split rule: see the C header)
    const int S = a.num_splits, split = blockIdx.x, n_att = len - sp.lo16;
    const int per = (n_att + S - 1) / S;
    const int chunk = (per + kSplitGranule - 1) / kSplitGranule * kSplitGranule;
    t0 = sp.lo16 + (int)min((long long)split * chunk, (long long)n_att);
    t1 = min(t0 + chunk, len);
    o_out = a.o_partial + (((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g) * D;
    lse_out = a.lse_partial + ((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g;
    if (t1 <= t0) {  // empty split: o = 0, lse = -inf
      for (int i = threadIdx.x; i < g * D; i += kThreads) o_out[i] = 0.f;
      for (int i = threadIdx.x; i < g; i += kThreads) lse_out[i] = -INFINITY;
      return;
    }
  } else {
    seg_tiles = (int)min(end - pos, (long long)(pair_tiles - tile));
    t0 = sp.lo16 + tile * kTile;
    t1 = min(t0 + seg_tiles * kTile, len);
    const bool whole = seg_tiles == pair_tiles;
    if (whole) {
      o_out = a.o_final + ((size_t)b * a.n_q_heads + (size_t)kvh * g) * D;
      lse_out = a.lse_final + (size_t)b * a.n_q_heads + (size_t)kvh * g;
    } else {
      const size_t part = 2 * (size_t)blockIdx.x + (tile == 0 ? 1 : 0);
      o_out = a.o_partial + part * g * D;
      lse_out = a.lse_partial + part * g;
    }
    if (a.batch > kNoteBeyond && tile == 0 && threadIdx.x == 0) {
      const int last = last_block >= 0 ? last_block : block_of(sh, pos + pair_tiles - 1);
      a.pair_blocks[(size_t)b * n_kv + kvh] = make_int2(blockIdx.x, last);
    }
  }
  const int n_tiles = (t1 - t0 + kTile - 1) / kTile;
  const int my_tiles = col < n_tiles ? (n_tiles - col + team - 1) / team : 0;

  // ================= this warp's ring =================
  // Half 2 j is K and half 2 j + 1 is V of the warp's tile j (the block's tile
  // col + j team).
  const int32_t* table =
      a.c.block_table ? a.c.block_table + (size_t)b * a.c.max_blocks_per_seq : nullptr;
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
  constexpr int kRowChunks = D / 16, kRowsAtOnce = 32 / kRowChunks;
  const uint32_t ring = smem_u32(smem + L::kRing + warp * L::kSlots * L::kHalfBytes);
  const uint32_t ring_sc = smem_u32(smem + L::kScale + warp * L::kSlots * L::kScaleBytes);
  const uint32_t put_off = (lane / kRowChunks) * D +
                           (((lane % kRowChunks) ^ swizzle<D>(lane / kRowChunks)) << 4);
  const uint8_t* k_base = a.c.k + (lane % kRowChunks) * 16;
  const uint8_t* v_base = a.c.v + (lane % kRowChunks) * 16;
  int next_a = 0, next_b = 0;             // entries of the next two tiles to be asked for
  uint32_t my_row = kNoRow, my_scale = 0;  // this lane's row (of all heads) and scale
  int put_slot = 0, put_tile = 0;
  bool put_v = false;
  // Asks for the next half, if there is one; one group of copies either way.
  auto put = [&]() {
    if (put_tile < my_tiles) {
      const int base = t0 + (col + put_tile * team) * kTile, t = base + lane;
      const bool ok = t >= lo_tok && t < t1;
      if (!put_v) {
        int blk = next_a;
        next_a = next_b;
        next_b = entry(put_tile + 2);
        if (table && (blk < 0 || blk >= a.c.num_blocks)) {
          atomicOr(kp.err_word, kErrBlockIndex);
          blk = 0;  // keep the copy in bounds; the result is flagged invalid
        }
        // rows and scales are counted in 32 bits (checked on the host)
        const uint32_t tok = table ? (uint32_t)blk * bs + (t - block_index(t) * bs)
                                   : (uint32_t)b * a.c.max_kv_len + t;
        my_row = ok ? tok * n_kv + kvh : kNoRow;
        const uint32_t sblk = table ? 0u : (uint32_t)b * ((a.c.max_kv_len + bs - 1) / bs);
        my_scale = (sblk + blk) * n_kv + kvh;
      }
      const uint32_t dst = ring + put_slot * L::kHalfBytes;
      const uint8_t* src = put_v ? v_base : k_base;
      if (base >= lo_tok && base + kTile <= t1) {
#pragma unroll
        for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
          const uint32_t row =
              __shfl_sync(0xffffffffu, my_row, i * kRowsAtOnce + lane / kRowChunks);
          cp_async16(dst + (put_off ^ (swizzle<D>(i * kRowsAtOnce) << 4)) + i * kRowsAtOnce * D,
                     src + (uint64_t)row * D);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
          const uint32_t row =
              __shfl_sync(0xffffffffu, my_row, i * kRowsAtOnce + lane / kRowChunks);
          cp_async16_or_zero(
              dst + (put_off ^ (swizzle<D>(i * kRowsAtOnce) << 4)) + i * kRowsAtOnce * D,
              src + (uint64_t)(row == kNoRow ? 0u : row) * D, row != kNoRow);
        }
      }
      cp_async4(ring_sc + put_slot * L::kScaleBytes + 4 * lane,
                (put_v ? a.c.v_scales : a.c.k_scales) + my_scale, ok);
      if (++put_slot == L::kSlots) put_slot = 0;
      put_tile += put_v;
      put_v = !put_v;
    }
    cp_async_commit();
  };
  if (my_tiles > 0) {
    next_a = entry(0);
    next_b = entry(1);
  }
  if (to_wait) grid_dep_wait();
  to_wait = false;
  if (my_tiles > 0) {
#pragma unroll 1
    for (int h = 0; h < L::kSlots; ++h) put();
  }

  // ================= q's fragments =================
  // A fragments (rows gid and gid + 8, columns 4 quad .. + 3 and 16 + 4 quad .. +
  // 3 of each 32): hi and lo parts of 8 rows in one, or of 16 in two.
  uint4 qf[kQSmem ? 1 : kSteps];
  uint4* qs = reinterpret_cast<uint4*>(smem + L::kQ) + rg * kSteps * 32 * (kWide ? 2 : 1);
  // The finer terms, for tiles with a K scale above fine_ks: behind the coarse ones, where
  // the first tile that needs them puts them (every warp for itself: they are the
  // same), or made again from q.
  const bool fine_smem = fine_in_smem(D, G);
  uint4* qt = reinterpret_cast<uint4*>(
                  smem + L::kQ + (kQSmem ? (kWide ? G : 1) * D * (kWide ? 32 : 16) : 0)) +
              rg * kSteps * 32 * (kWide ? 2 : 1);
  float fine_ks = INFINITY;
  float* row_up = reinterpret_cast<float*>(smem + L::kMerge) + row0 + gid;  // `up`, till the merge
  float sl2[kRows], cap_in[kRows];
  {
    float up[kRows];  // 2^(7 - e) of a row whose largest value is 2^e .. 2^(e + 1)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      uint32_t tops[2] = {0u, 0u};  // two halves each
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i) {
        tops[0] = __vmaxu2(tops[0], qx[r][i].x & 0x7fff7fffu);
        tops[1] = __vmaxu2(tops[1], qx[r][i].y & 0x7fff7fffu);
      }
      uint32_t top = __vmaxu2(tops[0], tops[1]);
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(top >> 7) - 127, -110), 127);
      // How many values lie below 2^(e - 14) = `limit` but for zeros: bit 15 of `from` -
      // (x - 1) says x < limit; a zero less 1 is made the largest (its borrow from
      // the upper half costs that one step of the format).
      const uint32_t limit = (uint32_t)(e + 127 - 14) << 7;
      const uint32_t from = (0x8000u + limit - 2u) * 0x00010001u;
      uint32_t counts[2] = {0u, 0u};  // times 128
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t x = (w ? qx[r][i].y : qx[r][i].x) & 0x7fff7fffu;
          const uint32_t y = __vminu2(x - 0x00010001u, 0x7fff7fffu);
          counts[w] = __dp4a((from - y) & 0x80008000u, 0x01000100u, counts[w]);
        }
      uint32_t count = counts[0] + counts[1];
      count += __shfl_xor_sync(0xffffffffu, count, 1);
      count += __shfl_xor_sync(0xffffffffu, count, 2);
      up[r] = __int_as_float((7 - e + 127) << 23);            // 2^(7 - e)
      float down = __int_as_float((e - 7 + 127) << 23);
      if (top >= 0x7f80u) down = __int_as_float(0x7fc00000);  // an infinity or NaN: the row is NaN
      // Keys whose scale is above this take the second pass (0 * inf: none do).
      const float left = (float)count * (448.f / 128.f / 32768.f) * fabsf(a.scale * kLog2e) * down;
      if (left > 0.f) fine_ks = fminf(fine_ks, __fdividef(kQNoise, left));
      sl2[r] = a.scale * kLog2e * down;
      cap_in[r] = 0.f;
      if (a.softcap > 0.f) {
        cap_in[r] = a.scale * down / a.softcap;
        sl2[r] = a.softcap * kLog2e;
      }
    }
    fine_ks = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(fine_ks)));
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint4 f;
      if constexpr (kWide) {
        uint4 fl;
        coarse_terms(qx[0][2 * i], up[0], f.x, fl.x);
        coarse_terms(qx[1][2 * i], up[1], f.y, fl.y);
        coarse_terms(qx[0][2 * i + 1], up[0], f.z, fl.z);
        coarse_terms(qx[1][2 * i + 1], up[1], f.w, fl.w);
        if (col == 0) {
          qs[(2 * i) * 32 + lane] = f;
          qs[(2 * i + 1) * 32 + lane] = fl;
        }
      } else {
        coarse_terms(qx[0][2 * i], up[0], f.x, f.y);
        coarse_terms(qx[0][2 * i + 1], up[0], f.z, f.w);
        if constexpr (kQSmem) {
          if (col == 0) qs[i * 32 + lane] = f;
        } else {
          qf[i] = f;
        }
      }
    }
    if (fine_ks < INFINITY) {  // (every warp of these rows the same)
#pragma unroll
      for (int r = 0; r < kRows; ++r) row_up[8 * r] = up[r];
      __syncwarp();
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

  // Where ldmatrix's lane reads, before the k step's chunk is XORed in.  K: tiles
  // n = 2 h and 2 h + 1 (by lane >> 4) of 16 tokens 16 h ..: column 2 q + e of tile
  // n is token 16 h + 4 q + 2 (n & 1) + e.
  const int k_tok = ((lane & 6) << 1) + (lane & 1) + ((lane >> 4) << 1);
  const uint32_t k_off = k_tok * D + ((((lane >> 3) & 1) ^ swizzle<D>(k_tok)) << 4);
  const uint32_t v_off = lane * D + (swizzle<D>(lane) << 4);

  float m[kRows], mr[kRows], l[kRows];  // reference, reference - kShift (0 at first), sum
  float2 acc[D / 8][kRows];  // n tile j: columns 8 j + 2 quad, + 1 of each row
#pragma unroll
  for (int r = 0; r < kRows; ++r) m[r] = -INFINITY, mr[r] = 0.f, l[r] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[j][r] = make_float2(0.f, 0.f);

  int slot = 0;
  // The next half: its copies have landed.
  auto take = [&](uint32_t& half, const float4*& scales) {
    cp_async_wait<L::kSlots - 1>();
    __syncwarp();
    half = ring + slot * L::kHalfBytes;
    scales = reinterpret_cast<const float4*>(smem + L::kScale +
                                             (warp * L::kSlots + slot) * L::kScaleBytes);
    if (++slot == L::kSlots) slot = 0;
  };
  // Puts q's finer terms where a tile looks for them.
  auto make_fine = [&]() {
    if (!fine_smem) return;
    float up[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) up[r] = row_up[8 * r];
#pragma unroll 1
    for (int i = 0; i < kSteps; ++i) {
      uint4 f, fl;
      fine_terms(load_q(0, 2 * i), up[0], f.x, fl.x);
      fine_terms(load_q(0, 2 * i + 1), up[0], f.z, fl.z);
      if constexpr (kWide) {
        fine_terms(load_q(1, 2 * i), up[1], f.y, fl.y);
        fine_terms(load_q(1, 2 * i + 1), up[1], f.w, fl.w);
        qt[(2 * i) * 32 + lane] = f;
        qt[(2 * i + 1) * 32 + lane] = fl;
      } else {
        qt[i * 32 + lane] = make_uint4(f.x, fl.x, f.z, fl.z);
      }
    }
    __syncwarp();
  };
  // The tiles.  With up to 8 heads one loop looks at each tile whether it needs the
  // finer terms.  The forms with more, which are short of registers, have the loop
  // twice: the first ends at the first tile that needs them, the second has them in
  // every tile (8 sequences, 4 kv heads of 128 / 256, 64 heads each: 116 / 213 us, as one
  // loop 120 / 281).
  int j = 0;
  bool made = false;
  auto stream = [&](auto mode) {
  constexpr int kMode = decltype(mode)::value;  // 0: without, 1: with, 2: as each tile needs
  auto needs_fine = [&](const float4* sc) {
    return fine_ks < INFINITY &&
           __any_sync(0xffffffffu, reinterpret_cast<const float*>(sc)[lane] > fine_ks);
  };
  for (; j < my_tiles; ++j) {
    const int first = t0 + (col + j * team) * kTile;
    const bool ragged = first + kTile > t1 || first < lo_tok;
    uint32_t half;
    const float4* sc;
    take(half, sc);  // K
    if (kMode == 0 && needs_fine(sc)) {
      slot = slot == 0 ? L::kSlots - 1 : slot - 1;  // this half is taken again
      return;
    }

    // ---- scores of 32 tokens: four n tiles of 8 ----
    float s[4][4], sl[kWide ? 4 : 1][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t at = half + (k_off ^ (uint32_t)(2 * i << 4));
      uint32_t x[4], y[4];  // tiles 0 and 1, both halves of the step's 32 columns; tiles 2, 3
      ldsm_x4(at, x);
      ldsm_x4(at + 16 * D, y);
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
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 2 * kRows; ++e)
        s[n][e] = fmaf(kWide ? sl[kWide ? n : 0][e] : s[n][2 + e], 1.f / kQLo, s[n][e]);
    // ---- what hi and lo leave of q ----
    if (kMode == 1 || (kMode == 2 && needs_fine(sc))) {
      if (kMode == 2 && !made) {
        make_fine();
        made = true;
      }
      float ft[kWide ? 8 : 4][4];
#pragma unroll
      for (int n = 0; n < (kWide ? 8 : 4); ++n) ft[n][0] = ft[n][1] = ft[n][2] = ft[n][3] = 0.f;
#pragma unroll (kWide && D != 128 ? 1 : kSteps)
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t at = half + (k_off ^ (uint32_t)(2 * i << 4));
        uint32_t x[4], y[4];
        ldsm_x4(at, x);
        ldsm_x4(at + 16 * D, y);
        uint4 f, f4;
        if (fine_smem) {
          f = qt[(kWide ? 2 * i : i) * 32 + lane];
          if constexpr (kWide) f4 = qt[(2 * i + 1) * 32 + lane];
        } else {
          fine_terms(load_q(0, 2 * i), row_up[0], f.x, f4.x);
          fine_terms(load_q(1, 2 * i), row_up[8 * (kRows - 1)], f.y, f4.y);
          fine_terms(load_q(0, 2 * i + 1), row_up[0], f.z, f4.z);
          fine_terms(load_q(1, 2 * i + 1), row_up[8 * (kRows - 1)], f.w, f4.w);
        }
        mma16832_e4m3(ft[0], false, f, x[0], x[1]);
        mma16832_e4m3(ft[1], false, f, x[2], x[3]);
        mma16832_e4m3(ft[2], false, f, y[0], y[1]);
        mma16832_e4m3(ft[3], false, f, y[2], y[3]);
        if constexpr (kWide) {
          mma16832_e4m3(ft[4], false, f4, x[0], x[1]);
          mma16832_e4m3(ft[5], false, f4, x[2], x[3]);
          mma16832_e4m3(ft[6], false, f4, y[0], y[1]);
          mma16832_e4m3(ft[7], false, f4, y[2], y[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2 * kRows; ++e)
          s[n][e] = fmaf(fmaf(kWide ? ft[kWide ? 4 + n : 0][e] : ft[n][2 + e], 1.f / kQLo, ft[n][e]),
                         1.f / kQFine, s[n][e]);
    }
    // ---- in log2 units, with K's scales ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 k4 = sc[4 * h + quad];
      const float ks[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 2 * h + (i >> 1), e = i & 1;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float& x = s[n][2 * r + e];
          if (capped)
            x = tanhf(x * (cap_in[r] * ks[i])) * sl2[r];
          else
            x *= sl2[r] * ks[i];
        }
      }
    }
    __syncwarp();
    put();
    const int t_quad = first + 4 * quad;  // the thread's tokens: t_quad + 16 h + 0 .. 3
    if (alibi) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            s[n][2 * r + e] =
                fmaf(-al2[r], (float)(len - 1 - (t_quad + 16 * (n >> 1) + 2 * (n & 1) + e)),
                     s[n][2 * r + e]);
    }
    if (ragged) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = t_quad + 16 * (n >> 1) + 2 * (n & 1) + e;
          if (t < lo_tok || t >= t1) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) s[n][2 * r + e] = -INFINITY;
          }
        }
    }
    // ---- online softmax, V's scales in the reference and the weights ----
    take(half, sc);  // V
    float vs[4][2];
    float mx[kRows];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < kRows; ++r) mx[r] = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v4 = sc[4 * h + quad];
      vs[2 * h][0] = v4.x, vs[2 * h][1] = v4.y, vs[2 * h + 1][0] = v4.z, vs[2 * h + 1][1] = v4.w;
#pragma unroll
      for (int n = 2 * h; n < 2 * h + 2; ++n)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          mx[r] = fmax3(mx[r], s[n][2 * r] + exponent_of(vs[n][0]),
                        s[n][2 * r + 1] + exponent_of(vs[n][1]));
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) grow |= mx[r] > m[r] + kGrow;
    if (__any_sync(0xffffffffu, grow)) {
      float corr[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float now = fmaxf(m[r], mx[r]);
        corr[r] = now == -INFINITY ? 1.f : ex2_approx(m[r] - now);  // 0 at the first token
        l[r] = scaled_sum(l[r], now == -INFINITY ? 0.f : m[r] - now, corr[r]);
        m[r] = now;
        mr[r] = now == -INFINITY ? 0.f : now - kShift;
      }
#pragma unroll
      for (int j8 = 0; j8 < D / 8; ++j8)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          acc[j8][r].x *= corr[r];
          acc[j8][r].y *= corr[r];
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
    // ---- O += P V, 16 columns at a time ----
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t x[4];  // columns gid and gid + 8 of tokens 0-15, then of 16-31
      ldsm_b8_t(half + (v_off ^ (uint32_t)(c << 4)), x);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float o[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t b0, b1;
          e4m3x4_to_f16(x[2 * t + w], b0, b1);
          const int n = 2 * t;
          if constexpr (kWide) {
            mma16816(o, t == 0, hi[0][n], hi[1][n], hi[0][n + 1], hi[1][n + 1], b0, b1);
            mma16816(o, false, lo[0][n], lo[1][n], lo[0][n + 1], lo[1][n + 1], b0, b1);
          } else {
            mma16816(o, t == 0, hi[0][n], lo[0][n], hi[0][n + 1], lo[0][n + 1], b0, b1);
          }
        }
        float2(&to)[kRows] = acc[2 * c + w];
        if constexpr (kWide) {
          to[0] = add2(to[0], make_float2(o[0], o[1]));
          to[1] = add2(to[1], make_float2(o[2], o[3]));
        } else {
          to[0] = add2(to[0], add2(make_float2(o[0], o[1]), make_float2(o[2], o[3])));
        }
      }
    }
    __syncwarp();
    put();
  }
  };
  if constexpr (kWide) {
    stream(std::integral_constant<int, 0>{});
    if (j < my_tiles) {
      make_fine();
      stream(std::integral_constant<int, 1>{});
    }
  } else {
    stream(std::integral_constant<int, 2>{});
  }

  // ================= merge the warps' states =================
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  // Every half that was asked for has landed and been read: the rings are free
  // once the warps meet.
  __syncthreads();
  float* mm = reinterpret_cast<float*>(smem + L::kMerge);  // [warp][16]
  float* ml = mm + kWarps * 16;
  float* mf = ml + kWarps * 16;
  constexpr int kWarpRows = kWide ? 16 : 8;
  float* mo = reinterpret_cast<float*>(smem + L::kRing);  // [warp][kWarpRows][kPitch]
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = gid + 8 * r;
    if (quad == 0) {
      mm[warp * 16 + row] = m[r];
      ml[warp * 16 + row] = l[r];
    }
    float* to = mo + (warp * kWarpRows + row) * L::kPitch + quad * 2;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) *reinterpret_cast<float2*>(to + 8 * j) = acc[j][r];
  }
  __syncthreads();
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
      const float d = mm[w * 16 + lr] == -INFINITY ? 0.f : mm[w * 16 + lr] - mt;
      const float f = ex2_approx(d);
      sum += scaled_sum(ml[w * 16 + lr], d, f);
      mf[w * 16 + lr] = f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // 0: every score is -inf
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
  // ---- the next segment of the share ----
  if (a.parts == 0) return;
  pos += seg_tiles;
  if (pos >= end) return;
  tile = 0;
  if (++kvh == n_kv) {
    kvh = 0;
    do {
      ++b;
      sp = span_of(a, a.kv_lens[b], nullptr);
      pair_tiles = tiles_of(sp);
    } while (pair_tiles == 0);
  }
  __syncthreads();  // the merged rows have been read: the rings are free again
  }
}

// ---------------------------------------------------------------------------
// Combine of the shares: one block per (sequence, query head, kCols columns)
// merges the pair's partials, those of blocks first .. last of the list, by their
// LSE weights.  Each warp takes every 16th (8th), kAtOnce at a time (their
// loads in flight together), with a running maximum; then the warps' states are
// merged.  Narrow slices of columns where that makes no more blocks than SMs (one
// sequence of 30720 tokens, 28 rows of 76 partials each: 1.1 us less than in whole
// rows); more of them cost more than they hide (8 sequences, 64 heads of 64: 2.9 us
// more).
//
// It does not let the next kernel start early: a decode whose blocks came in
// while this grid's still hold their places would not find all SMs free, and the
// blocks that came last would run behind the others (paged batch of 16: 139
// against 106 us).
// ---------------------------------------------------------------------------
constexpr int kAtOnce = 8;
constexpr int combine_warps(int cols) { return cols == 32 ? 16 : 8; }

template <int D, int kCols>
__global__ void __launch_bounds__(32 * combine_warps(kCols))
combine_shares_kernel(const DecodeFp8Args a) {
  constexpr int kCombineWarps = combine_warps(kCols);
  constexpr int kVec = kCols / 32;  // columns of a lane
  __shared__ float s_m[kCombineWarps], s_l[kCombineWarps], s_o[kCombineWarps][kCols];
  const int h = blockIdx.x, b = blockIdx.y, col0 = blockIdx.z * kCols;
  const int g = a.n_q_heads / a.c.n_kv_heads, kvh = h / g, row = h % g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int first, n;  // the pair's blocks
  if (a.batch <= kNoteBeyond) {
    // The lengths are there before the decode ends: the kernels in front of the call
    // had ended before the decode's blocks let this one start.
    const int len = lane < a.batch ? a.kv_lens[lane] : 0;
    const int tiles = lane < a.batch ? tiles_of(span_of(a, len, nullptr)) : 0;
    const int n_kv = a.c.n_kv_heads;
    const Shares sh = shares_of(a.parts, (long long)__reduce_add_sync(0xffffffffu, tiles) * n_kv,
                                (long long)a.batch * n_kv, __reduce_max_sync(0xffffffffu, tiles));
    const int count = sh.own ? (tiles + sh.most - 1) / sh.most : tiles;
    const int mine = __shfl_sync(0xffffffffu, count, b);
    const long long at =
        (long long)__reduce_add_sync(0xffffffffu, lane < b ? count : 0) * n_kv + (long long)kvh * mine;
    if (mine == 0) {
      first = n = 0;
    } else if (sh.own) {
      first = (int)at;
      n = mine;
    } else {
      first = block_of(sh, at);
      n = block_of(sh, at + mine - 1) - first + 1;
    }
    grid_dep_wait();
  } else {
    grid_dep_wait();
    const int2 blocks = a.pair_blocks[(size_t)b * a.c.n_kv_heads + kvh];
    first = blocks.x;
    n = blocks.y - blocks.x + 1;
  }
  if (n <= 1) return;  // the result is already there
  float m = -INFINITY, l = 0.f, o[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) o[e] = 0.f;
  for (int i0 = warp; i0 < n; i0 += kCombineWarps * kAtOnce) {
    float w[kAtOnce], x[kAtOnce][kVec];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kCombineWarps;
      w[u] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[u][e] = 0.f;
      if (i < n) {
        const size_t part = (2 * (size_t)(first + i) + (i == 0 ? 1 : 0)) * g + row;
        w[u] = a.lse_partial[part] * kLog2e;
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[u][e] = a.o_partial[part * D + col0 + e * 32 + lane];
      }
    }
    float now = m;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) now = fmax_nan(now, w[u]);
    const float ref = now == -INFINITY ? 0.f : now;
    const float c = ex2_approx(m - ref);  // 0 at first
    l *= c;
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] *= c;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const float p = ex2_approx(w[u] - ref);
      l += p;
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = fmaf(p, x[u][e], o[e]);
    }
    m = now;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < kVec; ++e) s_o[warp][e * 32 + lane] = o[e];
  __syncthreads();
  if (threadIdx.x >= kCols) return;
  float top = s_m[0];
#pragma unroll
  for (int w = 1; w < kCombineWarps; ++w) top = fmax_nan(top, s_m[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float v = 0.f, sum = 0.f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    const float f = ex2_approx(s_m[w] - ref);  // 0 for a warp that had none
    sum = fmaf(f, s_l[w], sum);
    v = fmaf(f, s_o[w][threadIdx.x], v);
  }
  const size_t at = (size_t)b * a.n_q_heads + h;
  a.o_final[at * D + col0 + threadIdx.x] = sum == 0.f ? 0.f : v / sum;
  if (threadIdx.x == 0 && col0 == 0) a.lse_final[at] = (top + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <int D, bool kWide>
cudaError_t launch_t(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  using L = Smem<D, kWide>;
  const int g = a.n_q_heads / a.c.n_kv_heads;  // at most 64 (validated)
  const int groups = g <= 16 ? 1 : (g <= 32 ? 2 : 4);
  DecodeFp8KParams kp;
  kp.a = a;
  kp.err_word = ctx.err_word;
  kp.bs_mul = 0u;
  kp.bs_shift = -1;
  const uint32_t bs = (uint32_t)a.c.block_size;
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
                                         L::total(q_smem_bytes(D, kWide, kWide ? 4 : 1)));
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = a.parts > 0 ? dim3(a.parts) : dim3(a.num_splits, a.c.n_kv_heads, a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::total(q_smem_bytes(D, kWide, groups));
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<D, kWide>, kp);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  return a.n_q_heads / a.c.n_kv_heads <= 8 ? launch_t<D, false>(a, ctx) : launch_t<D, true>(a, ctx);
}

}  // namespace

int decode_fp8_max_parts(int head_dim, int num_sms) {
  return blocks_per_sm(head_dim) * num_sms;
}

cudaError_t launch_combine_fp8(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int D = a.c.head_dim;
  // 32 columns a block, or whole rows (see the kernel).
  const bool slices = (long long)a.n_q_heads * a.batch * (D / 32) <= ctx.num_sms;
  cfg.gridDim = dim3(a.n_q_heads, a.batch, slices ? D / 32 : 1);
  cfg.blockDim = dim3(32 * combine_warps(slices ? 32 : D));
  auto run = [&](auto slice, auto row) {
    return slices ? cudaLaunchKernelEx(&cfg, slice, a) : cudaLaunchKernelEx(&cfg, row, a);
  };
  if (D == 256) return run(combine_shares_kernel<256, 32>, combine_shares_kernel<256, 256>);
  return D == 128 ? run(combine_shares_kernel<128, 32>, combine_shares_kernel<128, 128>)
                  : run(combine_shares_kernel<64, 32>, combine_shares_kernel<64, 64>);
}

cudaError_t launch_decode_fp8(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  if (a.c.head_dim == 256) return launch_d<256>(a, ctx);
  return a.c.head_dim == 128 ? launch_d<128>(a, ctx) : launch_d<64>(a, ctx);
}

}  // namespace attn
