// Writing a key/value cache held in 8 bits, and reading it back, sm_103a.
//
// A cache block (block_size tokens of one kv head, K or V) has one scale
// 2^k, k the smallest integer with amax <= 448 * 2^k, and e4m3 codes
// e4m3(x * 2^-k).  The power of two costs no precision (e4m3 is a floating
// format: its relative step does not depend on the scale) and makes every
// step but the one rounding exact: x * 2^-k is exact, so a code is the same in
// any arithmetic; a value read back, code * 2^k with 4 significant bits, is a
// bf16 number; and when a token that needs a larger scale joins a block, the
// codes already there move by whole exponents and are rounded again only where
// they fall among e4m3's subnormals.
//
// Work split: one unit per (block touched, kv head, K or V).  Which blocks a
// call touches is known on the device only (kv_lens and cu_seqlens are there),
// so units are numbered by slots that every warp can place by itself: sequence
// s owns the slots from cu[s] / block_size + 2 s on, at least
// n_s / block_size + 2 of them, and touches no more blocks than that.  A warp
// finds its sequence by a search over cu_seqlens that takes 32 probes at once
// (one round trip for up to 32 sequences, two for up to 1024), so no table has
// to be scanned first and the launch needs one kernel.
//
// Both kernels are bound by HBM on long inputs and by the latency of the
// chain cu_seqlens -> kv_lens -> block table -> rows on short ones.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunkRows = 16;  // rows of a block that a warp holds in registers

struct RowsKParams {
  CacheRowsArgs a;
  int warps_per_unit;  // 1, 2, 4 or 8
  long long units;
  uint32_t* err_word;
};

// One unit's place, the same in every lane of its warps.
struct Unit {
  int rows;             // rows of the call in this block (0: nothing to do)
  int before;           // write: rows of the block in front of them
  long long src_row;    // first row in the packed tensor
  long long cache_row;  // first row in the cache, in rows of all kv heads
  long long block_row;  // the block's first row
  long long scale;      // index into the scales
  int head;
  bool is_v;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// First slot of sequence s.
__device__ __forceinline__ long long first_slot(const CacheRowsArgs& a, int s) {
  return (long long)(clampi(a.cu_seqlens[s], 0, a.total_tokens) / a.c.block_size) + 2LL * s;
}

__device__ Unit find_unit(const RowsKParams& p, long long u, int lane) {
  const CacheRowsArgs& a = p.a;
  Unit r;
  r.rows = 0;
  r.is_v = (u & 1) != 0;
  r.head = (int)((u >> 1) % a.c.n_kv_heads);
  const long long slot = (u >> 1) / a.c.n_kv_heads;
  if (u >= p.units) return r;
  int s = 0, c0 = 0, n = 1, j = 0;
  if (a.cu_seqlens == nullptr) {
    s = c0 = (int)slot;
  } else {
    int lo = 0, hi = a.num_seqs;  // the sequence is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int probe = lo + lane * step;
      const bool at_or_before = probe < hi && (lane == 0 || first_slot(a, probe) <= slot);
      const int top = 31 - __clz(__ballot_sync(0xffffffffu, at_or_before));
      lo += top * step;
      hi = min(hi, lo + step);
    }
    s = lo;
    c0 = clampi(a.cu_seqlens[s], 0, a.total_tokens);
    n = clampi(a.cu_seqlens[s + 1], 0, a.total_tokens) - c0;
    const long long off = slot - first_slot(a, s);
    if (n <= 0 || off < 0 || off > n / a.c.block_size + 1) return r;
    j = (int)off;
  }
  const int start = a.starts ? a.starts[s] : 0;
  const long long cap = a.c.capacity();
  if (start < 0 || (long long)start + n > cap) {
    if (lane == 0) atomicOr(p.err_word, kErrKvLen);
    return r;
  }
  const int blk = start / a.c.block_size + j;
  const long long b0 = (long long)blk * a.c.block_size;
  const long long w0 = max((long long)start, b0);
  const long long w1 = min((long long)start + n, b0 + a.c.block_size);
  if (w0 >= w1) return r;
  if (a.c.block_table != nullptr) {
    const int phys = a.c.block_table[(size_t)s * a.c.max_blocks_per_seq + blk];
    if (phys < 0 || phys >= a.c.num_blocks) {
      if (lane == 0) atomicOr(p.err_word, kErrBlockIndex);
      return r;
    }
    r.block_row = (long long)phys * a.c.block_size;
    r.scale = (long long)phys * a.c.n_kv_heads + r.head;
  } else {
    const int per_seq = (a.c.max_kv_len + a.c.block_size - 1) / a.c.block_size;
    r.block_row = (long long)s * a.c.max_kv_len + b0;
    r.scale = ((long long)s * per_seq + blk) * a.c.n_kv_heads + r.head;
  }
  r.rows = (int)(w1 - w0);
  r.before = (int)(w0 - b0);
  r.cache_row = r.block_row + r.before;
  r.src_row = c0 + (w0 - start);
  return r;
}

// cu_seqlens has to start at 0 and not decrease up to total_tokens; one block
// of the grid looks at all of it.
__device__ void check_cu_seqlens(const RowsKParams& p) {
  if (blockIdx.x != 0 || p.a.cu_seqlens == nullptr) return;
  bool bad = false;
  for (int i = threadIdx.x; i < p.a.num_seqs; i += kThreads) {
    const int x = p.a.cu_seqlens[i], y = p.a.cu_seqlens[i + 1];
    bad |= x > y || x < 0 || y > p.a.total_tokens || (i == 0 && x != 0);
  }
  if (bad) atomicOr(p.err_word, kErrSeqLens);
}

// ---- e4m3 conversions of eight values ----
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2_pack(b, a) | (e4m3x2_pack(d, c) << 16);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Largest finite |x| of a packed pair against m, both as bf16 bit patterns
// (their order is that of the magnitudes).
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t pair) {
  const uint32_t lo = pair & 0x7fffu, hi = (pair >> 16) & 0x7fffu;
  if (lo < 0x7f80u) m = max(m, lo);
  if (hi < 0x7f80u) m = max(m, hi);
  return m;
}

// 2^k for a block whose largest finite magnitude has these bf16 bits:
// 448 = 1.75 * 2^8, and 1.75 is the mantissa 0x60.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  int k = kScaleExpMin;
  if (amax_bits != 0u) {
    const int e = (int)(amax_bits >> 7) - 127;
    k = e - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
    k = min(max(k, kScaleExpMin), kScaleExpMax);
  }
  return __int_as_float((k + 127) << 23);
}

// ---------------------------------------------------------------------------
// Write: amax over the unit's rows, the block's scale, the codes.  Up to
// kChunkRows rows a warp stay in registers between the two (blocks of up to
// 128 tokens are read once); larger blocks are read again, from L2.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads) cache_write_fp8_kernel(const RowsKParams p) {
  constexpr int kLanes = D / 8;             // lanes of a row, 8 values each
  constexpr int kRowsPerStep = 32 / kLanes;
  constexpr int kSteps = kChunkRows / kRowsPerStep;
  __shared__ uint32_t s_amax[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  check_cu_seqlens(p);
  const int wpu = p.warps_per_unit;
  const int sub = warp % wpu;  // this warp among its unit's
  const Unit u = find_unit(p, ((long long)blockIdx.x * kWarps + warp) / wpu, lane);
  const CacheRowsArgs& a = p.a;
  const uint16_t* src = u.is_v ? a.v : a.k;
  const long long ts = u.is_v ? a.v_token_stride : a.k_token_stride;
  const long long hs = u.is_v ? a.v_head_stride : a.k_head_stride;
  uint8_t* codes = u.is_v ? a.c.v : a.c.k;
  float* scales = u.is_v ? a.c.v_scales : a.c.k_scales;
  const int lr = lane / kLanes, lc = lane % kLanes;
  const bool again = u.rows > kChunkRows * wpu;

  uint4 x[kSteps];
  uint32_t amax = 0u;
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = c + i * kRowsPerStep + lr;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < u.rows)
        x[i] = *reinterpret_cast<const uint4*>(src + (u.src_row + r) * ts + u.head * hs + lc * 8);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      amax = finite_max(amax, x[i].x);
      amax = finite_max(amax, x[i].y);
      amax = finite_max(amax, x[i].z);
      amax = finite_max(amax, x[i].w);
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  const float was = u.rows > 0 && u.before > 0 ? scales[u.scale] : 0.f;
  if (wpu > 1) {  // the unit's maximum; `was` is read by every warp before it is replaced
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();
    for (int w = 0; w < wpu; ++w) amax = max(amax, s_amax[warp - sub + w]);
  }
  if (u.rows <= 0) return;
  __syncwarp();
  const float scale = fmaxf(scale_of(amax), was);
  if (sub == 0 && lane == 0 && scale != was) scales[u.scale] = scale;

  const float inv = 1.f / scale;  // exact: a power of two
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = c + i * kRowsPerStep + lr;
      if (r >= u.rows) continue;
      if (again)
        x[i] = *reinterpret_cast<const uint4*>(src + (u.src_row + r) * ts + u.head * hs + lc * 8);
      uint2 out;
      out.x = e4m3x4(bf16_lo(x[i].x) * inv, bf16_hi(x[i].x) * inv, bf16_lo(x[i].y) * inv,
                     bf16_hi(x[i].y) * inv);
      out.y = e4m3x4(bf16_lo(x[i].z) * inv, bf16_hi(x[i].z) * inv, bf16_lo(x[i].w) * inv,
                     bf16_hi(x[i].w) * inv);
      *reinterpret_cast<uint2*>(codes + ((u.cache_row + r) * a.c.n_kv_heads + u.head) * D +
                                lc * 8) = out;
    }
  }
  // The block's earlier rows, when its scale grew.
  if (u.before > 0 && scale != was) {
    const float ratio = was * inv;
    for (int r = sub * kRowsPerStep + lr; r < u.before; r += kRowsPerStep * wpu) {
      uint2* at = reinterpret_cast<uint2*>(
          codes + ((u.block_row + r) * a.c.n_kv_heads + u.head) * D + lc * 8);
      const uint2 old = *at;
      const float2 f0 = from_e4m3x2(old.x), f1 = from_e4m3x2(old.x >> 16);
      const float2 f2 = from_e4m3x2(old.y), f3 = from_e4m3x2(old.y >> 16);
      *at = make_uint2(e4m3x4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio),
                       e4m3x4(f2.x * ratio, f2.y * ratio, f3.x * ratio, f3.y * ratio));
    }
  }
}

// ---------------------------------------------------------------------------
// Read: codes times their block's scale, as bf16 (exact for the scales that
// the write sets).
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_fp8_kernel(const RowsKParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kRowsPerStep = 32 / kLanes;
  constexpr int kSteps = kChunkRows / kRowsPerStep;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  check_cu_seqlens(p);
  const int wpu = p.warps_per_unit;
  const int sub = warp % wpu;
  const Unit u = find_unit(p, ((long long)blockIdx.x * kWarps + warp) / wpu, lane);
  if (u.rows <= 0) return;
  const CacheRowsArgs& a = p.a;
  uint16_t* dst = u.is_v ? a.v : a.k;
  const long long ts = u.is_v ? a.v_token_stride : a.k_token_stride;
  const long long hs = u.is_v ? a.v_head_stride : a.k_head_stride;
  const uint8_t* codes = u.is_v ? a.c.v : a.c.k;
  const float scale = (u.is_v ? a.c.v_scales : a.c.k_scales)[u.scale];
  const int lr = lane / kLanes, lc = lane % kLanes;
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
    uint2 x[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = c + i * kRowsPerStep + lr;
      x[i] = make_uint2(0, 0);
      if (r < u.rows)
        x[i] = *reinterpret_cast<const uint2*>(
            codes + ((u.cache_row + r) * a.c.n_kv_heads + u.head) * D + lc * 8);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = c + i * kRowsPerStep + lr;
      if (r >= u.rows) continue;
      const float2 f0 = from_e4m3x2(x[i].x), f1 = from_e4m3x2(x[i].x >> 16);
      const float2 f2 = from_e4m3x2(x[i].y), f3 = from_e4m3x2(x[i].y >> 16);
      *reinterpret_cast<uint4*>(dst + (u.src_row + r) * ts + u.head * hs + lc * 8) = make_uint4(
          pack_bf16x2(f0.x * scale, f0.y * scale), pack_bf16x2(f1.x * scale, f1.y * scale),
          pack_bf16x2(f2.x * scale, f2.y * scale), pack_bf16x2(f3.x * scale, f3.y * scale));
    }
  }
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const CacheRowsArgs& a, const LaunchCtx& ctx) {
  RowsKParams p;
  p.a = a;
  p.err_word = ctx.err_word;
  const int chunks = (a.c.block_size + kChunkRows - 1) / kChunkRows;
  p.warps_per_unit = chunks <= 1 ? 1 : (chunks <= 2 ? 2 : (chunks <= 4 ? 4 : 8));
  const long long slots = a.cu_seqlens
                              ? a.total_tokens / a.c.block_size + 2LL * a.num_seqs
                              : (long long)a.num_seqs;
  p.units = slots * a.c.n_kv_heads * 2;
  const long long blocks = (p.units * p.warps_per_unit + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;  // refused by the caller
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_cache_write_fp8(const CacheRowsArgs& a, const LaunchCtx& ctx) {
  if (a.c.head_dim == 256) return launch_rows(cache_write_fp8_kernel<256>, a, ctx);
  return a.c.head_dim == 128 ? launch_rows(cache_write_fp8_kernel<128>, a, ctx)
                             : launch_rows(cache_write_fp8_kernel<64>, a, ctx);
}

cudaError_t launch_cache_read_fp8(const CacheRowsArgs& a, const LaunchCtx& ctx) {
  if (a.c.head_dim == 256) return launch_rows(cache_read_fp8_kernel<256>, a, ctx);
  return a.c.head_dim == 128 ? launch_rows(cache_read_fp8_kernel<128>, a, ctx)
                             : launch_rows(cache_read_fp8_kernel<64>, a, ctx);
}

}  // namespace attn
