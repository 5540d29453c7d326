// Writing a key/value cache held in 8 bits, and reading it back, sm_103a.
//
// A cache block (block_size tokens of one kv head, K or V) has one scale
// 2^k, k the smallest integer with amax <= 448 * 2^k, and e4m3 codes
// e4m3(x * 2^-k).  e4m3 is a floating format, so its relative step does not depend on
// the scale; what the power of two costs against amax / 448 is that the scale may be
// nearly twice as large, and e4m3's subnormals (values 2^-15 of the largest and less)
// then begin up to one binade higher.  It makes every
// step but the one rounding exact: x * 2^-k is exact, so a code is the same in
// any arithmetic; a value read back, code * 2^k with 4 significant bits, is a
// bf16 number; and when a token that needs a larger scale joins a block, the
// codes already there move by whole exponents and are rounded again only where
// they fall among e4m3's subnormals.
//
// Work split: one unit per (block touched, kv head), K and V together, so that
// one search serves both and a warp has twice the bytes in flight.  Which blocks a
// call touches is known on the device only (kv_lens and cu_seqlens are there),
// so units are numbered by slots that every warp can place by itself: sequence
// s owns the slots from cu[s] / block_size + 2 s on, at least
// n_s / block_size + 2 of them, and touches no more blocks than that.  A warp
// finds its sequence by a search over cu_seqlens that takes 32 probes at once
// (one round trip for up to 32 sequences, two for up to 1024), so no table has
// to be scanned first and the launch needs one kernel.
//
// Both kernels are bound by HBM on long inputs and by the latency of the
// chain cu_seqlens, kv_lens -> block table -> rows on short ones; the write's rows
// do not wait for the block table.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Rows of a block, of K and of V, that a warp takes at a time.
constexpr int chunk_rows(int D) { return D == 256 ? 8 : 16; }

struct RowsKParams {
  CacheRowsArgs a;
  int warps_per_unit;  // 1, 2 or 4
  long long units;
  bool start_next;  // let the decode behind it start
  uint32_t* err_word;
};

// One unit's place, the same in every lane of its warps.
struct Unit {
  int rows;             // rows of the call in this block (0: nothing to do)
  int before;           // write: rows of the block in front of them
  int src_row;          // first row in the packed tensors
  int head;
  int entry;            // the block as the table has it (contiguous: unused)
  long long block_row;  // contiguous: the block's first row, of all kv heads
  long long scale;      // contiguous: index of its scales
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ Unit find_unit(const RowsKParams& p, long long u, int lane) {
  const CacheRowsArgs& a = p.a;
  const int bs = a.c.block_size, total = a.total_tokens;
  Unit r;
  r.rows = 0;
  r.head = (int)(u % a.c.n_kv_heads);
  const long long slot = u / a.c.n_kv_heads;
  if (u >= p.units) return r;
  int s = 0, c0 = 0, n = 1, j = 0, start = 0;
  auto first_slot = [&](int c, int i) { return (long long)(c / bs) + 2LL * i; };
  if (a.cu_seqlens == nullptr) {
    s = c0 = (int)slot;
    start = a.starts[s];
  } else {
    // The sequence is in [lo, hi); the last round's probes are neighbours, and
    // each lane has its probe's start at hand.
    int lo = 0, hi = a.num_seqs, step, top, c, c_next, st;
    do {
      step = (hi - lo + 31) / 32;
      const int probe = min(lo + lane * step, a.num_seqs - 1);
      c = clampi(a.cu_seqlens[probe], 0, total);
      c_next = clampi(a.cu_seqlens[probe + 1], 0, total);
      st = a.starts ? a.starts[probe] : 0;
      const bool at_or_before =
          lo + lane * step < hi && (lane == 0 || first_slot(c, probe) <= slot);
      top = 31 - __clz(__ballot_sync(0xffffffffu, at_or_before));
      lo += top * step;
      hi = min(hi, lo + step);
    } while (step > 1);
    s = lo;
    c0 = __shfl_sync(0xffffffffu, c, top);
    n = __shfl_sync(0xffffffffu, c_next, top) - c0;
    start = __shfl_sync(0xffffffffu, st, top);
    const long long off = slot - first_slot(c0, s);
    if (n <= 0 || off < 0 || off > n / bs + 1) return r;
    j = (int)off;
  }
  if (start < 0 || (long long)start + n > a.c.capacity()) {
    if (lane == 0) atomicOr(p.err_word, kErrKvLen);
    return r;
  }
  const int blk = start / bs + j;
  const long long b0 = (long long)blk * bs;
  const long long w0 = max((long long)start, b0);
  const long long w1 = min((long long)start + n, b0 + bs);
  if (w0 >= w1) return r;
  if (a.c.block_table != nullptr) {
    r.entry = a.c.block_table[(size_t)s * a.c.max_blocks_per_seq + blk];
  } else {
    const int per_seq = (a.c.max_kv_len + bs - 1) / bs;
    r.block_row = (long long)s * a.c.max_kv_len + b0;
    r.scale = ((long long)s * per_seq + blk) * a.c.n_kv_heads + r.head;
  }
  r.rows = (int)(w1 - w0);
  r.before = (int)(w0 - b0);
  r.src_row = c0 + (int)(w0 - start);
  return r;
}

// Follows the block table's entry; false where it leads outside the cache.
__device__ __forceinline__ bool resolve(const RowsKParams& p, Unit& u, int lane) {
  const CacheFp8& c = p.a.c;
  if (c.block_table == nullptr) return true;
  if (u.entry < 0 || u.entry >= c.num_blocks) {
    if (lane == 0) atomicOr(p.err_word, kErrBlockIndex);
    return false;
  }
  u.block_row = (long long)u.entry * c.block_size;
  u.scale = (long long)u.entry * c.n_kv_heads + u.head;
  return true;
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
// chunk_rows rows a warp stay in shared memory between the two, where blocks of up
// to 4 times that are read once; larger blocks are read again, from L2.  16 prompts
// of 256-4096 tokens (214 MB, 32 us at the measured copy rate): 50 us with the rows
// held in registers (16 warps an SM instead of 24), 43 us in shared memory, 36.5 us
// with the maximum taken two values at a time.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads) cache_write_fp8_kernel(const RowsKParams p) {
  constexpr int kLanes = D / 8;             // lanes of a row, 8 values each
  constexpr int kRowsPerStep = 32 / kLanes;
  constexpr int kChunkRows = chunk_rows(D), kSteps = kChunkRows / kRowsPerStep;
  __shared__ uint32_t s_amax[2][kWarps];
  __shared__ uint4 s_rows[kWarps * 2 * kSteps * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  if (p.start_next) grid_dep_launch();
  check_cu_seqlens(p);
  const int wpu = p.warps_per_unit;
  const int sub = warp % wpu;  // this warp among its unit's
  Unit u = find_unit(p, ((long long)blockIdx.x * kWarps + warp) / wpu, lane);
  const CacheRowsArgs& a = p.a;
  const int lr = lane / kLanes, lc = lane % kLanes;
  const bool again = u.rows > kChunkRows * wpu;
  const uint16_t* src[2] = {a.k + u.head * a.k_head_stride + lc * 8,
                            a.v + u.head * a.v_head_stride + lc * 8};
  const long long ts[2] = {a.k_token_stride, a.v_token_stride};

  // Each lane's own 16 bytes of a step, in shared memory: no other thread reads them.
  uint4* x = s_rows + (warp * 2 * kSteps) * 32 + lane;
  auto load = [&](int c) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = c + i * kRowsPerStep + lr;
        if (r < u.rows) cp_async16(smem_u32(x + (w * kSteps + i) * 32), src[w] + (u.src_row + r) * ts[w]);
      }
  };
  if (u.rows > 0) load(sub * kChunkRows);
  const bool found = u.rows <= 0 || resolve(p, u, lane);
  uint32_t amax[2] = {0u, 0u};
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
    if (c != sub * kChunkRows) load(c);
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // Both halves of each word at once; an infinity or NaN (0x7f80 and above)
      // sends the lane through them again.
      uint32_t two = 0u;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (c + i * kRowsPerStep + lr >= u.rows) continue;
        const uint4 y = x[(w * kSteps + i) * 32];
        two = __vmaxu2(two, y.x & 0x7fff7fffu);
        two = __vmaxu2(two, y.y & 0x7fff7fffu);
        two = __vmaxu2(two, y.z & 0x7fff7fffu);
        two = __vmaxu2(two, y.w & 0x7fff7fffu);
      }
      uint32_t top = max(two & 0xffffu, two >> 16);
      if (top >= 0x7f80u) {
        top = 0u;
#pragma unroll 1
        for (int i = 0; i < kSteps; ++i) {
          if (c + i * kRowsPerStep + lr >= u.rows) continue;
          const uint4 y = x[(w * kSteps + i) * 32];
          top = finite_max(finite_max(top, y.x), y.y);
          top = finite_max(finite_max(top, y.z), y.w);
        }
      }
      amax[w] = max(amax[w], top);
    }
  }
  if (!found) u.rows = 0;
  float was[2] = {0.f, 0.f};
  if (u.rows > 0 && u.before > 0) {
    was[0] = a.c.k_scales[u.scale];
    was[1] = a.c.v_scales[u.scale];
  }
  amax[0] = __reduce_max_sync(0xffffffffu, amax[0]);
  amax[1] = __reduce_max_sync(0xffffffffu, amax[1]);
  if (wpu > 1) {  // the unit's maximum; `was` is read by every warp before it is replaced
    if (lane == 0) s_amax[0][warp] = amax[0], s_amax[1][warp] = amax[1];
    __syncthreads();
    for (int i = 0; i < wpu; ++i) {
      amax[0] = max(amax[0], s_amax[0][warp - sub + i]);
      amax[1] = max(amax[1], s_amax[1][warp - sub + i]);
    }
  }
  if (u.rows <= 0) return;
  __syncwarp();
  const long long pitch = (long long)a.c.n_kv_heads * D;
  float inv[2], ratio[2];
  uint8_t* codes[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float scale = fmaxf(scale_of(amax[w]), was[w]);
    if (sub == 0 && lane == 0 && scale != was[w])
      (w ? a.c.v_scales : a.c.k_scales)[u.scale] = scale;
    inv[w] = 1.f / scale;  // exact for a power of two (a caller's own scale may be none)
    ratio[w] = scale != was[w] ? was[w] * inv[w] : 1.f;
    codes[w] = (w ? a.c.v : a.c.k) + u.block_row * pitch + u.head * D + lc * 8;
  }
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
    if (again) {
      load(c);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = c + i * kRowsPerStep + lr;
        if (r >= u.rows) continue;
        const uint4 y = x[(w * kSteps + i) * 32];
        const float f = inv[w];
        uint2 out;
        out.x = e4m3x4(bf16_lo(y.x) * f, bf16_hi(y.x) * f, bf16_lo(y.y) * f, bf16_hi(y.y) * f);
        out.y = e4m3x4(bf16_lo(y.z) * f, bf16_hi(y.z) * f, bf16_lo(y.w) * f, bf16_hi(y.w) * f);
        *reinterpret_cast<uint2*>(codes[w] + (u.before + r) * pitch) = out;
      }
    }
  }
  // The block's earlier rows, when its scale grew.
  if (u.before > 0) {
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      const float f = w ? ratio[1] : ratio[0];
      if (f == 1.f) continue;
      for (int r = sub * kRowsPerStep + lr; r < u.before; r += kRowsPerStep * wpu) {
        uint2* at = reinterpret_cast<uint2*>((w ? codes[1] : codes[0]) + r * pitch);
        const uint2 old = *at;
        const float2 f0 = from_e4m3x2(old.x), f1 = from_e4m3x2(old.x >> 16);
        const float2 f2 = from_e4m3x2(old.y), f3 = from_e4m3x2(old.y >> 16);
        *at = make_uint2(e4m3x4(f0.x * f, f0.y * f, f1.x * f, f1.y * f),
                         e4m3x4(f2.x * f, f2.y * f, f3.x * f, f3.y * f));
      }
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
  constexpr int kChunkRows = chunk_rows(D), kSteps = kChunkRows / kRowsPerStep;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  check_cu_seqlens(p);
  const int wpu = p.warps_per_unit;
  const int sub = warp % wpu;
  Unit u = find_unit(p, ((long long)blockIdx.x * kWarps + warp) / wpu, lane);
  if (u.rows <= 0 || !resolve(p, u, lane)) return;
  const CacheRowsArgs& a = p.a;
  const int lr = lane / kLanes, lc = lane % kLanes;
  const long long pitch = (long long)a.c.n_kv_heads * D;
  const long long from = (u.block_row + u.before) * pitch + u.head * D + lc * 8;
  const float scale[2] = {a.c.k_scales[u.scale], a.c.v_scales[u.scale]};
  uint16_t* dst[2] = {a.k + u.head * a.k_head_stride + lc * 8,
                      a.v + u.head * a.v_head_stride + lc * 8};
  const long long ts[2] = {a.k_token_stride, a.v_token_stride};
  for (int c = sub * kChunkRows; c < u.rows; c += kChunkRows * wpu) {
    uint2 x[2][kSteps];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = c + i * kRowsPerStep + lr;
        x[w][i] = make_uint2(0, 0);
        if (r < u.rows)
          x[w][i] = *reinterpret_cast<const uint2*>((w ? a.c.v : a.c.k) + from + r * pitch);
      }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = c + i * kRowsPerStep + lr;
        if (r >= u.rows) continue;
        const float2 f0 = from_e4m3x2(x[w][i].x), f1 = from_e4m3x2(x[w][i].x >> 16);
        const float2 f2 = from_e4m3x2(x[w][i].y), f3 = from_e4m3x2(x[w][i].y >> 16);
        const float f = scale[w];
        *reinterpret_cast<uint4*>(dst[w] + (u.src_row + r) * ts[w]) =
            make_uint4(pack_bf16x2(f0.x * f, f0.y * f), pack_bf16x2(f1.x * f, f1.y * f),
                       pack_bf16x2(f2.x * f, f2.y * f), pack_bf16x2(f3.x * f, f3.y * f));
      }
  }
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const CacheRowsArgs& a, const LaunchCtx& ctx) {
  RowsKParams p;
  p.a = a;
  p.err_word = ctx.err_word;
  const int rows = chunk_rows(a.c.head_dim);
  const int chunks = (a.c.block_size + rows - 1) / rows;
  p.warps_per_unit = chunks <= 1 ? 1 : (chunks <= 2 ? 2 : 4);
  const long long slots = a.cu_seqlens
                              ? a.total_tokens / a.c.block_size + 2LL * a.num_seqs
                              : (long long)a.num_seqs;
  p.units = slots * a.c.n_kv_heads;
  const long long blocks = (p.units * p.warps_per_unit + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;  // refused by the caller
  // A decode that starts while this grid holds places finds fewer SMs for its blocks
  // at first: worth it for small grids (decode steps of 1 / 16 sequences of 8 kv heads
  // and 4000-8000 tokens, 2 / 32 blocks here: 14.2 -> 12.3 / 50.4 -> 48.9 us; of 32,
  // 64 blocks: 85.7 -> 85.4), not for large ones (of 64, 128 blocks: 125 -> 129).
  p.start_next = a.before_decode && 2 * blocks <= ctx.num_sms;
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
