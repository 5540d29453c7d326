// Split-KV single-token decode over a key/value cache held in 8 bits, sm_103a.
//
// One thread block per (split, kv head, sequence): 32 tokens at a time, K and V
// dequantised into shared memory as floats, the scores, the online softmax and
// the products in fp32.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;

struct DecodeFp8KParams {
  DecodeFp8Args a;
  uint32_t* err_word;
};

__device__ __forceinline__ float from_e4m3(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}"
      : "=f"(f)
      : "r"(h));
  return f;
}

template <int D>
__global__ void __launch_bounds__(kThreads) decode_fp8_kernel(const DecodeFp8KParams kp) {
  const DecodeFp8Args& a = kp.a;
  extern __shared__ float sm[];
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int S = a.num_splits, n_kv = a.c.n_kv_heads, bs = a.c.block_size;
  const int g = a.n_q_heads / n_kv, tid = threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();

  const long long capacity = a.c.capacity();
  int len = a.kv_lens[b];
  if (len < 0 || (long long)len + a.append > capacity) {
    if (tid == 0 && split == 0) atomicOr(kp.err_word, kErrKvLen);
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

  float* o_out = a.o_partial + (((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g) * D;
  float* lse_out = a.lse_partial + ((size_t)split * a.batch + b) * a.n_q_heads + (size_t)kvh * g;

  float* sq = sm;                        // [g][D]
  float* so = sq + g * D;                // [g][D]
  float* sx = so + g * D;                // [kTile][D + 1]
  float* ss = sx + kTile * (D + 1);      // [g][kTile]
  float* sm_ = ss + g * kTile;           // [g] running maximum
  float* sl = sm_ + g;                   // [g] running sum
  float* sc = sl + g;                    // [g] correction
  for (int i = tid; i < g * D; i += kThreads) {
    sq[i] = __uint_as_float(
        (uint32_t)a.q[((size_t)b * a.n_q_heads + (size_t)kvh * g) * D + i] << 16);
    so[i] = 0.f;
  }
  for (int i = tid; i < g; i += kThreads) {
    sm_[i] = -INFINITY;
    sl[i] = 0.f;
  }

  auto load = [&](const uint8_t* codes, const float* scales, int base) {
    __syncthreads();
    for (int i = tid; i < kTile * D; i += kThreads) {
      const int r = i / D, c = i % D, t = base + r;
      float x = 0.f;
      if (t >= lo_tok && t < t1) {
        size_t row, sidx;
        if (a.c.block_table) {
          int blk = a.c.block_table[(size_t)b * a.c.max_blocks_per_seq + t / bs];
          if (blk < 0 || blk >= a.c.num_blocks) {
            atomicOr(kp.err_word, kErrBlockIndex);
            blk = 0;
          }
          row = (size_t)blk * bs + t % bs;
          sidx = (size_t)blk;
        } else {
          row = (size_t)b * a.c.max_kv_len + t;
          sidx = (size_t)b * ((a.c.max_kv_len + bs - 1) / bs) + t / bs;
        }
        x = from_e4m3(codes[(row * n_kv + kvh) * D + c]) * scales[sidx * n_kv + kvh];
      }
      sx[r * (D + 1) + c] = x;
    }
    __syncthreads();
  };

  for (int base = t0; base < t1; base += kTile) {
    load(a.c.k, a.c.k_scales, base);
    for (int i = tid; i < g * kTile; i += kThreads) {
      const int h = i / kTile, r = i % kTile, t = base + r;
      float s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(sq[h * D + c], sx[r * (D + 1) + c], s);
      s *= a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      if (a.alibi_slopes) s = fmaf(-a.alibi_slopes[kvh * g + h], (float)(len - 1 - t), s);
      ss[h * kTile + r] = t >= lo_tok && t < t1 ? s : -INFINITY;
    }
    __syncthreads();
    for (int h = tid; h < g; h += kThreads) {
      float m = sm_[h];
      for (int r = 0; r < kTile; ++r) m = fmaxf(m, ss[h * kTile + r]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float c = expf(sm_[h] - ref);
      float l = sl[h] * c;
      for (int r = 0; r < kTile; ++r) {
        const float e = expf(ss[h * kTile + r] - ref);
        ss[h * kTile + r] = e;
        l += e;
      }
      sm_[h] = m;
      sl[h] = l;
      sc[h] = c;
    }
    load(a.c.v, a.c.v_scales, base);
    for (int i = tid; i < g * D; i += kThreads) {
      const int h = i / D, c = i % D;
      float o = so[i] * sc[h];
      for (int r = 0; r < kTile; ++r) o = fmaf(ss[h * kTile + r], sx[r * (D + 1) + c], o);
      so[i] = o;
    }
  }
  __syncthreads();
  for (int i = tid; i < g * D; i += kThreads) {
    const float l = sl[i / D];
    o_out[i] = l > 0.f ? so[i] / l : l;
  }
  for (int i = tid; i < g; i += kThreads) lse_out[i] = sm_[i] + logf(sl[i]);
}

template <int D>
cudaError_t launch_t(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  DecodeFp8KParams kp{a, ctx.err_word};
  const int g = a.n_q_heads / a.c.n_kv_heads;
  const size_t smem = sizeof(float) * (2 * g * D + kTile * (D + 1) + g * kTile + 3 * g);
  cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<D>, kp);
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Args& a, const LaunchCtx& ctx) {
  if (a.c.head_dim == 256) return launch_t<256>(a, ctx);
  return a.c.head_dim == 128 ? launch_t<128>(a, ctx) : launch_t<64>(a, ctx);
}

}  // namespace attn
