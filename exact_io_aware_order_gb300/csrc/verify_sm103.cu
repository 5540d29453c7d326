// Verification of drafted tokens against the target's probabilities, sm_103a.
//
// From the root on, the children of the node reached are tried in index order.  With
// p and q the target's and the draft's probabilities there, w = p and Z = 1 at first,
// a child with token x is accepted where u q(x) Z < w(x); where it is not, w becomes
// max(w - q Z, 0) and Z its sum, and the next child is tried against those.  Where no
// child is left, the next token is the smallest v with w(0) + .. + w(v) > u' sum(w).
// A drafted token so accepted, or one so drawn, is distributed as the target's.
// Without q (drafts that are certain) a refused child only loses its weight: w(x) = 0,
// Z less that.  After several refusals w = max(p - q (Z_1 + Z_2 + ..), 0) (what has reached
// 0 stays there), so one product serves all of them.
//
// All of it in whole multiples of 2^-60: sums and products of 64-bit integers are the
// same in any order, so the drawn index is the same however the vocabulary is divided,
// and two probabilities that differ are never taken for equal by rounding (an fp32
// running sum over 128k entries moves a border by 1e-6, the size of many entries).
// 64-bit integer additions are two instructions; fp64 ones would run at 1/64 rate.  Sums end
// at 8 - 2^-60 (what probabilities never reach): such a sum is the same in any order too, and
// its products with numbers below 2 fit 64 bits.
//
// Work split: a cluster of blocks a sequence, the vocabulary in equal runs, a run a
// warp.  The walk itself is scalar: one thread of the first block does it on numbers that
// 64 threads gathered (a child's p and q do not depend on the walk), and asks the cluster
// for a pass over the vocabulary only where it needs one: a sum after a refusal that has a
// sibling behind it, and the last draw.  That thread decides for all blocks, so they meet
// at the same barriers whatever the memory holds.
// Bound by HBM for large batches (one row of p, and of q, a sequence), by the latency
// of the gathers and the cluster's barriers for small ones.  Measured: 64 trees of 10 - 41
// nodes over 128257 entries 60 us, of which some 9 are the rows' bytes: a sequence is a chain of
// gathers, a pass for each refusal that has a sibling behind it, and two for the last draw;
// a chain of 6 over 32000 entries 9 us.
#include <algorithm>
#include <cstdint>
#include <type_traits>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostNodes = 64;
constexpr int kMostBlocks = 8;
constexpr int kMostWarps = 16;
constexpr int kUnroll = 8;
constexpr unsigned long long kOne = 1ull << 60;
constexpr unsigned long long kMostC = 1ull << 63;
constexpr unsigned long long kMostSum = kMostC - 1;

// Multiples of 2^-60 in x, rounded down; 0 for what is not in [0, 2).
__device__ __forceinline__ unsigned long long fixed60(float x) {
  const uint32_t b = __float_as_uint(x), e = b >> 23;  // (a set sign makes it 256 or more)
  // The 24 bits of an exponent of 127, moved down.
  const unsigned long long top = (unsigned long long)(((b & 0x7fffffu) | 0x800000u) << 5) << 32;
  return top >> min(127u - e, 63u);  // (top is below 2^61: an e of 128 or more wraps, and leaves 0)
}
// a b / 2^60, rounded down.
__device__ __forceinline__ unsigned long long times60(unsigned long long a, unsigned long long b) {
  return (__umul64hi(a, b) << 4) | ((a * b) >> 60);
}

// The sum of a warp's numbers, each at most kMostSum and so the sum, in pieces of 21 bits (whose
// sums take 26).
__device__ __forceinline__ unsigned long long warp_sum60(unsigned long long x) {
  constexpr uint32_t kPiece = (1u << 21) - 1u;
  const uint32_t s0 = __reduce_add_sync(0xffffffffu, (uint32_t)x & kPiece);
  const uint32_t s1 = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 21) & kPiece) + (s0 >> 21);
  const uint32_t s2 = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 42)) + (s1 >> 21);
  if (s2 > kPiece) return kMostSum;
  return (unsigned long long)s2 << 42 | (unsigned long long)(s1 & kPiece) << 21 | (s0 & kPiece);
}

enum Command : int { kEnd = 0, kSum = 1, kFind = 2, kLook = 3 };

// What the first block tells the others.
struct Order {
  int kind;
  int node;       // whose rows (local index)
  int levels;     // with q: terms of C (0 for the plain p); without: refused tokens
  int rank;       // kFind: the block that holds the border
  unsigned long long rest;  // kFind: what of the drawn sum is left there
};

struct Shared {
  Order order;
  // with q: C, the sum of the Zs of the refusals so far, in terms below 8
  unsigned long long C[kMostNodes];
  int gone[kMostNodes];                  // without q: the refused tokens
  unsigned long long totals[kMostBlocks];  // the blocks' sums (in the first block)
  unsigned long long warp_sums[kMostWarps];
  // gathered
  int parent[kMostNodes], token[kMostNodes];
  unsigned long long p[kMostNodes], q[kMostNodes], u[kMostNodes];
};

// What a pass over the vocabulary computes for an entry, chosen once a pass so that its loops
// have no branches inside (with them 64 trees over 128257 entries took 67 us instead of 58).
enum Form : int {
  kPlain = 0,  // p
  kLess = 1,   // max(p - q, 0): after the first refusal
  kTerm = 2,   // max(p - q C, 0)
  kAny = 3     // several terms of C, or tokens that are gone
};

template <bool DRAFTS, int FORM>
__device__ __forceinline__ unsigned long long weight(float pv, float qv, int v, int levels,
                                                     unsigned long long c0,
                                                     const unsigned long long* C, const int* gone) {
  unsigned long long w = fixed60(pv);
  if constexpr (DRAFTS && FORM != kPlain) {
    const unsigned long long q = fixed60(qv);
    const unsigned long long y = FORM == kLess ? q : times60(q, c0);
    w = w > y ? w - y : 0ull;
    if constexpr (FORM == kAny) {
      for (int i = 1; i < levels; ++i) {
        const unsigned long long z = times60(q, C[i]);
        w = w > z ? w - z : 0ull;
      }
    }
  } else if constexpr (FORM == kAny) {
    for (int i = 0; i < levels; ++i)
      if (gone[i] == v) w = 0ull;
  }
  return w;
}

template <bool DRAFTS, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(const VerifyArgs a) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= kMostWarps, "warp_sums");
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Shared* first = cluster.map_shared_rank(&sh, 0);
  grid_dep_wait();

  const int x0 = a.cu_nodes[b], x1 = a.cu_nodes[b + 1];
  const int n0 = min(max(x0, 0), a.total_nodes), n1 = min(max(x1, n0), a.total_nodes);
  const int n = min(n1 - n0, kMostNodes);
  if (rank == 0) {
    if (threadIdx.x == 0 &&
        (x0 != n0 || x1 != n1 || n1 - n0 > kMostNodes || (b == 0 && x0 != 0)))
      atomicOr(a.err_word, kErrSeqLens);
    for (int i = threadIdx.x; i < kMostNodes; i += kThreads) {
      a.path[(size_t)b * kMostNodes + i] = i == 0 && n > 0 ? 0 : -1;
      int up = -1, tok = -1;
      if (i < n) {
        up = a.parents[n0 + i];
        if (i == 0 ? up != -1 : (up < 0 || up >= i)) {
          atomicOr(a.err_word, kErrSeqLens);
          up = -1;
        }
      }
      if (i > 0 && up >= 0) {
        tok = a.tokens[n0 + i];
        if (tok < 0 || tok >= a.vocab) {
          atomicOr(a.err_word, kErrSeqLens);
          up = -1;  // it cannot be accepted
        } else {
          const size_t at = (size_t)(n0 + up) * a.p_stride + tok;
          sh.p[i] = fixed60(a.target_probs[at]);
          if constexpr (DRAFTS) sh.q[i] = fixed60(a.draft_probs[(size_t)(n0 + up) * a.q_stride + tok]);
          sh.u[i] = fixed60(a.u_accept[n0 + i]);
        }
      }
      sh.parent[i] = up;
      sh.token[i] = tok;
    }
    __syncthreads();
  }

  // The walk, in the first block's first thread: it stands at node `at`, `levels` of
  // whose children were refused; `next` is the node to be looked at.
  int at = 0, next = 1, levels = 0, count = 0;
  unsigned long long Z = kOne;
  bool have_z = true, drawing = false;
  auto sum_of_totals = [&] {
    unsigned long long hi = 0ull, lo = 0ull;
    for (int r = 0; r < blocks; ++r) {
      const unsigned long long t = sh.totals[r];
      hi += t >> 32;
      lo += (uint32_t)t;
    }
    hi += lo >> 32;
    return hi >> 31 ? kMostSum : hi << 32 | (uint32_t)lo;
  };
  auto decide = [&]() -> Order {
    if (n == 0) {
      a.num_accepted[b] = 0;
      a.next_token[b] = -1;
      return Order{kEnd, 0, 0, 0, 0ull};
    }
    if (drawing) {  // the sums of the last draw are in
      const unsigned long long total = sum_of_totals();
      if (total == 0ull && levels > 0) {
        levels = 0;  // nothing is left: the target's own probabilities
        return Order{kSum, at, 0, 0, 0ull};
      }
      a.num_accepted[b] = count;
      const unsigned long long T = times60(total, fixed60(a.u_sample[b]));
      if (T >= total) {
        a.next_token[b] = a.vocab - 1;
        return Order{total == 0ull ? kLook : kEnd, at, 0, 0, 0ull};
      }
      unsigned long long c = 0ull;  // (T is below the largest sum: none that stays at or below it ended)
      int r = 0;
      while (r + 1 < blocks && c + sh.totals[r] <= T) c += sh.totals[r++];
      return Order{kFind, at, levels, r, T - c};
    }
    if (!have_z) {  // back from a sum for a sibling
      Z = sum_of_totals();
      have_z = true;
    }
    for (; next < n; ++next) {
      if (sh.parent[next] != at) continue;
      if (!have_z) return Order{kSum, at, levels, 0, 0ull};
      unsigned long long w = sh.p[next], qz = Z;
      if constexpr (DRAFTS) {
        for (int i = 0; i < levels; ++i) {
          const unsigned long long y = times60(sh.q[next], sh.C[i]);
          w = w > y ? w - y : 0ull;
        }
        qz = times60(sh.q[next], Z);
      } else {
        for (int i = 0; i < levels; ++i)
          if (sh.gone[i] == sh.token[next]) w = 0ull;
      }
      if (times60(qz, sh.u[next]) < w) {
        at = next;
        a.path[(size_t)b * kMostNodes + ++count] = at;
        levels = 0;
        Z = kOne;
      } else if constexpr (DRAFTS) {
        if (levels > 0 && sh.C[levels - 1] + Z < kMostC) sh.C[levels - 1] += Z;
        else sh.C[levels++] = Z;
        have_z = false;
      } else {
        sh.gone[levels++] = sh.token[next];
        Z = Z > w ? Z - w : 0ull;
      }
    }
    drawing = true;
    return Order{kSum, at, levels, 0, 0ull};
  };
  for (;;) {
    if (rank == 0 && threadIdx.x == 0) sh.order = decide();
    cluster.sync();
    const Order o = first->order;
    if (o.kind == kEnd) break;
    // This warp's run of the vocabulary.
    const int runs = blocks * kWarps, run = rank * kWarps + warp;
    const int v0 = (int)((long long)a.vocab * run / runs);
    const int v1 = (int)((long long)a.vocab * (run + 1) / runs);
    const float* p = a.target_probs + (size_t)(n0 + o.node) * a.p_stride;
    const float* q = DRAFTS ? a.draft_probs + (size_t)(n0 + o.node) * a.q_stride : nullptr;
    if (rank != 0 && o.kind == kSum) {  // the levels, into this block's memory
      for (int i = threadIdx.x; i < o.levels; i += kThreads) {
        if constexpr (DRAFTS) sh.C[i] = first->C[i];
        else sh.gone[i] = first->gone[i];
      }
      __syncthreads();
    }
    const bool use_q = DRAFTS && o.levels > 0;
    const unsigned long long c0 = use_q ? sh.C[0] : 0ull;
    if (o.kind == kSum) {
      unsigned long long sum = 0ull;
      bool carries = false;
      auto add = [&](auto form) {
        constexpr int FORM = decltype(form)::value;
        for (int v = v0 + lane; v < v1; v += 32 * kUnroll) {
          float x[kUnroll], y[kUnroll];
#pragma unroll
          for (int k = 0; k < kUnroll; ++k) {
            const int i = v + 32 * k;
            x[k] = i < v1 ? p[i] : 0.f;
            y[k] = DRAFTS && FORM != kPlain && i < v1 ? q[i] : 0.f;
          }
          unsigned long long some = 0ull;
          static_assert(kUnroll <= 8, "weights are below 2^61");
#pragma unroll
          for (int k = 0; k < kUnroll; ++k)
            some += weight<DRAFTS, FORM>(x[k], y[k], v + 32 * k, o.levels, c0, sh.C, sh.gone);
          sum += some;
          carries |= sum < some;
        }
      };
      if (o.levels == 0) {
        add(std::integral_constant<int, kPlain>{});
      } else if constexpr (!DRAFTS) {
        add(std::integral_constant<int, kAny>{});
      } else {
        if (o.levels > 1) add(std::integral_constant<int, kAny>{});
        else if (c0 == kOne) add(std::integral_constant<int, kLess>{});
        else add(std::integral_constant<int, kTerm>{});
      }
      sum = warp_sum60(carries ? kMostSum : min(sum, kMostSum));
      if (lane == 0) sh.warp_sums[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        sum = warp_sum60(lane < kWarps ? sh.warp_sums[lane] : 0ull);
        if (lane == 0) first->totals[rank] = sum;
      }
      cluster.sync();
    } else if (o.kind == kLook) {  // a row without weight: flagged where it holds no numbers
      bool bad = false;
      for (int v = v0 + lane; v < v1; v += 32) bad |= !(p[v] >= 0.f && p[v] < 2.f);
      if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.err_word, kErrProbs);
    } else if (rank == o.rank) {  // kFind: the warp, then the entry
      unsigned long long c = 0ull;
      int w = 0;
      while (w + 1 < kWarps && c + sh.warp_sums[w] <= o.rest) c += sh.warp_sums[w++];
      if (warp == w) {
        const unsigned long long T = o.rest - c;
        unsigned long long base = 0ull;
        bool found = false;
        for (int v = v0; v < v1 && !found; v += 32 * kUnroll) {
          float x[kUnroll], y[kUnroll];
#pragma unroll
          for (int k = 0; k < kUnroll; ++k) {
            const int i = v + lane + 32 * k;
            x[k] = i < v1 ? p[i] : 0.f;
            y[k] = use_q && i < v1 ? q[i] : 0.f;
          }
#pragma unroll
          for (int k = 0; k < kUnroll; ++k) {
            if (found) break;
            const int i = v + lane + 32 * k;
            unsigned long long s =
                weight<DRAFTS, kAny>(x[k], y[k], i, o.levels, c0, sh.C, sh.gone);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const unsigned long long up = __shfl_up_sync(0xffffffffu, s, d);
              if (lane >= d) s += up;
            }
            // (up to the entry looked for sums are below T + 2: nothing wraps)
            const uint32_t over = __ballot_sync(0xffffffffu, base + s > T);
            if (over != 0u) {
              found = true;
              if (lane == 0) a.next_token[b] = v + 32 * k + __ffs(over) - 1;
            } else {
              base += __shfl_sync(0xffffffffu, s, 31);
            }
          }
        }
        // (weights that changed between the two passes)
        if (!found && lane == 0) a.next_token[b] = v1 - 1;
      }
    }
    if (o.kind != kSum) break;
  }
  cluster.sync();  // nobody leaves while its memory may be read
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, const LaunchCtx& ctx) {
  // A cluster of 8 blocks from 8192 entries on: one block / 8, us: 8000 entries, a chain 11.7 / 8.5,
  // 16 trees of 20 nodes 21.0 / 17.8, 64 23 / 32, 200 27 / 39; 4000 entries 9.4 / 8.5, 17.9 / 18.4,
  // 21 / 32, 23 / 38; 16000 17.1 / 8.9, 29 / 18, 37 / 30, 43 / 46; 32000 28 / 9.8, 41 / 17, 52 / 31,
  // 72 / 57.  Sequences differ in how many passes they need
  // (one to four and more), so a batch that the GPU holds at once (two blocks of 512 threads
  // an SM, in clusters) is as fast as its slowest, and that as the SMs it gets to itself; of
  // larger ones more run side by side with blocks of 256.  128257 entries, blocks of 512 / 256
  // threads: 8 trees 26 / 29 us, 64 trees 59 / 59, 200 trees 147 / 118 (clusters of 4 with 512:
  // 36, 68, 132).
  const int blocks = a.vocab >= 8192 ? kMostBlocks : 1;
  const int threads = (long long)a.batch * blocks > 4LL * ctx.num_sms ? 256 : 512;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * (unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto* kernel = threads == 512 ? (a.draft_probs ? verify_kernel<true, 512> : verify_kernel<false, 512>)
                                : (a.draft_probs ? verify_kernel<true, 256> : verify_kernel<false, 256>);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace attn
