// Attention of a tree of drafted tokens over a cache, sm_103a: TMA + cp.async + tcgen05 + TMEM.
//
// A sequence's nodes (its last token and the drafted ones, at most 64) lie in the
// cache behind the kv_len tokens cached before them.  Node i's query sees those
// tokens, and the nodes whose bits are set in its mask word (its ancestors and
// itself):  O = softmax(scale q K^T) V  with the online softmax, over a paged or
// contiguous cache, all nodes and all query heads of a kv head together, so that a
// key or value is read once for up to 256 rows.
//
// What bounds it: HBM for up to about 150 rows a kv head (a tile of 128 tokens at
// head_dim 128 is 64 KB, 1.5 us of an SM's share of the copy rate; a row tile of 128
// rows takes the pipeline 0.85 us), the tensor cores and the exponentials beyond.
// Even a few rows go through 128-row products: they hide behind the copies, and one
// path serves every size.  Measured (bf16 outputs, head_dim 128): 16 sequences of 1024 -
// 32768 tokens in 16-token blocks, 1.12 GB, 203 us, 5.5 TB/s; one of 30720, 63 MB, 35 us (5
// before the first product; the first kernel alone 30); 300 tokens 10 us.
//
// Design:
//   * a row tile holds the g rows of 128 / g nodes (so a tiled copy of queries is one box),
//     an item two row tiles (one at head_dim 256);
//   * persistent blocks, one an SM.  The work of all (sequence, kv head, row group)
//     items is counted in key tiles on the device, from kv_lens and cu_nodes, and
//     every block takes an equal run of them, across items; an item that is cut
//     leaves a normalised partial and its log-sum-exp for each block, which a second
//     kernel joins.  A block starts at most one cut item in its run and ends at most
//     one, so there are two places a block.  Short caches (by max_kv_len) go whole
//     items to a block, without the second kernel;
//   * a producer warp for keys (and queries) and one for values fill a ring of tiles each,
//     128-byte-swizzled as the MMAs read them: runs of rows that all exist, in blocks of
//     whole runs, by tiled copies (TMA); the others, and blocks of any size, by
//     16-byte copies (cp.async) of rows from wherever the block table says, with zeros for
//     what is missing.  Both announce themselves on the slot's barrier; the issuing threads
//     fence what the second kind wrote against the async proxy.  The keys' producer plans
//     the block's run for all the other warps;
//   * S = Q K^T and O += P V by two issuing threads, S in two to four TMEM buffers, P over
//     S, one O a row tile; with two row tiles in an item they take turns, so the
//     tensor cores work on one while the other is in the softmax.  P comes in halves of a tile
//     of 128 keys: the first is multiplied while the second is in the softmax;
//   * the softmax is one row a thread (half a row at head_dim 256), four warps a row tile, 64
//     columns at a time, which stay in registers from the maximum to the exponentials (P
//     overwrites columns that have been read).  A row's first maximum is the reference of its
//     exponentials; it is raised, and O rescaled, only where scores outgrow it by 2^32, so
//     that most tiles have neither a second look at S nor a wait for O;
//   * P is rounded to bf16 for a bf16 O (2^-8 of a weight, no more than O's own
//     rounding), and split into three bf16 parts (2^-24) for an fp32 one.  In random data
//     one part makes a bf16 O's error 2.4e-3 relative instead of the 1.7e-3 of its own
//     rounding.  Two parts would take that away and cost the P V products once more: 16
//     sequences of 1024 - 32768 tokens 268 us against 204, with ALiBi 307 against 237, at
//     head_dim 64 252 against 184, one of 30720 39 against 35;
//   * row statistics, O and the partials are fp32;
//   * every wait is bounded, as in the other kernels.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kSoftmaxThreads = 128;   // a warpgroup's; two of them
constexpr int kProducerThreads = 64;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// How far (log2 units) scores may outgrow the reference of their row's exponentials before
// it is raised and O rescaled: weights up to 2^32, and their sums, are as exact as those
// up to 1 (floating point), and leave O room for values up to 2^60.
constexpr float kRescaleThreshold = 32.0f;
constexpr int kMostNodes = 64;
constexpr int kSegSlots = 4;
constexpr int kMostBox = 64;
constexpr int kLeastBox = 8;

// Row tiles of an item, keys of a tile.  TMEM (512 columns): an O of D columns a row tile,
// and S buffers in what is left: as many columns as keys, or with fp32 outputs 96 for 64 keys
// (three parts of P of 32).  Tiles of 128 keys cost the issuing threads half the waits and
// commits, some 100 clocks each, for a key: 16 sequences of 1024 - 32768 tokens, 32 / 8 heads, at
// head_dim 128: soft-capped 329 us against 403 with 64 and twice the buffers, with ALiBi 266
// against 293; at head_dim 64 184 against 207, soft-capped 284 against 302.  With ALiBi at
// head_dim 64 it is 224 against 240 there, but 100 against 80 for 8 sequences of 100 - 16000
// tokens and 32 heads a kv head, whose many ends cost a whole tile's pass each.
template <int D> __host__ __device__ constexpr int row_tiles() { return D == 256 ? 1 : 2; }
enum Variant : int { kPlain = 0, kCap = 1, kAlibi = 2 };  // (a window is in all of them)
template <int D, int VAR, bool WIDE> __host__ __device__ constexpr int key_tile() {
  return D == 256 || WIDE || (D == 64 && VAR == kAlibi) ? 64 : 128;
}
template <int D, int VAR, bool WIDE> __host__ __device__ constexpr int s_pitch() {
  return WIDE ? 96 : key_tile<D, VAR, WIDE>();
}
template <int D, int VAR, bool WIDE> __host__ __device__ constexpr int s_bufs() {
  return !WIDE && (D == 256 || (D == 64 && VAR == kAlibi)) ? 4 : D == 64 ? 3 : 2;
}
template <int D> __host__ __device__ constexpr int threads_of() {
  return 2 * kSoftmaxThreads + kProducerThreads + 64;
}

template <int D, int VAR, bool WIDE>
struct TreeSmem {
  static constexpr int kBN = key_tile<D, VAR, WIDE>();
  static constexpr int kQTileBytes = 128 * D * 2;
  static constexpr int kTileBytes = kBN * D * 2;
  static constexpr int kQChunkBytes = 128 * 128;  // 128 rows of one 128-byte span
  static constexpr int kChunkBytes = kBN * 128;
  static constexpr int kMaxSlots = 12;
  // barriers: full / empty for each slot, q_empty, s_full[row tile][half][4], p_full[half][4],
  // half_done[4], pv_done[4], o_full[2], drain[2], full / empty for each segment slot, exchange.
  // s_full is a row tile's own: one that sits out an item of fewer rows would otherwise miss
  // phases, and take an old one for its next.
  static constexpr int kNumBars = 2 * kMaxSlots + 1 + 16 + 8 + 4 + 4 + 2 + 2 + 2 * kSegSlots + 1;
  static constexpr int kMiscBytes = 1024;  // barriers, then the segment slots
  // A table of depths a warp; at head_dim 256 what the halves of a row tell each other.
  static constexpr int kDepthTabBytes = 8 * kMostNodes * 4;
  static constexpr int kDepthBytes = kDepthTabBytes + (D == 256 ? 2 * 2 * 128 * 4 : 0);
  // The rings take what the query tiles leave of 226 KB, up to kMaxSlots tiles.
  static constexpr int slots(int q_tiles) {
    const int room = 226 * 1024 - kMiscBytes - kDepthBytes - 1024 - q_tiles * kQTileBytes;
    const int n = room / kTileBytes;
    return n < kMaxSlots ? n : kMaxSlots;
  }
  static constexpr int total(int q_tiles) {
    return q_tiles * kQTileBytes + slots(q_tiles) * kTileBytes + kMiscBytes + kDepthBytes + 1024;
  }
};

struct TreeKParams {
  DecodeTreeArgs a;
  int g;                // query heads of a kv head
  int tile_nodes;       // nodes of a row tile: 128 / g (their g rows each)
  int q_tiles, slots;   // row tiles that an item may have here, ring slots
  int unit_shift;       // a unit of work is 2^unit_shift key tiles
  int blocks_a_tile, rest_a_tile;  // kBN tokens in blocks, and what is left
  int box;              // rows of a tiled copy's box; 0: no tiled copies
  float sl2;            // scale * log2(e)
  float cap_in, cap_l2; // soft-capping: scale / softcap, softcap * log2(e)
  uint32_t* err_word;
  uint64_t timeout_ns;
};

// A sequence as the kernel takes it (bad lengths clamped to nothing).
struct Seq {
  int q0, nodes;  // first packed row, nodes
  int kv_len;     // tokens in front of the nodes
  int end;        // tokens and nodes
  int first;      // first key that some node may see; keys are [first, end)
  int lo;         // where the key tiles begin, at or before `first`
  int tiles;      // key tiles, at least 1
  int groups;     // groups of nodes, an item each
  bool bad_nodes, bad_len;
};

template <int kBN>
__device__ __forceinline__ Seq seq_of(const TreeKParams& p, int b) {
  const DecodeTreeArgs& a = p.a;
  Seq s;
  const int x = a.cu_nodes[b], y = a.cu_nodes[b + 1];
  s.q0 = min(max(x, 0), a.total_nodes);
  const int e = min(max(y, s.q0), a.total_nodes);
  s.nodes = min(e - s.q0, kMostNodes);
  s.bad_nodes = x != s.q0 || y != e || e - s.q0 > kMostNodes || (b == 0 && x != 0);
  const int len = a.kv_lens[b];
  s.bad_len = len < 0 || (long long)len + s.nodes > a.capacity();
  s.kv_len = s.bad_len ? 0 : len;
  s.end = s.bad_len ? 0 : len + s.nodes;
  // Every node's position is kv_len or more: a window starts no earlier than this.
  s.first = a.window_left >= 0 ? max(0, s.kv_len - a.window_left) : 0;
  s.lo = s.first / kMostBox * kMostBox;
  s.tiles = max(1, (s.end - s.lo + kBN - 1) / kBN);
  const int group = p.tile_nodes * p.q_tiles;
  s.groups = (s.nodes + group - 1) / group;
  return s;
}

// Work is counted in units: a run of 2^unit_shift key tiles costs kFullRun, of an item with one
// row tile of two kHalfRun (16 sequences of 1024 - 32768 tokens, 17 - 256 rows a kv head: the
// copies set the pace of one, the products that of two).  A block gets the runs that begin in
// its share of the units, which is kFullRun at least, so that one does in each.  Where items go
// whole, each is a run of cost 1: while there are no more than blocks, each has a block of its
// own (16 sequences of 300 tokens, 8 kv heads, 6 nodes: 12.2 us, 18.2 with the other costs; 64
// sequences 35.0 against 36.1, 300 of 10 - 300 tokens 57 against 60).
constexpr uint32_t kFullRun = 4, kHalfRun = 3;
__device__ __forceinline__ uint32_t full_run(const TreeKParams& p) {
  return p.a.whole ? 1u : kFullRun;
}
__device__ __forceinline__ uint32_t runs_of(const TreeKParams& p, const Seq& s) {
  return p.a.whole ? 1u : (uint32_t)(s.tiles + (1 << p.unit_shift) - 1) >> p.unit_shift;
}
// Cost of a run in the last group of nodes, which may fill one row tile only.
__device__ __forceinline__ uint32_t last_run(const TreeKParams& p, const Seq& s) {
  if (p.a.whole) return 1u;
  const int group = p.tile_nodes * p.q_tiles;
  return p.q_tiles > 1 && s.nodes - (s.groups - 1) * group <= p.tile_nodes ? kHalfRun : kFullRun;
}
__device__ __forceinline__ uint32_t head_units(const TreeKParams& p, const Seq& s) {
  return s.groups > 0 ? runs_of(p, s) * (full_run(p) * (uint32_t)(s.groups - 1) + last_run(p, s)) : 0u;
}
__device__ __forceinline__ uint32_t units_of(const TreeKParams& p, const Seq& s) {
  return (uint32_t)p.a.n_kv_heads * head_units(p, s);
}
// The item that unit `local` of a sequence belongs to: its kv head and group of nodes, its
// runs and their cost, and how many of its units lie in front.
struct Item {
  uint32_t kvh, group, runs, cost, off;
};
__device__ __forceinline__ Item item_at(const TreeKParams& p, const Seq& s, uint32_t local) {
  Item it;
  const uint32_t h = head_units(p, s);
  it.kvh = local / h;
  it.off = local - it.kvh * h;
  it.runs = runs_of(p, s);
  const uint32_t full = it.runs * full_run(p);
  it.group = min(it.off / full, (uint32_t)s.groups - 1u);
  it.off -= it.group * full;
  it.cost = (int)it.group == s.groups - 1 ? last_run(p, s) : full_run(p);
  return it;
}

// A run of key tiles of one item, as the roles get it.
struct alignas(16) Seg {
  int b, kvh, q0, seq_nodes;   // sequence, kv head, its first packed row, its nodes
  int kv_len, end, first, lo;  // as Seq
  int node0, nodes, nr;        // nodes [node0, node0 + nodes) and their row tiles
  int t0, tiles;               // key tiles [t0, t0 + tiles); none: the end
  int place;                   // 0: a partial of an item that began before, 1: of one that begins
                               // here, 2: a whole item
  int full0, full1;            // of those t0 + [full0, full1) consist of keys that all exist
};
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
// The barrier receives this thread's arrival once all its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Rows 16 k .. 16 k + 15 of a tile of 128-byte-swizzled spans, D values each: lane i has the
// place of row i of the 32 around them in units of `pitch` values behind `base`, -1 for zeros.
template <int D, int kBN>
__device__ __forceinline__ void copy_rows(uint32_t tile, int k, const uint16_t* base,
                                          long long pitch, int row, int lane) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // of a row, rows at a time
  constexpr int kPasses = 16 / kRows, kBatch = kPasses < 8 ? kPasses : 8;
  // (all shuffles of a batch in front of its copies, which overlap then)
  const int c = lane % kLanes, r = lane / kLanes;
  const uint32_t dst0 = tile + (c >> 3) * kBN * 128;
  base += c * 8;
#pragma unroll 1
  for (int i = 0; i < kPasses; i += kBatch) {
    int src[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      src[u] = __shfl_sync(0xffffffffu, row, (k & 1) * 16 + (i + u) * kRows + r);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int at = 16 * k + (i + u) * kRows + r;
      cp_async16_or_zero(dst0 + at * 128 + (((c & 7) ^ (at & 7)) << 4),
                         base + max(src[u], 0) * pitch, src[u] >= 0);
    }
  }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// Ties registers that tcgen05.ld filled to the wait in front of it: what reads them stays
// behind.
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}

// N x 32 bytes of a thread to consecutive addresses, a whole sector a store where the
// address allows it (a row a thread: 16-byte stores would fill sectors by halves).
template <int N>
__device__ __forceinline__ void store_32B(void* dst, const uint32_t (&y)[8 * N]) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                       static_cast<char*>(dst) + 32 * k),
                   "r"(y[8 * k]), "r"(y[8 * k + 1]), "r"(y[8 * k + 2]), "r"(y[8 * k + 3]),
                   "r"(y[8 * k + 4]), "r"(y[8 * k + 5]), "r"(y[8 * k + 6]), "r"(y[8 * k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 2 * N; ++k)
      reinterpret_cast<uint4*>(dst)[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
  }
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// softcap tanh(s scale / softcap) of 32 scores, in log2 units.  Up to 0.45 tanh(u) / u is
// 1 - t/3 + 2 t^2/15 - ... in t = u^2 (its Taylor series; the first term left out is
// 1.5e-3 t^7, 2e-8 there), six packed FMAs for two scores; a warp with a larger |u| takes
// tanhf for all of them.  ex2.approx and rcp.approx would be as fast, but their 2e-7 is an
// absolute error of tanh, 1e-5 of a score at softcap 50.
__device__ __forceinline__ void soft_cap(uint32_t (&x)[32], float in, float out) {
  const float2 in2 = make_float2(in, in), out2 = make_float2(out, out);
  auto two = [](float c) { return make_float2(c, c); };
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const float2 u = mul2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), in2);
    const float2 t = mul2(u, u);
    float2 y = fma2(t, two(21844.f / 6081075.f), two(-1382.f / 155925.f));
    y = fma2(t, y, two(62.f / 2835.f));
    y = fma2(t, y, two(-17.f / 315.f));
    y = fma2(t, y, two(2.f / 15.f));
    y = fma2(t, y, two(-1.f / 3.f));
    const float2 v = mul2(u, out2);
    y = fma2(mul2(t, y), v, v);
    x[k] = __float_as_uint(y.x);
    x[k + 1] = __float_as_uint(y.y);
  }
}
__device__ __forceinline__ bool small_for_cap(const uint32_t (&x)[32], float in) {
  float top[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 32; k += 4)
#pragma unroll
    for (int q = 0; q < 2; ++q)
      top[q] = fmax3(top[q], fabsf(__uint_as_float(x[k + 2 * q])), fabsf(__uint_as_float(x[k + 2 * q + 1])));
  return !(fmaxf(top[0], top[1]) * in > 0.45f);
}
// The same where a warp's scores lie in TMEM, for any |u| (NaN too): a short loop, because 32
// copies of tanhf in a tile's way cost every tile the fetch around them.
__device__ __forceinline__ void soft_cap_large(uint32_t at, int cols, float in, float out) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 8) {
    uint32_t y[8];
    tmem_ld8(at + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(out * tanhf(__uint_as_float(y[k]) * in));
    tmem_st8(at + c, y);
  }
  tmem_wait_st();
}

// Whether 32 scores in TMEM are that small, without those whose bits in w are clear: what masked
// columns hold must not decide how the others are computed.  A short loop too: with the masks
// written out over the 32 registers, 16 sequences of 1024 - 32768 tokens take 345 us, not 314.
__device__ __forceinline__ bool small_where(uint32_t at, uint32_t w, float in) {
  float top = 0.f;
#pragma unroll 1
  for (int c = 0; c < 32; c += 8, w >>= 8) {
    uint32_t y[8];
    tmem_ld8(at + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if ((w >> k) & 1u) top = fmaxf(top, fabsf(__uint_as_float(y[k])));
  }
  return !(top * in > 0.45f);
}

// VAR: what happens to a score besides scale and window.  WIDE: fp32 O, P in three parts.
template <int D, int VAR, bool WIDE>
__global__ void __launch_bounds__(threads_of<D>(), 1) decode_tree_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
    const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ TreeKParams p) {
  using L = TreeSmem<D, VAR, WIDE>;
  constexpr int kBN = L::kBN, kPitch = s_pitch<D, VAR, WIDE>(), SB = s_bufs<D, VAR, WIDE>(), NQ = row_tiles<D>();
  // Keys of an S product.  An issuing thread pays some 59 clocks an MMA and 100 a wait or commit,
  // whatever the MMA's size, so a whole tile at once is cheaper for it (16 sequences of 1024 -
  // 32768 tokens, 32 / 8 heads: 205 us against 228 with halves, with ALiBi 238 against 265); with
  // soft-capping the softmax takes long, and starts sooner with halves (311 against 329 when
  // both wait for all of the last P).
  constexpr int kSKeys = VAR == kCap ? 64 : kBN;
  constexpr bool kSplit = NQ == 1;  // both warpgroups work on the one row tile
  constexpr int kProducerWarp = 8, kSWarp = kProducerWarp + 2, kPVWarp = kSWarp + 1;
  static_assert(SB * kPitch + NQ * D <= (int)kTmemCols, "TMEM budget");
  const DecodeTreeArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = p.slots, k_slots = (slots + 1) / 2;  // (the keys' slots are the first ones)
  uint8_t* ring = smem + p.q_tiles * L::kQTileBytes;
  uint8_t* misc = ring + slots * L::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  constexpr int kFull = 0, kEmpty = L::kMaxSlots, kQEmpty = 2 * L::kMaxSlots, kSFull = kQEmpty + 1,
                kPFull = kSFull + 16, kHalfDone = kPFull + 8, kPVDone = kHalfDone + 4, kOFull = kPVDone + 4,
                kDrain = kOFull + 2, kSegFull = kDrain + 2, kSegEmpty = kSegFull + kSegSlots,
                kExchange = kSegEmpty + kSegSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + L::kNumBars * 8);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(tmem_slot + 1);
  constexpr int kSegOffset = (L::kNumBars * 8 + 16 + 15) / 16 * 16;
  Seg* segs = reinterpret_cast<Seg*>(misc + kSegOffset);
  static_assert(kSegOffset + kSegSlots * sizeof(Seg) <= L::kMiscBytes, "misc");
  int* depth_tab = reinterpret_cast<int*>(misc + L::kMiscBytes);

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < slots; ++i) {
      mbar_init(bar(kFull + i), 32);
      mbar_init(bar(kEmpty + i), 1);
    }
    mbar_init(bar(kQEmpty), 1);
    for (int i = 0; i < SB; ++i) {
      for (int j = 0; j < 16; j += 4) mbar_init(bar(kSFull + j + i), 1);
      mbar_init(bar(kHalfDone + i), 1);
      mbar_init(bar(kPFull + i), kSplit ? 2 * kSoftmaxThreads : kSoftmaxThreads);
      mbar_init(bar(kPFull + 4 + i), kSoftmaxThreads);
      mbar_init(bar(kPVDone + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kOFull + i), 1);
      mbar_init(bar(kDrain + i), 1);
    }
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(bar(kSegFull + i), 1);
      mbar_init(bar(kSegEmpty + i), 3 + kProducerWarp);  // the values' producer, two issuers, softmax warps
    }
    mbar_init(bar(kExchange), 2 * kSoftmaxThreads);
    fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tmap(&tm_q);
    if (p.box > 0) {
      prefetch_tmap(&tm_k);
      if (p.box >= 16) prefetch_tmap(&tm_v);
    }
  }
  if (warp == kSWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem + SB * kPitch;
  const WaitCtl ctl{abort_flag, p.err_word, p.timeout_ns};
  const int g = p.g;

  // First key of the t-th tile that a segment visits.  ALiBi's bias grows toward the nodes:
  // in order the maxima would rise, and O be rescaled, tile after tile, so it goes backwards.
  auto first_key = [&](const Seg& sg, int t) {
    return sg.lo + (sg.t0 + (VAR == kAlibi ? sg.tiles - 1 - t : t)) * kBN;
  };
  // Whether all keys of a tile exist (tiled copies fill it then, where blocks allow them).
  auto full_tile = [&](const Seg& sg, int t) {
    const int j = VAR == kAlibi ? sg.tiles - 1 - t : t;
    return j >= sg.full0 && j < sg.full1;
  };
  // The steps of 16 keys of a tile that hold keys at all: what the products take, and the
  // producers fill.
  auto steps_of = [&](const Seg& sg, int t, int& k0, int& k1) {
    const int tile0 = first_key(sg, t);
    k0 = max(sg.first - tile0, 0) >> 4;
    k1 = max((min(sg.end - tile0, kBN) + 15) >> 4, k0);
  };
  // The keys' producer plans the segments; the other roles take them from its slots, in order
  // (`all`: by a whole warp).  S products count over all of them (n: buffer n % SB), and so
  // do the tiles of keys and of values, each in slots of their own: a slot's releases all come
  // from one issuer, in order, so that a producer that has waited for one release knows of all
  // before it.  In one ring of an odd number of slots, keys and values would take turns in each,
  // and with 5 slots the values' producer could take a release by the S issuer for the one that
  // the P V issuer still owed (phases are told apart by their parity alone).
  auto take = [&](Seg& sg, int& count, bool all) -> bool {
    const int i = count % kSegSlots;
    const uint32_t parity = (count / kSegSlots) & 1;
    ++count;
    if (!(all ? mbar_wait_warp(bar(kSegFull + i), parity, ctl) : mbar_wait(bar(kSegFull + i), parity, ctl)))
      return false;
    sg = segs[i];
    if (all) __syncwarp();
    if (lane == 0) mbar_arrive(bar(kSegEmpty + i));
    return sg.tiles > 0;
  };
  const uint32_t id_s = idesc_bf16_f32(128, kSKeys, false, false);
  const uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
  const uint32_t dhi = sw128_desc_hi(1024);

  if (warp >= kProducerWarp && warp < kSWarp) {
    // ============================ producers ============================
    // The first warp fills the keys' slots (and the queries), the second the values'.
    const bool keys = warp == kProducerWarp;
    const CUtensorMap* map = keys ? &tm_k : &tm_v;
    const CUtensorMap* map16 = keys ? &tm_k16 : &tm_v16;
    const uint16_t* cache = keys ? a.k_cache : a.v_cache;
    constexpr int kSpans = D / 64, kSets = kBN / 32;
    const int box = lane / kSpans, span = lane % kSpans;
    // Boxes of 8 rows for keys alone (see the launch).
    const bool tiled = p.box >= 16 || (p.box > 0 && keys);
    const bool mine = tiled && box * p.box < kBN;
    const int slot0 = keys ? 0 : k_slots, slot1 = keys ? k_slots : slots;
    int slot = slot0, phase = 0, n_seg = 0, issued = 0;
    bool again = false;                                    // slots have been used before
    Seg sg;
    int count = 0;
    // ---- the plan: this block's run of units, [u, u1) of all, from sequence b on ----
    uint32_t u = 0, u1 = 0, base = 0;
    int b = 0;
    Seq s{};
    if (keys) {
      bool bad_nodes = false, bad_len = false;
      uint32_t total = 0;
#pragma unroll 4
      for (int i = lane; i < a.batch; i += 32) {
        const Seq x = seq_of<kBN>(p, i);
        total += units_of(p, x);
        bad_nodes |= x.bad_nodes;
        bad_len |= x.bad_len;
      }
      if (blockIdx.x == 0) {
        if (bad_nodes) atomicOr(p.err_word, kErrSeqLens);
        if (bad_len) atomicOr(p.err_word, kErrKvLen);
      }
      total = __reduce_add_sync(0xffffffffu, total);
      // The first `more` blocks get one unit more than the others; blocks beyond the units get
      // none, so that those with some are neighbours.
      const uint32_t G = total ? min(gridDim.x, max(total / full_run(p), 1u)) : 0u, c = blockIdx.x;
      const uint32_t each = G ? total / G : 0, more = G ? total - each * G : 0;
      if (c < G) {
        u = c * each + min(c, more);
        u1 = u + each + (c < more ? 1 : 0);
        for (int i0 = 0; i0 < a.batch; i0 += 32) {
          uint32_t n = 0;
          if (i0 + lane < a.batch) n = units_of(p, seq_of<kBN>(p, i0 + lane));
          uint32_t incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, u < base + incl);
          if (past) {
            const int at = __ffs(past) - 1;
            base += __shfl_sync(0xffffffffu, incl - n, at);
            b = i0 + at;
            break;
          }
          base += __shfl_sync(0xffffffffu, incl, 31);
        }
        s = seq_of<kBN>(p, b);
      }
      if (!a.whole && lane == 0) {
        // What the second kernel joins: an item that ends here and began in another block.
        TreeJoin j{-1, 0, 0, 0, 0, 0, 0, 0};
        if (u < u1) {
          const Item it = item_at(p, s, u - base);
          const uint32_t at = u - it.off, last = at + (it.runs - 1) * it.cost;
          if (it.off > 0 && last >= u && last < u1) {
            const uint32_t rich = more * (each + 1);
            j.first_block = (int)(at < rich ? at / (each + 1) : more + (at - rich) / each);
            j.kvh = (int)it.kvh;
            const int node0 = (int)it.group * p.tile_nodes * p.q_tiles;
            j.rows = min(p.tile_nodes * p.q_tiles, s.nodes - node0) * g;
            j.q0 = s.q0;
            j.row0 = node0 * g;
          }
        }
        a.joins[blockIdx.x] = j;
      }
    }
    auto plan = [&]() -> bool {
      sg.tiles = 0;
      while (u < u1) {
        uint32_t n = units_of(p, s);
        while (u >= base + n && b + 1 < a.batch) {
          base += n;
          s = seq_of<kBN>(p, ++b);
          n = units_of(p, s);
        }
        if (u >= base + n) break;  // (lengths that changed under the call)
        const Item it = item_at(p, s, u - base);
        const uint32_t n_units = min(it.runs * it.cost - it.off, u1 - u);
        const uint32_t t = (it.off + it.cost - 1) / it.cost;
        const uint32_t t_end = min((it.off + n_units + it.cost - 1) / it.cost, it.runs);
        u += n_units;
        if (t >= t_end) continue;  // (no run begins here)
        const int group = p.tile_nodes * p.q_tiles;
        sg.b = b, sg.q0 = s.q0, sg.seq_nodes = s.nodes;
        sg.kv_len = s.kv_len, sg.end = s.end, sg.first = s.first, sg.lo = s.lo;
        sg.kvh = (int)it.kvh;
        sg.node0 = (int)it.group * group;
        sg.nodes = min(group, s.nodes - sg.node0);
        sg.nr = (sg.nodes + p.tile_nodes - 1) / p.tile_nodes;
        sg.t0 = a.whole ? 0 : (int)(t << p.unit_shift);
        sg.tiles = a.whole ? s.tiles : min((int)((t_end - t) << p.unit_shift), s.tiles - sg.t0);
        sg.place = t > 0 ? 0 : t_end < it.runs ? 1 : 2;
        const int key0 = s.lo + sg.t0 * kBN;
        sg.full0 = key0 < s.first ? 1 : 0;
        sg.full1 = min(max(s.end - key0, 0) / kBN, sg.tiles);
        break;
      }
      const int i = count % kSegSlots;
      if (count >= kSegSlots &&
          !mbar_wait_warp(bar(kSegEmpty + i), (count / kSegSlots - 1) & 1, ctl))
        return false;
      ++count;
      if (lane == 0) {
        segs[i] = sg;
        mbar_arrive(bar(kSegFull + i));
      }
      __syncwarp();
      return sg.tiles > 0;
    };
    bool ok = true;
    while (ok && (keys ? plan() : take(sg, count, true))) {
      const int32_t* table =
          a.block_table ? a.block_table + (size_t)sg.b * a.max_blocks_per_seq : nullptr;
      // Tiled copies of a whole tile: a box and span a lane.  Its block's number in the table,
      // the row in it, and what the table says, which is read a tile ahead.
      int blk = 0, row_in = first_key(sg, 0) + box * p.box, entry = sg.b;
      if (table != nullptr) {
        blk = row_in / a.block_size;
        row_in -= blk * a.block_size;
      }
      auto look = [&](int t) {
        if (table != nullptr && mine && t < sg.tiles && full_tile(sg, t)) entry = table[blk];
      };
      look(0);
      for (int t = 0; t < sg.tiles && ok; ++t) {
        const int tile0 = first_key(sg, t);
        const uint32_t dst = smem_u32(ring + slot * L::kTileBytes), full = bar(kFull + slot);
        // (every lane waits: a warp that one lane kept waiting copies rows ten times slower)
        if (again && !mbar_wait_warp(bar(kEmpty + slot), phase ^ 1, ctl)) { ok = false; break; }
        const bool q_too = keys && t == 0;
        // The last segment's S products have to be through with Q.
        if (q_too && n_seg > 0 && !mbar_wait_warp(bar(kQEmpty), (n_seg - 1) & 1, ctl)) {
          ok = false;
          break;
        }
        if (lane == 0 && q_too) {
          // Queries: tile_nodes nodes' g rows a row tile (rows past the nodes are not used).
          mbar_expect_tx(full, (uint32_t)(sg.nr * p.tile_nodes * g) * D * 2);
          for (int r = 0; r < sg.nr; ++r)
            for (int i = 0; i < kSpans; ++i)
              tma_load_3d(smem_u32(smem + r * L::kQTileBytes + i * L::kQChunkBytes), &tm_q, full,
                          i * 64, sg.kvh * g, sg.q0 + sg.node0 + r * p.tile_nodes);
        }
        if (tiled && full_tile(sg, t)) {
          int plane = entry;
          if (table != nullptr && mine && (plane < 0 || plane >= a.num_blocks)) {
            // A bad block becomes one past the cache, which reads as zeros.
            atomicOr(p.err_word, kErrBlockIndex);
            plane = a.num_blocks;
          }
          if (lane == 0) mbar_expect_tx(full, kBN * D * 2);
          __syncwarp();
          // Every lane its own: with one lane that issues them all, 16 paged sequences of up to
          // 32768 tokens take 315 us instead of 228.
          if (mine)
            tma_load_4d(dst + span * L::kChunkBytes + box * p.box * 128, map, full, span * 64, sg.kvh,
                        row_in, plane);
          if (lane == 0) mbar_arrive_n(full, 32);
        } else {
          // A tile that ends early or begins in front of a window, or blocks of other sizes: steps
          // of 16 rows.  Those that are all there by a tiled copy where blocks allow it, the
          // others row by row, 16 bytes a lane, zeros for rows that are not there (the products
          // multiply them by weights of 0).
          int k0, k1;
          steps_of(sg, t, k0, k1);
          auto whole = [&](int k) {
            return p.box >= 16 && tile0 + 16 * k >= sg.first && tile0 + 16 * k + 16 <= sg.end;
          };
          auto find = [&](int tok, int& in) {  // the plane of a token's row, -1 for a bad block
            in = tok;
            if (table == nullptr) return sg.b;
            const int j = tok / a.block_size, x = table[j];
            in = tok - j * a.block_size;
            if (x >= 0 && x < a.num_blocks) return x;
            atomicOr(p.err_word, kErrBlockIndex);
            return -1;
          };
          int n_boxes = 0;
          for (int k = k0; k < k1; ++k) n_boxes += whole(k);
          if (n_boxes > 0) {
            if (lane == 0) mbar_expect_tx(full, (uint32_t)(n_boxes * 16 * D * 2));
            __syncwarp();
            if (box >= k0 && box < k1 && whole(box)) {
              int in;
              const int plane = find(tile0 + 16 * box, in);
              tma_load_4d(dst + span * L::kChunkBytes + box * 16 * 128, map16, full, span * 64, sg.kvh,
                          in, plane < 0 ? a.num_blocks : plane);
            }
            __syncwarp();
          }
          if (n_boxes < k1 - k0) {
            // The places of rows lane, lane + 32, ..
            const int rows = table ? a.block_size : a.max_kv_len;
            int row[kSets];
#pragma unroll
            for (int i = 0; i < kSets; ++i) {
              const int tok = tile0 + lane + 32 * i;
              row[i] = -1;
              if (tok >= sg.first && tok < sg.end && !whole(2 * i + (lane >> 4))) {
                int in;
                const int plane = find(tok, in);
                if (plane >= 0) row[i] = plane * rows + in;
              }
            }
            __syncwarp();
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
              if (whole(k)) continue;
              int r = row[0];
#pragma unroll
              for (int i = 1; i < kSets; ++i)
                if ((k >> 1) == i) r = row[i];
              copy_rows<D, kBN>(dst, k, cache + (size_t)sg.kvh * D, (long long)a.n_kv_heads * D, r,
                                lane);
            }
          }
          cp_async_arrive(full);
        }
        ++issued;
        // The next tile of the walk.
        if (table == nullptr) {
          row_in += VAR == kAlibi ? -kBN : kBN;
        } else if (VAR == kAlibi) {
          blk -= p.blocks_a_tile;
          row_in -= p.rest_a_tile;
          if (row_in < 0) row_in += a.block_size, --blk;
        } else {
          blk += p.blocks_a_tile;
          row_in += p.rest_a_tile;
          if (row_in >= a.block_size) row_in -= a.block_size, ++blk;
        }
        look(t + 1);
        if (++slot == slot1) slot = slot0, phase ^= 1, again = true;
      }
      ++n_seg;
    }
    cp_async_commit();
    cp_async_wait<0>();
    if (*abort_flag && lane == 0) {
      // Tiled copies in flight land before the block's memory is released.
      volatile uint32_t no_abort = 0u;
      WaitCtl drain{&no_abort, p.err_word, p.timeout_ns};
      const int n = slot1 - slot0;
      for (int i = max(0, issued - n); i < issued; ++i)
        mbar_wait(bar(kFull + slot0 + i % n), (i / n) & 1, drain);
    }
    __syncwarp();
  } else if (warp == kSWarp) {
    // ============================ S = Q K^T issuer ============================
    if (lane == 0) {
      Seg sg;
      int count = 0;
      bool ok = true;
      int n = 0, slot = 0, phase = 0;
      const uint32_t q_lo0 = sw128_desc_lo(smem_u32(smem), 16);
      while (ok && take(sg, count, false)) {
        for (int t = 0; t < sg.tiles && ok; ++t) {
          if (!mbar_wait(bar(kFull + slot), phase, ctl)) { ok = false; break; }
          // The 16-byte copies' writes, before the MMAs that read them.
          const bool full = full_tile(sg, t);
          int k0, k1 = kBN / 16;
          if (!full || p.box == 0) fence_proxy_async_smem();
          if (!full) steps_of(sg, t, k0, k1);
          const uint32_t k_lo = sw128_desc_lo(smem_u32(ring + slot * L::kTileBytes), 16);
          for (int r = 0; r < sg.nr; ++r, ++n) {
            const int b = n % SB;
            const uint32_t dS = tmem + b * kPitch;
            const uint32_t q_lo = q_lo0 + (uint32_t)((r * L::kQTileBytes) >> 4);
#pragma unroll 1
            for (int h = 0; h < kBN / kSKeys; ++h) {
              // Buffer b last held P(n - SB), whose halves are done one after the other.
              const uint32_t held = bar((kSKeys < kBN && h == 0 ? kHalfDone : kPVDone) + b);
              if (n >= SB && !mbar_wait(held, (n / SB - 1) & 1, ctl)) { ok = false; break; }
              tc_fence_after();
              const int keys = full ? kSKeys : min(16 * k1 - kSKeys * h, kSKeys);
              const uint32_t id = full ? id_s : idesc_bf16_f32(128, max(keys, 16), false, false);
              if (keys > 0) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint32_t qoff = ((kk >> 2) * L::kQChunkBytes + (kk & 3) * 32) >> 4;
                  const uint32_t koff = ((kk >> 2) * L::kChunkBytes + (kk & 3) * 32) >> 4;
                  mma_ss_lo(dS + 64 * h, q_lo + qoff, k_lo + 512 * h + koff, dhi, id, kk > 0);
                }
              }
              mma_commit(bar(kSFull + 8 * r + 4 * h + b));
            }
            if (!ok) break;
          }
          mma_commit(bar(kEmpty + slot));
          if (++slot == k_slots) slot = 0, phase ^= 1;
        }
        mma_commit(bar(kQEmpty));
      }
      mma_commit(bar(kDrain));
      volatile uint32_t no_abort = 0u;
      WaitCtl drain{&no_abort, p.err_word, p.timeout_ns};
      mbar_wait(bar(kDrain), 0, drain);
    }
    __syncwarp();
  } else if (warp == kPVWarp) {
    // ============================ O += P V issuer ============================
    if (lane == 0) {
      Seg sg;
      int count = 0;
      bool ok = true;
      int n = 0, slot = k_slots, phase = 0;
      while (ok && take(sg, count, false)) {
        for (int t = 0; t < sg.tiles && ok; ++t) {
          if (!mbar_wait(bar(kFull + slot), phase, ctl)) { ok = false; break; }
          // The 16-byte copies' writes, before the MMAs that read them.
          const bool full = full_tile(sg, t);
          int k0 = 0, k1 = kBN / 16;
          if (!full || p.box < 16) fence_proxy_async_smem();
          if (!full) steps_of(sg, t, k0, k1);
          const uint32_t v_lo =
              sw128_desc_lo(smem_u32(ring + slot * L::kTileBytes), D > 64 ? L::kChunkBytes : 16);
          for (int r = 0; r < sg.nr; ++r, ++n) {
            const int b = n % SB;
            // P comes in halves of 64 keys.
            const uint32_t aP = tmem + b * kPitch, tOr = tO + r * D;
            uint32_t onto = t > 0 ? 1u : 0u;  // (the first product of a segment overwrites O)
#pragma unroll 1
            for (int h = 0; h < kBN / 64; ++h) {
              if (!mbar_wait(bar(kPFull + 4 * h + b), (n / SB) & 1, ctl)) { ok = false; break; }
              tc_fence_after();
              const uint32_t aH = aP + 64 * h, v_h = v_lo + 512 * h;
              auto product = [&](int part, int kk) {
                mma_ts_lo(tOr, aH + part * 32 + kk * 8, v_h + ((kk * 16 * 128) >> 4), dhi, id_pv, onto);
                onto = 1u;
              };
              if (full) {  // (straight code: each branch between MMAs shows)
#pragma unroll
                for (int part = 0; part < (WIDE ? 3 : 1); ++part)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) product(part, kk);
              } else {
#pragma unroll 1
                for (int kk = max(k0 - 4 * h, 0); kk < min(k1 - 4 * h, 4); ++kk)
                  for (int part = 0; part < (WIDE ? 3 : 1); ++part) product(part, kk);
              }
              if (kBN > 64 && h == 0) mma_commit(bar(kHalfDone + b));
            }
            if (!ok) break;
            mma_commit(bar(kPVDone + b));
            if (t == sg.tiles - 1) mma_commit(bar(kOFull + r));
          }
          mma_commit(bar(kEmpty + slot));
          if (++slot == slots) slot = k_slots, phase ^= 1;
        }
      }
      mma_commit(bar(kDrain + 1));
      volatile uint32_t no_abort = 0u;
      WaitCtl drain{&no_abort, p.err_word, p.timeout_ns};
      mbar_wait(bar(kDrain + 1), 0, drain);
    }
    __syncwarp();
  } else if (warp < kProducerWarp) {
    // ============================ softmax, epilogue ============================
    // A warpgroup a row tile; at head_dim 256 both on the one, 32 of a tile's 64 keys each,
    // with one reference for a row, and half of O's columns each in the end: 4 sequences of
    // 2000 - 9000 tokens, a window of 4096, soft-capping and fp32 outputs 58 us, 70 with one.
    const int r = kSplit ? 0 : warp >> 2;                   // row tile
    const int part = kSplit ? warp >> 2 : 0;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int trow = (warp & 3) * 32 + lane;                // row within the tile (TMEM lane)
    int* depths = depth_tab + warp * kMostNodes;            // the nodes' depths, each warp its own
    Seg sg;
    int count = 0;
    bool ok = true;
    int n0 = 0, n_seg = 0;  // S products before the segment, segments of this row tile
    uint32_t exchanges = 0;
    float* told = reinterpret_cast<float*>(depth_tab + L::kDepthTabBytes / 4);
    // What the other half of the row says (the lower half's value first).
    auto exchange = [&](float mine, float (&both)[2]) -> bool {
      float* at = told + (exchanges & 1) * 256 + trow;
      at[part * 128] = mine;
      tc_fence_before();
      mbar_arrive(bar(kExchange));
      if (!mbar_wait_warp(bar(kExchange), exchanges & 1, ctl)) return false;
      ++exchanges;
      tc_fence_after();
      both[0] = at[0], both[1] = at[128];
      return true;
    };
    uint32_t s_phase = 0;   // s_full's phases, a bit for each half and buffer
    for (; ok && take(sg, count, true); n0 += sg.tiles * sg.nr) {
      if (r >= sg.nr) continue;
      const int in_tile = trow / g;                         // this row's node in the row tile
      const int node = sg.node0 + r * p.tile_nodes + in_tile;
      const int head = sg.kvh * g + (trow - in_tile * g);
      const bool real = in_tile < p.tile_nodes && node < sg.node0 + sg.nodes;
      const int i = (r * p.tile_nodes + in_tile) * g + (trow - in_tile * g);  // row of the group
      // The nodes this row sees.
      const unsigned long long all =
          sg.seq_nodes >= 64 ? ~0ull : (1ull << sg.seq_nodes) - 1ull;
      auto word_of = [&](int u) {
        const unsigned long long w = a.tree_mask
                                         ? (unsigned long long)a.tree_mask[sg.q0 + u]
                                         : (2ull << u) - 1ull;
        return w & all;
      };
      unsigned long long word = real ? word_of(node) : 0ull;
      if (sg.end == 0) word = 0ull;                       // a length that was refused
      const int depth = max(__popcll(word) - 1, 0);
      float slope_l2 = 0.f;
      const bool near = a.window_left >= 0 && a.window_left < kMostNodes;
      if (near || VAR == kAlibi) {
        __syncwarp();                                       // the last segment's readers
        for (int u = lane; u < sg.seq_nodes; u += 32) depths[u] = max(__popcll(word_of(u)) - 1, 0);
        __syncwarp();
        if (near)
          for (int u = 0; u < sg.seq_nodes; ++u)
            if (depth - depths[u] > a.window_left) word &= ~(1ull << u);
      }
      if (VAR == kAlibi && real) slope_l2 = a.alibi_slopes[head] * kLog2e;
      const int pos = sg.kv_len + depth;
      // Rows of no node hold what the queries' tile held before, or other sequences' queries:
      // nothing in them may decide how the other rows of their warp are computed.
      const float vote = real ? p.cap_in : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < sg.tiles; ++t) {
        const int n = n0 + t * sg.nr + r, b = n % SB;
        const int kv0 = first_key(sg, t);
        // Visible columns, a bit each, where some may not be.
        const bool edge = kv0 + kBN > sg.kv_len ||
                          (a.window_left >= 0 && kv0 < sg.kv_len + kMostNodes - a.window_left);
        uint32_t vis[kBN / 32];
        if (edge) {
          const int sft = sg.kv_len - kv0;                // column of node 0
          const int lo_c =
              a.window_left >= 0 ? min(pos - a.window_left, sg.kv_len) - kv0 : 0;
#pragma unroll
          for (int c = 0; c < kBN / 32; ++c) {
            const int s = sft - 32 * c;
            uint32_t w = s >= 32 ? 0xffffffffu : s > 0 ? (1u << s) - 1u : 0u;
            if (s < 32) w |= s >= 0 ? (uint32_t)(word << s) : s > -64 ? (uint32_t)(word >> -s) : 0u;
            const int q = lo_c - 32 * c;
            if (q > 0) w &= q >= 32 ? 0u : ~((1u << q) - 1u);
            vis[c] = w;
          }
        }
        const uint32_t tS = tmem + b * kPitch + lane_base;
        auto wait_s = [&](int h) {
          if (h >= kBN / kSKeys) return true;               // (it came with the first half)
          const int i = 4 * h + b;
          if (!mbar_wait_warp(bar(kSFull + 8 * r + i), (s_phase >> i) & 1u, ctl)) return false;
          s_phase ^= 1u << i;
          tc_fence_after();
          return true;
        };
        if (edge) {
          // Soft-capping, masks, and ALiBi where nodes are among the keys: a pass of its own,
          // written back.
          for (int h = 0; h < kBN / 64 && ok; ++h) ok = wait_s(h);
          if (!ok) break;
#pragma unroll 1
          for (int c = kSplit ? part : 0; c < (kSplit ? part + 1 : kBN / 32); ++c) {
            uint32_t w = vis[0];
#pragma unroll
            for (int q = 1; q < kBN / 32; ++q)
              if (c == q) w = vis[q];
            uint32_t y[32];
            tmem_ld32(tS + c * 32, y);
            tmem_wait_ld();
            landed(y);
            if constexpr (VAR == kCap) {
              if (__all_sync(0xffffffffu, small_where(tS + c * 32, w, vote))) {
                soft_cap(y, p.cap_in, p.cap_l2);
              } else {
                soft_cap_large(tS + c * 32, 32, p.cap_in, p.cap_l2);
                tmem_ld32(tS + c * 32, y);
                tmem_wait_ld();
                landed(y);
              }
            }
            if constexpr (VAR == kAlibi) {
              const float d0 = (float)(pos - kv0 - 32 * c);
              const int u0 = kv0 + 32 * c - sg.kv_len;      // node of the first column
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float dist = u0 + k < 0
                                       ? d0 - (float)k
                                       : (float)(depth - depths[min(u0 + k, kMostNodes - 1)]);
                y[k] = __float_as_uint(fmaf(__uint_as_float(y[k]), p.sl2, -slope_l2 * dist));
              }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((w >> k) & 1u)) y[k] = 0xff800000u;     // -inf
            tmem_st32(tS + c * 32, y);
          }
          tmem_wait_st();
        }
        // 64 keys at a time, whose scores stay in registers (one copy of the code for all: it
        // is fetched anew for every tile, beside five other roles').
#pragma unroll 1
        for (int h = 0; h < kBN / 64; ++h) {
          if (!edge && !wait_s(h)) { ok = false; break; }
          const uint32_t tH = tS + 64 * h + 32 * part;
          // What turns the score of column k into log2 units: x sl2 + (base + slope k).
          float sl2 = VAR == kCap ? 1.f : p.sl2, slope = 0.f, base = 0.f;
          if constexpr (VAR == kAlibi) {
            slope = slope_l2;
            base = -slope_l2 * (float)(pos - kv0 - 64 * h - 32 * part);
            if (edge) sl2 = 1.f, slope = 0.f, base = 0.f;
          }
          constexpr int kSets = kSplit ? 1 : 2;
          uint32_t x[kSets][32];
          auto load = [&]() {
#pragma unroll
            for (int c = 0; c < kSets; ++c) tmem_ld32(tH + 32 * c, x[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kSets; ++c) landed(x[c]);
          };
          load();
          if (VAR == kCap && !edge) {
            const bool small = small_for_cap(x[0], vote) && small_for_cap(x[kSets - 1], vote);
            if (__all_sync(0xffffffffu, small)) {
#pragma unroll
              for (int c = 0; c < kSets; ++c) soft_cap(x[c], p.cap_in, p.cap_l2);
            } else {
              soft_cap_large(tH, 32 * kSets, p.cap_in, p.cap_l2);
              load();
            }
          }
          // ---- the row's maximum ----
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < kSets; ++c) {
            uint32_t (&y)[32] = x[c];
            if constexpr (VAR == kAlibi) {
              float2 steps[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                steps[q] = make_float2(slope * (float)(2 * q), slope * (float)(2 * q + 1));
              const float2 sl2v = make_float2(sl2, sl2);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                // slope k is that of the 8 columns' first and one of four pairs.
                const float b8 = fmaf(slope, (float)(32 * c + (k & ~7)), base);
                const float2 e = fma2(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])),
                                      sl2v, add2(make_float2(b8, b8), steps[(k >> 1) & 3]));
                y[k] = __float_as_uint(e.x);
                y[k + 1] = __float_as_uint(e.y);
              }
            }
            float mc[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mc[q] = fmaxf(__uint_as_float(y[q]), __uint_as_float(y[q + 4]));
#pragma unroll
            for (int k = 8; k < 32; k += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mc[q] = fmax3(mc[q], __uint_as_float(y[k + q]), __uint_as_float(y[k + q + 4]));
            mx = fmax3(mx, fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
          }
          if constexpr (VAR != kAlibi) mx *= sl2;
          if (!real) mx = -INFINITY;                        // (no vote on the reference)
          if constexpr (kSplit) {
            // (both have read their scores then, which P overwrites)
            float both[2];
            if (!exchange(mx, both)) { ok = false; break; }
            mx = fmaxf(both[0], both[1]);
          }
          // ---- the reference: the first maximum that a row sees; raised only when some row of
          // the warp has outgrown it ----
          if (m == -INFINITY) m = mx;                       // (O and l are 0)
          if (__any_sync(0xffffffffu, mx - m > kRescaleThreshold)) {
            const float m_new = fmaxf(m, mx);
            const float corr = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);
            m = m_new;
            l *= corr;
            if (t > 0 || h > 0) {
              // O has to hold this row tile's products so far: the tile before's, or this one's
              // first half.
              const int pn = n - sg.nr;
              if (!(h > 0 ? mbar_wait_warp(bar(kHalfDone + b), (n / SB) & 1, ctl)
                          : mbar_wait_warp(bar(kPVDone + pn % SB), (pn / SB) & 1, ctl))) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = part * (D / 16); c < (kSplit ? (part + 1) * (D / 16) : D / 8); ++c) {
                uint32_t y[8];
                const uint32_t at = tO + r * D + lane_base + c * 8;
                tmem_ld8(at, y);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * corr);
                tmem_st8(at, y);
              }
            }
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          // ---- P over S ----
          const float2 sl2w = make_float2(sl2, sl2), nmv = make_float2(nm, nm);
          float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < kSets; ++c) {
            const uint32_t (&y)[32] = x[c];
            uint32_t hi[16], mid[WIDE ? 16 : 1], lo[WIDE ? 16 : 1];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 v = make_float2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]));
              // (ALiBi's scores are in log2 units already)
              const float2 e = VAR == kAlibi ? add2(v, nmv) : fma2(v, sl2w, nmv);
              float2 pp = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              rs[k & 1] = add2(rs[k & 1], pp);
              hi[k] = pack_bf16x2(pp.x, pp.y);
              if constexpr (WIDE) {
                pp.x -= __uint_as_float(hi[k] << 16);
                pp.y -= __uint_as_float(hi[k] & 0xffff0000u);
                mid[k] = pack_bf16x2(pp.x, pp.y);
                lo[k] = pack_bf16x2(pp.x - __uint_as_float(mid[k] << 16),
                                    pp.y - __uint_as_float(mid[k] & 0xffff0000u));
              }
            }
            const uint32_t tP = tS + 64 * h + (c + part) * 16;
            tmem_st16(tP, hi);
            if constexpr (WIDE) {
              tmem_st16(tP + 32, mid);
              tmem_st16(tP + 64, lo);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kPFull + 4 * h + b));
          const float2 rsum = add2(rs[0], rs[1]);
          l += rsum.x + rsum.y;
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- epilogue of the segment ----
      if (!mbar_wait_warp(bar(kOFull + r), n_seg & 1, ctl)) { ok = false; break; }
      ++n_seg;
      tc_fence_after();
      if constexpr (kSplit) {
        float both[2];
        if (!exchange(l, both)) { ok = false; break; }
        l = both[0] + both[1];
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // (a NaN stays)
      const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      const bool whole = sg.place == 2;
      // A cut item's partial: place 0 of the block for one that began before, else 1.
      const size_t pplace = (size_t)blockIdx.x * 2 + sg.place, prow = pplace * a.part_rows + i;
      const size_t orow = (size_t)(sg.q0 + node) * a.n_q_heads + head;
      if (real && part == 0) {
        if (whole) a.lse[orow] = lse;
        else a.lse_part[prow] = lse;
      }
#pragma unroll 1
      for (int c = part * (D / 64); c < (kSplit ? (part + 1) * (D / 64) : D / 32); ++c) {
        uint32_t x[32];
        tmem_ld32(tO + r * D + lane_base + c * 32, x);
        tmem_wait_ld();
        if (!real) continue;
        // (a row that has seen nothing may find anything in O)
        auto f = [&](int k) { return l == 0.f ? 0.f : __uint_as_float(x[k]) * inv; };
        if (!WIDE && whole) {
          uint16_t* dst = static_cast<uint16_t*>(a.o) + orow * D + c * 32;
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = pack_bf16x2(f(2 * k), f(2 * k + 1));
          store_32B<2>(dst, y);
        } else {
          // A partial's values lie 8 columns of all rows together, so that a warp's stores are
          // consecutive; a row of O is D values.
          float* dst = whole ? static_cast<float*>(a.o) + orow * D + c * 32
                             : a.o_part + (pplace * (D / 8) + c * 4) * a.part_rows * 8 + (size_t)i * 8;
          const size_t apart = whole ? 8 : (size_t)a.part_rows * 8;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(f(8 * q + k));
            store_32B<1>(dst + q * apart, y);
          }
        }
      }
      tc_fence_before();
    }
  }

  // ---- teardown: the TMEM readers and both MMA drains are done ----
  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// The partials of cut items: O = sum w_i O_i / sum w_i with w_i = exp(lse_i - max),
// blocks in order (and, with many, eight running sums in order), so that the result does
// not depend on which came first.  The first kernel's blocks leave what ended in them; every
// block here counts through those and takes its share of the rows, four to a warp: lane l
// has 4 values of row (l / 2) % 4 in column group l / 8 and every fourth behind it, so that
// a load takes 128 consecutive bytes from each of four groups.  Up to kFewParts partials a
// warp does its rows alone; more are divided among the block's warps (one sequence of 30720
// tokens is cut 38 ways).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 4;
// (with 24 for the border 8: one sequence of 2000 tokens 31 us instead of 17.8, 4 of 1024 -
// 32768 80 instead of 77; with 2 55 instead of 58 at head_dim 256 with a window, 75 instead of 77
// for those 4, 209 instead of 204 for 16)
constexpr int kFewParts = 8;
constexpr int kMostBlocks = 256;  // of the first kernel's grid

template <int D, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32) join_tree_kernel(const DecodeTreeArgs a) {
  constexpr int kV = D / 32;  // 16-byte pieces of a lane
  __shared__ int s_units[kMostBlocks + 1];  // units in front of each block's item
  __shared__ int s_warp[kJoinWarps];
  __shared__ float4 s_o[kJoinWarps][kV][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  // Units: kJoinRows rows, or with few partials kJoinWarps times as many.
  {
    const int c = threadIdx.x;
    int units = 0;
    if (c < a.blocks) {
      const TreeJoin j = a.joins[c];
      const int few = c - j.first_block + 1 <= kFewParts ? kJoinWarps : 1;
      if (j.first_block >= 0) units = (j.rows + kJoinRows * few - 1) / (kJoinRows * few);
    }
    int incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
      if (w < warp) incl += s_warp[w];
    s_units[c + 1] = incl;
    if (c == 0) s_units[0] = 0;
    __syncthreads();
  }
  const int total = s_units[a.blocks];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int c = 0;
    for (int hi = a.blocks; hi - c > 1;) {
      const int mid = (c + hi) >> 1;
      if (s_units[mid] <= u) c = mid; else hi = mid;
    }
    const TreeJoin j = a.joins[c];
    const int parts = c - j.first_block + 1;
    const bool many = parts > kFewParts;
    const int row0 = (many ? u - s_units[c] : (u - s_units[c]) * kJoinWarps + warp) * kJoinRows;
    const int k0 = many ? warp : 0, step = many ? kJoinWarps : 1;
    auto place = [&](int k) {  // the first block left it at its place 1, the others at place 0
      return (size_t)(j.first_block + k) * 2 + (k == 0 ? 1 : 0);
    };
    // Each row's largest LSE, and the sum of the weights: lane l looks at row l % 4, partials
    // l / 4 and every eighth behind it.
    const int mine = min(row0 + (lane & 3), j.rows - 1);
    float top = -INFINITY, sum = 0.f;
    if (row0 < j.rows) {
      for (int k = lane >> 2; k < parts; k += 8)
        top = fmax_nan(top, a.lse_part[place(k) * a.part_rows + mine]);
    }
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref_mine = top == -INFINITY ? 0.f : top;
    if (row0 < j.rows) {
      for (int k = lane >> 2; k < parts; k += 8)
        sum += ex2_approx((a.lse_part[place(k) * a.part_rows + mine] - ref_mine) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int sub = (lane >> 1) & 3, row = row0 + sub;  // the row whose values this lane has
    const float ref = __shfl_sync(0xffffffffu, ref_mine, sub);
    sum = __shfl_sync(0xffffffffu, sum, sub);
    float4 acc[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool live = row < j.rows;
    if (live) {
#pragma unroll 4
      for (int k = k0; k < parts; k += step) {
        const float w = ex2_approx((a.lse_part[place(k) * a.part_rows + row] - ref) * kLog2e);
        const float* src =
            a.o_part + ((place(k) * (D / 8) + (lane >> 3)) * a.part_rows + row) * 8 + (lane & 1) * 4;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          const float4 x =
              *reinterpret_cast<const float4*>(src + (size_t)v * 4 * a.part_rows * 8);
          acc[v].x = fmaf(w, x.x, acc[v].x);
          acc[v].y = fmaf(w, x.y, acc[v].y);
          acc[v].z = fmaf(w, x.z, acc[v].z);
          acc[v].w = fmaf(w, x.w, acc[v].w);
        }
      }
    }
    if (many) {
#pragma unroll
      for (int v = 0; v < kV; ++v) s_o[warp][v][lane] = acc[v];
      __syncthreads();
      // Warp w joins the pieces v = w, w + 8, ..
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        if (v % kJoinWarps != warp) continue;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kJoinWarps; ++w) {
          const float4 x = s_o[w][v][lane];
          t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
        }
        acc[v] = t;
      }
      __syncthreads();
    }
    if (!live) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int g = a.n_q_heads / a.n_kv_heads;
    const int node = (j.row0 + row) / g, head = j.kvh * g + (j.row0 + row) % g;
    const size_t orow = (size_t)(j.q0 + node) * a.n_q_heads + head;
    if ((lane & ~6) == 0 && (!many || warp == 0))
      a.lse[orow] = sum == 0.f ? -INFINITY : ref + log2f(sum) * kLn2;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      if (many && v % kJoinWarps != warp) continue;
      const float4 x = make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
      const size_t at = orow * D + ((lane >> 3) + 4 * v) * 8 + (lane & 1) * 4;
      if constexpr (WIDE)
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = x;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + at) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
  }
}

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

// A (planes, rows, n_kv, D) bf16 cache with boxes of 64 dims x 1 head x box rows x 1.
bool make_cache_map(CUtensorMap* m, const void* base, int D, int n_kv, int rows, int planes,
                    int box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)D * 2, token = row * (cuuint64_t)n_kv;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n_kv, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[3] = {row, token, token * (cuuint64_t)rows};
  cuuint32_t boxes[4] = {64, 1, (cuuint32_t)box, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxes,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries (nodes, heads, D) bf16, boxes of 64 dims x heads x nodes.
bool make_q_map(CUtensorMap* m, const void* base, int D, int n_q, int nodes, int box_heads,
                int box_nodes) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)D * 2;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n_q, (cuuint64_t)nodes};
  cuuint64_t strides[2] = {row, row * (cuuint64_t)n_q};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_nodes};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int VAR, bool WIDE>
cudaError_t launch_t(const DecodeTreeArgs& a, const LaunchCtx& ctx) {
  using L = TreeSmem<D, VAR, WIDE>;
  constexpr int kBN = L::kBN;
  TreeKParams p;
  p.a = a;
  const int g = p.g = a.n_q_heads / a.n_kv_heads;
  p.tile_nodes = 128 / g;
  p.q_tiles = std::min(row_tiles<D>(), (std::min(a.total_nodes, kMostNodes) + p.tile_nodes - 1) /
                                           p.tile_nodes);
  p.slots = L::slots(p.q_tiles);
  {
    // Units are counted in 31 bits: more than one tile each where the cache's capacity
    // would allow for more.
    const int group = p.tile_nodes * p.q_tiles;
    const long long items = (long long)a.batch * a.n_kv_heads * ((kMostNodes + group - 1) / group);
    const long long tiles = (a.capacity() + kBN - 1) / kBN + 1;
    p.unit_shift = 0;
    while (items * kFullRun * ((tiles >> p.unit_shift) + 1) > 0x7fffffffLL) {
      if (tiles >> p.unit_shift == 0) return cudaErrorInvalidValue;
      ++p.unit_shift;
    }
  }
  p.sl2 = a.scale * kLog2e;
  p.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  p.cap_l2 = a.softcap * kLog2e;
  p.err_word = ctx.err_word;
  p.timeout_ns = ctx.timeout_ns;
  // Tiled copies where blocks are made of runs of 8 to 64 rows.  A tiled copy costs the SM's
  // copy unit some 50 clocks and 2.5 for each row of 128 bytes: boxes of 16 rows come to the
  // memory's rate only while the unit never idles, those of 8 to half of it.  Copies by rows
  // (16 bytes a lane) come to half of it too, by another way: with runs of 8 rows the keys go
  // by the one, the values by the other (16 sequences of 1024 - 32768 tokens in blocks of 24:
  // 383 us, 414 by rows alone).
  CUtensorMap mq, mk, mv, mk16, mv16;
  if (!make_q_map(&mq, a.q, D, a.n_q_heads, a.total_nodes, g, p.tile_nodes))
    return cudaErrorInvalidValue;
  std::memset(&mk, 0, sizeof(mk));
  std::memset(&mv, 0, sizeof(mv));
  std::memset(&mk16, 0, sizeof(mk16));
  std::memset(&mv16, 0, sizeof(mv16));
  p.box = kMostBox;
  if (a.block_table)
    while (p.box >= kLeastBox && a.block_size % p.box != 0) p.box /= 2;
  if (p.box >= kLeastBox) {
    const int rows = a.block_table ? a.block_size : a.max_kv_len;
    const int planes = a.block_table ? a.num_blocks : a.batch;
    if (!make_cache_map(&mk, a.k_cache, D, a.n_kv_heads, rows, planes, p.box) ||
        (p.box >= 16 &&
         (!make_cache_map(&mv, a.v_cache, D, a.n_kv_heads, rows, planes, p.box) ||
          !make_cache_map(&mk16, a.k_cache, D, a.n_kv_heads, rows, planes, 16) ||
          !make_cache_map(&mv16, a.v_cache, D, a.n_kv_heads, rows, planes, 16))))
      p.box = 0;  // (sizes that a tensor map cannot hold)
  } else {
    p.box = 0;
  }
  p.blocks_a_tile = a.block_table ? kBN / a.block_size : 0;
  p.rest_a_tile = a.block_table ? kBN % a.block_size : 0;
  auto kernel = decode_tree_kernel<D, VAR, WIDE>;
  static bool configured[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         std::max(L::total(1), L::total(row_tiles<D>())));
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.blocks);
  cfg.blockDim = dim3(threads_of<D>());
  cfg.dynamicSmemBytes = L::total(p.q_tiles);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, mk16, mv16, p);
  if (e != cudaSuccess || a.whole) return e;
  cfg.gridDim = dim3((unsigned)(4 * a.blocks));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_tree_kernel<D, WIDE>, a);
}

template <int D, bool WIDE>
cudaError_t launch_v(const DecodeTreeArgs& a, const LaunchCtx& ctx) {
  if (a.softcap > 0.f) return launch_t<D, kCap, WIDE>(a, ctx);
  if (a.alibi_slopes != nullptr) return launch_t<D, kAlibi, WIDE>(a, ctx);
  return launch_t<D, kPlain, WIDE>(a, ctx);
}

template <int D>
cudaError_t launch_d(const DecodeTreeArgs& a, const LaunchCtx& ctx) {
  return a.wide ? launch_v<D, true>(a, ctx) : launch_v<D, false>(a, ctx);
}

}  // namespace

int decode_tree_part_rows(int head_dim, int group, int max_nodes) {
  const int tile_nodes = 128 / group;
  return std::min((head_dim == 256 ? 1 : 2) * tile_nodes, max_nodes) * group;
}

cudaError_t launch_decode_tree(const DecodeTreeArgs& a, const LaunchCtx& ctx) {
  if (a.head_dim == 256) return launch_d<256>(a, ctx);
  if (a.head_dim == 128) return launch_d<128>(a, ctx);
  return launch_d<64>(a, ctx);
}

}  // namespace attn
