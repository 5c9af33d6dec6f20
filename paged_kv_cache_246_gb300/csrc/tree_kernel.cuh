// The kernels of paged_attn_decode_tree: every node of a tree of drafted tokens attends to its
// sequence's context, its ancestors and itself:
//     s_j = scale * q.k_j + slope_h * (pos_j - pos_i),   out = softmax(s) . V,
// where a context key's position is its place in the cache and a node's is the
// context's length plus its depth.
//
// Rows are (node, query head of the KV group) pairs, node by node, in tiles of
// 128: 128 / QPK nodes each.  The step reads the context's K and V once per KV
// head and row tile.  Of a 16-bit cache a key is 4 D bytes and, with both terms of
// the weights (below), 6 D flops a row: 192 flops a byte for a full tile, against
// 281 of the card, so one row tile is bound by HBM, and two by the products.  Of an
// 8-bit cache it is 2 D bytes and the time of 4 D 16-bit flops for bf16 queries (two
// E4M3 terms of q at twice that rate, one of the weights: 256 a byte), of 7 D for
// fp16 ones (three and two: 448, so HBM binds tiles of up to 80 rows).  mma.sync
// tiles of 16 rows, as the other decodes use, would read K and V from L2 once per
// tile.
//
// CTA = one per SM, persistent.  The work is the list of units (row tile,
// sequence, KV head, 128-key tile), in this order; every CTA takes an equal,
// contiguous share of it, found from seq_lens and cu_nodes on the device, and
// walks it segment by segment (a segment: its part of one item, a sequence's KV
// head and row tile).  A segment that is a whole item writes the output; a part
// writes its (o, m, l) in fp32, and combine_kernel merges the parts in order.
// So all SMs do the same amount whatever the lengths and trees are, and every
// CTA has at most two partial segments (its first and its last).  The first row
// tiles of all trees come first, then the second ones: the CTAs of each walk the
// same K and V side by side, from HBM once and from L2 for the others.
//
// Roles of the 16 warps:
//   warps 0, 2  TMA producers of K (and each segment's query rows) and of V: tiles
//               of 128 keys, one box (block_size rows x 64 channels, 128-byte
//               swizzle) per cache block; blocks out of the visible range are
//               loaded from an out-of-range coordinate and arrive as zeros.  (One
//               producer for both would hold the next K back until a V stage is
//               free, a product later than its own.)
//   warp 1      MMA issuer: S = Q K^T into one of two score buffers in tensor
//               memory, O += P V with P read from there.
//   warp 3      over an 8-bit cache: makes each segment's queries.
//   warps 4-7   look through the V tiles that some row sees only in part (the
//               tree's, and the window's edge): rows hidden from all are
//               zeroed, values that are not finite are zeroed and the segment
//               is marked, since 0 * NaN in the product would reach rows that
//               do not see them (the rows that do get them back at the end).
//               Over an 8-bit cache they also widen the V codes to fp16.  (In the
//               other tiles all rows see an infinite value, whose channel then
//               is not finite in any of them; which it is, since the two terms of a
//               weight make inf - inf and 0 * inf of it, is looked up at the
//               segment's end.  Looking through all tiles on the way costs heads of
//               64 8 %: 145 -> 157 us.)
//   warps 8-11, 12-15  softmax groups A and B: thread r owns row r.
// Of every key tile group A takes the first 64 keys and B the last, each with
// its own running maximum, sum and accumulator; the two are merged at the
// segment's end.  So a tile's softmax takes half as long as with a thread for
// all 128 keys, no group waits for the other, and two score buffers fit beside
// the two accumulators: the products of one tile run under the softmax of the
// next.
//
// The weights enter P V as two 16-bit terms (hi + lo): a single rounded term
// puts up to 2^-8 of a bf16 weight into the output, as much as the output's own
// rounding; two leave 2^-17.  (One term for all: four row tiles of 16384 keys
// 868 -> 750 us, one tree 55 -> 52.)  Over an 8-bit cache P is fp16: two terms
// for fp16 outputs, one, 2^-11 of a weight, for bf16 outputs.  It shows a little
// beside their rounding of 2^-8: 128 contexts of 100 .. 4096 tokens lie 1.672e-3 of
// the output's norm off the 64-bit definition, with two terms 1.660e-3 as 32-bit
// arithmetic with one rounding does; but the second takes 197 -> 230 us there, 366 -> 398
// for 64 contexts of 4096 .. 16384.
// Over an 8-bit cache q.k runs on the codes as they are (kind::f8f6f4), each
// query row scaled by a power of two to its own largest finite component and
// split into E4M3 terms (two for the 8 bits of bf16, three for the 11 of fp16).
//
// Every wait is bounded; a timeout raises a CTA-wide flag, the roles stop,
// copies and products in flight are drained, tensor memory is freed.
#pragma once

#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "tcgen05.cuh"
#include "tree.cuh"

namespace pkv {
namespace tree {

using tc5::AB;
using tc5::wait_or_abort;
using tc5::warp_wait;

constexpr int kThreads = 512;
constexpr int kGuards = 4;  // warps that look through V
constexpr int kMaskWords = PKV_TREE_MAX_NODES / 32;

// ---------------------------------------------------------------------------
// The list of work
// ---------------------------------------------------------------------------
struct Seq {
  int row, nodes, ctx, L, kv_lo, kv_start, tiles;
};

// Sequence b; false: nothing to do, `bad` where what the tensors say cannot be.
__device__ __forceinline__ bool seq_of(const Args &a, int b, Seq &s, bool &bad) {
  bad = !nodes_of(a.tb, b, s.row, s.nodes);
  s.L = __ldg(a.seq_lens + b);
  if (bad || s.nodes == 0) return false;
  bad = s.L < s.nodes || s.L > a.max_seq_len ||
        s.L > static_cast<int64_t>(a.max_blocks_per_seq) * a.BS;
  if (bad) return false;
  s.ctx = s.L - s.nodes;
  // the first position that a node of depth 0 sees: deeper ones see less
  s.kv_lo = a.window > 0 ? max(0, s.ctx - a.window + 1) : 0;
  s.kv_start = s.kv_lo / BN * BN;
  s.tiles = (s.L - s.kv_start + BN - 1) / BN;
  return true;
}

struct Seg {
  Seq s;
  int b, g, j0, n;  // tiles j0 .. j0 + n - 1 of KV head g
  int node0;        // the row tile's first node
  __device__ __forceinline__ bool whole() const { return n == s.tiles; }
  // Of the segment's tiles all rows see those from calm_from to before calm_to
  // whole: in front of them lies the window's edge (a node of depth nodes - 1
  // sees least), behind them the tree.
  __device__ __forceinline__ int calm_from(const Args &a) const {
    return a.window > 0 ? (max(0, s.ctx + s.nodes - a.window - s.kv_start) + BN - 1) / BN - j0 : 0;
  }
  __device__ __forceinline__ int calm_to() const { return (s.ctx - s.kv_start) / BN - j0; }
};

// Units of a (sequence, KV head): its tiles behind item_units more; one where
// items are not cut (item_units 0).
__device__ __forceinline__ int units_of(const Args &a, const Seq &s) {
  return a.item_units > 0 ? s.tiles + a.item_units : 1;
}

// A CTA's segments, in order: every role walks them by itself.
struct Walk {
  int row_tile, b, g, j;  // unit j of KV head g of sequence b
  int64_t left;           // units to go
  bool known = false;
  Seq s;
  __device__ __forceinline__ bool next(const Args &a, Seg &o) {
    while (left > 0 && row_tile < a.row_tiles) {
      if (b >= a.tb.num_seqs) {
        b = 0;
        ++row_tile;
        continue;
      }
      if (!known) {
        bool bad;
        if (!seq_of(a, b, s, bad) || s.nodes <= row_tile * a.tile_nodes) {
          ++b;
          continue;
        }
        known = true;
      }
      const int item = units_of(a, s);
      const int take = static_cast<int>(min(static_cast<int64_t>(item - j), left));
      o.s = s;
      o.b = b;
      o.g = g;
      o.node0 = row_tile * a.tile_nodes;
      o.j0 = max(j - a.item_units, 0);
      j += take;
      left -= take;
      o.n = a.item_units > 0 ? max(j - a.item_units, 0) - o.j0 : s.tiles;
      if (j == item) {
        j = 0;
        if (++g == a.KVH) {
          g = 0;
          ++b;
          known = false;
        }
      }
      if (o.n > 0) return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------------------
// Shared memory
// ---------------------------------------------------------------------------
template <class T, int D, bool KV8>
struct Lay {
  static constexpr int REG = 128 * 128;  // a 64-channel region of 128 rows
  static constexpr int NREG = D / 64;
  static constexpr int TILE = REG * NREG;
  static constexpr int TILE8 = BN * D;
  static constexpr int TERMS = std::is_same_v<T, FP16> ? 3 : 2;  // E4M3 terms of a query
  // rings, as large as fit
  static constexpr int NK = KV8 ? 0 : (D == 128 ? 2 : 4);
  static constexpr int NV = KV8 ? 2 : (D == 128 ? 2 : 4);
  static constexpr int N8K = !KV8 ? 0 : D == 64 ? 6 : TERMS == 2 ? 3 : 2;
  static constexpr int N8V = !KV8 ? 0 : D == 64 ? 4 : TERMS == 2 ? 2 : 1;
  static constexpr int NQ = 2;  // query buffers
  static constexpr int OFF_Q = 0;
  static constexpr int Q_BYTES = NQ * (KV8 ? TERMS * TILE8 : TILE);
  static constexpr int OFF_K = OFF_Q + Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_K8 = OFF_V + NV * TILE;
  static constexpr int OFF_V8 = OFF_K8 + N8K * TILE8;
  static constexpr int OFF_MASK = OFF_V8 + N8V * TILE8;  // [words + 2][256 threads]
  static constexpr int OFF_ML = OFF_MASK + (kMaskWords + 2) * 256 * 4;  // [2][128] float2
  static constexpr int OFF_EXP = OFF_ML + 2 * 128 * 8;  // [NQ][128] 2^e of the queries
  static constexpr int OFF_BAD = OFF_EXP + NQ * 128 * 4;                // [8][32] words of a pass that are not finite
  static constexpr int OFF_BAR = OFF_BAD + 8 * 32 * 4;
  // copies landed (K, V, Q), stages free again (EK, EV, EQ; EV also: both
  // products of that tile done), V looked through (VG), V codes widened (E8V),
  // scores ready (S, per buffer), weights ready (P, per buffer), both
  // groups' maxima written (ML), both accumulators read (EPI).
  // A wait names a phase by its parity, so every waiter of a barrier sees each
  // of its phases, or knows by another barrier that the one before has
  // completed and that the one after cannot have.
  static constexpr int NKT = KV8 ? N8K : NK, NVT = KV8 ? N8V : NV;
  static constexpr int B_K = 0, B_EK = B_K + NKT, B_V = B_EK + NKT, B_VG = B_V + NVT,
                       B_EV = B_VG + NV, B_E8V = B_EV + NV, B_Q = B_E8V + N8V, B_EQ = B_Q + NQ,
                       B_S = B_EQ + NQ, B_P = B_S + 2, B_ML = B_P + 2, B_EPI = B_ML + 1,
                       B_FIN = B_EPI + 1, NBAR = B_FIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int BYTES = OFF_MISC + 512;
  // one CTA owns an SM and its tensor memory
  static constexpr int ALLOC = std::max(BYTES + 1024, 118 * 1024);
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
};

// One arrival for the warp, behind what its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Whether the phase with the given parity is through, without waiting for it.
__device__ __forceinline__ bool mbar_look(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Registers of a thread at the launch (the most that 512 threads can have, and
// what the kernels use), and in the warpgroups of warps 0-3, 4-7 and 8-15.
// Taking more than the launch's pool holds would wait for ever, so launch()
// makes sure of the kernel's count.
constexpr int kLaunchRegs = 128, kIssueRegs = 72, kGuardRegs = 104, kSoftmaxRegs = 168;
static_assert(kIssueRegs + kGuardRegs + 2 * kSoftmaxRegs <= 4 * kLaunchRegs);

// Registers of this warpgroup's threads from here on: every warp of it calls.
template <bool MORE, int N>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Words of the MISC area.
enum { kTmem = 0, kAbort = 1, kIssuedK = 2, kIssuedV = 3, kIssuedQ = 4, kStart = 6, kFlags = 16, kScan = 32 };
constexpr int kFlagSlots = 16;  // twice as many as segments that can be under way at once

// The element of a 16-bit pair that is not finite: bits of its half, else 0.
template <class T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & T::kInf) == T::kInf ? 0xffffu : 0u) |
         ((w & (T::kInf << 16)) == T::kInf << 16 ? 0xffff0000u : 0u);
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Whether any of N elements is not finite.
template <class T, int N>
__device__ __forceinline__ bool any_not_finite(const void *row) {
  uint4 u[N / 8];
#pragma unroll
  for (int i = 0; i < N / 8; ++i) u[i] = __ldg(reinterpret_cast<const uint4 *>(row) + i);
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    any |= not_finite<T>(u[i].x) | not_finite<T>(u[i].y) | not_finite<T>(u[i].z) | not_finite<T>(u[i].w);
  return any != 0;
}

// The key (half 0) or the value (half 1) at position pos, in block pb, which is in range.
__device__ __forceinline__ const uint8_t *cache_row(const Args &a, const Seg &s, int half, int pb,
                                                    int pos, int D, int elem_bytes) {
  return a.cache + (((half * a.num_blocks + pb) * a.BS + pos % a.BS) * a.row_elems +
                    static_cast<int64_t>(s.g) * D) * elem_bytes;
}

// Values that are not finite, and the rows that see them.  Any weight times
// infinity is infinity, but for the weight 0 of a score of -infinity, which makes
// NaN.  Such a score's key is not finite either (a query that is not finite has no
// finite scores, and its row is NaN as it is), and a key that is not finite has no
// finite score: so where key and value both are not, all rows that see them are NaN
// in the value's channel.

// The tiles that all rows see whole: a value of theirs that is not finite decides
// its channel in every row.  Called by a warp, each lane with its row, where
// some row's accumulator is not finite; the channels are c0 .. c0 + D / 2 - 1.  A
// tile takes 5 us, 22 where all its values are infinite: the second that the
// other roles wait is some 5 million such keys of one segment.
template <class T, int D>
__device__ __noinline__ void set_not_finite(const Args &a, const Seg &seg, int c0, bool write,
                                            uint16_t *out, float *part) {
  constexpr int COLS = D / 2, WORDS = COLS / 32;
  const int32_t *trow = a.block_tables + static_cast<int64_t>(seg.b) * a.max_blocks_per_seq;
  const int start = seg.s.kv_start + seg.j0 * BN;
  const int end = start + min(seg.calm_to(), seg.n) * BN;
  uint32_t up[WORDS] = {}, down[WORDS] = {};  // channels that hold +infinity, -infinity (NaN: both)
#pragma unroll 2
  for (int pos = start + max(seg.calm_from(a), 0) * BN + (threadIdx.x & 31); pos < end; pos += 32) {
    const int pb = __ldg(trow + pos / a.BS);
    if (pb < 0 || pb >= a.num_blocks) continue;
    const uint8_t *row = cache_row(a, seg, 1, pb, pos, D, 2) + c0 * 2;
    if (!any_not_finite<T, COLS>(row)) continue;
    const bool key_too = any_not_finite<T, D>(cache_row(a, seg, 0, pb, pos, D, 2));
#pragma unroll
    for (int w = 0; w < WORDS; ++w)
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row) + 4 * w + i);
        uint32_t p = 0, n = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t e = word_of(u, c / 2) >> (c % 2 * 16) & 0xffffu;
          const bool bad = (e & T::kInf) == T::kInf, nan = key_too || (e & 0x7fffu) != T::kInf;
          if (bad && (nan || e < 0x8000u)) p |= 1u << c;
          if (bad && (nan || e >= 0x8000u)) n |= 1u << c;
        }
        up[w] |= p << (8 * i);
        down[w] |= n << (8 * i);
      }
  }
  __syncwarp();
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    up[w] = __reduce_or_sync(0xffffffffu, up[w]);
    down[w] = __reduce_or_sync(0xffffffffu, down[w]);
#pragma unroll 1
    for (int e = 0; write && e < 32; ++e) {
      const bool p = up[w] >> e & 1, n = down[w] >> e & 1;
      if (!p && !n) continue;
      const float v = p && n ? __int_as_float(0x7fffffff) : p ? INFINITY : -INFINITY;
      const int c = c0 + 32 * w + e;
      if (out)
        out[c] = static_cast<uint16_t>(T::from_f2(v, 0.f));
      else
        part[static_cast<int64_t>(c / 4) * 512 + c % 4] = v;
    }
  }
}

// The tiles that rows see in part: what the look through V took out of them goes
// back into the rows that see it; every visible value that is not finite is added
// to the row's elements as they stand in memory.  Rare, as the one above.
template <class T, int D, bool KV8>
__device__ __noinline__ void add_not_finite(const Args &a, const Seg &seg, int lo, int c0, int cols,
                                            const uint32_t *mask, uint16_t *out, float *part) {
  const int32_t *trow = a.block_tables + static_cast<int64_t>(seg.b) * a.max_blocks_per_seq;
  auto key = [&](int pos) {
    const int pb = __ldg(trow + pos / a.BS);
    if (pb < 0 || pb >= a.num_blocks) return;
    const uint8_t *row = cache_row(a, seg, 1, pb, pos, D, KV8 ? 1 : 2);
    bool key_too = false, known = KV8;
    for (int d = 0; d < cols; ++d) {
      float v;
      if constexpr (KV8)
        v = (row[c0 + d] & 0x7f) == 0x7f ? __int_as_float(0x7fffffff) : 0.f;
      else
        v = T::to_f(reinterpret_cast<const uint16_t *>(row)[c0 + d]);
      if (fabsf(v) < INFINITY) continue;
      if (!known) {
        key_too = any_not_finite<T, D>(cache_row(a, seg, 0, pb, pos, D, 2));
        known = true;
      }
      if (key_too) v = __int_as_float(0x7fffffff);
      if (out)
        out[c0 + d] = static_cast<uint16_t>(T::from_f2(T::to_f(out[c0 + d]) + v, 0.f));
      else
        part[static_cast<int64_t>((c0 + d) / 4) * 512 + (c0 + d) % 4] += v;
    }
  };
  for (int j = 0; j < seg.n; ++j) {
    if (j >= seg.calm_from(a) && j < seg.calm_to()) continue;
    const int kv0 = seg.s.kv_start + (seg.j0 + j) * BN;
    for (int pos = max(kv0, lo); pos < min(kv0 + BN, seg.s.ctx); ++pos) key(pos);
    for (int c = max(0, kv0 - seg.s.ctx); c < min(seg.s.nodes, kv0 + BN - seg.s.ctx); ++c)
      if (mask[(c / 32 + 1) * 256] >> (c % 32) & 1) key(seg.s.ctx + c);
  }
}

template <class T, int D, bool KV8, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const Args a, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ CUtensorMap kvmap) {
  using L = Lay<T, D, KV8>;
  using OPT = std::conditional_t<KV8, FP16, T>;  // operand type of P V
  constexpr bool TWO = !KV8 || std::is_same_v<T, FP16>;  // weights in two terms
  // fp16 weights are held 2^5 times as large: one is off by up to half of the
  // type's smallest step, 2^-25, so by 2^-30 of the row's largest, and 2^19 keys
  // by no more than the output's rounding (unscaled, 2^14 keys).  A row's 64 keys
  // then add up to 2^11 at most where its maximum is up to date, and to 2^15
  // where that is 4 to 10 steps (of log2) late: then it moves.  (The lift costs
  // nothing but with ALiBi, where scores rise tile by tile: 290 -> 303 us for 128
  // contexts over an 8-bit cache.)
  constexpr bool P16 = std::is_same_v<OPT, FP16>;
  constexpr float kLift = P16 ? 5.f : 0.f, kLate = P16 ? 3.f : 8.f;
  constexpr int NV = L::NV, NKT = L::NKT, NVT = L::NVT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
  volatile uint32_t *abort_flag = misc + kAbort;
  volatile uint32_t *flags = misc + kFlags;
  // warp-uniform to the compiler too
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int64_t where = blockIdx.x;
  const int tile_rows = a.tile_nodes * a.QPK;

  // ---- before the kernel ahead has completed: nothing that it may write ----
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      uint32_t count = 1;
      if (i >= L::B_VG && i < L::B_VG + NV) count = kGuards;
      if (KV8 && i >= L::B_E8V && i < L::B_E8V + L::N8V) count = kGuards;
      if (i >= L::B_EQ && i < L::B_EQ + L::NQ) count = 8;
      if (i == L::B_P || i == L::B_P + 1 || i == L::B_ML || i == L::B_EPI) count = 8;
      mbar_init(&bars[i], count);
    }
    misc[kAbort] = 0;
    misc[kIssuedK] = misc[kIssuedV] = misc[kIssuedQ] = 0;
    for (int i = 0; i < kFlagSlots; ++i) misc[kFlags + i] = 0;
    fence_mbar_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kvmap);
  }
  if (warp == 1) tc5::tmem_alloc<512>(misc + kTmem);
  if constexpr (!KV8) {
    // rows that no copy writes (128 is no multiple of QPK): finite once and for all
    for (int i = threadIdx.x; i < L::NQ * L::NREG * (BM - tile_rows) * 8; i += kThreads) {
      const int per = (BM - tile_rows) * 8;
      *reinterpret_cast<uint4 *>(smem + L::OFF_Q + (i / per) * L::REG + tile_rows * 128 +
                                 (i % per) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- this CTA's share of the units ----
  Walk walk;
  int64_t total = 0, u0, u1, per_share;
  // more_shares of the shares, evenly spread, have a unit more than per_share: so
  // the CTAs of equal row tiles begin at the same keys, and stay within L2's reach
  // of each other (with the longer shares first four row tiles of 2 sequences
  // read K and V 2.4 times from HBM)
  int shares, more_shares;
  auto share_start = [&](int i) -> int64_t { return i * per_share + i * more_shares / shares; };
  {
    int64_t *scan = reinterpret_cast<int64_t *>(misc + kScan);                 // [2][16 warps], by turns
    int turn = 0;
    int64_t *tile_units = reinterpret_cast<int64_t *>(smem + L::OFF_MASK);     // [row tiles], not in use yet
    int64_t *start = reinterpret_cast<int64_t *>(misc + kStart);               // sequence, units into it
    // a sequence's units in each of its first `n` row tiles
    auto units = [&](int b, int &n) -> int64_t {
      Seq s;
      bool bad = false;
      int64_t u = 0;
      n = 0;
      if (b < a.tb.num_seqs) {
        if (seq_of(a, b, s, bad)) {
          u = static_cast<int64_t>(units_of(a, s)) * a.KVH;
          n = (s.nodes + a.tile_nodes - 1) / a.tile_nodes;
        }
        if (bad && blockIdx.x == 0) record_error(PKV_ERR_BOUNDS, b);
      }
      return u;
    };
    auto warp_scan = [&](int64_t v) -> int64_t {
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      return v;
    };
    // inclusive sum over the CTA's threads; every thread gets the sum over all
    auto block_scan = [&](int64_t v, int64_t &all) -> int64_t {
      int64_t *sums = scan + (turn ^= 16);
      v = warp_scan(v);
      if (lane == 31) sums[warp] = v;
      __syncthreads();
      const int64_t w = warp_scan(lane < kThreads / 32 ? sums[lane] : 0);
      all = __shfl_sync(0xffffffffu, w, 31);
      const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
      return warp > 0 ? v + before : v;
    };
    // the units of each row tile, up to the last one that a tree has
    int my_tiles, tiles = 0;
    const int64_t mine = units(threadIdx.x, my_tiles);
    int64_t incl0 = 0;  // of the first row tile and the first kThreads sequences
    for (int t = 0; t < a.row_tiles; ++t) {
      int64_t v = my_tiles > t ? mine : 0, all;
      for (int b = threadIdx.x + kThreads; b < a.tb.num_seqs; b += kThreads) {
        int n;
        const int64_t u = units(b, n);
        if (n > t) v += u;
      }
      v = block_scan(v, all);
      if (t == 0) incl0 = v;
      if (all == 0) break;
      if (threadIdx.x == 0) tile_units[t] = all;
      total += all;
      tiles = t + 1;
    }
    const int slots = gridDim.x, slot = blockIdx.x;
    shares = static_cast<int>(min(static_cast<int64_t>(slots), total));  // no empty ones among them
    per_share = shares > 0 ? total / shares : 0;
    more_shares = static_cast<int>(total - per_share * shares);
    u0 = slot < shares ? share_start(slot) : total;
    u1 = slot < shares ? share_start(slot + 1) : total;
    // the row tile and the sequence that hold unit u0
    int tile = 0;
    int64_t into = u0, base = 0;
    if (tiles > 1) {
      __syncthreads();
      while (tile < tiles && into >= tile_units[tile]) into -= tile_units[tile++];
    }
    for (int b0 = 0; b0 < a.tb.num_seqs && base <= into; b0 += kThreads) {
      int64_t all = total, own = mine, incl = incl0;
      int n = my_tiles;
      if (b0 > 0) own = units(b0 + threadIdx.x, n);
      if (n <= tile) own = 0;
      // the sum at hand is the first row tile's where all sequences have a thread
      if (tile > 0 || a.tb.num_seqs > kThreads) incl = base + block_scan(own, all);
      if (into < incl && into >= incl - own) {
        start[0] = b0 + threadIdx.x;
        start[1] = into - (incl - own);
      }
      base += all;
    }
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    walk.left = u1 - u0;
    walk.row_tile = tile;
    walk.b = walk.g = walk.j = 0;
    if (walk.left > 0) {
      walk.b = static_cast<int>(start[0]);
      Seq s;
      bool bad;
      seq_of(a, walk.b, s, bad);
      const int item = units_of(a, s);
      walk.g = static_cast<int>(start[1] / item);
      walk.j = static_cast<int>(start[1] - static_cast<int64_t>(walk.g) * item);
    }
  }
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[kTmem], 0);

  // K and the queries (V = false), or V
  int issued = 0;  // copies of this role, to be drained after an abort
  auto producer = [&](auto is_v) {
    constexpr bool V = decltype(is_v)::value;
    constexpr int STAGES = V ? NVT : NKT, FULL = V ? L::B_V : L::B_K;
    constexpr int EMPTY = !V ? L::B_EK : KV8 ? L::B_E8V : L::B_EV;
    constexpr int BYTES = KV8 ? L::TILE8 : L::TILE;
    constexpr int OFF = KV8 ? (V ? L::OFF_V8 : L::OFF_K8) : (V ? L::OFF_V : L::OFF_K);
    const int TB = BN / a.BS, TPB = 32 / TB;  // blocks of a tile; tiles whose blocks a warp holds
    // Lane l: the table's entry for block l of the TPB tiles from the segment's
    // tile j on, loaded a batch ahead: a load under way for every 4 or 8 tiles.
    auto entry = [&](const Seg &s, int j) -> int {
      const int lb = (s.s.kv_start + (s.j0 + j) * BN) / a.BS + lane;
      const int p0 = lb * a.BS;
      return p0 < s.s.L && p0 + a.BS > s.s.kv_lo
                 ? __ldg(a.block_tables + static_cast<int64_t>(s.b) * a.max_blocks_per_seq + lb)
                 : -1;
    };
    // Where the lane's block lies, or an out-of-range row (zeros) outside the
    // visible range or for a bad entry.
    auto coord_of = [&](const Seg &s, int j, int pb) -> int {
      const int lb = (s.s.kv_start + (s.j0 + j) * BN) / a.BS + lane;
      const int p0 = lb * a.BS;
      if (p0 >= s.s.L || p0 + a.BS <= s.s.kv_lo) return -a.BS;
      if (pb >= 0 && pb < a.num_blocks) return pb * a.BS;
      if (j + lane / TB < s.n)
        record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(s.b) * a.max_blocks_per_seq + lb);
      return -a.BS;
    };
    Seg s, ahead;
    bool have = walk.next(a, s);
    int next = have ? entry(s, 0) : 0, coords = 0;
    int it = 0;  // key tiles
    for (int si = 0; have; ++si) {
      const bool more = walk.next(a, ahead);
      for (int j = 0; j < s.n; ++j, ++it) {
        if (j % TPB == 0) {
          coords = coord_of(s, j, next);
          next = j + TPB < s.n ? entry(s, j + TPB) : more ? entry(ahead, 0) : 0;
        }
        const int coord = __shfl_sync(0xffffffffu, coords, (j % TPB) * TB + lane % TB);
        const int st = it % STAGES;
        uint64_t *full = &bars[FULL + st];
        uint8_t *dst = smem + OFF + st * BYTES + lane * a.BS * (KV8 ? D : 128);
        // little is left to do when the stage is free: this warp shares its
        // scheduler with two of the softmax's
        if (it >= STAGES &&
            !warp_wait(&bars[EMPTY + st], ((it / STAGES) - 1) & 1, abort_flag, where))
          return;
        if (lane == 0) mbar_arrive_expect_tx(full, BYTES);
        __syncwarp();
        if (lane < TB) {
#pragma unroll
          for (int r = 0; r < (KV8 ? 1 : L::NREG); ++r)
            tma_load_4d(dst + r * L::REG, &kvmap, full, 64 * r, s.g, coord, V);
        }
        issued = it + 1;
        if (!KV8 && !V && j == 0) {
          const int q = si % L::NQ;
          if (si >= L::NQ &&
              !warp_wait(&bars[L::B_EQ + q], ((si / L::NQ) - 1) & 1, abort_flag, where))
            return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars[L::B_Q + q], L::NREG * tile_rows * 128);
            misc[kIssuedQ] = si + 1;
            for (int r = 0; r < L::NREG; ++r)
              tc5::tma_load_3d(smem + L::OFF_Q + q * L::TILE + r * L::REG, &qmap, &bars[L::B_Q + q],
                               64 * r, s.g * a.QPK, s.s.row + s.node0);
          }
          __syncwarp();
        }
      }
      have = more;
      s = ahead;
    }
  };

  // Over an 8-bit cache: each row's query as E4M3 terms of q * 2^-e, a segment
  // ahead of its scores.  Lane = 16 channels of a row; one pass's loads run
  // under the pass before.
  auto queries = [&]() {
    constexpr int LPR = D / 16, RPP = 32 / LPR;  // lanes of a row, rows of a pass
    float *q_exp = reinterpret_cast<float *>(smem + L::OFF_EXP);
    uint32_t *bad_q = reinterpret_cast<uint32_t *>(smem + L::OFF_BAD);
    const int c = lane % LPR;
    Seg s;
#pragma unroll 1
    for (int si = 0; walk.next(a, s); ++si) {
      const int q = si % L::NQ;
      if (si >= L::NQ && !warp_wait(&bars[L::B_EQ + q], ((si / L::NQ) - 1) & 1, abort_flag, where))
        return;
      uint8_t *dst = smem + L::OFF_Q + q * L::TERMS * L::TILE8;
      const int rows = min(tile_rows, (s.s.nodes - s.node0) * a.QPK);
      auto row_at = [&](int r) {
        return reinterpret_cast<const uint4 *>(
            a.query + (static_cast<int64_t>(s.s.row + s.node0 + r / a.QPK) * a.H + s.g * a.QPK +
                       r % a.QPK) * D + c * 16);
      };
      int r = min(lane / LPR, rows - 1);
      uint4 n0 = __ldg(row_at(r)), n1 = __ldg(row_at(r) + 1);
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += RPP) {
        const uint4 v0 = n0, v1 = n1;
        const int here = r;
        r = min(r0 + RPP + lane / LPR, rows - 1);
        n0 = __ldg(row_at(r));
        n1 = __ldg(row_at(r) + 1);
        // the row's largest |q| as a 16-bit value: whole numbers compare as the
        // values do
        uint32_t x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        auto largest = [&]() -> uint32_t {
          uint32_t two = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) two = __vmaxu2(two, x[k] & 0x7fff7fffu);
          uint32_t top = max(two & 0xffffu, two >> 16);
#pragma unroll
          for (int d = 1; d < LPR; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
          return top;
        };
        uint32_t top = largest();
        if (__any_sync(0xffffffffu, top >= T::kInf)) {
          // the largest finite one; infinities become NaN (their codes would be finite)
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const uint32_t w = k < 4 ? word_of(v0, k) : word_of(v1, k - 4);
            bad_q[k * 32 + lane] = without_infinities<T>(w);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = bad_q[k * 32 + lane] & ~not_finite<T>(bad_q[k * 32 + lane]);
          top = largest();
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = bad_q[k * 32 + lane];
        }
        // largest |q| 2^-e in [2^7, 2^8); queries below 2^-57 stay below that
        const int e = max(static_cast<int>(__float_as_uint(T::to_f(static_cast<uint16_t>(top))) >> 23) - 134, -64);
        const float mul = __int_as_float((127 - e) << 23);
        uint32_t w[L::TERMS][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t half[L::TERMS][2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // a pair as fp16: exact but for what lies 2^-31 below the row's largest
            const float2 f = T::to_f2(x[2 * k + h]);
            __half2 rest = __floats2half2_rn(f.x * mul, f.y * mul);
#pragma unroll
            for (int t = 0; t < L::TERMS; ++t) {
              const __half2_raw raw = rest;
              half[t][h] = __nv_cvt_halfraw2_to_fp8x2(raw, __NV_SATFINITE, __NV_E4M3);
              if (t + 1 < L::TERMS) {
                const __half2_raw code = __nv_cvt_fp8x2_to_halfraw2(half[t][h], __NV_E4M3);
                rest = __hsub2(rest, __half2(code));
              }
            }
          }
#pragma unroll
          for (int t = 0; t < L::TERMS; ++t) w[t][k] = half[t][0] | half[t][1] << 16;
        }
        const int off = D == 128 ? here * 128 + ((c ^ (here & 7)) << 4)
                                 : here * 64 + ((c ^ ((here >> 1) & 3)) << 4);
#pragma unroll
        for (int t = 0; t < L::TERMS; ++t)
          *reinterpret_cast<uint4 *>(dst + t * L::TILE8 + off) =
              make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        if (c == 0) q_exp[q * BM + here] = __int_as_float((127 + e) << 23);
      }
      fence_proxy_async_smem();
      warp_arrive(&bars[L::B_Q + q]);
    }
  };

  auto issuer = [&](const bool one) {
    constexpr uint32_t ID_QK = tc5::idesc_f16(KV8 ? 0 : AB<OPT>::v, 0, BM, BN);
    constexpr uint32_t ID_PV = tc5::idesc_f16(AB<OPT>::v, 1, BM, D);
    auto desc8 = [&](uint32_t off) -> uint64_t {
      return D == 128 ? tc5::sdesc_sw128(sbase + off, 16, 1024)
                      : tc5::sdesc_sw64(sbase + off, 16, 512);
    };
    const uint64_t q_desc = KV8 ? desc8(L::OFF_Q) : tc5::sdesc_sw128(sbase + L::OFF_Q, 16, 1024);
    const uint64_t k_desc = KV8 ? desc8(L::OFF_K8) : tc5::sdesc_sw128(sbase + L::OFF_K, 16, 1024);
    const uint64_t v_desc = tc5::sdesc_sw128(sbase + L::OFF_V, L::REG, 1024);
    // Scores run two tiles ahead of the products with V, across segments.  This
    // warp feeds the tensor core, whose queue is short: it waits as seldom as it
    // can, and its control flow is uniform, so that descriptors stay in uniform
    // registers (one lane on its own: 109 cycles a product against 64).
    Walk walk_q = walk;
    int tq = 0, jq = 0, nq = 0, segs = 0;  // scores: next tile, its place in its segment of nq
    bool keys = false;  // its keys have been seen to be there
    auto scores = [&]() -> bool {
      if (jq == nq) {
        Seg s;
        s.n = 0;
        walk_q.next(a, s);
        jq = 0;
        nq = __shfl_sync(0xffffffffu, s.n, 0);
        if (nq == 0) return true;  // no more
        if (!warp_wait(&bars[L::B_Q + segs % L::NQ], (segs / L::NQ) & 1, abort_flag, where))
          return false;
        ++segs;
      }
      const int sk = tq % NKT;
      if (!keys && !warp_wait(&bars[L::B_K + sk], (tq / NKT) & 1, abort_flag, where)) return false;
      tc5::fence_after_sync();
      const uint32_t sb = tmem + (tq & 1) * 128;
      if (one) {
        if constexpr (KV8) {
          const uint64_t qb = q_desc + static_cast<uint64_t>((((segs - 1) % L::NQ) * L::TERMS * L::TILE8) >> 4);
          const uint64_t kb = k_desc + static_cast<uint64_t>((sk * L::TILE8) >> 4);
#pragma unroll
          for (int e = 0; e < L::TERMS; ++e)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              tc5::mma_ss_f8(sb, qb + static_cast<uint64_t>((e * L::TILE8 + k * 32) >> 4),
                             kb + static_cast<uint64_t>(k * 2), ID_QK, (e | k) ? 1u : 0u);
        } else {
          const uint64_t qb = q_desc + static_cast<uint64_t>((((segs - 1) % L::NQ) * L::TILE) >> 4);
          const uint64_t kb = k_desc + static_cast<uint64_t>((sk * L::TILE) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = static_cast<uint64_t>(((k / 4) * L::REG + (k % 4) * 32) >> 4);
            tc5::mma_ss(sb, qb + off, kb + off, ID_QK, k > 0 ? 1u : 0u);
          }
        }
        tc5::commit(&bars[L::B_S + (tq & 1)]);
      }
      __syncwarp();
      ++tq;
      ++jq;
      return true;
    };
    // step u: the products with V of tile u - 2, then the scores of tile u
    int n = 0, j = 0;  // tiles of the products' segment, place in it
    for (int u = 0;; ++u) {
      if (u >= 2) {
        if (j == n) {
          Seg s;
          s.n = 0;
          walk.next(a, s);
          n = __shfl_sync(0xffffffffu, s.n, 0);
          j = 0;
          if (n == 0) return;
        }
        const int t = u - 2, sv = t % NV, buf = t & 1;
        // A wait costs this warp 120 cycles even where it is over: one look at the
        // three barriers of the step, a lane at each, and waits for those that were
        // not through (heads of 64 148 -> 145 us; over an 8-bit cache, whose weights
        // come later, 199 -> 205).
        uint32_t through = 0;
        if constexpr (!KV8) {
          uint64_t *bar = &bars[lane == 0 ? L::B_VG + sv : lane == 1 ? L::B_P + buf : L::B_K + tq % NKT];
          const uint32_t parity = (lane == 0 ? t / NV : lane == 1 ? t / 2 : tq / NKT) & 1;
          through = __ballot_sync(0xffffffffu, mbar_look(bar, parity));
          __syncwarp();
          keys = through & 4u;
        }
        if (!(through & 1u) && !warp_wait(&bars[L::B_VG + sv], (t / NV) & 1, abort_flag, where)) return;
        if (!(through & 2u) && !warp_wait(&bars[L::B_P + buf], (t / 2) & 1, abort_flag, where)) return;
        tc5::fence_after_sync();
        if (one) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t pb = tmem + buf * 128 + x * 64, ob = tmem + 256 + x * 128;
            // keys 64 x .. of the tile: 16 of them are 2048 bytes of V
            const uint64_t vb = v_desc + static_cast<uint64_t>((sv * L::TILE + x * 64 * 128) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc5::mma_ts(ob, pb + k * 8, vb + static_cast<uint64_t>(k * 128), ID_PV,
                          k > 0 || j > 0 ? 1u : 0u);
            if constexpr (TWO) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc5::mma_ts(ob, pb + 32 + k * 8, vb + static_cast<uint64_t>(k * 128), ID_PV, 1u);
            }
          }
          tc5::commit(&bars[L::B_EV + sv]);
        }
        __syncwarp();
        ++j;
      }
      if (!scores()) return;
    }
  };

  // Each of these warps takes ROWS of a V tile's rows.
  auto guard = [&]() {
    constexpr int ROWS = BN / kGuards;
    const int rows0 = (warp - 4) * ROWS;
    Seg s;
    int it = 0;
    for (int si = 0; walk.next(a, s); ++si) {
      const int calm0 = s.calm_from(a), calm1 = s.calm_to();
      // a mark that no segment under way uses: the other warps are at most NV tiles
      // ahead, and segments more than NV + 1 tiles ago have ended
      if (warp == 4 && lane == 0) flags[(si + kFlagSlots / 2) % kFlagSlots] = 0;
      for (int j = 0; j < s.n; ++j, ++it) {
        const int kv0 = s.s.kv_start + (s.j0 + j) * BN;
        const bool edge = j < calm0 || j >= calm1;
        const int lo = s.s.kv_lo - kv0, hi = s.s.L - kv0;  // rows outside [lo, hi) are hidden from all
        const int sv = it % NV;
        bool found = false;
        if constexpr (!KV8) {
          if (!warp_wait(&bars[L::B_V + sv], (it / NV) & 1, abort_flag, where)) return;
          if (edge) {
#pragma unroll 1
            for (int i = lane; i < L::NREG * ROWS * 8; i += 32) {
              const int r = rows0 + (i / 8) % ROWS;
              uint4 *p = reinterpret_cast<uint4 *>(smem + L::OFF_V + sv * L::TILE +
                                                   (i / (ROWS * 8)) * L::REG + r * 128) + i % 8;
              const uint4 u = *p;
              if (r < lo || r >= hi) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 m = make_uint4(not_finite<T>(u.x), not_finite<T>(u.y),
                                           not_finite<T>(u.z), not_finite<T>(u.w));
                if (m.x | m.y | m.z | m.w) {
                  *p = make_uint4(u.x & ~m.x, u.y & ~m.y, u.z & ~m.z, u.w & ~m.w);
                  found = true;
                }
              }
            }
            if (found) flags[si % kFlagSlots] = 1;
            fence_proxy_async_smem();
          }
        } else {
          // Lane (row r0, 16-channel group cc) widens 16 codes of a swizzled
          // row into two 16-byte chunks of the swizzled fp16 tile; lanes of
          // the upper half store them in the opposite order, so that the 8
          // lanes of a row never meet in a bank group.
          constexpr int LPR = D / 16, RPI = 32 / LPR;
          const int cc = lane % LPR, r0 = lane / LPR;
          const bool swap = cc >= LPR / 2;
          const int s8 = it % L::N8V;
          if (!warp_wait(&bars[L::B_V + s8], (it / L::N8V) & 1, abort_flag, where)) return;
          if (it >= NV && !warp_wait(&bars[L::B_EV + sv], ((it / NV) - 1) & 1, abort_flag, where))
            return;
          uint8_t *src = smem + L::OFF_V8 + s8 * L::TILE8 + rows0 * D;
          uint8_t *dst = smem + L::OFF_V + sv * L::TILE + (cc / 4) * L::REG + rows0 * 128;
          if (edge) {
            // bytes whose low 7 bits are all set are NaN
#pragma unroll 1
            for (int i = lane; i < ROWS * D / 4; i += 32) {
              uint32_t *p = reinterpret_cast<uint32_t *>(src) + i;
              const int r = rows0 + i / (D / 4);
              const uint32_t w = *p, t = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (r < lo || r >= hi) {
                *p = 0;
              } else if (t) {
                *p = w & ~((t >> 7) * 0xffu);
                found = true;
              }
            }
            __syncwarp();
          }
          const int k0 = (2 * cc) % 8;
#pragma unroll 2
          for (int i = 0; i < ROWS / RPI; ++i) {
            const int r = RPI * i + r0;  // rows0 is a multiple of 8
            const int chunk = D == 128 ? (cc ^ (r & 7)) : (cc ^ ((r >> 1) & 3));
            const uint4 u = *reinterpret_cast<const uint4 *>(src + r * D + chunk * 16);
            const uint2 h0 = e4m3x4_to_h4(u.x), h1 = e4m3x4_to_h4(u.y);
            const uint2 h2 = e4m3x4_to_h4(u.z), h3 = e4m3x4_to_h4(u.w);
            const uint4 c0 = make_uint4(h0.x, h0.y, h1.x, h1.y);
            const uint4 c1 = make_uint4(h2.x, h2.y, h3.x, h3.y);
            uint8_t *row = dst + r * 128;
            uint4 *p0 = reinterpret_cast<uint4 *>(row + ((k0 ^ (r & 7)) * 16));
            uint4 *p1 = reinterpret_cast<uint4 *>(row + (((k0 + 1) ^ (r & 7)) * 16));
            *(swap ? p1 : p0) = swap ? c1 : c0;
            *(swap ? p0 : p1) = swap ? c0 : c1;
          }
          if (found) flags[si % kFlagSlots] = 1;
          fence_proxy_async_smem();
          warp_arrive(&bars[L::B_E8V + s8]);
        }
        warp_arrive(&bars[L::B_VG + sv]);
      }
    }
  };

  auto softmax = [&]() {
    constexpr int HN = BN / 2;            // keys of a tile that this group takes
    const int x = warp >= 12 ? 1 : 0;     // the first ones or the last
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int row_node = r / a.QPK, row_head = r % a.QPK;
    const bool row_ok = r < tile_rows;
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem + L::OFF_MASK) + x * 128 + r;  // word w: [(w + 1) * 256]
    float2 *ml = reinterpret_cast<float2 *>(smem + L::OFF_ML);
    const bool rec = threadIdx.x == 256;
    if (rec && a.item_units > 0) a.record[blockIdx.x] = make_int4(0, 0, 0, 0);

    int here = 0;  // the node's position
    // The node's ancestors, those inside the window: a bit each.
    auto look_up = [&](const Seg &s, int node) {
#pragma unroll 1
      for (int w = 0; w < kMaskWords + 2; ++w) mask[w * 256] = 0;
      int depth = -1;
      if (row_ok && node < s.s.nodes) {
        for (int c = node; c >= 0;) {
          ++depth;
          if (a.window <= 0 || depth < a.window) mask[(c / 32 + 1) * 256] |= 1u << (c % 32);
          int p = __ldg(a.tb.parents + s.s.row + c);
          if (p < -1 || p >= c) {
            record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(s.s.row) + c);
            p = -1;
          }
          c = p;
        }
      }
      here = s.s.ctx + max(depth, 0);
    };

    const float *q_exp = reinterpret_cast<const float *>(smem + L::OFF_EXP);
    Seg s;
    int last_b = -1, last_node = -1;
    int base = 0;  // key tiles before the segment
    for (int si = 0; walk.next(a, s); ++si) {
      const int node = s.node0 + row_node;
      const bool valid = row_ok && node < s.s.nodes;
      const bool busy = __any_sync(0xffffffffu, valid);
      // a new sequence's path: behind the first tile's work where that can do without
      const bool fresh = s.b != last_b || s.node0 != last_node;
      const bool later = fresh && a.window <= 0 && !ALIBI && s.s.kv_start + (s.j0 + 1) * BN <= s.s.ctx;
      if (fresh && !later) look_up(s, node);
      last_b = s.b;
      last_node = s.node0;
      const int lo = a.window > 0 ? max(0, here - a.window + 1) : 0;
      const int head = s.g * a.QPK + row_head;
      float sl2 = a.scale_log2;
      const float slope = ALIBI && row_ok ? __ldg(a.alibi + head) * kLog2e : 0.f;
      // log2 units of a score and of the maximum: the scale is folded into the
      // exponent's FMA, with ALiBi into the scores
      float unit = ALIBI ? 1.f : sl2;
      float m = -INFINITY, l = 0.f;
      bool unset = true;  // some row of the warp has no maximum yet
      const int n = s.n, calm0 = s.calm_from(a), calm1 = s.calm_to();
      int kv0 = s.s.kv_start + s.j0 * BN + x * HN;
#pragma unroll 1
      for (int k = 0; k < n; ++k, kv0 += BN) {
        const int t = base + k, buf = t & 1;
        const uint32_t sb = tmem + lane_base + buf * 128 + x * HN;
        if (!warp_wait(&bars[L::B_S + buf], (t / 2) & 1, abort_flag, where)) return;
        // the scores are there: their keys are read.  (As a commit of the issuer's this
        // would hold the tensor core's queue.)
        if (rec) mbar_arrive(&bars[L::B_EK + t % NKT]);
        __syncwarp();
        tc5::fence_after_sync();
        if (KV8 && k == 0) {
          // scores are there, so their queries' scale is
          sl2 = fmaxf(sl2 * q_exp[si % L::NQ * BM + r], kTiniest);
          if (!ALIBI) unit = sl2;
        }
        if (busy) {
          uint32_t raw[HN];
#pragma unroll
          for (int c = 0; c < HN / 32; ++c)
            tc5::tmem_ld32(sb + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(raw + 32 * c));
          tc5::tmem_ld_wait();
          if (ALIBI) {
            const float b0 = slope * static_cast<float>(kv0 - here);
#pragma unroll
            for (int e = 0; e < HN; ++e)
              raw[e] = __float_as_uint(fmaf(__uint_as_float(raw[e]), sl2,
                                            fmaf(slope, static_cast<float>(e), b0)));
          }
          if (k < calm0 || k >= calm1) {
            const int off = kv0 - s.s.ctx;  // the node that stands at kv0
            // nodes of the row's path behind these keys: each puts a step of depth
            // between a key and the row
            int behind = 0;
            if (ALIBI) {
#pragma unroll 1
              for (int w = 0; w < kMaskWords; ++w) {
                const int z = off + HN - 32 * w;  // first bit behind
                const uint32_t b = mask[(w + 1) * 256];
                behind += __popc(z <= 0 ? b : z >= 32 ? 0u : b >> z);
              }
            }
#pragma unroll
            for (int c = HN / 32 - 1; c >= 0; --c) {
              const int p0 = kv0 + 32 * c, o = off + 32 * c;
              // the row's visible context positions and path nodes among these 32 keys
              const int from = max(lo - p0, 0), to = min(s.s.ctx - p0, 32);
              uint32_t in_ctx = 0, in_tree = 0;
              if (to > from) in_ctx = (to >= 32 ? ~0u : (1u << to) - 1u) & (~0u << from);
              if (o > -32 && o < 32 * kMaskWords) {
                const int w = (o + 32) / 32;  // one word of padding at each end
                in_tree = __funnelshift_r(mask[w * 256], mask[(w + 1) * 256], o & 31);
              }
              if (ALIBI && __any_sync(0xffffffffu, in_tree != 0)) {
#pragma unroll
                for (int e = 31; e >= 0; --e)
                  if (in_tree >> e & 1) {
                    // the key stands `behind` steps above the row, not at its place in the cache
                    const float place = static_cast<float>(p0 + e - here);
                    raw[32 * c + e] = __float_as_uint(__uint_as_float(raw[32 * c + e]) -
                                                      slope * (place + static_cast<float>(behind)));
                    ++behind;
                  }
              }
              const uint32_t seen = in_ctx | in_tree;
              if (__any_sync(0xffffffffu, seen != ~0u)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(seen >> e & 1)) raw[32 * c + e] = __float_as_uint(-INFINITY);
              }
            }
          }
          // p = 2^(score - mu), written over the scores as one or two terms; returns the sum
          auto exps = [&](float mu) -> float {
            const unsigned long long mul2 = f2pack(unit, unit), negmu2 = f2pack(-mu, -mu);
            const unsigned long long minus = f2pack(-1.f, -1.f);
            unsigned long long ps2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c = 0; c < HN / 32; ++c) {
              uint32_t hi[16], low[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float x0, x1;
                f2unpack(ffma2(f2pack(__uint_as_float(raw[32 * c + e]),
                                      __uint_as_float(raw[32 * c + e + 1])),
                               mul2, negmu2),
                         x0, x1);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                const unsigned long long p = f2pack(p0, p1);
                ps2[(e / 2) & 3] = fadd2(ps2[(e / 2) & 3], p);
                hi[e / 2] = OPT::from_f2(p0, p1);
                if constexpr (TWO) {
                  const float2 h = OPT::to_f2(hi[e / 2]);
                  float r0, r1;
                  f2unpack(ffma2(f2pack(h.x, h.y), minus, p), r0, r1);
                  low[e / 2] = OPT::from_f2(r0, r1);
                }
              }
              tc5::tmem_st16(sb + 16 * c, hi);
              if constexpr (TWO) tc5::tmem_st16(sb + HN / 2 + 16 * c, low);
            }
            float s0, s1;
            f2unpack(fadd2(fadd2(ps2[0], ps2[1]), fadd2(ps2[2], ps2[3])), s0, s1);
            return s0 + s1;
          };
          // The reference moves lazily: exponents are taken against m as it
          // stands; only where m is not set is the maximum looked for first, and
          // only where a row's sum is out of range again, and the pass repeated.
          auto largest = [&]() -> float {
            float pm[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) pm[q] = -INFINITY;
#pragma unroll
            for (int e = 0; e < HN; e += 2)
              pm[(e / 2) & 3] =
                  fmax3(pm[(e / 2) & 3], __uint_as_float(raw[e]), __uint_as_float(raw[e + 1]));
            return fmax3(pm[0], pm[1], fmaxf(pm[2], pm[3]));
          };
          if (unset) {
            const float mx = largest();
            if (m == -INFINITY) m = mx;
            unset = __any_sync(0xffffffffu, valid && m == -INFINITY);
          }
          float ps = exps(m == -INFINITY ? 0.f : m * unit - kLift);
          if (__any_sync(0xffffffffu, valid && !(ps <= 32768.f))) {
            float alpha = 1.f;
            const float mx = largest();
            const bool moved = valid && (mx - m) * unit > kLate;
            if (moved) {
              alpha = fast_exp2((m - mx) * unit);
              m = mx;
            }
            tc5::tmem_st_wait();  // a first pass's weights are written before they are replaced
            ps = exps(m == -INFINITY ? 0.f : m * unit - kLift);
            l *= alpha;
            if (__any_sync(0xffffffffu, moved) && k > 0) {
              // the accumulator holds the product before this one once that has completed
              // (the one before that has: these scores came after it)
              if (!warp_wait(&bars[L::B_EV + (t - 1) % NV], ((t - 1) / NV) & 1, abort_flag, where))
                return;
              tc5::fence_after_sync();
              const uint32_t ob = tmem + lane_base + 256 + x * 128;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc5::tmem_ld32(ob + 32 * c, o);
                tc5::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tc5::tmem_st32(ob + 32 * c, o);
              }
            }
          }
          l += ps;
          tc5::tmem_st_wait();
        }
        // the other group has read this accumulator's last segment
        if (k == 0 && si > 0 && !warp_wait(&bars[L::B_EPI], (si - 1) & 1, abort_flag, where))
          return;
        tc5::fence_before_sync();
        warp_arrive(&bars[L::B_P + buf]);
        if (k == 0 && later) look_up(s, node);
      }
      // after the last scores every warp is done with the queries and their scale
      warp_arrive(&bars[L::B_EQ + si % L::NQ]);
      base += n;

      // ---- the segment's end ----
      float top = m * unit;
      ml[x * 128 + r] = make_float2(top, l);
      warp_arrive(&bars[L::B_ML]);
      if (!warp_wait(&bars[L::B_ML], si & 1, abort_flag, where)) return;
      const float2 first = ml[r], last = ml[128 + r];
      top = fmaxf(first.x, last.x);
      // what the two accumulators are multiplied by
      float f0 = first.x == -INFINITY ? 0.f : fast_exp2(first.x - top);
      float f1 = last.x == -INFINITY ? 0.f : fast_exp2(last.x - top);
      l = f0 * first.y + f1 * last.y;
      if (!warp_wait(&bars[L::B_EV + (base - 1) % NV], ((base - 1) / NV) & 1, abort_flag, where))
        return;
      tc5::fence_after_sync();
      const bool whole = s.whole();
      if (whole) {
        const float inv = a.v_scale / l;  // l = 0: nothing but -infinity, NaN
        f0 *= inv;
        f1 *= inv;
      }
      const int at = blockIdx.x * 2 + (s.j0 > 0 ? 0 : 1);
      uint16_t *out = a.out + (static_cast<int64_t>(s.s.row + node) * a.H + head) * D;
      float *part = a.part_o + (static_cast<int64_t>(at) * (D / 4) * BM + r) * 4;
      constexpr int COLS = D / 2;  // each group stores its half of the row
      const int col0 = x * COLS;
      if (busy) {
        const uint32_t ob = tmem + lane_base + 256 + col0;
        // sums of 0 times the elements: NaN where one is not finite.  (Packed, as the merge
        // itself: ALiBi's kernels feel every instruction here, 64 contexts 594 us without the
        // look, 608 so, 650 with both in single ones.  An 8-bit cache needs no look, and
        // its merge is faster in single ones, 197 against 205 us for 128 contexts.)
        unsigned long long bad = 0ull;
#pragma unroll 1
        for (int c = 0; c < COLS / 32; ++c) {
          uint32_t o[32], o1[32];
          tc5::tmem_ld32(ob + 32 * c, o);
          tc5::tmem_ld32(ob + 128 + 32 * c, o1);
          tc5::tmem_ld_wait();
          if constexpr (KV8) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              auto pair = [&](const uint32_t *v) {
                return f2pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              };
              const unsigned long long both =
                  ffma2(pair(o1), f2pack(f1, f1), fmul2(pair(o), f2pack(f0, f0)));
              bad = ffma2(both, 0ull, bad);
              float even, odd;
              f2unpack(both, even, odd);
              o[e] = __float_as_uint(even);
              o[e + 1] = __float_as_uint(odd);
            }
          }
          if (valid && whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(out + col0 + 32 * c);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = T::from_f2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          } else if (valid) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4 *>(part + static_cast<int64_t>((col0 + 32 * c) / 4 + q) * BM * 4) =
                  make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
        if (!whole && x == 0 && valid)
          a.part_ml[static_cast<int64_t>(at) * BM + r] = make_float2(top, l);
        if constexpr (!KV8) {
          // of the rows with a finite score and no NaN or +infinity among them (the
          // others are NaN, or 0 here, as the formula says)
          const bool there = valid && l > 0.f && l < INFINITY;
          if (__any_sync(0xffffffffu, there && ((bad & 0x7fffffff7fffffffull) != 0)))
            set_not_finite<T, D>(a, s, col0, there, whole ? out : nullptr, part);
        }
        if (flags[si % kFlagSlots] && valid)
          add_not_finite<T, D, KV8>(a, s, lo, col0, COLS, mask, whole ? out : nullptr, part);
      }
      tc5::fence_before_sync();
      warp_arrive(&bars[L::B_EPI]);
      if (rec && s.j0 == 0 && !whole) {
        // how many of the following CTAs the rest of the item goes to
        const int64_t end = u1 - s.n + s.s.tiles;
        int parts = 0;
        const int next = blockIdx.x + 1;
        while (next + parts < shares && share_start(next + parts) < end) ++parts;
        a.record[blockIdx.x] = make_int4(s.b, s.g, parts, s.node0);
      }
    }
    tc5::fence_before_sync();
  };

  // the launch's registers, but where they are needed
  if (warp >= 8) {
    set_registers<true, kSoftmaxRegs>();
    softmax();
  } else if (warp >= 4) {
    set_registers<false, kGuardRegs>();
    guard();
  } else {
    set_registers<false, kIssueRegs>();
    if (warp == 0) {
      producer(std::false_type{});
      if (lane == 0) misc[kIssuedK] = issued;
    } else if (warp == 2) {
      producer(std::true_type{});
      if (lane == 0) misc[kIssuedV] = issued;
    } else if (KV8 && warp == 3) {
      queries();
    } else if (warp == 1) {
      const bool one = tc5::elect_one();
      issuer(one);
      __syncwarp();
      // every product that was issued has completed before tensor memory is released
      if (one) {
        tc5::commit(&bars[L::B_FIN]);
        mbar_wait_bounded(&bars[L::B_FIN], 0, where);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // copies in flight land before the CTA's memory goes away
    auto drain = [&](int bar, int stages, int issued) {
      for (int t = max(0, issued - stages); t < issued; ++t)
        mbar_wait_bounded(&bars[bar + t % stages], (t / stages) & 1, where);
    };
    drain(L::B_K, NKT, misc[kIssuedK]);
    drain(L::B_V, NVT, misc[kIssuedV]);
    if (!KV8) drain(L::B_Q, L::NQ, misc[kIssuedQ]);
  }
  __syncthreads();
  if (warp == 1) {
    tc5::fence_after_sync();
    tc5::tmem_dealloc<512>(tmem);
  }
}

// ---------------------------------------------------------------------------
// The parts of the items that were cut: block (CTA, 8 rows) merges
// those of the item that the CTA's last segment begins, if it begins one: the
// CTA's own second partial segment, then the first one of every following CTA.
// Thread = (row, four channels).
// ---------------------------------------------------------------------------
// An infinite value stays what it is where its part's weight vanishes.
__device__ __forceinline__ float scaled(float x, float w) {
  return fabsf(x) < INFINITY ? w * x : x;
}

template <class T, int D>
__global__ void __launch_bounds__(8 * D / 4) combine_kernel(const Args a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int cta = blockIdx.x;
  const int4 rec = a.record[cta];
  if (rec.z <= 0) return;
  const int r = blockIdx.y * 8 + threadIdx.x % 8;
  const int d4 = threadIdx.x / 8;
  const int node = rec.w + r / a.QPK;
  Seq s;
  bool bad;
  if (r >= a.tile_nodes * a.QPK || !seq_of(a, rec.x, s, bad) || node >= s.nodes) return;
  auto place = [&](int i) -> int64_t {
    return static_cast<int64_t>(cta + i) * 2 + (i == 0 ? 1 : 0);
  };
  float top = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int DEPTH = 8;  // parts whose loads are under way together
#pragma unroll 1
  for (int i0 = 0; i0 <= rec.z; i0 += DEPTH) {
    float2 ml[DEPTH];
    float4 p[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i <= rec.z) {
        ml[i] = a.part_ml[place(i0 + i) * BM + r];
        p[i] = *reinterpret_cast<const float4 *>(a.part_o + ((place(i0 + i) * (D / 4) + d4) * BM + r) * 4);
      }
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) now = fmaxf(now, ml[i].x);
    const float f = top == -INFINITY ? 0.f : fast_exp2(top - now);
    top = now;
    l *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = scaled(o[k], f);
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - top);
      l += w * ml[i].y;
      o[0] += scaled(p[i].x, w);
      o[1] += scaled(p[i].y, w);
      o[2] += scaled(p[i].z, w);
      o[3] += scaled(p[i].w, w);
    }
  }
  // nothing but -infinity is NaN, whatever the values
  const float inv = l > 0.f ? a.v_scale / l : __int_as_float(0x7fffffff);
  const int64_t row = static_cast<int64_t>(s.row + node) * a.H + rec.y * a.QPK + r % a.QPK;
  *reinterpret_cast<uint2 *>(a.out + row * D + d4 * 4) =
      make_uint2(T::from_f2(o[0] * inv, o[1] * inv), T::from_f2(o[2] * inv, o[3] * inv));
}

template <class T, int D, bool KV8, bool ALIBI>
static cudaError_t launch(const Args &a, int ctas, const CUtensorMap &qmap,
                          const CUtensorMap &kvmap, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> registers{0};
  auto kern = tree_tc_kernel<T, D, KV8, ALIBI>;
  cudaError_t e = allow_shared_memory(kern, done, 0);
  if (e != cudaSuccess) return e;
  if (registers.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    registers.store(at.numRegs, std::memory_order_release);
  }
  if (registers.load(std::memory_order_acquire) < kLaunchRegs) return cudaErrorLaunchOutOfResources;
  {
    PdlLaunch cfg(dim3(ctas), kThreads, Lay<T, D, KV8>::ALLOC, stream);
    e = cudaLaunchKernelEx(&cfg.c, kern, a, qmap, kvmap);
    if (e != cudaSuccess) return e;
  }
  if (a.item_units == 0) return cudaSuccess;  // no parts
  PdlLaunch cfg(dim3(ctas, BM / 8), 8 * D / 4, 0, stream);
  return cudaLaunchKernelEx(&cfg.c, combine_kernel<T, D>, a);
}

template <class T>
static cudaError_t launch_typed(const Args &a, int ctas, bool fp8, int D, const CUtensorMap &qmap,
                                const CUtensorMap &kvmap, cudaStream_t stream) {
#define PKV_TREE(DD, K8)                                                             \
  if (D == DD && fp8 == K8)                                                          \
    return a.alibi ? launch<T, DD, K8, true>(a, ctas, qmap, kvmap, stream)           \
                   : launch<T, DD, K8, false>(a, ctas, qmap, kvmap, stream);
  PKV_TREE(128, false)
  PKV_TREE(128, true)
  PKV_TREE(64, false)
  PKV_TREE(64, true)
#undef PKV_TREE
  return cudaErrorInvalidValue;
}

}  // namespace tree
}  // namespace pkv
