// Block bounds and block selection of the sparse decode.
//
// kv_block_bounds: per cache block and KV head the channelwise minimum lo and
// maximum hi of the block's keys.  paged_attn_select_blocks: per (sequence,
// KV head) the blocks with the largest
//     s_j = max_h sum_d max(q_hd lo_jd, q_hd hi_jd)  >=  max_h max_t q_h . k_jt,
// h over the query heads of the group, t over the keys of block j.
#include <climits>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

namespace pkv {
namespace sel {

// ---------------------------------------------------------------------------
// Packed minima and maxima that keep NaNs (a NaN key makes its channel's
// bounds NaN, as it makes the attention over that block NaN).
// ---------------------------------------------------------------------------
struct Bf16x2 {
  static __device__ __forceinline__ uint32_t mn(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mx(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};
struct F16x2 {
  static __device__ __forceinline__ uint32_t mn(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mx(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};

template <class T>
struct PackedOf;
template <>
struct PackedOf<BF16> {
  using type = Bf16x2;
};
template <>
struct PackedOf<FP16> {
  using type = F16x2;
};

struct BoundsArgs {
  uint8_t *bounds;
  const uint8_t *k_half;
  const int32_t *block_tables, *context_lens, *seq_lens;
  int64_t num_blocks;
  int64_t row_bytes;
  int max_blocks_per_seq, max_new, BS, D;
};

constexpr int kBoundsThreads = 128;

// A thread owns one 16-byte chunk of the key row of one touched block and runs
// down the block's written rows, 16 loads in flight; a sequence's chunks of its
// touched blocks are consecutive threads of grid row y.  Bound by reading the
// blocks' keys.  BULK: streaming loads, where the keys may be more than half of
// L2 (16 prompts of up to 8192 tokens, 8-bit, 77 MB: 14.8 against 16.2 us; a
// decode step's blocks, which L2 keeps, 3.8 against 2.4).
template <class P, bool KV8, bool BULK>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.y;
  const int L = __ldg(a.seq_lens + b);
  const int ctx = a.context_lens ? __ldg(a.context_lens + b) : 0;
  if (L < 0 || L > static_cast<int64_t>(a.max_blocks_per_seq) * a.BS || ctx < 0 || ctx > L ||
      L - ctx > a.max_new) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(PKV_ERR_BOUNDS, b);
    return;
  }
  if (ctx == L) return;
  const int chunks = static_cast<int>(a.row_bytes / 16);
  const int item = blockIdx.x * kBoundsThreads + threadIdx.x;
  const int lb = ctx / a.BS + item / chunks, c = item % chunks;
  if (lb > (L - 1) / a.BS) return;
  const int64_t at = static_cast<int64_t>(b) * a.max_blocks_per_seq + lb;
  const int pb = __ldg(a.block_tables + at);
  if (pb < 0 || pb >= a.num_blocks) {
    if (c == 0) record_error(PKV_ERR_BOUNDS, at);
    return;
  }
  const int rows = min(a.BS, L - lb * a.BS);
  const int head_bytes = KV8 ? a.D : 2 * a.D;
  const uint8_t *src = a.k_half + static_cast<int64_t>(pb) * a.BS * a.row_bytes + 16 * c;
  constexpr int W = KV8 ? 8 : 4;  // packed pairs per chunk
  uint32_t lo[W], hi[W];
  auto take = [&](const uint4 &u, uint32_t(&w)[W]) {
    if constexpr (KV8) {
      const uint32_t in[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 h = e4m3x4_to_h4(in[i]);
        w[2 * i] = h.x;
        w[2 * i + 1] = h.y;
      }
    } else {
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    }
  };
  constexpr int U = 16;  // rows in flight
  for (int r0 = 0; r0 < rows; r0 += U) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {  // rows past the end repeat the last one
      const uint4 *row = reinterpret_cast<const uint4 *>(src + min(r0 + i, rows - 1) * a.row_bytes);
      u[i] = BULK ? __ldcs(row) : *row;
    }
    if (r0 == 0) {
      take(u[0], lo);
      take(u[0], hi);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      uint32_t w[W];
      take(u[i], w);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        lo[k] = P::mn(lo[k], w[k]);
        hi[k] = P::mx(hi[k], w[k]);
      }
    }
  }
  const int h = 16 * c / head_bytes;
  uint8_t *dst = a.bounds + static_cast<int64_t>(pb) * 2 * a.row_bytes + h * 2 * head_bytes +
                 (16 * c - h * head_bytes);
  auto put = [&](uint8_t *p, const uint32_t(&w)[W]) {
    uint4 u;
    if constexpr (KV8) {  // back to the codes: exact, each is one's value
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t c01, c23;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c01) : "r"(w[2 * i]));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c23) : "r"(w[2 * i + 1]));
        o[i] = static_cast<uint32_t>(c01) | (static_cast<uint32_t>(c23) << 16);
      }
      u = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4 *>(p) = u;
  };
  put(dst, lo);
  put(dst + head_bytes, hi);
}

// ---------------------------------------------------------------------------
// Selection.  A cluster of C CTAs serves one (sequence, KV head): the candidate
// blocks (visible, not taken anyway) are cut into C consecutive pieces, every CTA
// scores one and writes the scores to the first CTA's shared memory, which alone
// goes on (barriers of one CTA cost a tenth of a cluster's).
//
// Scores.  With lo <= hi, max(q lo, q hi) = max(q, 0) hi + min(q, 0) lo, so the
// scores of 16 blocks and 8 query heads are one product of [16 blocks x 2D
// bounds] and [2D x 8 heads] on the tensor core (mma.sync m16n8k16: the step is
// bound by reading the bounds, 2D elements per block and KV head, and the
// tensor core keeps the instructions per bound low).  The 2D axis is taken in
// an order in which a lane's 16-byte loads are its A fragments as they stand.
//
// Exactness.  Products of 16-bit values are exact.  A product step sums 16 of
// them; how the tensor core rounds that is not documented, and it is taken to err
// by no more than 1.5 * 2^-19 of the largest (as if each term were cut at 2^-23 of it
// and the sum at 2^-24; the most measured, over random terms and those that a climb
// from them found, was half of that).  It starts from zero, so that errors scale with the step's terms, not the sum so far;
// the steps' sums are added in fp32, 8 at most in a row and the two rows' sums.
// With m_h the sum of the steps' largest |q| a score is within
//     E = max_h (1.5 * 2^-19 m_h + 9 * 2^-24 |q_h|_1) * max |bound|
// of the exact one, so only scores within 2E of the border can belong on its
// other side.  A histogram of 1024 equal bins finds the border's bin, everything
// above it and 2E is taken, and what lies in it or within 2E (one to five
// blocks as a rule) is listed and ranked.  Only where listed scores lie within
// 2E of the border's are those blocks scored again, in 64-bit fixed point (the
// FP64 units are few: the same in doubles took 8 us).  Where the list does not
// fit, all that is open is scored again and the border found digit by digit;
// where a score is not finite, the same in doubles.  That takes longer: one
// sequence of 2048 blocks 30 us with one score far outside the others' span, 480
// with all scores alike, against 12; 64 of 1024 .. 2048 blocks 231 and 1420
// against 79.
// ---------------------------------------------------------------------------
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;  // of the score histogram; later a bit per block
static_assert(PKV_SELECT_MAX_BLOCKS <= 32 * kBins, "a bit per block");
constexpr int kList = 256;   // open blocks that are ranked at once
constexpr size_t kStatic = 12 * 1024;  // the kernel's own shared memory, rounded up

struct Args {
  int32_t *selected;
  const uint16_t *query;
  const uint8_t *bounds;
  const int32_t *block_tables, *seq_lens;
  int64_t num_blocks;
  int max_selected, max_blocks_per_seq, max_seq_len, sink, recent;
  int H, KVH, QPK, BS, window;
  int cluster, keys_fit;
};

// Order-preserving 64-bit key of a score: NaN counts as +infinity, -0 as 0.
__device__ __forceinline__ unsigned long long key_of(double s) {
  if (s != s) s = INFINITY;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Exclusive prefix sum of v over the CTA's W warps.
template <int W>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // scratch may still be read from the last scan
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < warp) base += scratch[w];
  return base + x - v;
}

// One bound's value from its element.
template <class T, bool KV8>
__device__ __forceinline__ float bound_value(const uint8_t *p, int i) {
  if constexpr (KV8) {
    const uint2 h = e4m3x4_to_h4(p[i]);
    return FP16::to_f2(h.x).x;
  } else {
    return T::to_f(reinterpret_cast<const uint16_t *>(p)[i]);
  }
}

// The score of the block with bounds `row`, by a whole warp, as an order-preserving
// key.  In doubles, for scores that may not be finite: products exact, sums off
// by 2^-53 of their terms.
template <class T, int D, bool KV8>
__device__ __noinline__ unsigned long long key_double(const uint8_t *row, const uint16_t *q,
                                                      int qpk) {
  const int lane = threadIdx.x & 31;
  double best = -INFINITY;
  bool nan = false;
  for (int h = 0; h < qpk; ++h) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int d = lane + 32 * k;
      const double qd = T::to_f(__ldg(q + h * D + d));
      const double x = qd * bound_value<T, KV8>(row, d), y = qd * bound_value<T, KV8>(row, D + d);
      s += (x > y || x != x) ? x : y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = s > best ? s : best;
  }
  return key_of(nan ? INFINITY : best);
}

// A finite 16-bit value as m * 2^e.
__device__ __forceinline__ void split_value(uint32_t x, int &m, int &e, BF16) {
  const int f = (x >> 7) & 255;
  m = (x & 127) | (f ? 128 : 0);
  e = max(f, 1) - 134;
  if (x & 0x8000u) m = -m;
}
__device__ __forceinline__ void split_value(uint32_t x, int &m, int &e, FP16) {
  const int f = (x >> 10) & 31;
  m = (x & 1023) | (f ? 1024 : 0);
  e = max(f, 1) - 25;
  if (x & 0x8000u) m = -m;
}

// The same for finite scores, in 64-bit fixed point with 54 bits below 2^top,
// which no product reaches: sums of 128 products do not overflow and do not
// depend on their order.  Terms are cut below 2^(top - 54); products have 22 bits
// at most, so those within 2^32 of the largest possible one are exact.
template <class T, int D, bool KV8>
__device__ __noinline__ unsigned long long key_fixed(const uint8_t *row, const uint16_t *q, int qpk,
                                                     int top) {
  using MT = std::conditional_t<KV8, FP16, T>;
  constexpr int E = D / 32;  // channels per lane
  const int lane = threadIdx.x & 31;
  int mb[2][E], eb[2][E];  // this lane's minima and maxima as m * 2^e
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t w[(E + 1) / 2];
    if constexpr (KV8) {
      uint32_t c;  // E codes
      if constexpr (E == 4) c = __ldg(reinterpret_cast<const uint32_t *>(row + x * D) + lane);
      else c = __ldg(reinterpret_cast<const uint16_t *>(row + x * D) + lane);
      const uint2 h = e4m3x4_to_h4(c);
      w[0] = h.x;
      if constexpr (E == 4) w[1] = h.y;
    } else if constexpr (E == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + x * D * 2) + lane);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t *>(row + x * D * 2) + lane);
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
      split_value((w[k / 2] >> (16 * (k & 1))) & 0xffffu, mb[x][k], eb[x][k], MT{});
  }
  long long best = LLONG_MIN;
  for (int h0 = 0; h0 < qpk; h0 += 4) {  // four heads' chains side by side
    uint32_t w[4][E / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t *qh = q + min(h0 + i, qpk - 1) * D;
      if constexpr (E == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(qh) + lane);
        w[i][0] = v.x;
        w[i][1] = v.y;
      } else {
        w[i][0] = __ldg(reinterpret_cast<const uint32_t *>(qh) + lane);
      }
    }
    long long s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = 0;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const uint32_t qb = (w[i][k / 2] >> (16 * (k & 1))) & 0xffffu;
        const bool neg = qb & 0x8000u;  // max(q lo, q hi) is that of q's sign
        int mq, eq;
        split_value(qb, mq, eq, T{});
        const int p = mq * (neg ? mb[0][k] : mb[1][k]);
        const int sh = eq + (neg ? eb[0][k] : eb[1][k]) - top + 54;  // p * 2^sh is below 2^54
        const long long m = abs(p);
        const long long v = p == 0 ? 0 : sh >= 0 ? m << min(sh, 63) : m >> min(-sh, 63);
        s[i] += p < 0 ? -v : v;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    best = max(best, max(max(s[0], s[1]), max(s[2], s[3])));
  }
  return static_cast<unsigned long long>(best) ^ (1ull << 63);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// B fragments of one m16n8k16 step after another for heads 8 h8 .. + 7: k-step
// s of lane (g, tq) covers elements 4 u .. 4 u + 3 of the bounds row's 16-byte
// chunk 4 (s / P) + tq, u = s % P, P steps per chunk; min(q, 0) against minima,
// max(q, 0) against maxima.  Also for the lane's head: the error's factor
// 1.5 * 2^-19 m + 9 * 2^-24 |q|_1, the largest |q| and, where bf16 queries meet fp8 bounds,
// the power of two that they are scaled down by (the largest of a head becomes
// [2^14, 2^15) in fp16, which is exact for components within 2^28 of it and off
// by 2^-39 of it below).
template <class T, int D, bool KV8>
__device__ __forceinline__ void make_b(const Args &a, const uint16_t *q, int h8,
                                       uint2 (&bq)[2 * D / 16], float &factor, float &top,
                                       float &unit) {
  constexpr int kSteps = 2 * D / 16, kPer = KV8 ? 4 : 2, kElems = KV8 ? 16 : 8;
  using Q = typename PackedOf<T>::type;
  const int lane = threadIdx.x & 31, h = h8 * 8 + (lane >> 2);
  auto element = [&](int s) { return (4 * (s / kPer) + (lane & 3)) * kElems + 4 * (s % kPer); };
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    bq[s] = h < a.QPK ? __ldg(reinterpret_cast<const uint2 *>(q + h * D + (element(s) & (D - 1))))
                      : make_uint2(0u, 0u);
  // elements below D (minima) are the first half of the steps, and the same
  // channels come again in the second
  float sum = 0.f, steps = 0.f;
  top = 0.f;
#pragma unroll
  for (int s = 0; s < kSteps / 2; ++s) {
    const float2 x = T::to_f2(bq[s].x), y = T::to_f2(bq[s].y);
    const float m = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
    sum += (fabsf(x.x) + fabsf(x.y)) + (fabsf(y.x) + fabsf(y.y));
    // the largest of the step's 16 channels; 2 m covers both halves' step
    float st = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    st = fmaxf(st, __shfl_xor_sync(0xffffffffu, st, 2));
    steps += st;
    top = fmaxf(top, st);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  // (2 m: both halves; a little more for the sums made here)
  factor = 1.001f * (steps * 0x1.8p-18f + sum * 0x1.2p-21f);
  unit = 1.f;
  if constexpr (KV8 && std::is_same<T, BF16>::value) {
    const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // top in [2^e, 2^(e+1))
    if (top > 0.f && e < 128)
      unit = __uint_as_float(static_cast<uint32_t>(min(max(e - 14, -126), 126) + 127) << 23);
  }
  const float inv = 1.f / unit;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {  // NaNs stay
    if (s < kSteps / 2) bq[s] = make_uint2(Q::mn(bq[s].x, 0u), Q::mn(bq[s].y, 0u));
    else bq[s] = make_uint2(Q::mx(bq[s].x, 0u), Q::mx(bq[s].y, 0u));
    if constexpr (KV8 && std::is_same<T, BF16>::value) {
      const float2 x = T::to_f2(bq[s].x), y = T::to_f2(bq[s].y);
      bq[s] = make_uint2(FP16::from_f2(x.x * inv, x.y * inv), FP16::from_f2(y.x * inv, y.y * inv));
    }
  }
}

// Blocks p0 + i, i < n, for which taken(i) to `out` in order; tie(i): taken too
// as long as `left` of them are not used up.
template <int W, class F, class G>
__device__ __forceinline__ void put_taken(int32_t *out, uint32_t left, int p0, int n,
                                          uint32_t (*scratch)[2], const F &taken, const G &tie) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = (n + 32 * W - 1) / (32 * W) * 32;  // consecutive blocks per warp
  const int w0 = warp * seg, w1 = min(w0 + seg, n);
  uint32_t up = 0, at = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    up += __popc(__ballot_sync(0xffffffffu, i < w1 && taken(i)));
    at += __popc(__ballot_sync(0xffffffffu, i < w1 && tie(i)));
  }
  if (lane == 0) {
    scratch[warp][0] = up;
    scratch[warp][1] = at;
  }
  __syncthreads();
  uint32_t ties = 0, place = 0;
  for (int w = 0; w < warp; ++w) {
    place += scratch[w][0];
    ties += scratch[w][1];
  }
  place += min(ties, left);
  const uint32_t below = (1u << lane) - 1;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool t = i < w1 && tie(i);
    const uint32_t tm = __ballot_sync(0xffffffffu, t);
    const bool take = i < w1 && (taken(i) || (t && ties + __popc(tm & below) < left));
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (take) out[place + __popc(m & below)] = p0 + i;
    place += __popc(m);
    ties += __popc(tm);
  }
}

// W warps: 8, two CTAs to an SM, or 4, four of them.
template <class T, int D, bool KV8, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) select_kernel(const Args a) {
  constexpr int kWarps = W, kThreads = 32 * W;
  static_assert(kBins % (4 * kThreads) == 0 && 256 % kThreads == 0, "whole 16-byte loads of bins");
  using MT = std::conditional_t<KV8, FP16, T>;  // operand type
  constexpr int kRowBytes = 2 * D * (KV8 ? 1 : 2);
  constexpr int kSteps = 2 * D / 16;
  constexpr int kLoads = kRowBytes / 64;          // 16-byte loads of a lane per row
  constexpr int kStepsPerLoad = kSteps / kLoads;  // 2, or 4 of 8-bit codes
  constexpr bool kScaled = KV8 && std::is_same<T, BF16>::value;
  constexpr int U = 8 / kLoads;  // tiles of 16 blocks that a warp has in flight (64 registers' worth)
  using P = typename PackedOf<MT>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  const int heads8 = (a.QPK + 7) / 8;
  // of heads 8 and up: fragments [heads8 - 1][kSteps][32], scales [heads8 - 1][8]
  uint2 *sb = reinterpret_cast<uint2 *>(smem);
  float *sunit = reinterpret_cast<float *>(sb + static_cast<size_t>(heads8 - 1) * kSteps * 32);
  // the first CTA's: every candidate's score, or its 64-bit key
  float *score = sunit + (heads8 - 1) * 8;
  unsigned long long *keys = reinterpret_cast<unsigned long long *>(score);
  __shared__ __align__(16) uint32_t bins[kBins];
  // of every warp: -smallest, largest score, largest |bound|, flags
  __shared__ float4 span[kMaxCluster * kWarps];
  __shared__ float2 list[kList];            // open blocks: score, place (as bits)
  __shared__ unsigned long long list_key[kList];
  __shared__ uint32_t scratch[kWarps], warp_counts[kWarps][2];
  __shared__ float wred[2][kWarps];
  __shared__ uint32_t pick[2];  // the bin or digit found, the rank left within it
  __shared__ uint32_t s_up, s_open, s_sure, s_near;
  __shared__ float s_border;

  const int kvh = blockIdx.y, b = blockIdx.z;
  const uint32_t rank = cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
  if (tid == 0) s_up = s_open = s_sure = s_near = 0;
  int32_t *out = a.selected + (static_cast<int64_t>(b) * a.KVH + kvh) * a.max_selected;
  grid_dependency_wait();
  grid_launch_dependents();

  int L = __ldg(a.seq_lens + b);
  const uint16_t *qg = a.query + (static_cast<int64_t>(b) * a.H + kvh * a.QPK) * D;
  uint2 bq[kSteps];
  float factor, qtop, unit;  // of E, the largest of all heads; the largest |q|
  make_b<T, D, KV8>(a, qg, 0, bq, factor, qtop, unit);
  if (L < 0 || L > a.max_seq_len || L > static_cast<int64_t>(a.max_blocks_per_seq) * a.BS) {
    if (rank == 0 && kvh == 0 && tid == 0) record_error(PKV_ERR_BOUNDS, b);
    L = 0;
  }
  const int nblk = (L + a.BS - 1) / a.BS;
  const int first = a.window > 0 ? max(0, L - a.window) / a.BS : 0;
  if (nblk - first <= a.max_selected) {  // all of the visible blocks (none: L = 0)
    if (rank == 0)
      for (int i = tid; i < a.max_selected; i += kThreads) out[i] = first + i < nblk ? first + i : -1;
    return;
  }
  // taken anyway: [first, c_lo) and [c_hi, nblk); candidates [c_lo, c_hi)
  const int c_hi = max(first, nblk - a.recent);
  const int c_lo = min(max(a.sink, first), c_hi);
  const int n_front = c_lo - first, n_back = nblk - c_hi;
  const int need = a.max_selected - n_front - n_back;  // >= 0, < candidates
  if (rank == 0) {
    for (int i = tid; i < n_front; i += kThreads) out[i] = first + i;
    for (int i = tid; i < n_back; i += kThreads) out[a.max_selected - n_back + i] = c_hi + i;
  }
  if (need == 0) return;
  const bool alone = a.cluster == 1;
  if (!alone) cluster_arrive();  // this CTA runs: it may be written to
  const int n = c_hi - c_lo;
  // this CTA's piece
  const int per = (n + a.cluster - 1) / a.cluster;
  const int i0 = min(static_cast<int>(rank) * per, n), i1 = min(i0 + per, n);

  // ---- scores: a warp takes U tiles of 16 blocks at a time -----------------------
  const int32_t *table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq + c_lo;
  const int g = lane >> 2, tq = lane & 3;
  // (rows past the last block repeat it)
  auto entry = [&](int i) { return i0 < i1 ? __ldg(table + min(i, i1 - 1)) : 0; };
  int pb0[U], pb1[U];
#pragma unroll
  for (int v = 0; v < U; ++v) {
    pb0[v] = entry(i0 + (warp * U + v) * 16 + g);
    pb1[v] = entry(i0 + (warp * U + v) * 16 + g + 8);
  }
  factor = warp_max(factor);
  qtop = warp_max(qtop);
  const float unit0 = __shfl_sync(0xffffffffu, unit, 8 * tq);
  const float unit1 = __shfl_sync(0xffffffffu, unit, 8 * tq + 4);
  if (heads8 > 1) {
    for (int h8 = 1 + warp; h8 < heads8; h8 += kWarps) {
      uint2 bh[kSteps];
      float f, top;
      make_b<T, D, KV8>(a, qg, h8, bh, f, top, unit);
      factor = fmaxf(factor, warp_max(f));
      qtop = fmaxf(qtop, warp_max(top));
#pragma unroll
      for (int s = 0; s < kSteps; ++s) sb[((h8 - 1) * kSteps + s) * 32 + lane] = bh[s];
      if (tq == 0) sunit[(h8 - 1) * 8 + g] = unit;
    }
    if (lane == 0) {
      wred[0][warp] = factor;
      wred[1][warp] = qtop;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      factor = fmaxf(factor, wred[0][w]);
      qtop = fmaxf(qtop, wred[1][w]);
    }
  }
  float mn = INFINITY, mx = -INFINITY;
  float nan = 0.f;      // 0, or NaN after a score that is not finite
  bool bad = false;     // a bad entry
  // the smallest minima, the largest maxima (with 0), packed
  uint32_t blo[2] = {0, 0}, bhi[2] = {0, 0};
  bool started = alone;
  for (int t = i0 + warp * 16 * U; t < i1; t += kWarps * 16 * U) {
    uint4 u0[U][kLoads], u1[U][kLoads];
    bool bad0[U], bad1[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      bad0[v] = pb0[v] < 0 || pb0[v] >= a.num_blocks;
      bad1[v] = pb1[v] < 0 || pb1[v] >= a.num_blocks;
      if (bad0[v] || bad1[v]) {
        bad = true;
        const int at = t + 16 * v + g + (bad0[v] ? 0 : 8);
        if (at < i1 && tq == 0)
          record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(b) * a.max_blocks_per_seq + c_lo + at);
      }
      const uint4 *r0 = reinterpret_cast<const uint4 *>(
          a.bounds + (static_cast<int64_t>(bad0[v] ? 0 : pb0[v]) * a.KVH + kvh) * kRowBytes) + tq;
      const uint4 *r1 = reinterpret_cast<const uint4 *>(
          a.bounds + (static_cast<int64_t>(bad1[v] ? 0 : pb1[v]) * a.KVH + kvh) * kRowBytes) + tq;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {  // (read once: 404 MB in 80 us, 84 without the hint)
        u0[v][i] = __ldcs(r0 + 4 * i);
        u1[v][i] = __ldcs(r1 + 4 * i);
      }
    }
    // the next tiles' entries arrive while these are worked on
#pragma unroll
    for (int v = 0; v < U; ++v) {
      pb0[v] = entry(t + (kWarps * U + v) * 16 + g);
      pb1[v] = entry(t + (kWarps * U + v) * 16 + g + 8);
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      if (t + 16 * v >= i1) break;
      float best0 = -INFINITY, best1 = -INFINITY;
      for (int h8 = 0; h8 < heads8; ++h8) {
        unsigned long long c01[2] = {0, 0}, c23[2] = {0, 0};  // packed fp32 pairs, even and odd steps
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t w0[4] = {u0[v][i].x, u0[v][i].y, u0[v][i].z, u0[v][i].w};
          const uint32_t w1[4] = {u1[v][i].x, u1[v][i].y, u1[v][i].z, u1[v][i].w};
#pragma unroll
          for (int u = 0; u < kStepsPerLoad; ++u) {
            const int s = i * kStepsPerLoad + u;
            uint32_t f0[2], f1[2];
            if constexpr (KV8) {
              const uint2 x = e4m3x4_to_h4(w0[u]), y = e4m3x4_to_h4(w1[u]);
              f0[0] = x.x;
              f0[1] = x.y;
              f1[0] = y.x;
              f1[1] = y.y;
            } else {
              f0[0] = w0[2 * u];
              f0[1] = w0[2 * u + 1];
              f1[0] = w1[2 * u];
              f1[1] = w1[2 * u + 1];
            }
            if (h8 == 0) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (s < kSteps / 2) blo[k] = P::mn(blo[k], P::mn(f0[k], f1[k]));
                else bhi[k] = P::mx(bhi[k], P::mx(f0[k], f1[k]));
              }
            }
            float d[4];
            const uint2 q2 = h8 == 0 ? bq[s] : sb[((h8 - 1) * kSteps + s) * 32 + lane];
            mma_16816<MT>(d, f0[0], f1[0], f0[1], f1[1], q2.x, q2.y, 0.f, 0.f, 0.f, 0.f);
            c01[s & 1] = fadd2(c01[s & 1], f2pack(d[0], d[1]));
            c23[s & 1] = fadd2(c23[s & 1], f2pack(d[2], d[3]));
          }
        }
        // heads 8 h8 + 2 tq, + 1 of blocks g (c[0], c[1]) and g + 8
        float c[4];
        f2unpack(fadd2(c01[0], c01[1]), c[0], c[1]);
        f2unpack(fadd2(c23[0], c23[1]), c[2], c[3]);
        if constexpr (kScaled) {
          const float e0 = h8 == 0 ? unit0 : sunit[(h8 - 1) * 8 + 2 * tq];
          const float e1 = h8 == 0 ? unit1 : sunit[(h8 - 1) * 8 + 2 * tq + 1];
          c[0] *= e0;
          c[2] *= e0;
          c[1] *= e1;
          c[3] *= e1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) nan = fmaf(c[k], 0.f, nan);  // 0 times infinity or NaN
        if (h8 * 8 + 2 * tq < a.QPK) {
          best0 = fmaxf(best0, c[0]);
          best1 = fmaxf(best1, c[2]);
        }
        if (h8 * 8 + 2 * tq + 1 < a.QPK) {
          best0 = fmaxf(best0, c[1]);
          best1 = fmaxf(best1, c[3]);
        }
      }
      best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, 1));
      best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, 1));
      best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, 2));
      best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, 2));
      // (rows past the last block are the last block's)
      mn = fminf(mn, fminf(bad0[v] ? INFINITY : best0, bad1[v] ? INFINITY : best1));
      mx = fmaxf(mx, fmaxf(bad0[v] ? -INFINITY : best0, bad1[v] ? -INFINITY : best1));
      // a bad entry: -infinity, below every other score and taken last
      if (bad0[v]) best0 = -INFINITY;
      if (bad1[v]) best1 = -INFINITY;
      if (!started) {
        cluster_wait();  // the first CTA runs
        started = true;
      }
      // lanes 0 and 1 of a quad write its two blocks
      const int at = t + 16 * v + g + 8 * (tq & 1);
      const float mine = tq == 0 ? best0 : best1;
      if (tq < 2 && at < i1) {
        if (alone) score[at] = mine;
        else cluster_store(score + at, mine, 0);
      }
    }
  }
  if (!started) cluster_wait();
  {
    const float2 lo = MT::to_f2(P::mn(blo[0], blo[1])), hi = MT::to_f2(P::mx(bhi[0], bhi[1]));
    const float w[4] = {warp_max(-mn), warp_max(mx),
                        warp_max(fmaxf(fmaxf(-lo.x, -lo.y), fmaxf(hi.x, hi.y))),
                        __any_sync(0xffffffffu, nan != nan) ? 2.f
                        : __any_sync(0xffffffffu, bad)      ? 1.f
                                                            : 0.f};
    float *mine = reinterpret_cast<float *>(&span[rank * kWarps + warp]);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (alone) mine[k] = w[k];
        else cluster_store(mine + k, w[k], 0);
    }
  }
  if (alone) {
    __syncthreads();
  } else {
    cluster_arrive();
    if (rank != 0) return;  // nobody reads this CTA's shared memory
    cluster_wait();
  }

  // ---- the first CTA: the span of all scores ----------------------------------------
  float4 sp = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  for (int k = lane; k < a.cluster * kWarps; k += 32) {
    sp.x = fmaxf(sp.x, span[k].x);
    sp.y = fmaxf(sp.y, span[k].y);
    sp.z = fmaxf(sp.z, span[k].z);
    sp.w = fmaxf(sp.w, span[k].w);
  }
  mn = -warp_max(sp.x);
  mx = warp_max(sp.y);
  const float btop = warp_max(sp.z);
  const float flags = warp_max(sp.w);
  const bool odd = flags == 2.f;
  // (products below fp32's range may be lost altogether; none are if all are 0)
  const float err = qtop == 0.f || btop == 0.f ? 0.f : factor * btop + 1e-36f;
  if (flags == 0.f && err == 0.f) {  // all scores are 0
    for (int i = tid; i < need; i += kThreads) out[n_front + i] = c_lo + i;
    return;
  }
  const float inv = mx > mn ? kBins / (mx - mn) : 0.f;
  bool fits = !odd && mx >= mn && mx - mn < INFINITY && err < INFINITY && inv < INFINITY;
  float t_lo = -INFINITY, t_hi = INFINITY;  // above t_hi taken, below t_lo not
  // 2^top: more than any product
  const int top =
      static_cast<int>(__float_as_uint(qtop) >> 23) + static_cast<int>(__float_as_uint(btop) >> 23) - 252;
  auto key = [&](int i) -> unsigned long long {  // a bad entry's is below every score's
    const int pb = __ldg(table + i);
    if (pb < 0 || pb >= a.num_blocks) return 0;
    const uint8_t *row = a.bounds + (static_cast<int64_t>(pb) * a.KVH + kvh) * kRowBytes;
    return odd ? key_double<T, D, KV8>(row, qg, a.QPK) : key_fixed<T, D, KV8>(row, qg, a.QPK, top);
  };
  if (fits) {
    // ---- the border's bin -----------------------------------------------------------
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads)
      atomicAdd(&bins[max(0, min(kBins - 1, static_cast<int>((score[i] - mn) * inv)))], 1u);
    __syncthreads();
    constexpr int kPer = kBins / kThreads;  // bins per thread, from the highest down
    uint32_t cnt[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(&bins[kBins - kPer * (tid + 1) + k]);
      cnt[kPer - 1 - k] = v.x;
      cnt[kPer - 2 - k] = v.y;
      cnt[kPer - 3 - k] = v.z;
      cnt[kPer - 4 - k] = v.w;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += cnt[k];
    uint32_t above = block_scan<W>(sum, scratch);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (above < static_cast<uint32_t>(need) && static_cast<uint32_t>(need) <= above + cnt[k])
        pick[0] = kBins - 1 - kPer * tid - k;
      above += cnt[k];
    }
    __syncthreads();
    // the bin's edges, out by its arithmetic's rounding (a few 2^-24 of the
    // span and of the values) and by 2 E
    const float w = (mx - mn) / kBins;
    const float slack = 2.f * err + (mx - mn) * 0x1p-20f + fmaxf(fabsf(mn), fabsf(mx)) * 0x1p-21f;
    t_lo = pick[0] == 0 ? -INFINITY : mn + w * static_cast<float>(pick[0]) - slack;
    t_hi = mn + w * static_cast<float>(pick[0] + 1) + slack;
    // ---- taken (a bit each in `bins`), open, not taken ------------------------------
    uint32_t *taken = bins;
    uint32_t up = 0;
    for (int i = tid; i - lane < n; i += kThreads) {
      const float s = i < n ? score[i] : -INFINITY;
      const uint32_t m = __ballot_sync(0xffffffffu, i < n && s > t_hi);
      if (lane == 0) taken[i >> 5] = m;
      up += __popc(m);
      if (i < n && s <= t_hi && s >= t_lo) {
        const uint32_t at = atomicAdd(&s_open, 1u);
        if (at < kList) list[at] = make_float2(s, __int_as_float(i));
      }
    }
    if (lane == 0 && up) atomicAdd(&s_up, up);
    __syncthreads();
    const uint32_t open = s_open, left = need - s_up;
    fits = open <= kList;
    if (fits) {
      // the border: the left-th largest of the listed scores
      for (uint32_t k = tid; k < open; k += kThreads) {
        const float2 e = list[k];
        uint32_t ahead = 0;
        for (uint32_t j = 0; j < open; ++j)
          ahead += list[j].x > e.x ||
                   (list[j].x == e.x && __float_as_int(list[j].y) < __float_as_int(e.y));
        if (ahead == left - 1) s_border = e.x;
      }
      __syncthreads();
      const float hi = s_border + 2.f * err, lo = s_border - 2.f * err;
      for (uint32_t k = tid; k < open; k += kThreads) {
        if (list[k].x > hi) atomicAdd(&s_sure, 1u);
        else if (list[k].x >= lo) atomicAdd(&s_near, 1u);
      }
      __syncthreads();
      const bool all_near = s_sure + s_near == left;  // none of the near ones stays out
      if (!all_near) {
        for (uint32_t k = warp; k < open; k += kWarps) {
          const float s = list[k].x;
          unsigned long long x = s > hi ? ~0ull : 0;
          if (s <= hi && s >= lo) x = key(__float_as_int(list[k].y));
          if (lane == 0) list_key[k] = x;
        }
        __syncthreads();
      }
      for (uint32_t k = tid; k < open; k += kThreads) {
        const int at = __float_as_int(list[k].y);
        bool take = list[k].x >= lo;
        if (!all_near && take) {
          uint32_t ahead = 0;
          for (uint32_t j = 0; j < open; ++j)
            ahead += list_key[j] > list_key[k] ||
                     (list_key[j] == list_key[k] && __float_as_int(list[j].y) < at &&
                      list[j].x >= lo);
          take = ahead < left;
        }
        if (take) atomicOr(&taken[at >> 5], 1u << (at & 31));
      }
      __syncthreads();
      const int words = (n + 31) / 32, each = (words + kThreads - 1) / kThreads;
      const int k0 = min(tid * each, words), k1 = min(k0 + each, words);
      uint32_t count = 0;
      for (int k = k0; k < k1; ++k) count += __popc(taken[k]);
      uint32_t place = block_scan<W>(count, scratch);
      for (int k = k0; k < k1; ++k)
        for (uint32_t m = taken[k]; m; m &= m - 1)
          out[n_front + place++] = c_lo + 32 * k + __ffs(m) - 1;
      return;
    }
  }

  // ---- all that is open in 64 bits, the rest above or below all keys -------------------
  // where there is room the keys are kept (in place of the scores, from the last
  // block down: key i covers scores 2 i and 2 i + 1), else made again when asked for
  auto key_at = [&](int i) {  // by a whole warp
    const float s = score[i];
    return s > t_hi ? ~0ull : s < t_lo ? 0ull : key(i);
  };
  const bool kept = a.keys_fit != 0;
  if (kept) {
    for (int base = (n - 1) / kWarps * kWarps; base >= 0; base -= kWarps) {
      const int i = base + warp;
      unsigned long long x = 0;
      if (i < n) x = key_at(i);
      __syncthreads();  // scores base .. base + kWarps - 1 are read
      if (i < n && lane == 0) keys[i] = x;
      __syncthreads();
    }
  }
  // the need-th largest key, 8 bits at a time
  unsigned long long border = 0, mask = 0;
  uint32_t left = need;  // how many of the keys that match the prefix are taken
  for (int shift = 56; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int i = tid; i < 256; i += kThreads) bins[i] = 0;
    __syncthreads();
    if (kept) {
      for (int i = tid; i < n; i += kThreads)
        if ((keys[i] & mask) == border) atomicAdd(&bins[(keys[i] >> shift) & 255], 1u);
    } else {
      for (int i = warp; i < n; i += kWarps) {
        const unsigned long long x = key_at(i);
        if (lane == 0 && (x & mask) == border) atomicAdd(&bins[(x >> shift) & 255], 1u);
      }
    }
    __syncthreads();
    constexpr int kPer = 256 / kThreads > 0 ? 256 / kThreads : 1;
    uint32_t cnt[kPer], sum = 0;  // of digits 255 - kPer tid - k
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += cnt[k] = bins[255 - kPer * tid - k];
    uint32_t above = block_scan<W>(sum, scratch);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (above < left && left <= above + cnt[k]) {
        pick[0] = 255 - kPer * tid - k;
        pick[1] = left - above;
      }
      above += cnt[k];
    }
    __syncthreads();
    border |= static_cast<unsigned long long>(pick[0]) << shift;
    mask |= 255ull << shift;
    left = pick[1];
  }
  if (!kept) {
    // the scores are not needed any more: 2 above the border, 1 at it, 0 below
    for (int i = warp; i < n; i += kWarps) {
      const unsigned long long x = key_at(i);
      __syncwarp();
      if (lane == 0) score[i] = x > border ? 2.f : x == border ? 1.f : 0.f;
    }
    __syncthreads();
    put_taken<W>(out + n_front, left, c_lo, n, warp_counts, [&](int i) { return score[i] == 2.f; },
                 [&](int i) { return score[i] == 1.f; });
  } else {
    put_taken<W>(out + n_front, left, c_lo, n, warp_counts, [&](int i) { return keys[i] > border; },
                 [&](int i) { return keys[i] == border; });
  }
}

template <class T, int D, bool KV8, int W>
static cudaError_t launch_select_typed(const Args &a, int num_seqs, size_t smem,
                                       cudaStream_t stream) {
  auto kern = select_kernel<T, D, KV8, W>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(kern, allowed, kStatic);
  if (e != cudaSuccess) return e;
  PdlLaunch cfg(dim3(a.cluster, a.KVH, num_seqs), 32 * W, smem, stream, a.cluster);
  return cudaLaunchKernelEx(&cfg.c, kern, a);
}

}  // namespace sel

cudaError_t launch_block_bounds(void *bounds, const void *kv_cache, const int32_t *block_tables,
                                int max_blocks_per_seq, const int32_t *context_lens,
                                const int32_t *seq_lens, int num_seqs, int max_new_tokens,
                                const Geometry &g, cudaStream_t stream) {
  sel::BoundsArgs a{};
  a.bounds = static_cast<uint8_t *>(bounds);
  a.k_half = static_cast<const uint8_t *>(kv_cache);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.seq_lens = seq_lens;
  a.num_blocks = g.num_blocks;
  a.row_bytes = g.row_bytes;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_new = max_new_tokens;
  a.BS = g.BS;
  a.D = g.D;
  // new positions may start anywhere in a block
  const int64_t touched =
      std::min<int64_t>(max_blocks_per_seq, (int64_t{max_new_tokens} + g.BS - 2) / g.BS + 1);
  const int64_t items = touched * (g.row_bytes / 16);
  PdlLaunch cfg(dim3(static_cast<unsigned>((items + sel::kBoundsThreads - 1) / sel::kBoundsThreads),
                     num_seqs),
                sel::kBoundsThreads, 0, stream);
  const bool bulk = num_seqs * touched * g.block_bytes > 64 << 20;
#define PKV_BOUNDS(PP, KK)                                                              \
  return bulk ? cudaLaunchKernelEx(&cfg.c, sel::bounds_kernel<sel::PP, KK, true>, a)    \
              : cudaLaunchKernelEx(&cfg.c, sel::bounds_kernel<sel::PP, KK, false>, a)
  if (g.fp8) PKV_BOUNDS(F16x2, true);
  if (g.dtype == PKV_BF16) PKV_BOUNDS(Bf16x2, false);
  PKV_BOUNDS(F16x2, false);
#undef PKV_BOUNDS
}

cudaError_t launch_select(const SelectCall &s, const Geometry &g, cudaStream_t stream) {
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return e;
  sel::Args a{};
  a.selected = s.selected;
  a.query = static_cast<const uint16_t *>(s.query);
  a.bounds = static_cast<const uint8_t *>(s.bounds);
  a.block_tables = s.block_tables;
  a.seq_lens = s.seq_lens;
  a.num_blocks = g.num_blocks;
  a.max_selected = s.max_selected;
  a.max_blocks_per_seq = s.max_blocks_per_seq;
  a.max_seq_len = s.max_seq_len;
  a.sink = s.num_sink;
  a.recent = s.num_recent;
  a.H = g.H;
  a.KVH = g.KVH;
  a.QPK = g.QPK;
  a.BS = g.BS;
  a.window = g.window;
  // blocks a sequence can have candidates in: max_seq_len may be a captured step's
  // bound, far above what the table's width allows (64 sequences of 2k .. 4k under a
  // bound of 512k: 17 us, 42 sized by the bound)
  const int blocks = static_cast<int>(
      std::min<int64_t>(scored_blocks(s.max_seq_len, g), s.max_blocks_per_seq));
  const int64_t items = static_cast<int64_t>(s.num_seqs) * g.KVH;
  const size_t heads8 = (g.QPK + 7) / 8;
  const size_t fixed = (heads8 - 1) * (8 * 4 + (g.D / 8) * 32 * 8);
  const size_t room = static_cast<size_t>(dev.max_smem_optin) - sel::kStatic - fixed;
  if (static_cast<size_t>(blocks) * 4 > room) return cudaErrorInvalidValue;
  // More (sequence, KV head) pairs than 8-warp CTAs fit: 4 warps, four CTAs to an
  // SM (64 sequences of 2k .. 4k, 8 KV heads: 17 against 22 us; of 16k .. 32k: 80 both;
  // with fewer pairs 8 warps, 32 sequences: 12 against 14 and 45 against 60).
  const bool many = items > 2LL * dev.sms;
  // 64-bit keys for all candidates where that costs no resident CTA
  a.keys_fit = fixed + static_cast<size_t>(blocks) * 8 <= (many ? 40 : 96) * 1024;
  const size_t smem = fixed + static_cast<size_t>(blocks) * (a.keys_fit ? 8 : 4);
  // A CTA per SM or more, and 64 blocks or more to each.  Measured with 1 / 2 / 4 / 8
  // CTAs per (sequence, KV head), 8 KV heads, us: 64 sequences of 16k .. 32k 80 / 90 /
  // 101 / 143, 16 of them 36 / 28 / 31 / 40, 4 30 / 20 / 15 / 15, one of 32k 20 / 15 /
  // 12 / 10; 16 of 64k .. 128k, 8-bit heads of 64, 34 / 27 / 32 / 37.
  a.cluster = 1;
  while (a.cluster < sel::kMaxCluster && items * a.cluster < dev.sms && blocks / a.cluster >= 64)
    a.cluster *= 2;
  const bool bf = g.dtype == PKV_BF16;
#define PKV_SEL(TT, DD, KK)                                                             \
  if (g.D == DD && g.fp8 == KK)                                                         \
    return many ? sel::launch_select_typed<TT, DD, KK, 4>(a, s.num_seqs, smem, stream)  \
                : sel::launch_select_typed<TT, DD, KK, 8>(a, s.num_seqs, smem, stream);
  if (bf) {
    PKV_SEL(BF16, 128, false) PKV_SEL(BF16, 64, false)
    PKV_SEL(BF16, 128, true) PKV_SEL(BF16, 64, true)
  } else {
    PKV_SEL(FP16, 128, false) PKV_SEL(FP16, 64, false)
    PKV_SEL(FP16, 128, true) PKV_SEL(FP16, 64, true)
  }
#undef PKV_SEL
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_select(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
