// Block bounds and block selection of the sparse decode.
//
// kv_block_bounds: per cache block and KV head the channelwise minimum lo and
// maximum hi of the block's keys.  paged_attn_select_blocks: per (sequence,
// KV head) the blocks with the largest
//     s_j = max_h sum_d max(q_hd lo_jd, q_hd hi_jd)  >=  max_h max_t q_h . k_jt,
// h over the query heads of the group, t over the keys of block j.
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

struct BoundsArgs {
  uint8_t *bounds;
  const uint8_t *k_half;
  const int32_t *block_tables, *context_lens, *seq_lens;
  int64_t num_blocks;
  int64_t row_bytes;
  int max_blocks_per_seq, max_new, BS, D;
};

constexpr int kBoundsThreads = 128;

// CTA = (touched block x, sequence y): a thread owns 16-byte chunks of the
// key row and runs down the block's written rows.
template <class P, bool KV8>
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
  const int lb = ctx / a.BS + blockIdx.x;
  if (lb > (L - 1) / a.BS) return;
  const int64_t at = static_cast<int64_t>(b) * a.max_blocks_per_seq + lb;
  const int pb = __ldg(a.block_tables + at);
  if (pb < 0 || pb >= a.num_blocks) {
    if (threadIdx.x == 0) record_error(PKV_ERR_BOUNDS, at);
    return;
  }
  const int rows = min(a.BS, L - lb * a.BS);
  const int chunks = static_cast<int>(a.row_bytes / 16);
  const int head_bytes = KV8 ? a.D : 2 * a.D;
  for (int c = threadIdx.x; c < chunks; c += kBoundsThreads) {
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
      for (int i = 0; i < U; ++i)  // rows past the end repeat the last one
        u[i] = *reinterpret_cast<const uint4 *>(src + min(r0 + i, rows - 1) * a.row_bytes);
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
}

// ---------------------------------------------------------------------------
// Selection.  A cluster of C CTAs serves one (sequence, KV head): the
// candidate blocks (visible, not taken anyway) are cut into C consecutive
// pieces whose scores stay in the CTAs' shared memory; what the cluster has
// to know of all of them goes through distributed shared memory.
//
// Scores.  With lo <= hi, max(q lo, q hi) = max(q, 0) hi + min(q, 0) lo, so the
// scores of 16 blocks and 8 query heads are one product of [16 blocks x 2D
// bounds] and [2D x 8 heads] on the tensor core (mma.sync m16n8k16: the step is
// bound by reading the bounds, 2D elements per block and KV head, and the
// tensor core keeps the instructions per bound low).  The 2D axis is taken in
// an order in which a lane's 16-byte loads are its A fragments as they stand.
//
// Exactness.  Products of 16-bit values are exact; a product step sums 16 of
// them with an error of at most 2^-19 of their magnitudes' sum (each term cut
// at 2^-23 of the largest), and starts from zero, so that errors scale with the
// step's terms and not with the sum so far; the steps' sums are added in fp32.
// Altogether a score is within
//     E = 2^-18 * max_h |q_h|_1 * max |bound|
// of the exact one, so only scores within 2E of the border can belong on its
// other side.  A histogram of 1024 equal bins finds the border's bin; what lies
// in it or within 2E of it (one to three blocks as a rule) is scored again in 64
// bits and ranked, everything above is taken.  Where that list does not fit, or
// a score is not finite, all that is open is scored in 64 bits and the border
// found digit by digit.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;  // of the score histogram
constexpr int kList = 64;    // open blocks a CTA can list

struct Args {
  int32_t *selected;
  const uint16_t *query;
  const uint8_t *bounds;
  const int32_t *block_tables, *seq_lens;
  int64_t num_blocks;
  int max_selected, max_blocks_per_seq, max_seq_len, sink, recent;
  int H, KVH, QPK, BS, window;
  int cluster;
};

// Order-preserving 64-bit key of a score: NaN counts as +infinity, -0 as 0.
__device__ __forceinline__ unsigned long long key_of(double s) {
  if (s != s) s = INFINITY;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Exclusive prefix sum of v over the CTA's threads, and the total.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long *total,
                                                         unsigned long long *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // scratch may still be read from the last scan
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  unsigned long long base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += scratch[w];
    sum += scratch[w];
  }
  *total = sum;
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

// The score of one block in 64 bits, by a whole warp: products of bounds and
// queries are exact, sums off by 2^-53 of their terms.
template <class T, int D, bool KV8>
__device__ __forceinline__ double exact_score(const uint8_t *row, const float *q, int qpk) {
  const int lane = threadIdx.x & 31;
  double best = -INFINITY;
  bool nan = false;
  for (int h = 0; h < qpk; ++h) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int d = lane + 32 * k;
      const double qd = q[h * D + d];
      const double x = qd * bound_value<T, KV8>(row, d), y = qd * bound_value<T, KV8>(row, D + d);
      s += (x > y || x != x) ? x : y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = s > best ? s : best;
  }
  return nan ? INFINITY : best;
}

// acc = max(acc, |w|) on packed pairs (a NaN is left out: its score tells).
template <class MT>
__device__ __forceinline__ uint32_t max_abs(uint32_t acc, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_abs<BF16>(uint32_t acc, uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.bf16x2 %0, %1, t;\n\t}"
      : "=r"(d)
      : "r"(acc), "r"(w));
  return d;
}
template <>
__device__ __forceinline__ uint32_t max_abs<FP16>(uint32_t acc, uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\tabs.f16x2 t, %2;\n\tmax.f16x2 %0, %1, t;\n\t}"
      : "=r"(d)
      : "r"(acc), "r"(w));
  return d;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// What a CTA tells its cluster.
struct Shared {
  uint32_t hist[2][256];     // digit counts (the 64-bit path)
  uint32_t bins[kBins];
  float span[4];             // smallest, largest score; largest |bound|; 1: not finite
  uint32_t counts[2];        // blocks above the border, blocks at it
  uint32_t listed;           // blocks to rank
  unsigned long long list_key[kList];
  int32_t list_at[kList];
};

template <class T, int D, bool KV8>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const Args a) {
  using MT = std::conditional_t<KV8, FP16, T>;  // operand type
  constexpr int kRowBytes = 2 * D * (KV8 ? 1 : 2);
  constexpr int kSteps = 2 * D / 16;
  constexpr int kLoads = kRowBytes / 64;          // 16-byte loads of a lane per row
  constexpr int kStepsPerLoad = kSteps / kLoads;  // 2, or 4 of 8-bit codes
  extern __shared__ __align__(16) uint8_t smem[];
  const int heads8 = (a.QPK + 7) / 8;
  float *sq = reinterpret_cast<float *>(smem);                        // [QPK][D]
  float *sunit = sq + static_cast<size_t>(a.QPK) * D;                 // [heads8 * 8]
  uint2 *sb = reinterpret_cast<uint2 *>(sunit + heads8 * 8);          // [heads8][kSteps][32]
  // per candidate 8 bytes: its score as a float, or its 64-bit key
  unsigned long long *keys =
      reinterpret_cast<unsigned long long *>(sb + static_cast<size_t>(heads8) * kSteps * 32);
  __shared__ Shared sh;
  __shared__ unsigned long long scratch[kWarps];
  __shared__ uint32_t pick[2];  // the bin or digit found, the rank left within it
  __shared__ float wred[4][kWarps];
  __shared__ unsigned long long all_key[kMaxCluster * kList];
  __shared__ int32_t all_at[kMaxCluster * kList];

  grid_dependency_wait();
  grid_launch_dependents();
  const int kvh = blockIdx.y, b = blockIdx.z;
  const uint32_t rank = cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t *out = a.selected + (static_cast<int64_t>(b) * a.KVH + kvh) * a.max_selected;

  int L = __ldg(a.seq_lens + b);
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
  const int per = (c_hi - c_lo + a.cluster - 1) / a.cluster;
  const int p0 = min(c_lo + static_cast<int>(rank) * per, c_hi);
  const int n = min(per, c_hi - p0);

  // ---- the group's queries -------------------------------------------------
  const uint16_t *qg = a.query + (static_cast<int64_t>(b) * a.H + kvh * a.QPK) * D;
  for (int i = tid; i < a.QPK * D; i += kThreads) sq[i] = T::to_f(__ldg(qg + i));
  for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
  if (tid == 0) sh.listed = 0;
  __syncthreads();
  float q1 = 0.f;  // the largest sum of a head's |q|
  for (int h = warp; h < heads8 * 8; h += kWarps) {
    float s = 0.f, m = 0.f;
    if (h < a.QPK)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const float x = fabsf(sq[h * D + lane + 32 * k]);
        s += x;
        m = fmaxf(m, x);
      }
    m = warp_max(m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    q1 = fmaxf(q1, s);
    if (lane == 0) {
      // bf16 queries against fp8 bounds are taken as fp16 times a power of two
      // (the largest of a head in [2^14, 2^15)): exact for components within
      // 2^28 of it, off by 2^-39 of it below
      float unit = 1.f;
      if constexpr (KV8 && std::is_same<T, BF16>::value) {
        const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;  // m in [2^e, 2^(e+1))
        if (m > 0.f && e < 128) unit = __uint_as_float(static_cast<uint32_t>(min(max(e - 14, -126), 126) + 127) << 23);
      }
      sunit[h] = unit;
    }
  }
  if (lane == 0) wred[0][warp] = q1;
  __syncthreads();
  q1 = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) q1 = fmaxf(q1, wred[0][w]);
  // B fragments: k-step s of lane (g, tq) covers elements 4u .. 4u + 3 of the
  // row's 16-byte chunk 4 (s / steps per load) + tq, u = s % steps per load
  for (int i = tid; i < heads8 * kSteps * 32; i += kThreads) {
    const int ln = i & 31, s = (i >> 5) % kSteps, h = (i >> 5) / kSteps * 8 + (ln >> 2);
    const int chunk = 4 * (s / kStepsPerLoad) + (ln & 3);
    const int e = chunk * (KV8 ? 16 : 8) + 4 * (s % kStepsPerLoad);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (h < a.QPK) {
      const float inv = 1.f / sunit[h];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = sq[h * D + (e + k) % D] * inv;
        v[k] = e < D ? fminf(x, 0.f) : fmaxf(x, 0.f);
        if (x != x) v[k] = x;
      }
    }
    sb[i] = make_uint2(MT::from_f2(v[0], v[1]), MT::from_f2(v[2], v[3]));
  }
  __syncthreads();

  // ---- scores: a warp takes 16 blocks at a time --------------------------------
  const int32_t *table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
  const int g = lane >> 2, tq = lane & 3;
  uint2 bq[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) bq[s] = sb[s * 32 + lane];
  const float unit0 = sunit[2 * tq], unit1 = sunit[2 * tq + 1];
  // (rows past the last block repeat it)
  auto entry = [&](int i) { return n > 0 ? __ldg(table + p0 + min(i, n - 1)) : 0; };
  float mn = INFINITY, mx = -INFINITY;
  bool odd = false;  // a score that is not finite
  uint32_t mb = 0;   // largest |bound|, packed
  int pb0 = entry(warp * 16 + g), pb1 = entry(warp * 16 + g + 8);
  for (int t = warp * 16; t < n; t += kWarps * 16) {
    const bool in0 = t + g < n, in1 = t + g + 8 < n;
    const bool bad0 = pb0 < 0 || pb0 >= a.num_blocks, bad1 = pb1 < 0 || pb1 >= a.num_blocks;
    if (((in0 && bad0) || (in1 && bad1)) && tq == 0)
      record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(b) * a.max_blocks_per_seq + p0 + t + g +
                                       (in0 && bad0 ? 0 : 8));
    const uint4 *r0 = reinterpret_cast<const uint4 *>(
                          a.bounds + (static_cast<int64_t>(bad0 ? 0 : pb0) * a.KVH + kvh) * kRowBytes) + tq;
    const uint4 *r1 = reinterpret_cast<const uint4 *>(
                          a.bounds + (static_cast<int64_t>(bad1 ? 0 : pb1) * a.KVH + kvh) * kRowBytes) + tq;
    uint4 u0[kLoads], u1[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      u0[i] = __ldg(r0 + 4 * i);
      u1[i] = __ldg(r1 + 4 * i);
    }
    // the next tile's entries arrive while this one is worked on
    pb0 = entry(t + kWarps * 16 + g);
    pb1 = entry(t + kWarps * 16 + g + 8);
    float best0 = -INFINITY, best1 = -INFINITY;
    for (int h8 = 0; h8 < heads8; ++h8) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w0[4] = {u0[i].x, u0[i].y, u0[i].z, u0[i].w};
        const uint32_t w1[4] = {u1[i].x, u1[i].y, u1[i].z, u1[i].w};
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
            mb = max_abs<MT>(max_abs<MT>(mb, f0[0]), f0[1]);
            mb = max_abs<MT>(max_abs<MT>(mb, f1[0]), f1[1]);
          }
          float d[4];
          const uint2 q2 = h8 == 0 ? bq[s] : sb[(h8 * kSteps + s) * 32 + lane];
          mma_16816<MT>(d, f0[0], f1[0], f0[1], f1[1], q2.x, q2.y, 0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] += d[k];
        }
      }
      // heads 8 h8 + 2 tq, + 1 of blocks g (c[0], c[1]) and g + 8
      if constexpr (KV8 && std::is_same<T, BF16>::value) {
        const float e0 = h8 == 0 ? unit0 : sunit[h8 * 8 + 2 * tq], e1 = h8 == 0 ? unit1 : sunit[h8 * 8 + 2 * tq + 1];
        c[0] *= e0;
        c[2] *= e0;
        c[1] *= e1;
        c[3] *= e1;
      }
      const bool v0 = h8 * 8 + 2 * tq < a.QPK, v1 = h8 * 8 + 2 * tq + 1 < a.QPK;
      // x - x is 0 for finite x alone
      odd |= in0 && !bad0 && ((v0 && c[0] - c[0] != 0.f) || (v1 && c[1] - c[1] != 0.f));
      odd |= in1 && !bad1 && ((v0 && c[2] - c[2] != 0.f) || (v1 && c[3] - c[3] != 0.f));
      best0 = fmaxf(best0, fmaxf(v0 ? c[0] : -INFINITY, v1 ? c[1] : -INFINITY));
      best1 = fmaxf(best1, fmaxf(v0 ? c[2] : -INFINITY, v1 ? c[3] : -INFINITY));
    }
    best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, 1));
    best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, 1));
    best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, 2));
    best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, 2));
    // a bad entry: -infinity, below every other score and taken last
    if (tq == 0 && in0) keys[t + g] = __float_as_uint(bad0 ? -INFINITY : best0);
    if (tq == 0 && in1) keys[t + g + 8] = __float_as_uint(bad1 ? -INFINITY : best1);
    if (in0 && !bad0) {
      mn = fminf(mn, best0);
      mx = fmaxf(mx, best0);
    }
    if (in1 && !bad1) {
      mn = fminf(mn, best1);
      mx = fmaxf(mx, best1);
    }
  }
  // ---- the cluster's span of scores ----------------------------------------------
  {
    const float2 m2 = MT::to_f2(mb);
    const float w0 = warp_max(-mn), w1 = warp_max(mx), w2 = warp_max(fmaxf(m2.x, m2.y));
    const float w3 = __any_sync(0xffffffffu, odd) ? 1.f : 0.f;
    __syncthreads();
    if (lane == 0) {
      wred[0][warp] = w0;
      wred[1][warp] = w1;
      wred[2][warp] = w2;
      wred[3][warp] = w3;
    }
    __syncthreads();
    if (tid < 4) {
      float x = wred[tid][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) x = fmaxf(x, wred[tid][w]);
      sh.span[tid] = x;
    }
  }
  cluster_sync();
  float span[4] = {-INFINITY, -INFINITY, 0.f, 0.f};
  for (int c = 0; c < a.cluster; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      span[k] = fmaxf(span[k], __uint_as_float(cluster_load(&sh.span[k], c)));
  mn = -span[0];
  mx = span[1];
  // products below fp32's range may be lost altogether
  const float err = q1 * span[2] * 0x1p-18f + 1e-36f;
  bool slow = span[3] != 0.f || !(mx >= mn) || !(mx - mn < INFINITY) || !(err < INFINITY);
  float t_lo = -INFINITY, t_hi = INFINITY;  // above t_hi taken, below t_lo not
  const int each = (n + kThreads - 1) / kThreads;  // consecutive blocks per thread
  const int i0 = min(tid * each, n), i1 = min(i0 + each, n);
  if (!slow) {
    // ---- the border's bin -----------------------------------------------------------
    const float inv = mx > mn ? kBins / (mx - mn) : 0.f;
    if (inv < INFINITY) {
      for (int i = i0; i < i1; ++i) {
        const float s = __uint_as_float(static_cast<uint32_t>(keys[i]));
        atomicAdd(&sh.bins[max(0, min(kBins - 1, static_cast<int>((s - mn) * inv)))], 1u);
      }
      cluster_sync();
      constexpr int kPer = kBins / kThreads;
      uint32_t cnt[kPer], sum = 0;  // of bins kBins - 1 - kPer * tid - k, over the cluster
#pragma unroll
      for (int k = 0; k < kPer; ++k) cnt[k] = 0;
      for (int c = 0; c < a.cluster; ++c)
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          cnt[k] += cluster_load(&sh.bins[kBins - 1 - kPer * tid - k], c);
#pragma unroll
      for (int k = 0; k < kPer; ++k) sum += cnt[k];
      unsigned long long total;
      uint32_t above = static_cast<uint32_t>(block_scan(sum, &total, scratch));
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
    } else {
      slow = true;
    }
  }
  // ---- taken, open, not taken --------------------------------------------------------
  if (!slow) {
    uint32_t up = 0;
    for (int i = i0; i < i1; ++i) {
      const float s = __uint_as_float(static_cast<uint32_t>(keys[i]));
      up += s > t_hi;
      if (s <= t_hi && s >= t_lo) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kList) sh.list_at[at] = i;
      }
    }
    unsigned long long total;
    block_scan(up, &total, scratch);  // its barriers also complete the list
    if (tid == 0) sh.counts[0] = static_cast<uint32_t>(total);
    const int m = min(sh.listed, static_cast<uint32_t>(kList));
    for (int k = warp; k < m; k += kWarps) {
      const int i = sh.list_at[k];
      const int pb = __ldg(table + p0 + i);
      const bool bad = pb < 0 || pb >= a.num_blocks;
      const unsigned long long key =
          bad ? 0 : key_of(exact_score<T, D, KV8>(a.bounds + (static_cast<int64_t>(pb) * a.KVH + kvh) * kRowBytes, sq, a.QPK));
      if (lane == 0) sh.list_key[k] = key;
    }
    cluster_sync();
    uint32_t ups = 0, open = 0, ups_before = 0, open_before = 0;
    for (int c = 0; c < a.cluster; ++c) {
      const uint32_t l = cluster_load(&sh.listed, c), u = cluster_load(&sh.counts[0], c);
      slow |= l > kList;
      if (c < static_cast<int>(rank)) {
        ups_before += u;
        open_before += l;
      }
      ups += u;
      open += l;
    }
    if (!slow) {
      // every CTA ranks all of the open blocks
      uint32_t base = 0;
      for (int c = 0; c < a.cluster; ++c) {
        const uint32_t l = cluster_load(&sh.listed, c);
        for (uint32_t k = tid; k < l; k += kThreads) {
          const uint32_t lo = cluster_load(&sh.list_key[k], c);
          const uint32_t hi = cluster_load(reinterpret_cast<uint32_t *>(&sh.list_key[k]) + 1, c);
          all_key[base + k] = static_cast<unsigned long long>(hi) << 32 | lo;
          all_at[base + k] = c * per + static_cast<int>(cluster_load(&sh.list_at[k], c));
        }
        base += l;
      }
      cluster_arrive();  // this CTA reads no other's shared memory any more
      if (tid == 0) sh.counts[1] = 0;
      __syncthreads();
      const uint32_t left = need - ups;
      uint32_t taken_before = 0;
      for (uint32_t k = tid; k < open; k += kThreads) {
        uint32_t ahead = 0;
        const unsigned long long key = all_key[k];
        const int at = all_at[k];
        for (uint32_t j = 0; j < open; ++j)
          ahead += all_key[j] > key || (all_key[j] == key && all_at[j] < at);
        const bool take = ahead < left;
        taken_before += take && k < open_before;
        if (k >= open_before && at < static_cast<int>(rank) * per + n)  // this CTA's own
          keys[at - rank * per] = __float_as_uint(take ? INFINITY : -INFINITY);
      }
      if (taken_before) atomicAdd(&sh.counts[1], taken_before);
      __syncthreads();
      uint32_t mine = 0;
      for (int i = i0; i < i1; ++i) mine += __uint_as_float(static_cast<uint32_t>(keys[i])) > t_hi;
      uint32_t place = n_front + ups_before + sh.counts[1] +
                       static_cast<uint32_t>(block_scan(mine, &total, scratch));
      for (int i = i0; i < i1; ++i)
        if (__uint_as_float(static_cast<uint32_t>(keys[i])) > t_hi) out[place++] = p0 + i;
      cluster_wait();
      return;
    }
    cluster_sync();  // the counts are read: they are written again below
  }

  // ---- 64 bits: what is open as its exact key, the rest above or below all keys --------
  for (int i = warp; i < n; i += kWarps) {
    const float s = __uint_as_float(static_cast<uint32_t>(keys[i]));
    unsigned long long key = s > t_hi ? ~0ull : 0;
    if (!(s > t_hi || s < t_lo)) {
      const int pb = __ldg(table + p0 + i);
      if (pb >= 0 && pb < a.num_blocks)
        key = key_of(exact_score<T, D, KV8>(a.bounds + (static_cast<int64_t>(pb) * a.KVH + kvh) * kRowBytes, sq, a.QPK));
    }
    __syncwarp();
    if (lane == 0) keys[i] = key;
  }

  // the need-th largest key of the cluster, 8 bits at a time
  unsigned long long border = 0, mask = 0;
  uint32_t left = need;  // how many of the keys that match the prefix are taken
  for (int shift = 56, p = 0; shift >= 0; shift -= 8, p ^= 1) {
    sh.hist[p][tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if ((keys[i] & mask) == border) atomicAdd(&sh.hist[p][(keys[i] >> shift) & 255], 1u);
    cluster_sync();
    uint32_t cnt = 0;  // of digit 255 - tid, over the cluster
    for (int c = 0; c < a.cluster; ++c) cnt += cluster_load(&sh.hist[p][255 - tid], c);
    unsigned long long total;
    const uint32_t above = static_cast<uint32_t>(block_scan(cnt, &total, scratch));
    if (above < left && left <= above + cnt) {
      pick[0] = 255 - tid;
      pick[1] = left - above;
    }
    __syncthreads();
    border |= static_cast<unsigned long long>(pick[0]) << shift;
    mask |= 255ull << shift;
    left = pick[1];
  }

  // taken: keys above the border, and the first `left` at it
  unsigned long long mine = 0;  // above << 32 | at the border
  for (int i = i0; i < i1; ++i)
    mine += keys[i] > border ? 1ull << 32 : keys[i] == border ? 1ull : 0ull;
  unsigned long long total;
  unsigned long long before = block_scan(mine, &total, scratch);
  if (tid == 0) {
    sh.counts[0] = static_cast<uint32_t>(total >> 32);
    sh.counts[1] = static_cast<uint32_t>(total);
  }
  cluster_sync();
  uint32_t ties = 0, place = n_front;  // ties and taken blocks of the CTAs before this one
  for (uint32_t c = 0; c < rank; ++c) {
    const uint32_t up = cluster_load(&sh.counts[0], c), at = cluster_load(&sh.counts[1], c);
    place += up + min(at, left - min(left, ties));
    ties += at;
  }
  cluster_arrive();  // this CTA reads no other's shared memory any more
  const uint32_t own_left = left - min(left, ties);
  uint32_t tie = static_cast<uint32_t>(before);
  place += static_cast<uint32_t>(before >> 32) + min(tie, own_left);
  for (int i = i0; i < i1; ++i) {
    const bool at = keys[i] == border;
    if (keys[i] > border || (at && tie < own_left)) out[place++] = p0 + i;
    tie += at;
  }
  cluster_wait();
}

template <class T, int D, bool KV8>
static cudaError_t launch_select_typed(const Args &a, int num_seqs, size_t smem,
                                       cudaStream_t stream) {
  auto kern = select_kernel<T, D, KV8>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  PdlLaunch cfg(dim3(a.cluster, a.KVH, num_seqs), kThreads, smem, stream, a.cluster);
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
  const int touched = std::min(max_blocks_per_seq, (max_new_tokens - 1 + g.BS - 1) / g.BS + 1);
  PdlLaunch cfg(dim3(touched, num_seqs), sel::kBoundsThreads, 0, stream);
  if (g.fp8) return cudaLaunchKernelEx(&cfg.c, sel::bounds_kernel<sel::F16x2, true>, a);
  return g.dtype == PKV_BF16 ? cudaLaunchKernelEx(&cfg.c, sel::bounds_kernel<sel::Bf16x2, false>, a)
                             : cudaLaunchKernelEx(&cfg.c, sel::bounds_kernel<sel::F16x2, false>, a);
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
  // blocks a sequence can have candidates in
  int64_t span = s.max_seq_len;
  if (g.window > 0) span = std::min<int64_t>(span, static_cast<int64_t>(g.window) + g.BS);
  const int blocks = static_cast<int>((span + g.BS - 1) / g.BS);
  const int64_t items = static_cast<int64_t>(s.num_seqs) * g.KVH;
  const size_t heads8 = (g.QPK + 7) / 8;
  const size_t fixed = static_cast<size_t>(g.QPK) * g.D * 4 + heads8 * 8 * 4 + heads8 * (g.D / 8) * 32 * 8;
  // clusters grow while the grid leaves SMs idle and a CTA still has a few
  // tiles of blocks, or while the keys do not fit
  constexpr size_t kStatic = 20 * 1024;  // the kernel's own shared memory, rounded up
  int c = 1;
  while (c < sel::kMaxCluster &&
         ((items * c < 2LL * dev.sms && blocks / c >= 128) ||
          fixed + (static_cast<size_t>(blocks) / c + 1) * 8 > static_cast<size_t>(dev.max_smem_optin) - kStatic))
    c *= 2;
  a.cluster = c;
  const size_t smem = fixed + (static_cast<size_t>(blocks) / c + 1) * 8;
  if (smem > static_cast<size_t>(dev.max_smem_optin) - kStatic) return cudaErrorInvalidValue;
  const bool bf = g.dtype == PKV_BF16;
#define PKV_SEL(TT, DD)                                                                    \
  if (g.D == DD)                                                                           \
    return g.fp8 ? sel::launch_select_typed<TT, DD, true>(a, s.num_seqs, smem, stream)     \
                 : sel::launch_select_typed<TT, DD, false>(a, s.num_seqs, smem, stream);
  if (bf) {
    PKV_SEL(BF16, 128) PKV_SEL(BF16, 64)
  } else {
    PKV_SEL(FP16, 128) PKV_SEL(FP16, 64)
  }
#undef PKV_SEL
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_select(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
