// Block bounds and block selection of the sparse decode.
//
// kv_block_bounds: per cache block and KV head the channelwise minimum lo and
// maximum hi of the block's keys.  paged_attn_select_blocks: per (sequence,
// KV head) the blocks with the largest
//     s_j = max_h sum_d max(q_hd lo_jd, q_hd hi_jd)  >=  max_h max_t q_h . k_jt,
// h over the query heads of the group, t over the keys of block j.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

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
// pieces, each CTA keeps its piece's scores as order-preserving 64-bit keys
// in shared memory, and the cluster finds the r-th largest key digit by
// digit: every CTA counts its keys' digits, all counts are summed through
// distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

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

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit word at `p` of CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t cluster_load(const void *p, uint32_t rank) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

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

template <class T, int D, bool KV8>
__global__ void __launch_bounds__(kThreads) select_kernel(const Args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  float *sq = reinterpret_cast<float *>(smem);  // [QPK][D]
  unsigned long long *keys =
      reinterpret_cast<unsigned long long *>(smem + static_cast<size_t>(a.QPK) * D * 4);
  __shared__ uint32_t hist[2][256];
  __shared__ unsigned long long scratch[kWarps];
  __shared__ uint32_t pick[2];    // the digit found, the rank left within it
  __shared__ uint32_t counts[2];  // this CTA's keys above the border, at it

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

  for (int i = tid; i < a.QPK * D; i += kThreads)
    sq[i] = T::to_f(__ldg(a.query + (static_cast<int64_t>(b) * a.H + kvh * a.QPK) * D + i));
  __syncthreads();

  // ---- scores ---------------------------------------------------------------
  constexpr int kRowBytes = 2 * D * (KV8 ? 1 : 2);
  const int32_t *table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
  for (int i = warp; i < n; i += kWarps) {
    const int pb = __ldg(table + p0 + i);
    unsigned long long key = 0;  // a bad entry: taken last
    if (pb >= 0 && pb < a.num_blocks) {
      key = key_of(exact_score<T, D, KV8>(
          a.bounds + (static_cast<int64_t>(pb) * a.KVH + kvh) * kRowBytes, sq, a.QPK));
    } else if (lane == 0) {
      record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(b) * a.max_blocks_per_seq + p0 + i);
    }
    if (lane == 0) keys[i] = key;
  }

  // ---- the need-th largest key of the cluster, 8 bits at a time -----------------
  unsigned long long border = 0, mask = 0;
  uint32_t left = need;  // how many of the keys that match the prefix are taken
  for (int shift = 56, p = 0; shift >= 0; shift -= 8, p ^= 1) {
    hist[p][tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if ((keys[i] & mask) == border) atomicAdd(&hist[p][(keys[i] >> shift) & 255], 1u);
    cluster_sync();
    uint32_t cnt = 0;  // of digit 255 - tid, over the cluster
    for (int c = 0; c < a.cluster; ++c) cnt += cluster_load(&hist[p][255 - tid], c);
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

  // ---- taken: keys above the border, and the first `left` at it ------------------
  const int each = (n + kThreads - 1) / kThreads;  // consecutive keys per thread
  const int i0 = min(tid * each, n), i1 = min(i0 + each, n);
  unsigned long long mine = 0;  // above << 32 | at the border
  for (int i = i0; i < i1; ++i)
    mine += keys[i] > border ? 1ull << 32 : keys[i] == border ? 1ull : 0ull;
  unsigned long long total;
  unsigned long long before = block_scan(mine, &total, scratch);
  if (tid == 0) {
    counts[0] = static_cast<uint32_t>(total >> 32);
    counts[1] = static_cast<uint32_t>(total);
  }
  cluster_sync();
  uint32_t ties = 0, place = n_front;  // ties and taken blocks of the CTAs before this one
  for (uint32_t c = 0; c < rank; ++c) {
    const uint32_t up = cluster_load(&counts[0], c), at = cluster_load(&counts[1], c);
    place += up + min(at, left - min(left, ties));
    ties += at;
  }
  cluster_sync();  // no CTA leaves while its counts are read
  const uint32_t own_left = left - min(left, ties);
  uint32_t tie = static_cast<uint32_t>(before);
  place += static_cast<uint32_t>(before >> 32) + min(tie, own_left);
  for (int i = i0; i < i1; ++i) {
    const bool at = keys[i] == border;
    if (keys[i] > border || (at && tie < own_left)) out[place++] = p0 + i;
    tie += at;
  }
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
  const size_t fixed = static_cast<size_t>(g.QPK) * g.D * 4;
  // clusters grow while the grid leaves SMs idle and a CTA still has a few
  // tiles of blocks, or while the keys do not fit
  int c = 1;
  while (c < sel::kMaxCluster &&
         ((items * c < 2LL * dev.sms && blocks / c >= 128) ||
          fixed + (static_cast<size_t>(blocks) / c + 1) * 8 > static_cast<size_t>(dev.max_smem_optin) - 4096))
    c *= 2;
  a.cluster = c;
  const size_t smem = fixed + (static_cast<size_t>(blocks) / c + 1) * 8;
  if (smem > static_cast<size_t>(dev.max_smem_optin) - 4096) return cudaErrorInvalidValue;
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
