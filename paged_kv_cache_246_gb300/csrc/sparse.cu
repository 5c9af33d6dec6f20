// paged_attn_decode_sparse: one query token per sequence attending to the
// selected blocks of its KV head,
//     s_j = scale * q.k_j + slope_h * (j - i),   out = softmax(s) . V
// over the keys j of the selected blocks with j <= i = L - 1 inside the
// sliding window.
//
// The plain form of it: CTA = (query head, sequence), a warp takes every
// fourth selected block key by key, a lane D / 32 channels; one pass with the
// running maximum and sum of the softmax, the warps merged at the end.
#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace sparse {

constexpr int kWarps = 4;

struct Args {
  void *out;
  const uint16_t *query;
  const uint8_t *cache;
  const int32_t *block_tables, *seq_lens, *selected;
  const float *alibi;
  int64_t num_blocks, half_bytes;
  int max_blocks_per_seq, max_selected, H, KVH, QPK, BS, window;
  float scale_log2, v_scale;
};

template <class T, int D, bool KV8>
__device__ __forceinline__ float element(const uint8_t *row, int d) {
  if constexpr (KV8) {
    return FP16::to_f2(e4m3x4_to_h4(row[d]).x).x;
  } else {
    return T::to_f(reinterpret_cast<const uint16_t *>(row)[d]);
  }
}

template <class T, int D, bool KV8>
__global__ void __launch_bounds__(kWarps * 32) sparse_kernel(const Args a) {
  constexpr int E = D / 32;
  constexpr int EB = KV8 ? 1 : 2;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  grid_dependency_wait();
  grid_launch_dependents();
  const int h = blockIdx.x, b = blockIdx.y, kvh = h / a.QPK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > static_cast<int64_t>(a.max_blocks_per_seq) * a.BS) {
    if (h == 0 && threadIdx.x == 0) record_error(PKV_ERR_BOUNDS, b);
    L = 0;
  }
  const int nblk = (L + a.BS - 1) / a.BS, lo = a.window > 0 ? max(0, L - a.window) : 0;
  const int64_t row0 = (static_cast<int64_t>(b) * a.KVH + kvh) * a.max_selected;
  const float slope = a.alibi ? __ldg(a.alibi + h) * kLog2e : 0.f;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = T::to_f(a.query[(static_cast<int64_t>(b) * a.H + h) * D + lane + 32 * e]);
    o[e] = 0.f;
  }
  for (int i = warp; i < a.max_selected; i += kWarps) {
    const int s = __ldg(a.selected + row0 + i), prev = i ? __ldg(a.selected + row0 + i - 1) : -1;
    if (s < 0 || L == 0) continue;
    if (s >= nblk || (i && (prev < 0 || prev >= s))) {
      if (lane == 0) record_error(PKV_ERR_BOUNDS, row0 + i);
      continue;
    }
    const int64_t at = static_cast<int64_t>(b) * a.max_blocks_per_seq + s;
    const int pb = __ldg(a.block_tables + at);
    if (pb < 0 || pb >= a.num_blocks) {
      if (lane == 0) record_error(PKV_ERR_BOUNDS, at);
      continue;
    }
    for (int t = 0; t < a.BS; ++t) {
      const int j = s * a.BS + t;
      if (j >= L || j < lo) continue;
      const uint8_t *kr =
          a.cache + ((static_cast<int64_t>(pb) * a.BS + t) * a.KVH + kvh) * (D * EB);
      float x = 0.f;
      for (int e = 0; e < E; ++e) x = fmaf(q[e], element<T, D, KV8>(kr, lane + 32 * e), x);
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      x = x * a.scale_log2 + slope * static_cast<float>(j - (L - 1));
      const float mn = fmaxf(m, x);
      const float al = m == -INFINITY ? 0.f : exp2f(m - mn), p = x == -INFINITY ? 0.f : exp2f(x - mn);
      m = mn;
      l = l * al + p;
      for (int e = 0; e < E; ++e)
        o[e] = fmaf(p, element<T, D, KV8>(kr + a.half_bytes, lane + 32 * e), o[e] * al);
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float num = 0.f, den = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float e = sl[w] == 0.f ? 0.f : exp2f(sm[w] - M);
      num = fmaf(e, so[w][d], num);
      den = fmaf(e, sl[w], den);
    }
    static_cast<uint16_t *>(a.out)[(static_cast<int64_t>(b) * a.H + h) * D + d] =
        static_cast<uint16_t>(T::from_f2(den == 0.f ? 0.f : num / den * a.v_scale, 0.f) & 0xffffu);
  }
}

}  // namespace sparse

cudaError_t launch_sparse_decode(void *out, const void *query, int num_seqs, const void *kv_cache,
                                 const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *selected,
                                 int max_selected, const Geometry &g, cudaStream_t stream) {
  sparse::Args a{};
  a.out = out;
  a.query = static_cast<const uint16_t *>(query);
  a.cache = static_cast<const uint8_t *>(kv_cache);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.selected = selected;
  a.alibi = g.alibi;
  a.num_blocks = g.num_blocks;
  a.half_bytes = g.num_blocks * g.block_bytes;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_selected = max_selected;
  a.H = g.H;
  a.KVH = g.KVH;
  a.QPK = g.QPK;
  a.BS = g.BS;
  a.window = g.window;
  a.scale_log2 = g.scale * kLog2e * g.k_scale;
  a.v_scale = g.v_scale;
  PdlLaunch cfg(dim3(g.H, num_seqs), sparse::kWarps * 32, 0, stream);
  const bool bf = g.dtype == PKV_BF16;
#define PKV_SP(TT, DD)                                                            \
  if (g.D == DD)                                                                  \
    return g.fp8 ? cudaLaunchKernelEx(&cfg.c, sparse::sparse_kernel<TT, DD, true>, a) \
                 : cudaLaunchKernelEx(&cfg.c, sparse::sparse_kernel<TT, DD, false>, a);
  if (bf) {
    PKV_SP(BF16, 128) PKV_SP(BF16, 64)
  } else {
    PKV_SP(FP16, 128) PKV_SP(FP16, 64)
  }
#undef PKV_SP
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_sparse(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
