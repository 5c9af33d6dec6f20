// paged_attn_decode_tree: every node of a tree of drafted tokens attends to its
// sequence's context, its ancestors and itself:
//     s_j = scale * q.k_j + slope_h * (pos_j - pos_i),   out = softmax(s) . V,
// where a context key's position is its place in the cache and a node's is the
// context's length plus its depth.
//
// The plainest form: CTA = (node, query head), four warps take the keys in
// turn, each lane D / 32 channels, with a running maximum and sum.
#include <algorithm>

#include <cuda_fp8.h>

#include "tree.cuh"

namespace pkv {
namespace tree {

struct Args {
  TreeBatch tb;
  uint16_t *out;
  const uint16_t *query;
  const uint8_t *cache;
  const int32_t *block_tables, *seq_lens;
  const float *alibi;
  int64_t num_blocks, row_elems;
  int max_blocks_per_seq, max_seq_len, H, QPK, BS, window;
  float scale_log2, v_scale;
};

constexpr int kMax = PKV_TREE_MAX_NODES;

template <class T, int D, bool KV8>
__global__ void __launch_bounds__(128) simple_kernel(const Args a) {
  __shared__ int depth[kMax];
  __shared__ uint32_t seen[kMax / 32];
  __shared__ float part[4][D + 2];
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.z, t = blockIdx.y, h = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int row, n;
  bool ok = nodes_of(a.tb, b, row, n);
  const int L = __ldg(a.seq_lens + b);
  ok = ok && L >= n && L <= a.max_seq_len &&
       L <= static_cast<int64_t>(a.max_blocks_per_seq) * a.BS;
  if (!ok) {
    if (threadIdx.x == 0 && t == 0 && h == 0) record_error(PKV_ERR_BOUNDS, b);
    return;
  }
  if (t >= n) return;
  const int ctx = L - n;
  auto parent = [&](int c) -> int {
    const int p = __ldg(a.tb.parents + row + c);
    if (p >= -1 && p < c) return p;
    record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(row) + c);
    return -1;
  };
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    int d = -1;
    for (int p = c; p >= 0; p = parent(p)) ++d;
    depth[c] = d;
  }
  if (threadIdx.x < kMax / 32) seen[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int p = t; p >= 0; p = parent(p)) seen[p / 32] |= 1u << (p % 32);
  __syncthreads();
  const int mine = ctx + depth[t];
  const float slope = a.alibi ? __ldg(a.alibi + h) * kLog2e : 0.f;
  constexpr int E = D / 32;
  float q[E], o[E];
  const uint16_t *qr = a.query + (static_cast<int64_t>(row + t) * a.H + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = T::to_f(qr[e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int g = h / a.QPK;
  const int lo = a.window > 0 ? max(0, mine - a.window + 1) : 0;
  auto value = [&](int64_t elem) -> float {
    if constexpr (KV8) {
      const __half_raw x = __nv_cvt_fp8_to_halfraw(a.cache[elem], __NV_E4M3);
      return __half2float(__half(x));
    } else {
      return T::to_f(reinterpret_cast<const uint16_t *>(a.cache)[elem]);
    }
  };
  for (int j = warp; j < L; j += 4) {
    int pos = j;
    if (j < ctx) {
      if (j < lo) continue;
    } else {
      const int c = j - ctx;
      pos = ctx + depth[c];
      if (!(seen[c / 32] >> (c % 32) & 1) || pos < lo) continue;
    }
    const int pb = __ldg(a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq + j / a.BS);
    if (pb < 0 || pb >= a.num_blocks) {
      if (lane == 0) record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(b) * a.max_blocks_per_seq + j / a.BS);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(pb) * a.BS + j % a.BS) * a.row_elems + g * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * value(at + e);
#pragma unroll
    for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
    s = s * a.scale_log2 + slope * static_cast<float>(pos - mine);
    const float top = fmaxf(m, s);
    const float up = m == -INFINITY ? 0.f : exp2f(m - top);
    const float p = s == -INFINITY ? 0.f : exp2f(s - top);
    m = top;
    l = l * up + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * up + p * value(at + e + a.num_blocks * a.BS * a.row_elems);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = o[e];
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][D]);
    for (int w = 0; w < 4; ++w) {
      if (part[w][D + 1] == 0.f) continue;
      const float f = exp2f(part[w][D] - top);
      sum += f * part[w][D + 1];
      acc += f * part[w][threadIdx.x];
    }
    const float r = acc / sum * a.v_scale;
    a.out[(static_cast<int64_t>(row + t) * a.H + h) * D + threadIdx.x] =
        static_cast<uint16_t>(T::from_f2(r, 0.f));
  }
}

}  // namespace tree

size_t tree_workspace_bytes(int, int, int, const Geometry &, int) { return 0; }

cudaError_t launch_tree_decode(void *out, const void *query, const TreeBatch &t,
                               const void *kv_cache, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens, int max_seq_len,
                               const Geometry &g, void *, cudaStream_t stream) {
  tree::Args a{};
  a.tb = t;
  a.out = static_cast<uint16_t *>(out);
  a.query = static_cast<const uint16_t *>(query);
  a.cache = static_cast<const uint8_t *>(kv_cache);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.alibi = g.alibi;
  a.num_blocks = g.num_blocks;
  a.row_elems = g.row_elems;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.H = g.H;
  a.QPK = g.QPK;
  a.BS = g.BS;
  a.window = g.window;
  a.scale_log2 = g.scale * kLog2e * g.k_scale;
  a.v_scale = g.v_scale;
  PdlLaunch cfg(dim3(g.H, t.max_nodes, t.num_seqs), 128, 0, stream);
#define PKV_TREE(TT, DD)                                                                  \
  if (g.D == DD)                                                                          \
    return g.fp8 ? cudaLaunchKernelEx(&cfg.c, tree::simple_kernel<TT, DD, true>, a)       \
                 : cudaLaunchKernelEx(&cfg.c, tree::simple_kernel<TT, DD, false>, a);
  if (g.dtype == PKV_BF16) {
    PKV_TREE(BF16, 128) PKV_TREE(BF16, 64)
  } else {
    PKV_TREE(FP16, 128) PKV_TREE(FP16, 64)
  }
#undef PKV_TREE
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_tree(unsigned long long *out) { return read_and_clear_unit_error(out); }

}  // namespace pkv
