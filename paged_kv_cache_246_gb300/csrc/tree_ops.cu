// What follows a verify step over trees of drafted tokens: the walk down the
// tokens that the model would have taken (paged_attn_tree_accept), and the
// move of their keys and values behind the context (kv_commit_tree).
#include <algorithm>

#include "tree.cuh"

namespace pkv {
namespace tree {

constexpr int kMax = PKV_TREE_MAX_NODES;

// ---------------------------------------------------------------------------
// paged_attn_tree_accept: CTA = one warp = one sequence.  first[p] = the lowest
// child c of node p with draft[c] == target[p]: each lane looks at the nodes
// lane, lane + 32, ... at once; then one lane follows first[] from node 0.
// A tree of 64 nodes is 1.3 KB: bound by latency (three dependent loads and
// the path's steps of one shared-memory access each).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(32)
accept_kernel(const TreeBatch tb, int32_t *accepted, int max_accepted, int32_t *num_accepted,
              int64_t *next_token, const int64_t *draft, const int64_t *target) {
  __shared__ int64_t goal[kMax];
  __shared__ int first[kMax], path[kMax];
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x;
  int row, n;
  if (!nodes_of(tb, b, row, n)) {
    if (lane == 0) record_error(PKV_ERR_BOUNDS, b);
    n = 0;
  }
  for (int c = lane; c < n; c += 32) {
    goal[c] = __ldg(target + row + c);
    first[c] = kMax;
  }
  __syncwarp();
  for (int c = lane; c < n; c += 32) {
    const int p = __ldg(tb.parents + row + c);
    if (p < -1 || p >= c)
      record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(row) + c);
    else if (p >= 0 && __ldg(draft + row + c) == goal[p])
      atomicMin(&first[p], c);
  }
  __syncwarp();
  int count = 0;
  if (lane == 0 && n > 0) {
    // children come behind their parents: the walk ascends and ends
    int c = 0;
    do {
      path[count++] = c;
      c = first[c];
    } while (c < kMax && count < max_accepted);
  }
  count = __shfl_sync(0xffffffffu, count, 0);
  __syncwarp();
  int32_t *out = accepted + static_cast<int64_t>(b) * max_accepted;
  for (int i = lane; i < max_accepted; i += 32) out[i] = i < count ? path[i] : -1;
  if (lane == 0) {
    num_accepted[b] = count;
    next_token[b] = count > 0 ? goal[path[count - 1]] : -1;
  }
}

// ---------------------------------------------------------------------------
// kv_commit_tree: row positions ctx + path[i] -> ctx + i.  CTA (sequence,
// layer, piece of the row) moves the same 16-byte chunks of all the path's
// rows, thread by thread, in the path's order and eight at a time: path
// ascends, so path[i] >= i, and a row that is read later (path[j] > path[i] >=
// i) has not been written yet.  So a thread's order alone makes the move as if
// all were read first; no two threads touch the same bytes.
// ---------------------------------------------------------------------------
constexpr int kMaxLayers = 256;
struct Layers {
  uint4 *p[kMaxLayers];
};
constexpr int kCommitThreads = 256;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kCommitThreads)
commit_kernel(const __grid_constant__ Layers caches, const TreeBatch tb, const int32_t *accepted,
              int max_accepted, const int32_t *block_tables, int max_blocks_per_seq,
              const int32_t *seq_lens, int64_t num_blocks, int BS, int row_chunks) {
  __shared__ int64_t src[kMax], dst[kMax];
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.y;
  int row, n;
  bool ok = nodes_of(tb, b, row, n);
  const int L = __ldg(seq_lens + b);
  ok = ok && L >= n && L <= static_cast<int64_t>(max_blocks_per_seq) * BS;
  const int ctx = L - n;
  const int32_t *path = accepted + static_cast<int64_t>(b) * max_accepted;
  const int32_t *trow = block_tables + static_cast<int64_t>(b) * max_blocks_per_seq;
  bool bad = !ok, end = false;
  // max_accepted <= kMax = the CTA's threads: thread i looks at entry i
  const int i = threadIdx.x;
  int node = -1;
  if (ok && i < max_accepted) {
    node = __ldg(path + i);
    end = node < 0;
    if (!end) {
      const int before = i > 0 ? __ldg(path + i - 1) : -1;
      // behind the end of the path (before < 0) nothing is moved, whatever stands there
      if (i > 0 && before < 0) bad = true;
      if (node <= before || node >= n) bad = true;
      if (!bad) {
        auto slot = [&](int pos) -> int64_t {
          const int pb = __ldg(trow + pos / BS);
          if (pb < 0 || pb >= num_blocks) {
            bad = true;
            return 0;
          }
          return static_cast<int64_t>(pb) * BS + pos % BS;
        };
        src[i] = slot(ctx + node);
        dst[i] = slot(ctx + i);
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) record_error(PKV_ERR_BOUNDS, b);
    return;
  }
  const int count = __syncthreads_count(node >= 0);
  // chunk c of the two halves' rows: keys, then values
  const int64_t half = num_blocks * BS * row_chunks;
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kCommitThreads + threadIdx.x;
       c < 2 * row_chunks; c += static_cast<int64_t>(gridDim.x) * kCommitThreads) {
    uint4 *base = caches.p[blockIdx.z] + (c < row_chunks ? c : half + c - row_chunks);
    for (int k = 0; k < count; k += kBatch) {
      uint4 r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (k + u < count && src[k + u] != dst[k + u]) r[u] = base[src[k + u] * row_chunks];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (k + u < count && src[k + u] != dst[k + u]) base[dst[k + u] * row_chunks] = r[u];
    }
  }
}

}  // namespace tree

cudaError_t launch_tree_accept(int32_t *accepted, int max_accepted, int32_t *num_accepted,
                               int64_t *next_token, const int64_t *draft_tokens,
                               const int64_t *target_tokens, const TreeBatch &t,
                               cudaStream_t stream) {
  PdlLaunch cfg(dim3(t.num_seqs), 32, 0, stream);
  return cudaLaunchKernelEx(&cfg.c, tree::accept_kernel, t, accepted, max_accepted, num_accepted,
                            next_token, draft_tokens, target_tokens);
}

cudaError_t launch_commit_tree(void *const *caches, int num_layers, const int32_t *accepted,
                               int max_accepted, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens, const TreeBatch &t,
                               const Geometry &g, cudaStream_t stream) {
  static_assert(tree::kCommitThreads >= tree::kMax, "a thread per entry of the path");
  tree::Layers layers;
  for (int l = 0; l < tree::kMaxLayers; ++l)
    layers.p[l] = l < num_layers ? static_cast<uint4 *>(caches[l]) : nullptr;
  const int row_chunks = static_cast<int>(g.row_bytes / 16);
  const unsigned pieces = static_cast<unsigned>(std::min<int64_t>(
      (2LL * row_chunks + tree::kCommitThreads - 1) / tree::kCommitThreads, 1024));
  PdlLaunch cfg(dim3(pieces, t.num_seqs, num_layers), tree::kCommitThreads, 0, stream);
  return cudaLaunchKernelEx(&cfg.c, tree::commit_kernel, layers, t, accepted, max_accepted,
                            block_tables, max_blocks_per_seq, seq_lens, g.num_blocks, g.BS,
                            row_chunks);
}

cudaError_t read_device_error_tree_ops(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
