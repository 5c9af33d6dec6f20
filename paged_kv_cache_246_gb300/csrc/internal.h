// Host-side interfaces between the libpkv translation units.  Arguments are
// validated by the front end (abi.cu) before any of these is called.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pkv.h"

namespace pkv {

// Validated, derived view of pkv_attn_params.
struct Geometry {
  int H, KVH, QPK, D, BS;
  int dtype;  // pkv_dtype
  float scale;
  const float *alibi;
  int window;            // <= 0: none
  int non_causal;        // 1: every query row sees its whole sequence
  int64_t num_blocks;    // blocks per cache half
  int64_t row_elems;     // KVH * D
  int64_t block_elems;   // BS * KVH * D
  bool fp8;              // cache holds E4M3 codes (1 byte per element)
  float k_scale, v_scale;
  int64_t elem_bytes;    // of the cache: 2, or 1 for fp8
  int64_t row_bytes;     // one token row of the cache
  int64_t block_bytes;   // one block of one cache half
};

// Streams/devices: the SM count and opt-in shared memory of the current device.
struct DeviceInfo {
  int device;
  int sms;
  int max_smem_optin;
};
cudaError_t current_device_info(DeviceInfo *out);

// Driver entry point for cuTensorMapEncodeTiled, resolved once.
CUresult encode_tensor_map(CUtensorMap *map, CUtensorMapDataType dtype, cuuint32_t rank,
                           void *base, const cuuint64_t *dims, const cuuint64_t *strides_bytes,
                           const cuuint32_t *box, CUtensorMapSwizzle swizzle,
                           CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);

// kv_ops.cu
cudaError_t launch_kv_write(const void *key, const void *value, int64_t num_tokens, void *kv_cache,
                            const int64_t *slot_mapping, const Geometry &g, cudaStream_t stream);
cudaError_t launch_kv_copy(void *const *caches, int num_layers, const int64_t *pairs,
                           int64_t num_pairs, const Geometry &g, cudaStream_t stream);
cudaError_t launch_kv_swap(const void *src, int64_t src_blocks, void *dst, int64_t dst_blocks,
                           const int64_t *pairs_host, int64_t num_pairs, const Geometry &g,
                           cudaStream_t stream);
cudaError_t read_device_error_kv_ops(unsigned long long *out);
cudaError_t launch_wait_timeout_check(int64_t tag, cudaStream_t stream);

// decode.cu (single- and multi-token decode)
struct DecodePlan {
  int row_groups;   // 16-row groups of (token, head) rows per KV head
  int split_units;  // 16-key units per split
  int max_splits;   // grid extent over splits (1 = no split, no workspace)
  size_t workspace_bytes;
};
// Decode context parallelism: this rank's place in the group and, for a
// rank's share, where its (o, m, l) go instead of the output (world 1, rank
// 0 and null pointers: a plain decode).
struct DcpShare {
  int world = 1, rank = 0;
  float *res_o = nullptr, *res_ml = nullptr;
};
DecodePlan plan_decode(int num_seqs, int query_len, int max_seq_len, const Geometry &g, int sms,
                       int dcp_world = 1);
cudaError_t launch_decode(void *out, const void *query, int num_seqs, int query_len,
                          const void *kv_cache, const int32_t *block_tables,
                          int max_blocks_per_seq, const int32_t *seq_lens, const Geometry &g,
                          const DecodePlan &plan, void *workspace, cudaStream_t stream,
                          const DcpShare &dcp = DcpShare{});
cudaError_t launch_dcp_combine(void *out, const float *parts_o, const float *parts_ml,
                              int num_parts, int64_t num_rows, const Geometry &g,
                              cudaStream_t stream);
cudaError_t read_device_error_decode(unsigned long long *out);
// Device address and size of the static decode scratch of `device`, which
// must be the current device (looked up on the first call per device).
cudaError_t static_decode_scratch(int device, void **ptr, size_t *bytes);

// rope.cu
struct RopeCall {
  void *query_out;
  int64_t query_out_stride;
  const void *query;
  int64_t query_stride;
  const void *key;
  int64_t key_stride;
  const void *value;
  int64_t value_stride;
  int64_t num_tokens;
  const int64_t *positions;
  const float *cos_sin;
  int64_t max_position;
  int32_t rot_dim, interleaved;
  void *kv_cache;
  const int64_t *slot_mapping;
  // positions of several axes: each pair's (host array), elements between them; null: one
  const uint8_t *pair_axes = nullptr;
  int64_t positions_stride = 0;
};
cudaError_t launch_rope_write(const RopeCall &r, const Geometry &g, cudaStream_t stream);
cudaError_t read_device_error_rope(unsigned long long *out);

// select.cu
cudaError_t launch_block_bounds(void *bounds, const void *kv_cache, const int32_t *block_tables,
                                int max_blocks_per_seq, const int32_t *context_lens,
                                const int32_t *seq_lens, int num_seqs, int max_new_tokens,
                                const Geometry &g, cudaStream_t stream);
struct SelectCall {
  int32_t *selected;
  int max_selected;
  const void *query;
  int num_seqs;
  const void *bounds;
  const int32_t *block_tables;
  int max_blocks_per_seq;
  const int32_t *seq_lens;
  int max_seq_len, num_sink, num_recent;
};
// Blocks of a sequence of max_seq_len tokens that a selection may score: those
// that the sliding window can reach.
inline int64_t scored_blocks(int64_t max_seq_len, const Geometry &g) {
  const int64_t window = static_cast<int64_t>(g.window) + g.BS;
  const int64_t span = g.window > 0 && window < max_seq_len ? window : max_seq_len;
  return (span + g.BS - 1) / g.BS;
}
cudaError_t launch_select(const SelectCall &s, const Geometry &g, cudaStream_t stream);
cudaError_t read_device_error_select(unsigned long long *out);

// sparse.cu
cudaError_t launch_sparse_decode(void *out, const void *query, int num_seqs, const void *kv_cache,
                                 const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *selected,
                                 int max_selected, const Geometry &g, cudaStream_t stream);
cudaError_t read_device_error_sparse(unsigned long long *out);

// tree.cu, tree_ops.cu (speculative decoding over trees)
struct TreeBatch {
  const int32_t *cu_nodes, *parents;
  int64_t num_tokens;
  int num_seqs, max_nodes;
};
cudaError_t launch_tree_decode(void *out, const void *query, const TreeBatch &t,
                               const void *kv_cache, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens, int max_seq_len,
                               const Geometry &g, void *workspace, cudaStream_t stream);
size_t tree_workspace_bytes(int num_seqs, int max_nodes, int max_seq_len, const Geometry &g,
                            int sms);
cudaError_t read_device_error_tree(unsigned long long *out);
cudaError_t launch_tree_accept(int32_t *accepted, int max_accepted, int32_t *num_accepted,
                               int64_t *next_token, const int64_t *draft_tokens,
                               const int64_t *target_tokens, const TreeBatch &t,
                               cudaStream_t stream);
cudaError_t launch_commit_tree(void *const *caches, int num_layers, const int32_t *accepted,
                               int max_accepted, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens, const TreeBatch &t,
                               const Geometry &g, cudaStream_t stream);
cudaError_t read_device_error_tree_ops(unsigned long long *out);

// Lets a kernel take as much dynamic shared memory as the device grants beside
// its static `reserved` bytes; asked once per kernel and device (`done`: a bit
// per device).
template <class K>
cudaError_t allow_shared_memory(K *kernel, std::atomic<uint64_t> &done, size_t reserved) {
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << dev.device;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           dev.max_smem_optin - static_cast<int>(reserved));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A kernel launch as a programmatic dependent of the kernel before it in the
// stream, in clusters of `cluster` CTAs along x (0: none).
struct PdlLaunch {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[2];
  PdlLaunch(dim3 grid, int threads, size_t smem, cudaStream_t stream, unsigned cluster = 0) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = at;
    c.numAttrs = 1;
    if (cluster) {
      at[1].id = cudaLaunchAttributeClusterDimension;
      at[1].val.clusterDim.x = cluster;
      at[1].val.clusterDim.y = 1;
      at[1].val.clusterDim.z = 1;
      c.numAttrs = 2;
    }
  }
  PdlLaunch(const PdlLaunch &) = delete;
};

// prefill.cu
cudaError_t launch_prefill(void *out, const void *query, int64_t num_q_tokens, int num_seqs,
                           const int32_t *cu_q, const int32_t *cu_k, int max_query_len,
                           int max_seq_len, const void *kv_cache, const int32_t *block_tables,
                           int max_blocks_per_seq, const Geometry &g, cudaStream_t stream);
cudaError_t read_device_error_prefill(unsigned long long *out);

}  // namespace pkv
