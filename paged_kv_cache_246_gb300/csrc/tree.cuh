// What the units of speculative decoding over trees share: a sequence's tree
// among the step's tokens, and the arguments of its attention.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace tree {

// Sequence b's nodes: `nodes` of them from row `row` on.  False where cu_nodes
// says something that cannot be.
__device__ __forceinline__ bool nodes_of(const TreeBatch &t, int b, int &row, int &nodes) {
  row = __ldg(t.cu_nodes + b);
  const int end = __ldg(t.cu_nodes + b + 1);
  nodes = end - row;
  return row >= 0 && end >= row && end <= t.num_tokens && nodes <= t.max_nodes;
}

// paged_attn_decode_tree (tree.cu): rows of a query tile, keys of a key tile.
constexpr int BM = 128, BN = 128;

// The least that scores are multiplied by: 0 would make NaN of the hidden ones' -infinity.
constexpr float kTiniest = 0x1p-149f;

struct Args {
  TreeBatch tb;
  uint16_t *out;
  const uint16_t *query;
  const uint8_t *cache;
  const int32_t *block_tables, *seq_lens;
  const float *alibi;
  float *part_o;     // [CTA][2][D / 4][128][4]
  float2 *part_ml;   // [CTA][2][128]: maximum (log2 units), sum
  int4 *record;      // [CTA]: sequence, KV head, further CTAs, first node of the item that its last segment begins
  int64_t num_blocks, row_elems;
  int max_blocks_per_seq, max_seq_len, H, KVH, QPK, BS, window;
  int tile_nodes;  // nodes of a row tile: 128 / QPK
  int row_tiles;   // of the widest tree that may come
  int item_units;  // what an item costs beside its tiles, in tiles (0: items are not cut)
  float scale_log2, v_scale;
};

// tree_bf16.cu, tree_fp16.cu: the attention and the merge of its parts, `ctas` CTAs.
cudaError_t launch_bf16(const Args &a, int ctas, bool fp8, int D, const CUtensorMap &qmap,
                        const CUtensorMap &kvmap, cudaStream_t stream);
cudaError_t launch_fp16(const Args &a, int ctas, bool fp8, int D, const CUtensorMap &qmap,
                        const CUtensorMap &kvmap, cudaStream_t stream);

}  // namespace tree

cudaError_t read_device_error_tree_bf16(unsigned long long *out);
cudaError_t read_device_error_tree_fp16(unsigned long long *out);

}  // namespace pkv
