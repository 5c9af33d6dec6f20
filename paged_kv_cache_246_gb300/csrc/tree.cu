// Host side of paged_attn_decode_tree: sizes, tensor maps, dispatch (the kernels
// are in tree_kernel.cuh).
#include <algorithm>

#include "tree.cuh"

namespace pkv {
namespace tree {

struct Plan {
  int tile_nodes, row_tiles, ctas, item_units;
  size_t part_o, part_ml, bytes;  // offsets behind the records, and the whole
};

static Plan plan(int num_seqs, int max_nodes, int max_seq_len, const Geometry &g, int sms) {
  Plan p{};
  p.tile_nodes = BM / g.QPK;
  p.row_tiles = (max_nodes + p.tile_nodes - 1) / p.tile_nodes;
  int64_t keys = max_seq_len;
  if (g.window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(g.window) + max_nodes + BN);
  const int64_t tiles = std::max<int64_t>(1, (keys + BN - 1) / BN);
  // Items (a sequence's KV head) of up to 2 tiles are not cut: the CTAs take
  // whole ones, and the merge of parts is not launched (one context of 250
  // tokens, 8 KV heads: 10.9 us, cut 12.6; of 500 14.0, cut 13.3).
  // What an item costs beside its tiles, in tiles: the softmax of its first and
  // last ones, the accumulators' way out, instructions that are not at hand
  // (3000 to 6000 cycles, a tile 2000).  These units come before the item's
  // tiles, so that a CTA whose share is short contexts has no more to do than the
  // others.  With 1 / 2 / 3 / 4 / 5 / 6 / 8 units (us), 16-bit cache: one context of
  // 32768 59 / 58 / 57 / 55 / 55 / 55 / 55, 64 of 4096 .. 16384 448 / 445 / 441 / 437 /
  // 434 / 435 / 431, 128 of 100 .. 4096 242 / 226 / 222 / 218 / 217 / 217 / 221, heads of 64
  // 145 / 145 / 146 / 145 / 146 / 146 / 147: equal within a hundredth from 4 to 6.  8-bit
  // cache: 128 contexts 251 / 235 / 221 / 210 / 201 / 197 / 195, 64 378 / 375 / 371 / 369 / 369 /
  // 365 / 364; fp16 queries 298 / 283 / 283 / 290 / 293 / 296 / 304.
  p.item_units = tiles <= 2 ? 0 : g.fp8 ? 6 : 4;
  const int64_t items = static_cast<int64_t>(num_seqs) * g.KVH * p.row_tiles;
  const int64_t units = p.item_units == 0 ? items : items * (tiles + p.item_units);
  p.ctas = static_cast<int>(std::min<int64_t>(sms, units));
  if (p.item_units == 0) return p;
  const size_t parts = static_cast<size_t>(p.ctas) * 2 * BM;
  p.part_ml = (static_cast<size_t>(p.ctas) * sizeof(int4) + 255) / 256 * 256;
  p.part_o = p.part_ml + parts * sizeof(float2);
  p.bytes = p.part_o + parts * g.D * sizeof(float);
  return p;
}

}  // namespace tree

size_t tree_workspace_bytes(int num_seqs, int max_nodes, int max_seq_len, const Geometry &g,
                            int sms) {
  return tree::plan(num_seqs, max_nodes, max_seq_len, g, sms).bytes;
}

cudaError_t launch_tree_decode(void *out, const void *query, const TreeBatch &t,
                               const void *kv_cache, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens, int max_seq_len,
                               const Geometry &g, void *workspace, cudaStream_t stream) {
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return e;
  const tree::Plan p = tree::plan(t.num_seqs, t.max_nodes, max_seq_len, g, dev.sms);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  tree::Args a{};
  a.tb = t;
  a.out = static_cast<uint16_t *>(out);
  a.query = static_cast<const uint16_t *>(query);
  a.cache = static_cast<const uint8_t *>(kv_cache);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.alibi = g.alibi;
  a.record = reinterpret_cast<int4 *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(ws + p.part_ml);
  a.part_o = reinterpret_cast<float *>(ws + p.part_o);
  a.num_blocks = g.num_blocks;
  a.row_elems = g.row_elems;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = std::min(max_seq_len, 0x7fff0000);  // tiles' ends stay within 32 bits
  a.H = g.H;
  a.KVH = g.KVH;
  a.QPK = g.QPK;
  a.BS = g.BS;
  a.window = g.window;
  a.tile_nodes = p.tile_nodes;
  a.row_tiles = p.row_tiles;
  a.item_units = p.item_units;
  a.scale_log2 = std::max(g.scale * kLog2e * g.k_scale, tree::kTiniest);
  a.v_scale = g.v_scale;
  const bool bf = g.dtype == PKV_BF16;
  const CUtensorMapDataType dt =
      bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap qmap, kvmap;
  {
    // the rows of 128 / QPK nodes and one KV head's query heads, 64 channels
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(g.D), static_cast<cuuint64_t>(g.H),
                                static_cast<cuuint64_t>(t.num_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(g.D) * 2,
                                   static_cast<cuuint64_t>(g.H) * g.D * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(g.QPK),
                               static_cast<cuuint32_t>(tree::BM / g.QPK)};
    if (encode_tensor_map(&qmap, dt, 3, const_cast<void *>(query), dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  {
    // 16-bit: 64-channel swizzled boxes of a cache block's rows; 8-bit: its whole
    // rows, swizzled by their length
    const cuuint64_t eb = static_cast<cuuint64_t>(g.elem_bytes);
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(g.D), static_cast<cuuint64_t>(g.KVH),
                                static_cast<cuuint64_t>(g.num_blocks * g.BS), 2};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(g.D) * eb,
                                   static_cast<cuuint64_t>(g.row_elems) * eb,
                                   static_cast<cuuint64_t>(g.num_blocks * g.block_elems) * eb};
    const cuuint32_t box[4] = {g.fp8 ? static_cast<cuuint32_t>(g.D) : 64u, 1,
                               static_cast<cuuint32_t>(g.BS), 1};
    const CUtensorMapSwizzle swz = !g.fp8 || g.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                         : CU_TENSOR_MAP_SWIZZLE_64B;
    // L2 fetches no more than the head's row: the next head's is another item's
    // (256 bytes at rows of 128: 64 contexts of 4096 .. 16384 over an 8-bit cache 396 us
    // against 369, with heads of 64 in 16 bits 318 against 296)
    const CUtensorMapL2promotion fetch = g.D * eb >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : g.D * eb == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                           : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    if (encode_tensor_map(&kvmap, g.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : dt, 4,
                          const_cast<void *>(kv_cache), dims, strides, box, swz, fetch) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return bf ? tree::launch_bf16(a, p.ctas, g.fp8, g.D, qmap, kvmap, stream)
            : tree::launch_fp16(a, p.ctas, g.fp8, g.D, qmap, kvmap, stream);
}

cudaError_t read_device_error_tree(unsigned long long *out) {
  // both are cleared; the first one that holds something is told
  unsigned long long other = 0;
  cudaError_t e = read_device_error_tree_bf16(out);
  if (e == cudaSuccess) e = read_device_error_tree_fp16(&other);
  if (*out == 0) *out = other;
  return e;
}

}  // namespace pkv
