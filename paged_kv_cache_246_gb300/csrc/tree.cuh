// What the kernels of speculative decoding over trees (tree.cu, tree_ops.cu)
// share: a sequence's tree among the step's tokens.
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

}  // namespace tree
}  // namespace pkv
