// paged_attn_decode_tree for fp16 queries: a unit of its own, to be compiled beside the other.
#include "tree_kernel.cuh"

namespace pkv {
namespace tree {

cudaError_t launch_fp16(const Args &a, int ctas, bool fp8, int D, const CUtensorMap &qmap,
                        const CUtensorMap &kvmap, cudaStream_t stream) {
  return launch_typed<FP16>(a, ctas, fp8, D, qmap, kvmap, stream);
}

}  // namespace tree

cudaError_t read_device_error_tree_fp16(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
