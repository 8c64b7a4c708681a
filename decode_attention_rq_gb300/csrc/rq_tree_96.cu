// rq_tree_attention, heads of width 96 (a translation unit of its own: the two widths compile in parallel).
#include "rq_tree_kernels.cuh"

namespace rq {

cudaError_t launch_tree_mma_96(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream) {
  return launch_tree_d<96>(a, nb, num_sms, stream);
}

}  // namespace rq
