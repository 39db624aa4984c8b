// split_rows.cu -- the split kernel for the rows of a tree or of a padded batch.
#define DATTN_ROWS 1
#include "split_kernel.cuh"

namespace dattn {

cudaError_t launch_split_rows(const CUtensorMap& k_map, const CUtensorMap& v_map, const SplitArgs& a,
                              bool cluster_merge, cudaStream_t stream) {
  return launch_narrow(k_map, v_map, a, cluster_merge, stream);
}

}  // namespace dattn
