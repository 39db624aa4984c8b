// wide_rows.cu -- the tcgen05 kernel for the rows of a tree or of a padded batch.
#define DATTN_ROWS 1
#include "wide_kernel.cuh"

namespace dattn {

cudaError_t launch_wide_rows(const CUtensorMap& k_map, const CUtensorMap& v_map, const SplitArgs& a,
                             cudaStream_t stream) {
  return a.kv_fp8 ? launch_wide_t<DA_CACHE_FP8_E4M3>({k_map, v_map}, a, stream)
                  : launch_wide_t<DA_CACHE_BF16>({k_map, v_map}, a, stream);
}

cudaError_t launch_wide_fp4_rows(const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream) {
  return launch_wide_t<DA_CACHE_FP4_E2M1>({maps}, a, stream);
}

}  // namespace dattn
