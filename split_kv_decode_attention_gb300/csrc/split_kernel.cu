// split_kernel.cu -- launch of the split kernel (split_kernel.cuh), and what the
// planner asks about it.

#include "split_kernel.cuh"

namespace dattn {

cudaError_t launch_split(const CUtensorMap& k_map, const CUtensorMap& v_map, const SplitArgs& a,
                         bool cluster_merge, cudaStream_t stream) {
  if (a.rows > kMaxNarrowRows) return launch_wide(k_map, v_map, a, stream);
  if (a.own.on) return launch_split_rows(k_map, v_map, a, cluster_merge, stream);
  return launch_narrow(k_map, v_map, a, cluster_merge, stream);
}

int split_box_tokens(int rows, bool fp8, bool paged, int64_t ctas) {
  if (paged || rows > kMaxNarrowRows) return kTileTokens;  // pages, or the tcgen05 kernel
  if (fp8) return kTileTokens * (rows <= 8 ? Variant<1, false, true>::kTps
                                           : Variant<2, false, true>::kTps);
  return kTileTokens * (deep_grid(false, ctas) ? Variant<1, false, false, true>::kTps
                                               : Variant<1, false, false>::kTps);
}

int split_ctas_per_sm(int rows, bool fp8) {
  if (rows > kMaxNarrowRows) return wide_ctas_per_sm();
  if (fp8) return rows <= 8 ? ctas_per_sm_nt<1, true>() : ctas_per_sm_nt<2, true>();
  return rows <= 8 ? ctas_per_sm_nt<1, false>() : ctas_per_sm_nt<2, false>();
}

bool split_cluster_merge_fits(int rows, bool fp8, int num_splits, int64_t num_clusters) {
  if (num_splits < 2 || num_splits > kMaxCluster || num_clusters < 1 || rows > kMaxNarrowRows)
    return false;
  const bool deep = deep_grid(fp8, num_splits * num_clusters);  // as launch_split decides
  const int n = fp8 ? (rows <= 8 ? max_active_clusters<1, true>(num_splits)
                                 : max_active_clusters<2, true>(num_splits))
                    : deep ? (rows <= 8 ? max_active_clusters<1, false, true>(num_splits)
                                        : max_active_clusters<2, false, true>(num_splits))
                           : (rows <= 8 ? max_active_clusters<1, false>(num_splits)
                                        : max_active_clusters<2, false>(num_splits));
  // all clusters resident at once: in multi-wave grids the idle CTAs of short
  // requests hold slots (GB300 sweeps: 1.5-2x slower than partials + combine)
  return n >= num_clusters;
}

}  // namespace dattn
