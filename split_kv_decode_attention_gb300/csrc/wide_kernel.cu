// wide_kernel.cu -- launch of the tcgen05 kernel (wide_kernel.cuh), and what the
// planner asks about it.

#include "wide_kernel.cuh"

namespace dattn {

cudaError_t launch_wide(const CUtensorMap& k_map, const CUtensorMap& v_map, const SplitArgs& a,
                        cudaStream_t stream) {
  if (a.own.on) return launch_wide_rows(k_map, v_map, a, stream);
  return a.kv_fp8 ? launch_wide_t<DA_CACHE_FP8_E4M3>({k_map, v_map}, a, stream)
                  : launch_wide_t<DA_CACHE_BF16>({k_map, v_map}, a, stream);
}

cudaError_t launch_wide_fp4(const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream) {
  if (a.own.on) return launch_wide_fp4_rows(maps, a, stream);
  return launch_wide_t<DA_CACHE_FP4_E2M1>({maps}, a, stream);
}

int wide_ctas_per_sm() {
  static int cached[64];  // per device, queried once
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (ensure_wide_attrs<DA_CACHE_BF16>(nullptr) != cudaSuccess) return 1;
  {
    std::lock_guard<std::mutex> lk(g_wide_mu);
    if (cached[dev] > 0) return cached[dev];
  }
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, wide_kernel<DA_CACHE_BF16, false, false>,
                                                    WCfg<DA_CACHE_BF16>::kThreads,
                                                    WCfg<DA_CACHE_BF16>::kSmemBytes) != cudaSuccess ||
      n < 1)
    return 1;
  std::lock_guard<std::mutex> lk(g_wide_mu);
  cached[dev] = n;
  return n;
}

}  // namespace dattn
