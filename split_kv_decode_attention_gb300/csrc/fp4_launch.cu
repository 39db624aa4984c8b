// fp4_launch.cu -- choice and launch of the variants of the 4-bit kernel.

#include <mutex>

#include "kernels.cuh"

namespace dattn {
namespace fp4 {
// (fp4_kernel.cuh; one translation unit per row-tile count defines each)
template <int NT>
struct Variants {
  static cudaError_t launch(int hg, bool cluster, const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream);
  static cudaError_t prepare(int hg, int* ctas);
  static cudaError_t clusters(int splits, int* n);
  static int warps();
};
}  // namespace fp4

namespace {

constexpr int kMaxDev = 64;
constexpr int kMaxCluster = 16;
std::mutex g_mu;
int g_ctas[3][4][kMaxDev];                    // resident CTAs per SM by row tiles and heads; 0: not prepared
int g_clusters[3][kMaxCluster + 1][kMaxDev];  // clusters that fit, plus one; 0: not asked

int variant_of(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : 2; }

cudaError_t current(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  return *dev < 0 || *dev >= kMaxDev ? cudaErrorInvalidDevice : cudaSuccess;
}

cudaError_t prepare(int rows, int hg, int* ctas) {
  int dev = 0;
  cudaError_t e = current(&dev);
  if (e != cudaSuccess) return e;
  const int v = variant_of(rows);
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = g_ctas[v][hg == 8 ? 3 : hg >> 1][dev];
  if (n == 0) {
    int got = 0;
    e = v == 0 ? fp4::Variants<1>::prepare(hg, &got)
        : v == 1 ? fp4::Variants<2>::prepare(hg, &got) : fp4::Variants<4>::prepare(hg, &got);
    if (e != cudaSuccess) return e;
    n = got > 0 ? got : 1;
  }
  if (ctas != nullptr) *ctas = n;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_fp4(const Fp4Maps& maps, const SplitArgs& a, int heads_per_cta, bool cluster_merge,
                       cudaStream_t stream) {
  const cudaError_t e = prepare(a.rows, heads_per_cta, nullptr);
  if (e != cudaSuccess) return e;
  switch (variant_of(a.rows)) {
    case 0: return fp4::Variants<1>::launch(heads_per_cta, cluster_merge, maps, a, stream);
    case 1: return fp4::Variants<2>::launch(heads_per_cta, cluster_merge, maps, a, stream);
    default: return fp4::Variants<4>::launch(heads_per_cta, cluster_merge, maps, a, stream);
  }
}

int fp4_warps(int rows) {
  switch (variant_of(rows)) {
    case 0: return fp4::Variants<1>::warps();
    case 1: return fp4::Variants<2>::warps();
    default: return fp4::Variants<4>::warps();
  }
}

int fp4_ctas_per_sm(int rows, int heads_per_cta) {
  int n = 0;
  return prepare(rows, heads_per_cta, &n) == cudaSuccess ? n : 1;
}

bool fp4_cluster_merge_fits(int rows, int num_splits, int64_t num_clusters) {
  int dev = 0;
  if (num_splits < 2 || num_splits > kMaxCluster || current(&dev) != cudaSuccess) return false;
  const int v = variant_of(rows);
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = g_clusters[v][num_splits][dev];
  if (n == 0) {
    int got = 0;
    const cudaError_t e = v == 0 ? fp4::Variants<1>::clusters(num_splits, &got)
                          : v == 1 ? fp4::Variants<2>::clusters(num_splits, &got)
                                   : fp4::Variants<4>::clusters(num_splits, &got);
    if (e != cudaSuccess) return false;
    n = got + 1;
  }
  return num_clusters < n;
}

}  // namespace dattn
