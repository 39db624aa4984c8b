// fp4_launch.cu -- choice and launch of the variants of the 4-bit kernel.

#include <mutex>

#include "kernels.cuh"

namespace dattn {
namespace fp4 {
// (fp4_kernel.cuh; one translation unit per row-tile count defines each)
template <int NT, bool TR>
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
int g_ctas[2][3][4][kMaxDev];                    // resident CTAs per SM by form, row tiles and heads; 0: not prepared
int g_clusters[2][3][kMaxCluster + 1][kMaxDev];  // clusters that fit, plus one; 0: not asked

int variant_of(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : 2; }

cudaError_t current(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  return *dev < 0 || *dev >= kMaxDev ? cudaErrorInvalidDevice : cudaSuccess;
}

// f(Variants) for the row-tile count of `rows` and the form of the rows.
template <typename F>
auto with_variant(int rows, bool own_rows, F f) {
  switch (variant_of(rows)) {
    case 0: return own_rows ? f(fp4::Variants<1, true>()) : f(fp4::Variants<1, false>());
    case 1: return own_rows ? f(fp4::Variants<2, true>()) : f(fp4::Variants<2, false>());
    default: return own_rows ? f(fp4::Variants<4, true>()) : f(fp4::Variants<4, false>());
  }
}

cudaError_t prepare(int rows, bool own_rows, int hg, int* ctas) {
  int dev = 0;
  cudaError_t e = current(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = g_ctas[own_rows][variant_of(rows)][hg == 8 ? 3 : hg >> 1][dev];
  if (n == 0) {
    int got = 0;
    e = with_variant(rows, own_rows, [&](auto v) { return v.prepare(hg, &got); });
    if (e != cudaSuccess) return e;
    n = got > 0 ? got : 1;
  }
  if (ctas != nullptr) *ctas = n;
  return cudaSuccess;
}

bool clusters_fit(int rows, bool own_rows, int num_splits, int64_t num_clusters) {
  int dev = 0;
  if (num_splits < 2 || num_splits > kMaxCluster || current(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  int& n = g_clusters[own_rows][variant_of(rows)][num_splits][dev];
  if (n == 0) {
    int got = 0;
    if (with_variant(rows, own_rows, [&](auto v) { return v.clusters(num_splits, &got); }) != cudaSuccess)
      return false;
    n = got + 1;
  }
  return num_clusters < n;
}

}  // namespace

cudaError_t launch_fp4(const Fp4Maps& maps, const SplitArgs& a, int heads_per_cta, bool cluster_merge,
                       cudaStream_t stream) {
  const bool own_rows = a.own.on != 0;
  cudaError_t e = prepare(a.rows, own_rows, heads_per_cta, nullptr);
  // (the cluster form of the plain rows was prepared when the planner asked whether it fits)
  if (e == cudaSuccess && own_rows && cluster_merge && !clusters_fit(a.rows, true, a.num_splits, 1))
    return cudaErrorInvalidConfiguration;
  if (e != cudaSuccess) return e;
  return with_variant(a.rows, own_rows,
                      [&](auto v) { return v.launch(heads_per_cta, cluster_merge, maps, a, stream); });
}

// (the plans ask about the plain form; the other has its launch shape)
int fp4_warps(int rows) {
  return with_variant(rows, false, [](auto v) { return v.warps(); });
}

int fp4_ctas_per_sm(int rows, int heads_per_cta) {
  int n = 0;
  return prepare(rows, false, heads_per_cta, &n) == cudaSuccess ? n : 1;
}

bool fp4_cluster_merge_fits(int rows, int num_splits, int64_t num_clusters) {
  return clusters_fit(rows, false, num_splits, num_clusters);
}

}  // namespace dattn
