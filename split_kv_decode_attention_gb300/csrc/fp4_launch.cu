// fp4_launch.cu -- choice and launch of the variants of the 4-bit kernel.

#include <mutex>

#include "kernels.cuh"

namespace dattn {
namespace fp4 {
template <int NT>
struct Variants {
  static cudaError_t launch(int hg, const Fp4Maps& maps, const SplitArgs& a, cudaStream_t stream);
  static cudaError_t prepare(int hg, int* ctas);
  static int warps();
};
}  // namespace fp4

namespace {

constexpr int kMaxDev = 64;
std::mutex g_mu;
int g_ctas[3][4][kMaxDev];  // resident CTAs per SM by row tiles and heads; 0: not prepared

cudaError_t prepare(int rows, int hg, int* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  const int v = rows <= 8 ? 0 : rows <= 16 ? 1 : 2;
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

cudaError_t launch_fp4(const Fp4Maps& maps, const SplitArgs& a, int heads_per_cta, cudaStream_t stream) {
  const cudaError_t e = prepare(a.rows, heads_per_cta, nullptr);
  if (e != cudaSuccess) return e;
  return a.rows <= 8 ? fp4::Variants<1>::launch(heads_per_cta, maps, a, stream)
         : a.rows <= 16 ? fp4::Variants<2>::launch(heads_per_cta, maps, a, stream)
                        : fp4::Variants<4>::launch(heads_per_cta, maps, a, stream);
}

int fp4_warps(int rows) {
  return rows <= 8 ? fp4::Variants<1>::warps() : rows <= 16 ? fp4::Variants<2>::warps() : fp4::Variants<4>::warps();
}

int fp4_ctas_per_sm(int rows, int heads_per_cta) {
  int n = 0;
  return prepare(rows, heads_per_cta, &n) == cudaSuccess ? n : 1;
}

}  // namespace dattn
