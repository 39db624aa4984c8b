// fp4_rows32.cu -- the 4-bit kernel for tiles of 32 query rows per KV head.
#include "fp4_kernel.cuh"

namespace dattn {
namespace fp4 {
DATTN_FP4_VARIANTS(4)
}  // namespace fp4
}  // namespace dattn
