// fp4_rows16.cu -- the 4-bit kernel for tiles of 16 query rows per KV head.
#include "fp4_kernel.cuh"

namespace dattn {
namespace fp4 {
DATTN_FP4_VARIANTS(2)
}  // namespace fp4
}  // namespace dattn
