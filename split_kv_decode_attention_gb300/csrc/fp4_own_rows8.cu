// fp4_own_rows8.cu -- the 4-bit kernel for tiles of 8 query rows per KV head, of a
// tree or a padded batch.
#define DATTN_ROWS 1
#include "fp4_kernel.cuh"

namespace dattn {
namespace fp4 {
DATTN_FP4_VARIANTS(1)
}  // namespace fp4
}  // namespace dattn
