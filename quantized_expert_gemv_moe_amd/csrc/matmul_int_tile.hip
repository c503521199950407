// Large tiles of the 8-bit integer products: their instantiations (the kernel is in matmul_tile.h).
#include "matmul_tile.h"

namespace moe {

void launch_matmul_int_tile(const MatmulIntArgs &a, const MatmulChoice &c, hipStream_t s) {
    launch_tile_dtype<MOE_DTYPE_I8>(a, c, s);
}

}  // namespace moe
