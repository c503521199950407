// Large tiles of the unquantised products: their instantiations (the kernel is in matmul_tile.h).
#include "matmul_tile.h"

namespace moe {

void launch_matmul_tile(int dtype, const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_tile_dtype<MOE_DTYPE_BF16>(a, c, s); break;
        case MOE_DTYPE_F16: launch_tile_dtype<MOE_DTYPE_F16>(a, c, s); break;
        default: launch_tile_dtype<MOE_DTYPE_F32>(a, c, s); break;
    }
}

}  // namespace moe
