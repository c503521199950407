// Small tiles of the unquantised products: their instantiations (the kernel is in matmul_deep.h).
#include "matmul_deep.h"

namespace moe {

void launch_matmul_deep(int dtype, const MatmulArgs &a, const MatmulChoice &c, void *ws, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_deep_dtype<MOE_DTYPE_BF16>(a, c, ws, s); break;
        case MOE_DTYPE_F16: launch_deep_dtype<MOE_DTYPE_F16>(a, c, ws, s); break;
        default: launch_deep_dtype<MOE_DTYPE_F32>(a, c, ws, s); break;
    }
}

}  // namespace moe
