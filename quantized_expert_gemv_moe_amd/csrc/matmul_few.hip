// Few rows, unquantised: the instantiations of the kernel in matmul_few.h.
#include "matmul_few.h"

namespace moe {

void launch_matmul_few(int dtype, const MatmulArgs &a, const MatmulChoice &c, hipStream_t s) {
    switch (dtype) {
        case MOE_DTYPE_BF16: launch_few_dtype<MOE_DTYPE_BF16>(a, c, s); break;
        case MOE_DTYPE_F16: launch_few_dtype<MOE_DTYPE_F16>(a, c, s); break;
        default: launch_few_dtype<MOE_DTYPE_F32>(a, c, s); break;
    }
}

}  // namespace moe
