// The 128 x 128 tile of the 8-bit integer products: its instantiations (the kernel is in matmul_tile.h).
#include "matmul_tile.h"

namespace moe {

void launch_matmul_int_tile4(const MatmulIntArgs &a, const MatmulChoice &c, hipStream_t s) {
    a.w_up ? launch_tile<MOE_DTYPE_I8, true, 4, 4>(a, c, s) : launch_tile<MOE_DTYPE_I8, false, 4, 4>(a, c, s);
}

}  // namespace moe
