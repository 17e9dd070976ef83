// Instances of the tiled op kernel for bf16 inputs, products with bias, activation and residual (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_FORWARD, true, true, 64>(OpParams);

int launch_forward_bf16(bool ta, bool tb, int tile, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (ta)
        return tb ? launch_op_tile<IN_BF16, OP_FORWARD, true, true>(tile, p, s)
                  : launch_op_tile<IN_BF16, OP_FORWARD, true, false>(tile, p, s);
    return tb ? launch_op_tile<IN_BF16, OP_FORWARD, false, true>(tile, p, s)
              : launch_op_tile<IN_BF16, OP_FORWARD, false, false>(tile, p, s);
}

}  // namespace mpg
