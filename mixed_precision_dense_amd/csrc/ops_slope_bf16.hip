// Instances of the tiled op kernel for bf16 inputs, gradients through an activation (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_SLOPE, true, true, 64>(OpParams);

int launch_slope_bf16(bool ta, bool tb, int tile, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (ta)
        return tb ? launch_op_tile<IN_BF16, OP_SLOPE, true, true>(tile, p, s)
                  : launch_op_tile<IN_BF16, OP_SLOPE, true, false>(tile, p, s);
    return tb ? launch_op_tile<IN_BF16, OP_SLOPE, false, true>(tile, p, s)
              : launch_op_tile<IN_BF16, OP_SLOPE, false, false>(tile, p, s);
}

}  // namespace mpg
