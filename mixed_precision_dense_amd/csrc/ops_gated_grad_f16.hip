// Instances of the tiled op kernel for f16 inputs, gradients of gated products (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, false, 256>(OpParams);
template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, false, 128>(OpParams);
template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, false, 64>(OpParams);
template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_F16, OP_GATED_GRAD, false, true, 64>(OpParams);

int launch_gated_grad_f16(bool tb, int tile, const OpParams &p, void *stream) {
    return tb ? launch_op_tile<IN_F16, OP_GATED_GRAD, false, true>(tile, p, (hipStream_t)stream)
              : launch_op_tile<IN_F16, OP_GATED_GRAD, false, false>(tile, p, (hipStream_t)stream);
}

}  // namespace mpg
