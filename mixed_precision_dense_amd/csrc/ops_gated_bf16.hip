// Instances of the tiled op kernel for bf16 inputs, gated products (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_BF16, OP_GATED, false, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_GATED, false, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_GATED, false, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_GATED, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_GATED, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_GATED, false, true, 64>(OpParams);

int launch_gated_bf16(bool tb, int tile, const OpParams &p, void *stream) {
    return tb ? launch_op_tile<IN_BF16, OP_GATED, false, true>(tile, p, (hipStream_t)stream)
              : launch_op_tile<IN_BF16, OP_GATED, false, false>(tile, p, (hipStream_t)stream);
}

}  // namespace mpg
