// Instances of the tiled op kernel for the cross entropy, both input types (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_F16, OP_CE_STATS, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_F16, OP_CE_STATS, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_F16, OP_CE_STATS, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_F16, OP_CE_PROBS, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_F16, OP_CE_PROBS, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_F16, OP_CE_PROBS, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_STATS, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_STATS, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_STATS, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_PROBS, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_PROBS, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, OP_CE_PROBS, false, true, 64>(OpParams);

template <int IN>
static int by_mode(int tile, const OpParams &p, hipStream_t s) {
    return p.mode == OP_CE_STATS ? launch_op_tile<IN, OP_CE_STATS, false, true>(tile, p, s)
                                 : launch_op_tile<IN, OP_CE_PROBS, false, true>(tile, p, s);
}

int launch_ce(bool bf16, int tile, const OpParams &p, void *stream) {
    return bf16 ? by_mode<IN_BF16>(tile, p, (hipStream_t)stream) : by_mode<IN_F16>(tile, p, (hipStream_t)stream);
}

}  // namespace mpg
