// Instances of the tiled op kernel for bf16 inputs (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_ops_kernel.hpp"

namespace mpg {

template __global__ void op_kernel<IN_BF16, false, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, false, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, false, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, false, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, false, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, false, true, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, true, false, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, true, false, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, true, false, 64>(OpParams);
template __global__ void op_kernel<IN_BF16, true, true, 256>(OpParams);
template __global__ void op_kernel<IN_BF16, true, true, 128>(OpParams);
template __global__ void op_kernel<IN_BF16, true, true, 64>(OpParams);

template <bool TA, bool TB>
static int by_tile(int tile, const OpParams &p, hipStream_t s) {
    switch (tile) {
    case 256: return launch_op<IN_BF16, TA, TB, 256>(p, s);
    case 128: return launch_op<IN_BF16, TA, TB, 128>(p, s);
    case 64: return launch_op<IN_BF16, TA, TB, 64>(p, s);
    default: return (int)hipErrorInvalidValue;
    }
}

int launch_op_bf16(bool ta, bool tb, int tile, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (ta) return tb ? by_tile<true, true>(tile, p, s) : by_tile<true, false>(tile, p, s);
    return tb ? by_tile<false, true>(tile, p, s) : by_tile<false, false>(tile, p, s);
}

}  // namespace mpg
