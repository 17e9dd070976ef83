// Instances of the op kernel for few rows, bf16 inputs (instantiated explicitly: host code that
// only reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_skinny_kernel.hpp"

namespace mpg {

template __global__ void skinny_kernel<IN_BF16, false, false, 1, 1>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, false, 1, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, false, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, false, 2, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, false, 4, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, true, 1, 1>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, true, 1, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, true, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, true, 2, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, false, true, 4, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, false, 1, 1>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, false, 1, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, false, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, false, 2, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, false, 4, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, true, 1, 1>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, true, 1, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, true, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, true, 2, 2>(OpParams);
template __global__ void skinny_kernel<IN_BF16, true, true, 4, 2>(OpParams);

template <bool TA, bool TB>
static int by_shape(int fm, int w, const OpParams &p, hipStream_t s) {
    switch (10 * fm + w) {
    case 11: return launch_skinny<IN_BF16, TA, TB, 1, 1>(p, s);
    case 12: return launch_skinny<IN_BF16, TA, TB, 1, 2>(p, s);
    case 14: return launch_skinny<IN_BF16, TA, TB, 1, 4>(p, s);
    case 22: return launch_skinny<IN_BF16, TA, TB, 2, 2>(p, s);
    case 42: return launch_skinny<IN_BF16, TA, TB, 4, 2>(p, s);
    default: return (int)hipErrorInvalidValue;
    }
}

int launch_skinny_bf16(bool ta, bool tb, int fm, int w, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (ta) return tb ? by_shape<true, true>(fm, w, p, s) : by_shape<true, false>(fm, w, p, s);
    return tb ? by_shape<false, true>(fm, w, p, s) : by_shape<false, false>(fm, w, p, s);
}

}  // namespace mpg
