// Instances of the op kernel for few rows, f16 inputs (instantiated explicitly: host code that
// only reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_skinny_kernel.hpp"

namespace mpg {

template __global__ void skinny_kernel<IN_F16, false, false, 1, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, false, 1, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, false, 1, 4, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, false, 2, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, false, 2, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, false, 4, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 1, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 1, 1, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 1, 4, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 2, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 2, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, false, true, 4, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, false, 1, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, false, 1, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, false, 2, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, false, 2, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, false, 4, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 1, 1, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 1, 1, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 1, 4, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 2, 2, 4>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 2, 2, 8>(OpParams);
template __global__ void skinny_kernel<IN_F16, true, true, 4, 2, 8>(OpParams);

template <bool TA, bool TB>
static int by_shape(int fm, int w, int waves, const OpParams &p, hipStream_t s) {
    if (fm == 4 && w == 2) return launch_skinny_shape<IN_F16, TA, TB, 4, 2, 8>(p, s);
    if (fm == 2 && w == 2) return launch_skinny<IN_F16, TA, TB, 2, 2>(waves, p, s);
    if constexpr (!TA || TB)   // (k x n operands in 64 columns: experts' rows only, which are never transposed)
        if (fm == 1 && w == 4) return launch_skinny_shape<IN_F16, TA, TB, 1, 4, 4>(p, s);
    if (fm == 1 && w == (TB ? 1 : 2)) return launch_skinny<IN_F16, TA, TB, 1, TB ? 1 : 2>(waves, p, s);
    return (int)hipErrorInvalidValue;
}

int launch_skinny_f16(bool ta, bool tb, int fm, int w, int waves, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (ta) return tb ? by_shape<true, true>(fm, w, waves, p, s) : by_shape<true, false>(fm, w, waves, p, s);
    return tb ? by_shape<false, true>(fm, w, waves, p, s) : by_shape<false, false>(fm, w, waves, p, s);
}

}  // namespace mpg
