// Instances of the gated product's kernel for few rows (instantiated explicitly: host code that only
// reaches a kernel through an inlined launcher does not reliably emit its launch stub).
#include "mpgemm_skinny_gated_kernel.hpp"

namespace mpg {

template __global__ void gated_skinny_kernel<IN_F16, false, 1, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, false, 1, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, false, 2, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, false, 2, 2, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, false, 2, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 1, 1, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 1, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 1, 2, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 2, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 2, 2, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 2, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_F16, true, 4, 2, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, false, 1, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, false, 1, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, false, 2, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, false, 2, 2, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, false, 2, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 1, 1, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 1, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 1, 2, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 2, 1, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 2, 2, 8>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 2, 4, 4>(OpParams);
template __global__ void gated_skinny_kernel<IN_BF16, true, 4, 2, 8>(OpParams);

template <int IN, bool TB>
static int by_shape(int fm, int w, int waves, const OpParams &p, hipStream_t s) {
    if constexpr (TB)
        if (fm == 1 && w == 1 && waves == 4) return launch_gated_skinny_shape<IN, TB, 1, 1, 4>(p, s);
    if (fm == 1 && w == 1 && waves == 8) return launch_gated_skinny_shape<IN, TB, 1, 1, 8>(p, s);
    if constexpr (TB)
        if (fm == 1 && w == 2 && waves == 4) return launch_gated_skinny_shape<IN, TB, 1, 2, 4>(p, s);
    if constexpr (!TB)
        if (fm == 1 && w == 4 && waves == 4) return launch_gated_skinny_shape<IN, TB, 1, 4, 4>(p, s);
    if (fm == 2 && w == 1 && waves == 8) return launch_gated_skinny_shape<IN, TB, 2, 1, 8>(p, s);
    if (fm == 2 && w == 2 && waves == 8) return launch_gated_skinny_shape<IN, TB, 2, 2, 8>(p, s);
    if (fm == 2 && w == 4 && waves == 4) return launch_gated_skinny_shape<IN, TB, 2, 4, 4>(p, s);
    if constexpr (TB)
        if (fm == 4 && w == 2 && waves == 8) return launch_gated_skinny_shape<IN, TB, 4, 2, 8>(p, s);
    return (int)hipErrorInvalidValue;
}

int launch_gated_skinny(bool bf16, bool tb, int fm, int w, int waves, const OpParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (bf16) return tb ? by_shape<IN_BF16, true>(fm, w, waves, p, s) : by_shape<IN_BF16, false>(fm, w, waves, p, s);
    return tb ? by_shape<IN_F16, true>(fm, w, waves, p, s) : by_shape<IN_F16, false>(fm, w, waves, p, s);
}

}  // namespace mpg
