// mpgemm_ops_host.hpp -- host-only rules of the epilogue, grouped and linear cross entropy
// products: which kernel takes a product and how the workspaces are laid out.  Plain C++.
#pragma once

#include <stdint.h>

#include "mpgemm.h"

namespace mpg_host {

constexpr int64_t kOpMaxSize = (int64_t)INT32_MAX - 255;   // sizes, rounded up to a tile, stay 32-bit

// The kernel of one product: the kernel for few rows (fm x w blocks of 16, four or eight waves) or a tile edge.
struct OpPlan {
    bool skinny;
    int fm, w, waves;
    int rows, cols;   // of D per workgroup
    int64_t tiles_m, tiles_n;
};
// How much an epilogue adds to a tile's time, for the rules below.
double forward_weight(int act, bool aux, bool c);
double slope_weight(int act);
constexpr double kStatsWeight = 0.7, kProbsWeight = 1.0;
// A product of m rows and n columns with a summed length k.
OpPlan op_plan(int64_t m, int64_t n, int64_t k, bool tb, double weight);
// A product of `rows` rows divided among `groups` experts; tiles_m is the most row tiles that
// any division can take.
OpPlan grouped_plan(int64_t rows, int64_t groups, int64_t n, int64_t k, bool tb, double weight);
// The products of each expert's rows summed: D is m x n for each.
OpPlan wgrad_plan(int64_t groups, int64_t rows, int64_t m, int64_t n);

// Rows of partial column sums, and their row length.
int64_t colsum_rows(int64_t groups, int64_t m);
inline int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

struct CeLayout {
    OpPlan logits;            // m x piece (or m x n without gradients)
    int parts;                // row statistics per row
    int64_t piece, pieces;    // vocabulary columns per piece of the gradient
    OpPlan dx, dw;
    bool outer;               // dW by the kernel for few summed rows instead of dw
    int splits;               // of the piece, in dX's product
    int64_t k_split;
    // Gradients of more rows first list those whose target counts and gather their X, so that rows
    // that do not (padding, a prompt) cost nothing in the products and nothing of their X reaches dW.
    bool listed;
    uint64_t off_lse, off_target, off_source, off_place, off_scale, off_x, off_probs, off_dx;   // bytes; weights at 0
    uint64_t total;           // also covers the row statistics of the forward pass, which start at 0
};
bool ce_layout(int64_t m, int64_t n, int64_t k, bool train, CeLayout &L);

}  // namespace mpg_host
