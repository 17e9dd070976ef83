// mpgemm_ops.hpp -- what the host side and the kernels of the epilogue, grouped and linear
// cross entropy products share: the kernel arguments, the launchers and the rules that choose a
// kernel (plain C++, so that the rules also build as ordinary host code).
#pragma once

#include <stdint.h>

#include "mpgemm_kinds.hpp"

namespace mpg {

// The activations of mpgemm_act_t, in its order.
enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// What a tile's epilogue makes of v = alpha * acc.
enum OpMode {
    OP_FORWARD = 0,   // D = act(v + bias) + beta C, v + bias kept in aux
    OP_SLOPE = 1,     // D = v act'(aux), column sums of D per tile
    OP_CE_STATS = 2,  // per row: maximum and sum of exponentials over the tile's columns
    OP_CE_PROBS = 3,  // D = (exp(v - lse) - [column == target]) * row weight
    OP_GATED = 4,     // B is a pair: D = act(v + bias) * (v2 + bias2), both factors kept in aux
    OP_GATED_GRAD = 5,  // D = v u act'(g) and v act(g) with g, u from aux, column sums of both per tile
};
// How the rows of a product are divided among experts.
enum OpGroups {
    GROUPS_NONE = 0,
    GROUPS_ROWS = 1,  // rows of A and D are cut by the offsets, B and bias are the expert's own
    GROUPS_K = 2,     // the summed index is cut by the offsets, D is the expert's own
};

// Row statistics of one column range: the largest value (in units of log 2) and the sum of
// exp2(value - largest).
struct CeStat {
    float top, sum;
};

// Arguments of the op kernels (one struct, passed by value).
struct OpParams {
    const void *A, *B;
    int64_t lda, ldb;            // elements
    int m, n, k;                 // GROUPS_ROWS: m = all rows; GROUPS_K: k = all summed rows
    int tiles_m, tiles_n;        // GROUPS_ROWS: tiles_m = upper bound over all offsets
    float alpha, beta;
    int mode, act;
    const void *bias;            // nullptr: none
    int bias_f32;                // else the inputs' type
    int64_t bias_stride;         // elements between two experts' biases
    void *aux;                   // OP_FORWARD: written; OP_SLOPE: read; the inputs' type; or nullptr
    int64_t ld_aux;
    const void *C;               // nullptr: not read
    int c_f32;
    int64_t ldc;                 // (C is laid out over experts and ranges as D is)
    void *D;
    int d_f32;                   // else the inputs' type
    int64_t ldd;
    int lines;                   // D's (and aux's) rows are whole 128-byte lines
    int wide;                    // D's rows are a multiple of 32 KB apart
    float *colsum;               // OP_SLOPE: two rows of partial sums per row tile, or nullptr
    int64_t ld_colsum;
    int groups_kind, groups;
    const int *offsets;          // groups + 1
    int64_t stride_b, stride_d;  // elements between two experts' B (GROUPS_ROWS), D (GROUPS_K)
    int splits, k_split;         // the summed index in `splits` ranges of k_split, each with its D
    int64_t stride_split;        // elements between two ranges' D
    const float *scale;          // device factor of alpha, or nullptr
    const int *count;            // device count of the rows (count_k: of the summed index) that take
    int count_k;                 // part, at most m (k); nullptr: all of them
    // cross entropy
    const int64_t *target;
    const float *lse, *weight;
    CeStat *stats;               // stats[row * parts + part]
    int parts;
    int col0;                    // vocabulary index of column 0
    // gated products: elements from the gate's matrix to the up projection's of B, of aux (G, U), of D
    // (OP_GATED_GRAD: dG, dU) and of colsum
    int64_t stride_up, stride_aux, stride_du, stride_colsum;
    const void *bias_up;         // of bias's type and stride
    void *H;                     // OP_GATED_GRAD: receives act(g) u in the inputs' type, or nullptr
    int64_t ldh;
};

// ------------------------------------------------------------------------------- launchers
// (declared with void * streams so that this header stays free of HIP)
// the tiled kernel for p.mode; the cross entropy's are for A stored m x k and B stored n x k
int launch_forward_f16(bool ta, bool tb, int tile, const OpParams &p, void *stream);
int launch_forward_bf16(bool ta, bool tb, int tile, const OpParams &p, void *stream);
int launch_slope_f16(bool ta, bool tb, int tile, const OpParams &p, void *stream);
int launch_slope_bf16(bool ta, bool tb, int tile, const OpParams &p, void *stream);
int launch_ce(bool bf16, int tile, const OpParams &p, void *stream);
int launch_skinny_f16(bool ta, bool tb, int fm, int w, int waves, const OpParams &p, void *stream);
int launch_skinny_bf16(bool ta, bool tb, int fm, int w, int waves, const OpParams &p, void *stream);
int launch_gated_f16(bool tb, int tile, const OpParams &p, void *stream);
int launch_gated_bf16(bool tb, int tile, const OpParams &p, void *stream);
int launch_gated_grad_f16(bool tb, int tile, const OpParams &p, void *stream);
int launch_gated_grad_bf16(bool tb, int tile, const OpParams &p, void *stream);
int launch_gated_skinny(bool bf16, bool tb, int fm, int w, int waves, const OpParams &p, void *stream);
// D = alpha A^T B in the inputs' type for p.k <= 128, A and B stored k x m and k x n; rows of B whose
// p.target is negative are taken as zeros; no other operand
int launch_outer(bool bf16, const OpParams &p, void *stream);
// dbias from the tiles' partial column sums (rows_per_tile partial rows a tile); halves: 2 for a gated
// product, whose second sums lie stride_colsum further and whose dbias are n and n values an expert
int launch_colsum(const OpParams &p, int tile_rows, int rows_per_tile, int halves, float *dbias, void *stream);
// loss and log-sum-exp from the row statistics; X and W give the target's logit
int launch_ce_merge(bool bf16, const CeStat *stats, int parts, int m, int n, int k, float alpha,
                    const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                    float *loss, float *lse, void *stream);
// What the cross entropy's gradient takes from its rows, m entries each.
struct CeRows {
    float *weight, *lse;   // of a row; weight 0: its target does not count
    int64_t *target;       // -1: does not count
    int *place;            // row r is entry place[r] (-1: its target does not count)
    int *source;           // nullptr: rows stay where they are.  Else only those that count are listed: entry j is
                           // row source[j]
    float *scale;          // one factor common to the weights
    int *count;            // number of entries
};
// mass: nullptr, or what stands in for the targets: rows of mass 0 do not count, the others' exponentials are
// multiplied by theirs and no column is a target (kNoColumn)
int launch_ce_rows(bool bf16, int m, int n, const int64_t *target, const float *mass, const float *lse, const float *grad,
                   const CeRows &rows, void *stream);
constexpr int64_t kNoColumn = INT64_MAX / 2;
constexpr int kMostTop = 1024;   // entries of a teacher's row
// A teacher's top logits, as mpgemm_teacher_t gives them.
struct Teacher {
    int top;
    const int64_t *index;
    const float *logit;
    int64_t ld;
    float scale;
    const float *lse;   // or nullptr
};
// the loss from the statistics and the logits at the teacher's columns, which are formed and kept too: by the
// kernel that joins the statistics (itself) or by one before it
constexpr int kMergePicks = 32;   // entries of a row that the joining kernel's waves form in one turn
int launch_distill_merge(bool bf16, const Teacher &t, const CeStat *stats, int parts, int m, int n, int k, float alpha, const void *X,
                         int64_t ldx, const void *W, int64_t ldw, float *picked, float *loss, float *lse, bool itself, void *stream);
int launch_mass(const Teacher &t, int m, int n, float *level, float *mass, void *stream);
int launch_scatter(bool bf16, const Teacher &t, int m, int n, int first, int have, const float *level, const float *mass,
                   const float *lse, const float *picked, const int *place, const float *weight, void *P, int64_t ldp, void *stream);
// out row j (16-byte blocks, ld_out) = in row source[j], for count[0] rows of at most m
int launch_gather_rows(const void *in, int64_t ld_in, const int *source, const int *count, int m, int k, void *out, int64_t ld_out,
                       void *stream);
// out (rows x cols, 16 bit) = alpha * scale[0] * sum of `splits` FP32 parts; row r's are in row place[r], and
// a row without one is 0
int launch_sum_parts(bool bf16, const float *parts, int splits, int64_t stride, int64_t ld_part, const int *place, int rows,
                     int cols, float alpha, const float *scale, void *out, int64_t ld_out, void *stream);

// Log probabilities of m rows of n stored logits (ldz elements apart), each in `parts` of part_vectors
// 16-byte vectors.
constexpr int kLogprobPart = 131072;   // most elements of a part
enum LogitsType { LOGITS_F16 = 0, LOGITS_BF16 = 1, LOGITS_F32 = 2 };
struct LogprobParams {
    const void *Z;
    int64_t ldz;
    int m, n;
    float alpha;
    const int64_t *target;
    float *logprob, *lse, *entropy;   // each nullptr: not asked for
    int top;                          // 0: no alternatives
    int64_t *top_index;
    float *top_logprob;
    int64_t ld_top;
    int parts, part_vectors;
    float *stats;                     // parts > 1: four values a part
    uint64_t *keys;                   // and `top` keys a part
};
int launch_logprobs(int type, int waves, const LogprobParams &p, void *stream);

}  // namespace mpg
