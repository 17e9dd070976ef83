// mpgemm_ops_api.hip -- the device-facing part of the epilogue, grouped and linear cross entropy
// products: each entry point checks its arguments, fills the kernels' arguments and queues its
// kernels.  No device memory is allocated and nothing waits for the device.
#include <hip/hip_runtime.h>

#include <string.h>

#include "mpgemm.h"
#include "mpgemm_handle.hpp"
#include "mpgemm_host.hpp"
#include "mpgemm_ops.hpp"
#include "mpgemm_ops_host.hpp"

using namespace mpg_host;

namespace {

// Rows of `ld` elements that start and end on 128-byte lines: whole tiles of them are stored past
// the caches, which are left to the operands.
bool lines(const void *base, int64_t ld, int bytes) { return ((uintptr_t)base & 127) == 0 && (ld * bytes) % 128 == 0; }

mpg::OpParams product(const OpPlan &plan, int64_t m, int64_t n, int64_t k, float alpha, const void *A, int64_t lda,
                      const void *B, int64_t ldb, void *D, bool d_f32, int64_t ldd) {
    mpg::OpParams p = {};
    p.A = A;
    p.B = B;
    p.lda = lda;
    p.ldb = ldb;
    p.m = (int)m;
    p.n = (int)n;
    p.k = (int)k;
    p.tiles_m = (int)plan.tiles_m;
    p.tiles_n = (int)plan.tiles_n;
    p.alpha = alpha;
    p.mode = mpg::OP_FORWARD;
    p.D = D;
    p.d_f32 = d_f32;
    p.ldd = ldd;
    p.splits = 1;
    p.k_split = (int)k;
    p.lines = lines(D, ldd, d_f32 ? 4 : 2);
    return p;
}

void set_epilogue(mpg::OpParams &p, const mpgemm_epilogue_t *e) {
    p.act = e->act;
    p.bias = e->bias;
    p.bias_f32 = e->bias_type == MPGEMM_R_32F;
    p.bias_stride = e->bias_stride;
    p.aux = e->aux;
    p.ld_aux = e->ld_aux;
    if (e->aux && !lines(e->aux, e->ld_aux, 2)) p.lines = 0;
}

void set_slope(mpg::OpParams &p, mpgemm_act_t act, const void *Z, int64_t ldz, float *dbias, void *workspace) {
    p.mode = mpg::OP_SLOPE;
    p.act = act;
    p.aux = act == MPGEMM_ACT_NONE ? nullptr : const_cast<void *>(Z);
    p.ld_aux = ldz;
    p.colsum = dbias ? (float *)workspace : nullptr;
    p.ld_colsum = round8(p.n);
}

mpgemm_status_t queued(int e) { return e == 0 ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_LAUNCH_FAILED; }

mpgemm_status_t launch(const OpPlan &plan, bool bf16, bool ta, bool tb, const mpg::OpParams &p, void *stream) {
    if (plan.skinny)
        return queued((bf16 ? mpg::launch_skinny_bf16 : mpg::launch_skinny_f16)(ta, tb, plan.fm, plan.w, plan.waves, p, stream));
    if (p.mode == mpg::OP_CE_STATS || p.mode == mpg::OP_CE_PROBS) return queued(mpg::launch_ce(bf16, plan.rows, p, stream));
    const auto f = p.mode == mpg::OP_SLOPE ? (bf16 ? mpg::launch_slope_bf16 : mpg::launch_slope_f16)
                                           : (bf16 ? mpg::launch_forward_bf16 : mpg::launch_forward_f16);
    return queued(f(ta, tb, plan.rows, p, stream));
}

mpgemm_status_t launch_dbias(const OpPlan &plan, const mpg::OpParams &p, float *dbias, void *stream) {
    return queued(mpg::launch_colsum(p, plan.rows, plan.skinny ? 1 : 2, dbias, stream));
}

}  // namespace

#define MPGEMM_TRY(call)                              \
    do {                                              \
        const mpgemm_status_t st_ = (call);           \
        if (st_ != MPGEMM_STATUS_SUCCESS) return st_; \
    } while (0)

extern "C" {

mpgemm_status_t mpgemm_run_epilogue(mpgemm_handle_t handle, mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n,
                                    int64_t k, const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                    const void *B, mpgemm_dtype_t b_type, int64_t ldb, const mpgemm_epilogue_t *epilogue,
                                    const float *beta, const void *C, mpgemm_dtype_t c_type, int64_t ldc, void *D,
                                    mpgemm_dtype_t d_type, int64_t ldd, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_epilogue(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, epilogue, beta, C, c_type,
                                     ldc, D, d_type, ldd));
    if (m == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const bool ta = transa == MPGEMM_OP_T, tb = transb == MPGEMM_OP_T;
    const bool read_c = !beta_is_zero(beta, MPGEMM_R_32F);
    const OpPlan plan = op_plan(m, n, k, tb, forward_weight(epilogue->act, epilogue->aux != nullptr, read_c));
    mpg::OpParams p = product(plan, m, n, k, *alpha, A, lda, B, ldb, D, d_type == MPGEMM_R_32F, ldd);
    set_epilogue(p, epilogue);
    if (read_c) {
        p.beta = *beta;
        p.C = C;
        p.c_f32 = c_type == MPGEMM_R_32F;
        p.ldc = ldc;
    }
    return launch(plan, a_type == MPGEMM_R_16BF, ta, tb, p, stream);
}

mpgemm_status_t mpgemm_run_epilogue_grad(mpgemm_handle_t handle, mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n,
                                         int64_t k, const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                         const void *B, mpgemm_dtype_t b_type, int64_t ldb, mpgemm_act_t act, const void *Z,
                                         int64_t ldz, void *D, mpgemm_dtype_t d_type, int64_t ldd, float *dbias, void *workspace,
                                         uint64_t workspace_bytes, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_epilogue_grad(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, act, Z, ldz, D, d_type,
                                          ldd, dbias, workspace, workspace_bytes));
    if (n == 0 || (m == 0 && !dbias)) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const bool ta = transa == MPGEMM_OP_T, tb = transb == MPGEMM_OP_T;
    const OpPlan plan = op_plan(m, n, k, tb, slope_weight(act));
    mpg::OpParams p = product(plan, m, n, k, *alpha, A, lda, B, ldb, D, d_type == MPGEMM_R_32F, ldd);
    set_slope(p, act, Z, ldz, dbias, workspace);
    if (m == 0) {
        p.tiles_m = 0;   // no rows: only their sum is written
    } else {
        // one row tile of the few rows' kernel: its partial sums are the sums
        const bool direct = dbias && plan.skinny && plan.tiles_m == 1;
        if (direct) {
            p.colsum = dbias;
            p.ld_colsum = 0;
        }
        MPGEMM_TRY(launch(plan, a_type == MPGEMM_R_16BF, ta, tb, p, stream));
        if (direct) return MPGEMM_STATUS_SUCCESS;
    }
    return dbias ? launch_dbias(plan, p, dbias, stream) : MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t mpgemm_run_grouped(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                   const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda, const int32_t *offsets,
                                   const void *B, mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                   const mpgemm_epilogue_t *epilogue, void *D, mpgemm_dtype_t d_type, int64_t ldd, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_grouped(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b, epilogue,
                                    D, d_type, ldd));
    if (groups == 0 || rows == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const bool tb = transb == MPGEMM_OP_T;
    const OpPlan plan = grouped_plan(rows, groups, n, k, tb, forward_weight(epilogue->act, epilogue->aux != nullptr, false));
    mpg::OpParams p = product(plan, rows, n, k, *alpha, A, lda, B, ldb, D, d_type == MPGEMM_R_32F, ldd);
    set_epilogue(p, epilogue);
    p.groups_kind = mpg::GROUPS_ROWS;
    p.groups = (int)groups;
    p.offsets = offsets;
    p.stride_b = stride_b;
    return launch(plan, a_type == MPGEMM_R_16BF, false, tb, p, stream);
}

mpgemm_status_t mpgemm_run_grouped_grad(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n,
                                        int64_t k, const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                        const int32_t *offsets, const void *B, mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                        mpgemm_act_t act, const void *Z, int64_t ldz, void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                        float *dbias, void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_grouped_grad(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b, act,
                                         Z, ldz, D, d_type, ldd, dbias, workspace, workspace_bytes));
    if (groups == 0 || n == 0 || (rows == 0 && !dbias)) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const bool tb = transb == MPGEMM_OP_T;
    const OpPlan plan = grouped_plan(rows, groups, n, k, tb, slope_weight(act));
    mpg::OpParams p = product(plan, rows, n, k, *alpha, A, lda, B, ldb, D, d_type == MPGEMM_R_32F, ldd);
    set_slope(p, act, Z, ldz, dbias, workspace);
    p.groups_kind = mpg::GROUPS_ROWS;
    p.groups = (int)groups;
    p.offsets = offsets;
    p.stride_b = stride_b;
    if (rows > 0) MPGEMM_TRY(launch(plan, a_type == MPGEMM_R_16BF, false, tb, p, stream));
    return dbias ? launch_dbias(plan, p, dbias, stream) : MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t mpgemm_run_grouped_wgrad(mpgemm_handle_t handle, int64_t groups, int64_t rows, int64_t m, int64_t n,
                                         const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda, const void *X,
                                         mpgemm_dtype_t x_type, int64_t ldx, const int32_t *offsets, const float *beta, void *D,
                                         mpgemm_dtype_t d_type, int64_t ldd, int64_t stride_d, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_grouped_wgrad(groups, rows, m, n, alpha, A, a_type, lda, X, x_type, ldx, offsets, beta, D, d_type, ldd,
                                          stride_d));
    if (groups == 0 || m == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const OpPlan plan = wgrad_plan(groups, rows, m, n);
    mpg::OpParams p = product(plan, m, n, rows, *alpha, A, lda, X, ldx, D, d_type == MPGEMM_R_32F, ldd);
    p.groups_kind = mpg::GROUPS_K;
    p.groups = (int)groups;
    p.offsets = offsets;
    p.stride_d = stride_d;
    if (!beta_is_zero(beta, MPGEMM_R_32F)) {
        p.beta = *beta;
        p.C = D;
        p.c_f32 = p.d_f32;
        p.ldc = ldd;
    }
    return launch(plan, a_type == MPGEMM_R_16BF, true, false, p, stream);
}

mpgemm_status_t mpgemm_run_linear_ce(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k, const float *alpha, const void *X,
                                     mpgemm_dtype_t type, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                     float *loss, float *lse, void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_linear_ce(m, n, k, alpha, X, type, ldx, W, ldw, target, loss, lse, workspace, workspace_bytes));
    if (m == 0) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    CeLayout L;
    if (!ce_layout(m, n, k, false, L)) return MPGEMM_STATUS_INTERNAL_ERROR;   // checked above
    const bool bf16 = type == MPGEMM_R_16BF;
    mpg::OpParams p = product(L.logits, m, n, k, *alpha, X, ldx, W, ldw, nullptr, true, 0);
    p.mode = mpg::OP_CE_STATS;
    p.stats = (mpg::CeStat *)workspace;
    p.parts = L.parts;
    MPGEMM_TRY(launch(L.logits, bf16, false, true, p, stream));
    return queued(mpg::launch_ce_merge(bf16, p.stats, L.parts, (int)m, (int)n, (int)k, *alpha, X, ldx, W, ldw, target, loss, lse,
                                       stream));
}

mpgemm_status_t mpgemm_run_linear_ce_grad(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k, const float *alpha,
                                          const void *X, mpgemm_dtype_t type, int64_t ldx, const void *W, int64_t ldw,
                                          const int64_t *target, const float *lse, const float *grad, void *dX, int64_t lddx,
                                          void *dW, int64_t lddw, void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!handle || !handle_live(handle)) return MPGEMM_STATUS_NOT_INITIALIZED;
    MPGEMM_TRY(mpgemm_check_linear_ce_grad(m, n, k, alpha, X, type, ldx, W, ldw, target, lse, grad, dX, lddx, dW, lddw, workspace,
                                           workspace_bytes));
    if (k == 0 || (!dX && !dW) || (m == 0 && !dW)) return MPGEMM_STATUS_SUCCESS;
    MPGEMM_TRY(handle_on_device(handle));
    const bool bf16 = type == MPGEMM_R_16BF;
    if (m == 0) {   // a sum over no rows
        const OpPlan plan = op_plan(n, k, 0, false, 0.0);
        return launch(plan, bf16, true, false, product(plan, n, k, 0, 0.0f, nullptr, 8, nullptr, 8, dW, false, lddw), stream);
    }
    CeLayout L;
    if (!ce_layout(m, n, k, true, L)) return MPGEMM_STATUS_INTERNAL_ERROR;   // checked above
    char *ws = (char *)workspace;
    const mpg::CeRows rows = {(float *)ws, (float *)(ws + L.off_lse), (int64_t *)(ws + L.off_target), (int *)(ws + L.off_place),
                              L.listed ? (int *)(ws + L.off_source) : nullptr, (float *)(ws + L.off_scale),
                              (int *)(ws + L.off_scale) + 1};
    float *part = (float *)(ws + L.off_dx);
    void *probs = ws + L.off_probs;
    const int64_t ld_part = round8(k);
    MPGEMM_TRY(queued(mpg::launch_ce_rows(bf16, (int)m, (int)n, target, lse, grad, rows, stream)));
    const int *count = L.listed ? rows.count : nullptr;
    if (L.listed) {   // from here on X is its rows that count
        MPGEMM_TRY(queued(mpg::launch_gather_rows(X, ldx, rows.source, rows.count, (int)m, (int)k, ws + L.off_x, round8(k), stream)));
        X = ws + L.off_x;
        ldx = round8(k);
    }
    for (int64_t c = 0; c < L.pieces; ++c) {
        const int64_t first = c * L.piece, have = n - first < L.piece ? n - first : L.piece;
        const char *w = (const char *)W + first * ldw * 2;
        const OpPlan lp = op_plan(m, have, k, true, kProbsWeight);
        mpg::OpParams p = product(lp, m, have, k, *alpha, X, ldx, w, ldw, probs, false, L.piece);
        p.mode = mpg::OP_CE_PROBS;
        p.target = rows.target;
        p.lse = rows.lse;
        p.weight = rows.weight;
        p.count = count;
        p.col0 = (int)first;
        MPGEMM_TRY(launch(lp, bf16, false, true, p, stream));
        if (dW) {
            const OpPlan plan = op_plan(have, k, m, false, 0.0);
            mpg::OpParams q = product(plan, have, k, m, *alpha, probs, L.piece, X, ldx, (char *)dW + first * lddw * 2, false, lddw);
            q.scale = rows.scale;
            q.count = count;
            q.count_k = 1;
            q.target = rows.target;
            MPGEMM_TRY(L.outer ? queued(mpg::launch_outer(bf16, q, stream)) : launch(plan, bf16, true, false, q, stream));
        }
        if (dX) {
            mpg::OpParams q = product(L.dx, m, k, have, 1.0f, probs, L.piece, w, ldw, part, true, ld_part);
            q.splits = (int)((have + L.k_split - 1) / L.k_split);
            q.k_split = (int)L.k_split;
            q.stride_split = m * ld_part;
            q.count = count;
            if (c > 0) {   // added to what the pieces before have summed
                q.beta = 1.0f;
                q.C = part;
                q.c_f32 = 1;
                q.ldc = ld_part;
            }
            MPGEMM_TRY(launch(L.dx, bf16, false, false, q, stream));
        }
    }
    if (!dX) return MPGEMM_STATUS_SUCCESS;
    return queued(mpg::launch_sum_parts(bf16, part, L.splits, m * ld_part, ld_part, rows.place, (int)m, (int)k, *alpha, rows.scale, dX,
                                        lddx, stream));
}

}  // extern "C"
