// mpgemm_ops_host.cpp -- host-only part of the epilogue, grouped and linear cross entropy
// products declared in include/mpgemm.h: argument checks, the rules that choose a kernel and the
// workspaces' layouts.  No device call and no HIP header.
#include "mpgemm_ops_host.hpp"

#include "mpgemm_host.hpp"
#include "mpgemm_kinds.hpp"

namespace mpg_host {
namespace {

constexpr int kCus = 256;   // a whole MI355X: workspace sizes depend on the rules, not on a handle

bool aligned(const void *p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }
int64_t at_least1(int64_t v) { return v > 1 ? v : 1; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Largest leading dimension of elements of eb bytes (256 rows span less than 2^31 bytes).
int64_t max_ld(int eb) { return (((int64_t)1 << 31) - 4096) / (256 * (int64_t)eb); }
bool op_valid(mpgemm_op_t t) { return t == MPGEMM_OP_N || t == MPGEMM_OP_T; }
bool half_type(mpgemm_dtype_t t) { return t == MPGEMM_R_16F || t == MPGEMM_R_16BF; }
// Types of outputs and of what epilogues read: the inputs' type or FP32.
bool out_type(int t, mpgemm_dtype_t in) { return t == in || t == MPGEMM_R_32F; }
bool act_valid(int a) { return a >= MPGEMM_ACT_NONE && a <= MPGEMM_ACT_SILU; }
// A stride that the kernels' addressing covers, in whole 16-byte blocks.
bool stride_ok(int64_t ld, int eb) { return ld <= max_ld(eb) && (ld * eb) % 16 == 0; }

OpPlan tiled(int64_t m, int64_t n, int edge) {
    return OpPlan{false, 0, 0, 0, edge, edge, ceil_div(m, edge), ceil_div(n, edge)};
}

// The kernel for few rows: tiles_m row tiles of 16 fm rows, columns in blocks of 16 w.  Eight waves share
// k where there are at most two workgroups per CU (1 x 4096 x 4096: 9.4 us, 11.3 with four), else
// four, whose shorter ends overlap with other workgroups' loads (64 rows over 32 experts, 1408 x
// 2048: 32 us, 40 with eight).
OpPlan skinny(int64_t tiles_m, int64_t n, int fm, int w) {
    const int64_t tiles_n = ceil_div(n, 16 * w);
    const int waves = fm == 4 || (w < 4 && tiles_m * tiles_n <= 2 * kCus) ? 8 : 4;
    return OpPlan{true, fm, w, waves, 16 * fm, 16 * w, tiles_m, tiles_n};
}

// Estimated time (us) of tiles of an edge with a summed length k and an epilogue of a weight.  A
// 256-wide tile has a CU to itself; two workgroups of 128-wide ones or four of 64-wide ones share
// a CU, which hides their epilogues but reads the LDS more often per product.  Fitted to BF16 products
// of 512^2 to 4096^2 with k of 256, 1024 and 3000 (stages come in pairs of 128 k): a round of a tile per CU,
// and one that fills the CUs, take (us)
//   256: 18 - 22, 28 - 36, 57 - 78        128: 9, 14, 36 and 10, 21, 52
//    64: 5, 7, 22 and 8, 17, 46
// and in between a round grows with every 256 tiles.
double tiles_time(int edge, int64_t tiles, int64_t k, double weight) {
    struct Fit { int per_cu; double alone, alone_k, full, full_k, per_weight; };
    const Fit f = edge == 256 ? Fit{1, 15.5, 0.0195, 15.5, 0.0195, 5.0}
                  : edge == 128 ? Fit{2, 6.0, 0.0098, 6.0, 0.0155, 1.7} : Fit{4, 3.2, 0.006, 4.0, 0.014, 1.0};
    const double kk = (double)ceil_div(k, 128) * 128.0, epilogue = f.per_weight * weight;
    const double alone = f.alone + f.alone_k * kk + epilogue, full = f.full + f.full_k * kk + epilogue;
    const int64_t slots = f.per_cu * kCus, left = tiles % slots;
    double last = 0.0;
    if (left > 0) last = f.per_cu == 1 ? alone : alone + (full - alone) * (double)(ceil_div(left, kCus) - 1) / (double)(f.per_cu - 1);
    return (double)(tiles / slots) * full + last;
}

// The edge with the least estimated time; tiles(edge) counts the tiles.
template <typename Tiles>
int best_edge(int64_t k, double weight, Tiles &&tiles) {
    int best = 256;
    for (int e = 128; e >= 64; e /= 2)
        if (tiles_time(e, tiles(e), k, weight) < tiles_time(best, tiles(best), k, weight)) best = e;
    return best;
}

// Launches have a 32-bit number of lanes: at most this many workgroups of 256 or 512.
bool launchable(const OpPlan &p, int64_t times) {
    const int64_t most = (int64_t)UINT32_MAX / (p.skinny ? 512 : 256);
    return p.tiles_m <= most && p.tiles_n <= most && times <= most && p.tiles_m * p.tiles_n <= most &&
           p.tiles_m * p.tiles_n * times <= most;
}

}  // namespace

// Weights measured per 256-wide tile, in units of 5 us.
double forward_weight(int act, bool aux, bool c) {
    const double acts[] = {0.0, 0.0, 1.5, 0.7, 0.5};
    return acts[act] + (aux ? 0.7 : 0.0) + (c ? 1.4 : 0.0);
}
double slope_weight(int act) {
    const double acts[] = {0.0, 0.5, 2.2, 1.7, 1.2};
    return acts[act];
}

// Few rows go to their own kernel as long as its workgroups are few: beyond that the tiled kernel's
// stages stream B faster.  Measured (us, few rows' kernel / 64-wide tiles):
//   up to 16 rows:  1 x 4096 x 4096 9.4 with 16 columns a workgroup (13.9 with 32);
//                   8 x 32000 x 4096 57 / 61 where B is n x k and a workgroup takes 64 columns (63 with
//                   16), 50 / 45 where B is k x n
//   up to 32 rows:  32 x 8192 x 4096 23 / 29; 16 x 32000 x 4096 70 / 61
//   up to 64 rows:  37 x 5000 x 1001 7.4 / 8.4; 64 x 4096 x 4096 27 / 28; 64 x 8192 x 4096 30 / 30;
//                   64 x 117760 x 1725 185 / 96
//   more rows:      108 x 751 x 1408 10 / 6
OpPlan op_plan(int64_t m, int64_t n, int64_t k, bool tb, double weight) {
    const int64_t cols64 = ceil_div(n, 64);
    if (m <= 16 && n <= ((int64_t)1 << 22) && (tb || cols64 < 384)) return skinny(1, n, 1, cols64 >= 384 ? 4 : (tb ? 1 : 2));
    if (m <= 32 && cols64 < 384) return skinny(1, n, 2, 2);
    if (m <= 64 && ceil_div(n, 32) <= kCus) return skinny(1, n, 4, 2);
    return tiled(m, n, best_edge(k, weight, [&](int64_t e) { return ceil_div(m, e) * ceil_div(n, e); }));
}

// The same for experts' rows (us, few rows' kernel / best tiled one):
//   64 rows of 32 experts, 1408 x 2048: 32 with 16 columns (41 with 64) / 46 where B is n x k,
//   33 with 64 columns (36 with 32) / 37 where it is k x n; 256 rows: 45 / 49 and 37 / 41;
//   512 rows: 54 / 49 and 48 / 42; 215 rows of 4 experts, 504 x 1832: 10.6 with 32 rows / 13.2
OpPlan grouped_plan(int64_t rows, int64_t groups, int64_t n, int64_t k, bool tb, double weight) {
    const int64_t mean = ceil_div(rows, groups > 0 ? groups : 1);
    const int64_t owners = groups < rows ? groups : rows;   // an expert's last tile may be short
    const bool many = owners * ceil_div(n, 64) >= 384;
    if (mean <= 10 && n <= ((int64_t)1 << 22))
        return skinny(rows / 16 + owners, n, 1, many && (!tb || mean > 5) ? 4 : (tb ? 1 : 2));
    if (mean <= 64 && (rows / 32 + owners) * ceil_div(n, 32) <= kCus) return skinny(rows / 32 + owners, n, 2, 2);
    // half a tile per expert is lost on average
    OpPlan p = tiled(rows, n, best_edge(k, weight, [&](int64_t e) { return (rows / e + owners / 2) * ceil_div(n, e); }));
    p.tiles_m = rows / p.rows + owners;
    return p;
}

OpPlan wgrad_plan(int64_t groups, int64_t rows, int64_t m, int64_t n) {
    return tiled(m, n, best_edge(rows / (groups > 0 ? groups : 1), 0.0,
                                 [&](int64_t e) { return groups * ceil_div(m, e) * ceil_div(n, e); }));
}

int64_t colsum_rows(int64_t groups, int64_t m) {
    // two partial rows per row tile of at least 64 rows, or one per tile of at least 16
    return m / 16 + 2 * (groups > 0 ? groups : 1);
}

// dW over few rows is bound by its stores (us, tiles / the kernel for few summed rows):
//   24 x 100112 x 1781 165 / 108; 16 x 100112 x 2048 177 / 87; 64 x 32000 x 4096 111 / 72;
//   96 x 32000 x 4096 117 / 80; 128 x 32000 x 4096 119 / 96; 128 x 4096 x 1024 8.3 / 6.3
// More rows leave it one wave per SIMD (160 x 32000 x 4096 137 / 141).  Its grid is a multiple of
// eight times k's strips.
static bool outer_plan(int64_t m, int64_t k) { return m <= 128 && k <= ((int64_t)1 << 20); }

bool ce_layout(int64_t m, int64_t n, int64_t k, bool train, CeLayout &L) {
    if (m < 0 || n < 1 || k < 0 || m > kOpMaxSize || n > kOpMaxSize || k > kOpMaxSize) return false;
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    L.logits = op_plan(m, n, k, true, kStatsWeight);
    L.parts = (int)(L.logits.tiles_n * (L.logits.skinny ? 1 : 2));
    const uint64_t stats = up((uint64_t)m * (uint64_t)L.parts * 8);
    L.piece = n;
    L.pieces = 1;
    L.splits = 1;
    L.k_split = n;
    L.listed = false;
    L.outer = false;
    L.off_lse = L.off_target = L.off_source = L.off_place = L.off_scale = L.off_x = L.off_probs = L.off_dx = 0;
    L.total = stats;
    if (!train || m == 0) return true;
    // Probabilities of one piece at a time, at most 128 MiB of them (or 256 columns): half of the
    // memory-side cache, and enough columns for products of full speed.
    int64_t most = ((int64_t)128 << 20) / (2 * m) / 256 * 256;
    most = most < 256 ? 256 : (most > ((int64_t)1 << 20) ? (int64_t)1 << 20 : most);
    L.pieces = ceil_div(n, most);
    L.piece = ceil_div(ceil_div(n, L.pieces), 256) * 256;
    L.pieces = ceil_div(n, L.piece);
    L.logits = op_plan(m, L.piece, k, true, kProbsWeight);
    L.dw = op_plan(L.piece, k, m, false, 0.0);
    L.outer = outer_plan(m, k);
    // dX sums over a whole piece, which is cut into ranges where its tiles do not fill the CUs; their
    // FP32 parts are written and read once more, at 4 TB/s.
    const int64_t have = n < L.piece ? n : L.piece;
    const int64_t most_splits = ceil_div(have, 512) < 128 ? ceil_div(have, 512) : 128;
    // (The few rows' kernel needs as many ranges and reads lines by halves: 24 rows, k = 1781, 100112 columns
    // 115 us with 13 ranges, 83 with 64-wide tiles and 16; 16 rows, 4096, 32000: 44 against 42.)
    double least = 0.0;
    for (int e = 256; e >= 64; e /= 2)
        for (int64_t s = 1; s <= most_splits; s += 1 + s / 8) {
            const double t = tiles_time(e, ceil_div(m, e) * ceil_div(k, e) * s, ceil_div(have, s), 1.4) +
                             (double)s * (double)m * (double)k * 8.0 / 4.0e6;
            if (least == 0.0 || t < least) {
                least = t;
                L.dx = tiled(m, k, e);
                L.splits = (int)s;
            }
        }
    L.k_split = ceil_div(ceil_div(have, L.splits), 64) * 64;
    L.splits = (int)ceil_div(have, L.k_split);
    // (The kernel for few summed rows leaves them out by itself.)  Loss and gradient, us with rows as they
    // are / listed: 256 x 32000 x 4096 375 / 381 where all count, 371 / 360 where half do; 200 x 5000 x 512
    // 42.5 / 47.2; 500 x 32000 x 2048 290 / 295, 288 / 271 with 3 in 10 left out.
    L.listed = !L.outer;
    const uint64_t rows = (uint64_t)m, row_x = L.listed ? (uint64_t)round8(k) * 2 : 0;
    L.off_lse = up(rows * 4);
    L.off_target = L.off_lse + up(rows * 4);
    L.off_source = L.off_target + up(rows * 8);
    L.off_place = L.off_source + (L.listed ? up(rows * 4) : 0);
    L.off_scale = L.off_place + up(rows * 4);
    L.off_x = L.off_scale + 256;
    L.off_probs = L.off_x + up(rows * row_x);
    L.off_dx = L.off_probs + up(rows * (uint64_t)L.piece * 2);
    const unsigned __int128 total = (unsigned __int128)L.off_dx + (unsigned __int128)L.splits * (uint64_t)m * (uint64_t)round8(k) * 4;
    if (total > ((unsigned __int128)1 << 62)) return false;
    L.total = (uint64_t)total > stats ? (uint64_t)total : stats;
    return true;
}

}  // namespace mpg_host

using namespace mpg_host;

namespace {

// What every product checks of its operands: types, leading dimensions, and (once there is
// something to compute) pointers, alignment and strides.
mpgemm_status_t check_types(mpgemm_dtype_t a, mpgemm_dtype_t b, mpgemm_dtype_t d) {
    return a == b && half_type(a) && out_type(d, a) ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_NOT_SUPPORTED;
}

mpgemm_status_t check_epilogue_arg(const mpgemm_epilogue_t *e, mpgemm_dtype_t in, int64_t n, bool grouped) {
    if (!e || !act_valid(e->act)) return MPGEMM_STATUS_INVALID_VALUE;
    if (e->bias && !out_type(e->bias_type, in)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (e->bias && grouped && e->bias_stride < 0) return MPGEMM_STATUS_INVALID_VALUE;
    if (e->aux && e->ld_aux < at_least1(n)) return MPGEMM_STATUS_INVALID_VALUE;
    return MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t check_epilogue_layout(const mpgemm_epilogue_t *e) {
    if (e->bias && !aligned(e->bias, e->bias_type == MPGEMM_R_32F ? 4 : 2)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (e->aux && (!aligned(e->aux, 16) || !stride_ok(e->ld_aux, 2))) return MPGEMM_STATUS_NOT_SUPPORTED;
    return MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t check_workspace(const void *ws, uint64_t bytes, uint64_t need) {
    if (need == 0) return MPGEMM_STATUS_SUCCESS;
    if (!ws || bytes < need) return MPGEMM_STATUS_INVALID_VALUE;
    return aligned(ws, 256) ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_NOT_SUPPORTED;
}

}  // namespace

#define MPGEMM_TRY(call)                                          \
    do {                                                          \
        const mpgemm_status_t st_ = (call);                       \
        if (st_ != MPGEMM_STATUS_SUCCESS) return st_;             \
    } while (0)

extern "C" {

mpgemm_status_t mpgemm_check_epilogue(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                      const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                      const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                      const mpgemm_epilogue_t *epilogue, const float *beta, const void *C,
                                      mpgemm_dtype_t c_type, int64_t ldc, const void *D, mpgemm_dtype_t d_type,
                                      int64_t ldd) {
    if (!op_valid(transa) || !op_valid(transb) || m < 0 || n < 0 || k < 0 || !alpha || !beta) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_types(a_type, b_type, d_type));
    const bool read_c = !beta_is_zero(beta, MPGEMM_R_32F);
    if (read_c && !out_type(c_type, a_type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    MPGEMM_TRY(check_epilogue_arg(epilogue, a_type, n, false));
    const bool ta = transa == MPGEMM_OP_T, tb = transb == MPGEMM_OP_T;
    if (lda < at_least1(ta ? m : k) || ldb < at_least1(tb ? k : n) || ldd < at_least1(n) || (read_c && ldc < at_least1(n)))
        return MPGEMM_STATUS_INVALID_VALUE;
    if (m == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    if (!D || (k > 0 && (!A || !B)) || (read_c && !C)) return MPGEMM_STATUS_INVALID_VALUE;
    if (m > kOpMaxSize || n > kOpMaxSize || k > kOpMaxSize || !launchable(op_plan(m, n, k, tb, forward_weight(epilogue->act, epilogue->aux != nullptr, read_c)), 1))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if ((k > 0 && (!aligned(A, 16) || !aligned(B, 16))) || !aligned(D, 16) || (read_c && !aligned(C, 16)))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(lda, 2) || !stride_ok(ldb, 2) || !stride_ok(ldd, elem_bytes(d_type)) ||
        (read_c && !stride_ok(ldc, elem_bytes(c_type))))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return check_epilogue_layout(epilogue);
}

uint64_t mpgemm_epilogue_grad_workspace_size(int64_t groups, int64_t m, int64_t n) {
    if (groups < 1 || m < 1 || n < 1 || m > kOpMaxSize || n > kOpMaxSize || groups > 65535) return 0;
    return (uint64_t)colsum_rows(groups, m) * (uint64_t)round8(n) * 4;
}

mpgemm_status_t mpgemm_check_epilogue_grad(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                           const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                           const void *B, mpgemm_dtype_t b_type, int64_t ldb, mpgemm_act_t act,
                                           const void *Z, int64_t ldz, const void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                           const float *dbias, const void *workspace, uint64_t workspace_bytes) {
    if (!op_valid(transa) || !op_valid(transb) || m < 0 || n < 0 || k < 0 || !alpha || !act_valid(act)) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_types(a_type, b_type, d_type));
    const bool ta = transa == MPGEMM_OP_T, tb = transb == MPGEMM_OP_T, read_z = act != MPGEMM_ACT_NONE;
    if (lda < at_least1(ta ? m : k) || ldb < at_least1(tb ? k : n) || ldd < at_least1(n) || (read_z && ldz < at_least1(n)))
        return MPGEMM_STATUS_INVALID_VALUE;
    if (n == 0 || (m == 0 && !dbias)) return MPGEMM_STATUS_SUCCESS;
    if (m > kOpMaxSize || n > kOpMaxSize || k > kOpMaxSize || !launchable(op_plan(m, n, k, tb, slope_weight(act)), 1))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!aligned(dbias, 4)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (m == 0) return MPGEMM_STATUS_SUCCESS;   // (the sum of no rows is written)
    if (!D || (k > 0 && (!A || !B)) || (read_z && !Z)) return MPGEMM_STATUS_INVALID_VALUE;
    if ((k > 0 && (!aligned(A, 16) || !aligned(B, 16))) || !aligned(D, 16) || (read_z && !aligned(Z, 16)))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(lda, 2) || !stride_ok(ldb, 2) || !stride_ok(ldd, elem_bytes(d_type)) || (read_z && !stride_ok(ldz, 2)))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return dbias ? check_workspace(workspace, workspace_bytes, mpgemm_epilogue_grad_workspace_size(1, m, n)) : MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t mpgemm_check_grouped(mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n, int64_t k, const float *alpha,
                                     const void *A, mpgemm_dtype_t a_type, int64_t lda, const int32_t *offsets, const void *B,
                                     mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b, const mpgemm_epilogue_t *epilogue,
                                     const void *D, mpgemm_dtype_t d_type, int64_t ldd) {
    if (!op_valid(transb) || groups < 0 || rows < 0 || n < 0 || k < 0 || !alpha || stride_b < 0) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_types(a_type, b_type, d_type));
    MPGEMM_TRY(check_epilogue_arg(epilogue, a_type, n, true));
    const bool tb = transb == MPGEMM_OP_T;
    if (lda < at_least1(k) || ldb < at_least1(tb ? k : n) || ldd < at_least1(n)) return MPGEMM_STATUS_INVALID_VALUE;
    if (groups == 0 || rows == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    if (!D || !offsets || (k > 0 && (!A || !B))) return MPGEMM_STATUS_INVALID_VALUE;
    if (rows > kOpMaxSize || n > kOpMaxSize || k > kOpMaxSize || groups > 65535 || 
        !launchable(grouped_plan(rows, groups, n, k, tb, forward_weight(epilogue->act, epilogue->aux != nullptr, false)), 1))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if ((k > 0 && (!aligned(A, 16) || !aligned(B, 16))) || !aligned(D, 16) || !aligned(offsets, 4)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(lda, 2) || !stride_ok(ldb, 2) || !stride_ok(ldd, elem_bytes(d_type)) || stride_b % 8 || stride_b > INT64_MAX / 131072)
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return check_epilogue_layout(epilogue);
}

mpgemm_status_t mpgemm_check_grouped_grad(mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                          const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                          const int32_t *offsets, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                          int64_t stride_b, mpgemm_act_t act, const void *Z, int64_t ldz, const void *D,
                                          mpgemm_dtype_t d_type, int64_t ldd, const float *dbias, const void *workspace,
                                          uint64_t workspace_bytes) {
    if (!act_valid(act)) return MPGEMM_STATUS_INVALID_VALUE;
    const mpgemm_epilogue_t none = {MPGEMM_ACT_NONE, nullptr, MPGEMM_R_32F, 0, nullptr, 0};
    MPGEMM_TRY(mpgemm_check_grouped(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b, &none, D,
                                    d_type, ldd));
    const bool read_z = act != MPGEMM_ACT_NONE;
    if (read_z && ldz < at_least1(n)) return MPGEMM_STATUS_INVALID_VALUE;
    if (groups == 0 || n == 0 || (rows == 0 && !dbias)) return MPGEMM_STATUS_SUCCESS;
    if (groups > 65535 || n > kOpMaxSize || !aligned(dbias, 4)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (rows == 0) return offsets ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_INVALID_VALUE;
    if (read_z && !Z) return MPGEMM_STATUS_INVALID_VALUE;
    if (read_z && (!aligned(Z, 16) || !stride_ok(ldz, 2))) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!launchable(grouped_plan(rows, groups, n, k, transb == MPGEMM_OP_T, slope_weight(act)), 1)) return MPGEMM_STATUS_NOT_SUPPORTED;
    return dbias ? check_workspace(workspace, workspace_bytes, mpgemm_epilogue_grad_workspace_size(groups, rows, n)) : MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t mpgemm_check_grouped_wgrad(int64_t groups, int64_t rows, int64_t m, int64_t n, const float *alpha, const void *A,
                                           mpgemm_dtype_t a_type, int64_t lda, const void *X, mpgemm_dtype_t x_type, int64_t ldx,
                                           const int32_t *offsets, const float *beta, const void *D, mpgemm_dtype_t d_type,
                                           int64_t ldd, int64_t stride_d) {
    if (groups < 0 || rows < 0 || m < 0 || n < 0 || !alpha || !beta) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_types(a_type, x_type, d_type));
    if (lda < at_least1(m) || ldx < at_least1(n) || ldd < at_least1(n)) return MPGEMM_STATUS_INVALID_VALUE;
    if (groups == 0 || m == 0 || n == 0) return MPGEMM_STATUS_SUCCESS;
    if (!D || !offsets || (rows > 0 && (!A || !X))) return MPGEMM_STATUS_INVALID_VALUE;
    if (rows > kOpMaxSize || m > kOpMaxSize || n > kOpMaxSize || groups > 65535 || !launchable(wgrad_plan(groups, rows, m, n), groups))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    const int ed = elem_bytes(d_type);
    if ((rows > 0 && (!aligned(A, 16) || !aligned(X, 16))) || !aligned(D, 16) || !aligned(offsets, 4)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(lda, 2) || !stride_ok(ldx, 2) || !stride_ok(ldd, ed)) return MPGEMM_STATUS_NOT_SUPPORTED;
    // the experts' D must not overlap: they are written at the same time
    if (groups > 1 && stride_d < (m - 1) * ldd + n) return MPGEMM_STATUS_INVALID_VALUE;
    if (stride_d < 0 || stride_d > INT64_MAX / 131072 || (groups > 1 && (stride_d * ed) % 16)) return MPGEMM_STATUS_NOT_SUPPORTED;
    return MPGEMM_STATUS_SUCCESS;
}

uint64_t mpgemm_linear_ce_workspace_size(int64_t m, int64_t n, int64_t k, mpgemm_dtype_t type, int train) {
    CeLayout L;
    if (!half_type(type) || !ce_layout(m, n, k, train != 0, L)) return 0;
    return m == 0 ? 0 : L.total;
}

mpgemm_status_t mpgemm_check_linear_ce(int64_t m, int64_t n, int64_t k, const float *alpha, const void *X, mpgemm_dtype_t type,
                                       int64_t ldx, const void *W, int64_t ldw, const int64_t *target, const float *loss,
                                       const float *lse, const void *workspace, uint64_t workspace_bytes) {
    if (m < 0 || n < 1 || k < 0 || !alpha) return MPGEMM_STATUS_INVALID_VALUE;
    if (!half_type(type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (ldx < at_least1(k) || ldw < at_least1(k)) return MPGEMM_STATUS_INVALID_VALUE;
    if (m == 0) return MPGEMM_STATUS_SUCCESS;
    if ((k > 0 && (!X || !W)) || !target || !loss || !lse) return MPGEMM_STATUS_INVALID_VALUE;
    CeLayout L;
    if (!ce_layout(m, n, k, false, L) || !launchable(L.logits, 1)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (k > 0 && (!aligned(X, 16) || !aligned(W, 16))) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(ldx, 2) || !stride_ok(ldw, 2) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return check_workspace(workspace, workspace_bytes, L.total);
}

mpgemm_status_t mpgemm_check_linear_ce_grad(int64_t m, int64_t n, int64_t k, const float *alpha, const void *X, mpgemm_dtype_t type,
                                            int64_t ldx, const void *W, int64_t ldw, const int64_t *target, const float *lse,
                                            const float *grad, const void *dX, int64_t lddx, const void *dW, int64_t lddw,
                                            const void *workspace, uint64_t workspace_bytes) {
    if (m < 0 || n < 1 || k < 0 || !alpha) return MPGEMM_STATUS_INVALID_VALUE;
    if (!half_type(type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (ldx < at_least1(k) || ldw < at_least1(k) || (dX && lddx < at_least1(k)) || (dW && lddw < at_least1(k)))
        return MPGEMM_STATUS_INVALID_VALUE;
    if (k == 0 || (!dX && !dW) || (m == 0 && !dW)) return MPGEMM_STATUS_SUCCESS;
    if (m > 0 && (!X || !W || !target || !lse || !grad)) return MPGEMM_STATUS_INVALID_VALUE;
    CeLayout L;
    if (!ce_layout(m, n, k, true, L)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (m > 0 && (!launchable(L.logits, 1) || !launchable(L.dx, L.splits) || !launchable(L.dw, 1))) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (m == 0 && !launchable(op_plan(n, k, 0, false, 0.0), 1)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (m > 0 && (!aligned(X, 16) || !aligned(W, 16) || !stride_ok(ldx, 2) || !stride_ok(ldw, 2) || !aligned(target, 8) ||
                  !aligned(lse, 4) || !aligned(grad, 4)))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (dX && (!aligned(dX, 16) || !stride_ok(lddx, 2))) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (dW && (!aligned(dW, 16) || !stride_ok(lddw, 2))) return MPGEMM_STATUS_NOT_SUPPORTED;
    return m == 0 ? MPGEMM_STATUS_SUCCESS : check_workspace(workspace, workspace_bytes, L.total);
}

}  // extern "C"
