// mpgemm_ops_host.cpp -- host-only part of the epilogue, grouped and linear cross entropy
// products declared in include/mpgemm.h: argument checks, the rules that choose a kernel and the
// workspaces' layouts.  No device call and no HIP header.
#include "mpgemm_ops_host.hpp"

#include "mpgemm_host.hpp"
#include "mpgemm_kinds.hpp"
#include "mpgemm_ops.hpp"

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
// and in between a round grows with every 256 tiles.  crowded: what an epilogue of 64-wide tiles that fill the
// CUs costs, times one of its own (the gated products', which move two to five times as much as they compute).
double tiles_time(int edge, int64_t tiles, int64_t k, double weight, double crowded = 1.0) {
    struct Fit { int per_cu; double alone, alone_k, full, full_k, per_weight; };
    const Fit f = edge == 256 ? Fit{1, 15.5, 0.0195, 15.5, 0.0195, 5.0}
                  : edge == 128 ? Fit{2, 6.0, 0.0098, 6.0, 0.0155, 1.7} : Fit{4, 3.2, 0.006, 4.0, 0.014, 1.0};
    const double kk = (double)ceil_div(k, 128) * 128.0, epilogue = f.per_weight * weight;
    const double alone = f.alone + f.alone_k * kk + epilogue, full = f.full + f.full_k * kk + epilogue * (edge == 64 ? crowded : 1.0);
    const int64_t slots = f.per_cu * kCus, left = tiles % slots;
    double last = 0.0;
    if (left > 0) last = f.per_cu == 1 ? alone : alone + (full - alone) * (double)(ceil_div(left, kCus) - 1) / (double)(f.per_cu - 1);
    return (double)(tiles / slots) * full + last;
}

// The edge with the least estimated time; tiles(edge) counts the tiles.
template <typename Tiles>
int best_edge(int64_t k, double weight, Tiles &&tiles, double crowded = 1.0) {
    int best = 256;
    for (int e = 128; e >= 64; e /= 2)
        if (tiles_time(e, tiles(e), k, weight, crowded) < tiles_time(best, tiles(best), k, weight, crowded)) best = e;
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

double gated_weight(int act, bool kept) { return 0.5 * forward_weight(act, false, false) + (kept ? 0.7 : 0.0); }
double gated_grad_weight(int act, bool h) { return slope_weight(act) + 1.5 + (h ? 0.7 : 0.0); }

// The shape of the gated product's kernel for few rows.  Measured (us; rows of 16 / columns of 16 /
// waves of a workgroup; BF16, B stored n x k unless "k x n"):
//   few workgroups (below 384 of 16 columns): eight waves and 16 columns, and above 16 rows 32 rows each
//     8 x 2501 x 1001 1/1/8 6.3, 1/2/8 7.1;  24 x 2501 x 1001 2/1/8 6.4, 2/2/8 8.0;  40 x 1408 x 2048 2/1/8 11.1,
//     4/2/8 17;  64 x 2501 x 1001 2/2/8 8.2, 2/1/8 above 9.9, 4/2/8 9.9;  k x n 8 x 1408 x 2048 1/1/8 10.3, 1/2/8 11.0
//   more of them: 1 x 8192 x 4096 1/1/4 27.3, 1/1/8 29.0;  16 x 8192 x 4096 1/2/4 31.2, 1/1/4 32.9;  8 x 14336 x 4096
//     1/2/4 53.7, 1/1/4 above 54;  24 x 14336 x 4096 2/4/4 56.1, 64-wide tiles 58.1;  64 x 8192 x 4096 4/2/8 42.6,
//     tiles 45.3;  k x n, whose rows come in pieces of 32 w bytes: 8 x 14336 x 4096 1/4/4 51.7, 1/2/4 70.5;
//     24 x 14336 x 4096 2/4/4 56.1, 2/2/8 76.6;  40 x 8192 x 4096 2/4/4 42.0, 4/2/8 42.8
//   experts, 1408 x 2048, 32 of them: 64 rows 1/1/4 60, 1/2/4 63 (k x n 1/4/4 61, 1/2/4 67);  256 rows 1/2/4 78, 1/1/4
//     81 (66, 84);  512 rows 2/4/4 88, 64-wide tiles 87 (78, 91)
static bool gated_few(int64_t groups, int64_t rows, int64_t n, bool tb, OpPlan &p) {
    const int64_t owners = groups < rows ? groups : rows;   // an expert's last tile may be short
    const int64_t mean = groups > 0 ? ceil_div(rows, groups) : rows;
    if (mean > 64 || n > ((int64_t)1 << 22)) return false;
    auto shape = [&](int fm, int w, int waves) {
        p = OpPlan{true, fm, w, waves, 16 * fm, 16 * w, groups > 0 ? rows / (16 * fm) + owners : ceil_div(rows, 16 * fm), ceil_div(n, 16 * w)};
        return true;
    };
    const int64_t strips = ceil_div(n, 16) * (groups > 0 ? owners : 1);
    if (strips < 384) {
        if (mean <= 16) return shape(1, 1, 8);
        return mean <= 32 || strips <= 128 ? shape(2, 1, 8) : shape(2, 2, 8);
    }
    if (mean <= (groups > 0 ? 10 : 16)) {
        if (!tb) return shape(1, 4, 4);
        return mean <= (groups > 0 ? 5 : 8) && (groups > 0 || strips < 768) ? shape(1, 1, 4) : shape(1, 2, 4);
    }
    if (groups > 0) return mean <= 16 && shape(2, 4, 4);
    if (mean <= 32) return strips < 640 ? shape(2, 2, 8) : shape(2, 4, 4);
    return strips <= 512 && (tb ? shape(4, 2, 8) : shape(2, 4, 4));
}

// (us, 64 / 128 / 256: 1000 x 2048 x 512 with both kept 14.8 / 10.4 / 22.7;  its gradient 15.4 / 19.4 / 45;  gradient
// 4096 x 1024 x 256 28 / 21.6 / 42, 4000 rows of 16 experts 704 x 1024 31 / 26 / 55;  8192 x 4096 x 2048 488 / 249 / 225,
// gradient 354 / 190 / 164)
constexpr double kGatedCrowded = 3.5;

OpPlan gated_plan(int64_t groups, int64_t rows, int64_t n, int64_t k, bool tb, double weight) {
    const int64_t owners = groups < rows ? groups : rows;
    OpPlan p;
    if (gated_few(groups, rows, n, tb, p)) return p;
    // (an edge's tile holds half as many outputs a row; half a tile per expert is lost on average)
    const int e = best_edge(k, weight, [&](int64_t t) {
        return (groups > 0 ? rows / t + owners / 2 : ceil_div(rows, t)) * ceil_div(n, t / 2);
    }, kGatedCrowded);
    return OpPlan{false, 0, 0, 0, e, e / 2, groups > 0 ? rows / e + owners : ceil_div(rows, e), ceil_div(n, e / 2)};
}

OpPlan gated_grad_plan(int64_t groups, int64_t rows, int64_t n, int64_t k, double weight) {
    const int64_t owners = groups < rows ? groups : rows;
    const int e = best_edge(k, weight, [&](int64_t t) {
        return (groups > 0 ? rows / t + owners / 2 : ceil_div(rows, t)) * ceil_div(n, t);
    }, kGatedCrowded);
    OpPlan p = tiled(rows, n, e);
    if (groups > 0) p.tiles_m = rows / e + owners;
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

LogprobLayout logprob_layout(int64_t m, int64_t n, int bytes, int64_t top) {
    const int64_t vectors = ceil_div(n, 16 / bytes);
    // A row in parts costs a second launch and a search in every part, so that rows are cut only where they
    // leave CUs idle, into two workgroups a CU (us with 20 alternatives, whole / 512 / 4096 parts in all):
    //   16 x 32000 FP32 12.8 / 17.1 / 17.9;  300 x 32000 16.6 / 24.7 / 30.9;  256 x 128000 30.3 / 37.8 / 45.3
    //   (BF16 27.3 / 30.2 / 46.4);  64 x 128000 - / 22.1 / 28.7;  16 x 128000 - / 18.7 / 18.2
    int64_t parts = 1;
    if (m > 0 && m < kCus && n > 32768) {
        parts = ceil_div(2 * kCus, m);
        if (parts > ceil_div(n, 4096)) parts = ceil_div(n, 4096);
    }
    if (parts < ceil_div(n, mpg::kLogprobPart)) parts = ceil_div(n, mpg::kLogprobPart);
    LogprobLayout L;
    // A wave a row where rows are short (four would have little each and meet twice) or many (us with 20
    // alternatives, one wave / four):
    //   16 x 4096 FP32 8.3 / 9.1;  128 x 8192 10.2 / 9.6;  1024 x 8192 13.9 / 15.5;  1024 x 16384 BF16 17.0 / 17.5;
    //   1024 x 32000 25.5 / 22.8;  4096 x 1000 14.0 / 34.3;  4096 x 32000 59.9 / 77.4 (FP32 107 / 103)
    // But with many alternatives 64 lanes' maxima bound them too loosely: of random rows about 64 log(64 / (64 - top))
    // elements reach the bound (44 for 32, 75 for 44, 266 and more for 64), and where these lie in more than 64 of the
    // lanes' turns (2 a lane at 4096 columns, 16 at 32768) the row is gone through again with lists.  256 lanes' maxima
    // bound any number of them well enough; below 2560 columns most of these have nothing to read (BF16, one wave / four):
    //   4096 x 2048, 48 alternatives 23 / 43, 64 40 / 91;  4096 x 2560, 64 39 / 49 (FP32 48 / 44, 64 rows 22 / 14)
    //   4096 x 3504, 44 30 / 39, 48 38 / 40, 56 45 / 42;  64 x 3504, 48 22 / 12;  4096 x 4096, 40 21 / 38, 48 42 / 40, 64 50 / 42
    //   (FP32 28 / 34, 54 / 37, 61 / 38);  4096 x 6000, 36 24 / 36, 40 38 / 38, 48 58 / 40;  1024 x 8192, 36 15 / 14, 40 32 / 14
    //   2048 x 16384, 32 25 / 27, 36 58 / 28;  4096 x 32000, 32 57 / 59, 36 120 / 61, 64 192 / 73
    const int64_t most = n < 2560 ? kMaxAlternatives : n <= 4096 ? 44 : n <= 8192 ? 36 : 32;   // of one wave
    int64_t one = 8 * m < (bytes == 2 ? 32768 : 16384) ? 8 * m : (bytes == 2 ? 32768 : 16384);
    if (one < 4096) one = 4096;
    L.waves = n <= one && top <= most ? 1 : 4;
    L.part_vectors = (int)(ceil_div(ceil_div(vectors, parts), 64) * 64);
    L.parts = (int)(vectors > 0 ? ceil_div(vectors, L.part_vectors) : 1);
    L.off_keys = L.total = 0;
    if (L.parts > 1) {
        L.off_keys = ((uint64_t)m * (uint64_t)L.parts * 16 + 255) / 256 * 256;
        L.total = L.off_keys + (uint64_t)m * (uint64_t)L.parts * (uint64_t)top * 8;
    }
    return L;
}

bool distill_layout(int64_t m, int64_t n, int64_t k, bool train, DistillLayout &D) {
    if (!ce_layout(m, n, k, train, D.ce)) return false;
    D.off_level = (D.ce.total + 255) / 256 * 256;
    D.off_mass = D.off_level + ((uint64_t)m * 4 + 255) / 256 * 256;
    D.total = train && m > 0 ? D.off_mass + (uint64_t)m * 4 : D.ce.total;
    return true;
}

// That saves a launch where a workgroup's waves have a turn of entries at most, or where there is a row for every CU, work
// that outweighs the launch, and k enough for the lanes of a wave.  Below 256 rows the others idle.  Measured (us of
// the loss, apart / itself):
//   n = 32000, k = 4096: 8 rows of 20 entries 73 / 66, 8 of 128 72 / 86
//   n = 8192, k = 4096: 8 of 1024 53 / 196, 16 of 512 46 / 113, 64 of 64 41 / 44, 64 of 128 46 / 56, 128 of 64 47 / 47, 128 of 512
//     114 / 132, 256 of 48 52.7 / 51.5, 256 of 128 77 / 73, 512 of 128 122 / 115, 1024 of 64 142 / 135;  k = 8192: 8 of 1024 73 / 344
//   k = 2048: 256 of 512 99.5 / 97.6, 4096 of 64 255 / 236;  k = 1024: 512 of 1000 147 / 142, 2048 of 64 74.5 / 74.9
//   k = 512: 1024 of 48 29.9 / 29.9;  k = 256: 4096 of 40 71 / 85
bool merge_picks(int64_t m, int64_t top, int64_t k) {
    return top <= mpg::kMergePicks || (m >= kCus && k >= 512 && m * top >= ((int64_t)1 << 25) / k);
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

namespace {

// A pair of matrices `stride` elements apart: how far, and (for one that is written) that it does not overlap itself.
constexpr int64_t kMaxStride = INT64_MAX / 131072;
mpgemm_status_t check_pair(int64_t m, int64_t n, int64_t ld, int64_t stride, int eb, bool written) {
    if (stride < 0) return MPGEMM_STATUS_INVALID_VALUE;
    if (stride > kMaxStride || (stride * eb) % 16) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!written) return MPGEMM_STATUS_SUCCESS;
    // (of sizes and leading dimensions that have been checked: no overflow)
    const bool beside = stride >= n && stride <= ld - n, after = stride >= (m - 1) * ld + n;
    return beside || after ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_INVALID_VALUE;
}

// What the four gated calls share: sizes, types, operands and where D goes.  groups < 0: one product.
struct GatedArgs {
    mpgemm_op_t transb;
    int64_t groups, rows, n, k;
    const float *alpha;
    const void *A;
    mpgemm_dtype_t a_type;
    int64_t lda;
    const int32_t *offsets;
    const void *B;
    mpgemm_dtype_t b_type;
    int64_t ldb, stride_b;
    const void *D;
    mpgemm_dtype_t d_type;
    int64_t ldd;
    bool empty() const { return groups == 0 || rows == 0 || n == 0; }
};

mpgemm_status_t check_gated_sizes(const GatedArgs &a) {
    if (!op_valid(a.transb) || a.rows < 0 || a.n < 0 || a.k < 0 || !a.alpha || a.stride_b < 0) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_types(a.a_type, a.b_type, a.d_type));
    const bool tb = a.transb == MPGEMM_OP_T;
    if (a.lda < at_least1(a.k) || a.ldb < at_least1(tb ? a.k : a.n) || a.ldd < at_least1(a.n)) return MPGEMM_STATUS_INVALID_VALUE;
    return MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t check_gated_operands(const GatedArgs &a, const OpPlan &plan) {
    if (!a.D || (a.groups > 0 && !a.offsets) || (a.k > 0 && (!a.A || !a.B))) return MPGEMM_STATUS_INVALID_VALUE;
    if (a.rows > kOpMaxSize || a.n > kOpMaxSize || a.k > kOpMaxSize || a.groups > 65535 || !launchable(plan, 1))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if ((a.k > 0 && (!aligned(a.A, 16) || !aligned(a.B, 16))) || !aligned(a.D, 16) || (a.groups > 0 && !aligned(a.offsets, 4)))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(a.lda, 2) || !stride_ok(a.ldb, 2) || !stride_ok(a.ldd, elem_bytes(a.d_type)) || a.stride_b % 8 ||
        a.stride_b > kMaxStride)
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return MPGEMM_STATUS_SUCCESS;
}

mpgemm_status_t check_gated_call(const GatedArgs &a, int64_t stride_up, const mpgemm_gated_t *g) {
    MPGEMM_TRY(check_gated_sizes(a));
    if (!g || !act_valid(g->act) || stride_up < 0) return MPGEMM_STATUS_INVALID_VALUE;
    if ((g->bias_gate || g->bias_up) && !out_type(g->bias_type, a.a_type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if ((g->bias_gate || g->bias_up) && a.groups >= 0 && g->bias_stride < 0) return MPGEMM_STATUS_INVALID_VALUE;
    if (g->kept && g->ld_kept < at_least1(a.n)) return MPGEMM_STATUS_INVALID_VALUE;
    if (a.empty()) return MPGEMM_STATUS_SUCCESS;
    const bool sized = a.rows <= kOpMaxSize && a.n <= kOpMaxSize && a.k <= kOpMaxSize && a.groups <= 65535;
    if (!sized) return a.D ? MPGEMM_STATUS_NOT_SUPPORTED : MPGEMM_STATUS_INVALID_VALUE;
    const int64_t groups = a.groups > 0 ? a.groups : 0;
    MPGEMM_TRY(check_gated_operands(a, gated_plan(groups, a.rows, a.n, a.k, a.transb == MPGEMM_OP_T, gated_weight(g->act, g->kept != nullptr))));
    if (stride_up % 8 || stride_up > ((int64_t)1 << 30) || 256 * 2 * a.ldb + 2 * stride_up > ((int64_t)1 << 31) - 4096)
        return MPGEMM_STATUS_NOT_SUPPORTED;
    const unsigned be = g->bias_type == MPGEMM_R_32F ? 4 : 2;
    if (!aligned(g->bias_gate, be) || !aligned(g->bias_up, be) || ((g->bias_gate || g->bias_up) && g->bias_stride > kMaxStride && a.groups > 0))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!g->kept) return MPGEMM_STATUS_SUCCESS;
    if (!aligned(g->kept, 16) || !stride_ok(g->ld_kept, 2)) return MPGEMM_STATUS_NOT_SUPPORTED;
    return check_pair(a.rows, a.n, g->ld_kept, g->stride_kept, 2, true);
}

mpgemm_status_t check_gated_grad_call(const GatedArgs &a, const mpgemm_gated_grad_t *g, int64_t stride_d, const void *workspace,
                                      uint64_t workspace_bytes) {
    MPGEMM_TRY(check_gated_sizes(a));
    if (!g || !act_valid(g->act)) return MPGEMM_STATUS_INVALID_VALUE;
    if (g->ld_kept < at_least1(a.n) || (g->H && g->ldh < at_least1(a.n))) return MPGEMM_STATUS_INVALID_VALUE;
    if (a.groups == 0 || a.n == 0 || (a.rows == 0 && !g->dbias)) return MPGEMM_STATUS_SUCCESS;
    if (a.rows > kOpMaxSize || a.n > kOpMaxSize || a.k > kOpMaxSize || a.groups > 65535 || !aligned(g->dbias, 4))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (a.rows == 0)   // (the sum of no rows is written)
        return a.groups > 0 && !a.offsets ? MPGEMM_STATUS_INVALID_VALUE : MPGEMM_STATUS_SUCCESS;
    if (!g->kept) return MPGEMM_STATUS_INVALID_VALUE;
    const int64_t groups = a.groups > 0 ? a.groups : 0;
    MPGEMM_TRY(check_gated_operands(a, gated_grad_plan(groups, a.rows, a.n, a.k, gated_grad_weight(g->act, g->H != nullptr))));
    if (!aligned(g->kept, 16) || !stride_ok(g->ld_kept, 2) || (g->H && (!aligned(g->H, 16) || !stride_ok(g->ldh, 2))))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    MPGEMM_TRY(check_pair(a.rows, a.n, g->ld_kept, g->stride_kept, 2, false));
    MPGEMM_TRY(check_pair(a.rows, a.n, a.ldd, stride_d, elem_bytes(a.d_type), true));
    return g->dbias ? check_workspace(workspace, workspace_bytes, mpgemm_gated_grad_workspace_size(a.groups > 0 ? a.groups : 1, a.rows, a.n))
                    : MPGEMM_STATUS_SUCCESS;
}

}  // namespace

uint64_t mpgemm_gated_grad_workspace_size(int64_t groups, int64_t m, int64_t n) {
    return 2 * mpgemm_epilogue_grad_workspace_size(groups, m, n);
}

mpgemm_status_t mpgemm_check_gated(mpgemm_op_t transb, int64_t m, int64_t n, int64_t k, const float *alpha, const void *A,
                                   mpgemm_dtype_t a_type, int64_t lda, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                   int64_t stride_up, const mpgemm_gated_t *gated, const void *D, mpgemm_dtype_t d_type,
                                   int64_t ldd) {
    return check_gated_call({transb, -1, m, n, k, alpha, A, a_type, lda, nullptr, B, b_type, ldb, 0, D, d_type, ldd}, stride_up, gated);
}

mpgemm_status_t mpgemm_check_grouped_gated(mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                           const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                           const int32_t *offsets, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                           int64_t stride_b, int64_t stride_up, const mpgemm_gated_t *gated, const void *D,
                                           mpgemm_dtype_t d_type, int64_t ldd) {
    if (groups < 0) return MPGEMM_STATUS_INVALID_VALUE;
    return check_gated_call({transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b, D, d_type, ldd},
                            stride_up, gated);
}

mpgemm_status_t mpgemm_check_gated_grad(mpgemm_op_t transb, int64_t m, int64_t n, int64_t k, const float *alpha, const void *A,
                                        mpgemm_dtype_t a_type, int64_t lda, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                        const mpgemm_gated_grad_t *grad, const void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                        int64_t stride_d, const void *workspace, uint64_t workspace_bytes) {
    return check_gated_grad_call({transb, -1, m, n, k, alpha, A, a_type, lda, nullptr, B, b_type, ldb, 0, D, d_type, ldd}, grad, stride_d,
                                 workspace, workspace_bytes);
}

mpgemm_status_t mpgemm_check_grouped_gated_grad(mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n, int64_t k,
                                                const float *alpha, const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                                const int32_t *offsets, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                                int64_t stride_b, const mpgemm_gated_grad_t *grad, const void *D,
                                                mpgemm_dtype_t d_type, int64_t ldd, int64_t stride_d, const void *workspace,
                                                uint64_t workspace_bytes) {
    if (groups < 0) return MPGEMM_STATUS_INVALID_VALUE;
    return check_gated_grad_call({transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b, D, d_type, ldd},
                                 grad, stride_d, workspace, workspace_bytes);
}

namespace {

mpgemm_status_t check_teacher(const mpgemm_teacher_t *t) {
    if (!t || t->top < 1 || t->ld < t->top) return MPGEMM_STATUS_INVALID_VALUE;
    if (!(t->scale >= -1.0e30f && t->scale <= 1.0e30f)) return MPGEMM_STATUS_INVALID_VALUE;   // (NaN too)
    return t->top <= mpg::kMostTop && t->ld <= kOpMaxSize ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_NOT_SUPPORTED;
}

mpgemm_status_t check_teacher_layout(const mpgemm_teacher_t *t) {
    return aligned(t->index, 8) && aligned(t->logit, 4) && aligned(t->lse, 4) ? MPGEMM_STATUS_SUCCESS : MPGEMM_STATUS_NOT_SUPPORTED;
}

}  // namespace

uint64_t mpgemm_linear_distill_workspace_size(int64_t m, int64_t n, int64_t k, int64_t top, mpgemm_dtype_t type, int train) {
    DistillLayout D;
    if (!half_type(type) || top < 1 || top > mpg::kMostTop || !distill_layout(m, n, k, train != 0, D)) return 0;
    return m == 0 ? 0 : D.total;
}

mpgemm_status_t mpgemm_check_linear_distill(int64_t m, int64_t n, int64_t k, const float *alpha, const void *X, mpgemm_dtype_t type,
                                            int64_t ldx, const void *W, int64_t ldw, const mpgemm_teacher_t *teacher,
                                            const float *loss, const float *lse, const float *picked, const void *workspace,
                                            uint64_t workspace_bytes) {
    if (m < 0 || n < 1 || k < 0 || !alpha) return MPGEMM_STATUS_INVALID_VALUE;
    if (!half_type(type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (ldx < at_least1(k) || ldw < at_least1(k)) return MPGEMM_STATUS_INVALID_VALUE;
    MPGEMM_TRY(check_teacher(teacher));
    if (m == 0) return MPGEMM_STATUS_SUCCESS;
    if ((k > 0 && (!X || !W)) || !teacher->index || !teacher->logit || !loss || !lse || !picked) return MPGEMM_STATUS_INVALID_VALUE;
    DistillLayout D;
    if (!distill_layout(m, n, k, false, D) || !launchable(D.ce.logits, 1)) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (k > 0 && (!aligned(X, 16) || !aligned(W, 16))) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!stride_ok(ldx, 2) || !stride_ok(ldw, 2) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(picked, 4))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    MPGEMM_TRY(check_teacher_layout(teacher));
    return check_workspace(workspace, workspace_bytes, D.total);
}

mpgemm_status_t mpgemm_check_linear_distill_grad(int64_t m, int64_t n, int64_t k, const float *alpha, const void *X,
                                                 mpgemm_dtype_t type, int64_t ldx, const void *W, int64_t ldw,
                                                 const mpgemm_teacher_t *teacher, const float *lse, const float *picked,
                                                 const float *grad, const void *dX, int64_t lddx, const void *dW, int64_t lddw,
                                                 const void *workspace, uint64_t workspace_bytes) {
    if (m < 0 || n < 1 || k < 0 || !alpha) return MPGEMM_STATUS_INVALID_VALUE;
    if (!half_type(type)) return MPGEMM_STATUS_NOT_SUPPORTED;
    MPGEMM_TRY(check_teacher(teacher));
    const bool rows = m > 0 && k > 0 && (dX || dW);
    if (rows && (!teacher->index || !teacher->logit || !picked)) return MPGEMM_STATUS_INVALID_VALUE;
    // everything else is as for the cross entropy (whose targets the teacher's columns stand for)
    DistillLayout D = {};
    const bool fits = rows && distill_layout(m, n, k, true, D);
    MPGEMM_TRY(mpgemm_check_linear_ce_grad(m, n, k, alpha, X, type, ldx, W, ldw, rows ? teacher->index : nullptr, lse, grad, dX, lddx, dW,
                                           lddw, workspace, workspace_bytes));
    if (!rows) return MPGEMM_STATUS_SUCCESS;
    if (!fits || !aligned(picked, 4)) return MPGEMM_STATUS_NOT_SUPPORTED;
    MPGEMM_TRY(check_teacher_layout(teacher));
    return check_workspace(workspace, workspace_bytes, D.total);
}

uint64_t mpgemm_logprobs_workspace_size(int64_t m, int64_t n, mpgemm_dtype_t z_type, int64_t top) {
    if (m < 1 || n < 1 || m > kOpMaxSize || n > kOpMaxSize || top < 0 || top > kMaxAlternatives) return 0;
    if (!half_type(z_type) && z_type != MPGEMM_R_32F) return 0;
    return logprob_layout(m, n, elem_bytes(z_type), top).total;
}

mpgemm_status_t mpgemm_check_logprobs(int64_t m, int64_t n, const float *alpha, const void *Z, mpgemm_dtype_t z_type, int64_t ldz,
                                      const int64_t *target, const float *logprob, const float *lse, const float *entropy,
                                      int64_t top, const int64_t *top_index, const float *top_logprob, int64_t ld_top,
                                      const void *workspace, uint64_t workspace_bytes) {
    if (m < 0 || n < 1 || !alpha || top < 0) return MPGEMM_STATUS_INVALID_VALUE;
    if (!half_type(z_type) && z_type != MPGEMM_R_32F) return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!(*alpha > 0.0f) || *alpha > 1.0e30f || ldz < n || (top > 0 && ld_top < top)) return MPGEMM_STATUS_INVALID_VALUE;
    if (m == 0) return MPGEMM_STATUS_SUCCESS;
    if (!Z || (logprob && !target) || (top > 0 && (!top_index || !top_logprob))) return MPGEMM_STATUS_INVALID_VALUE;
    const int64_t most = INT64_MAX / ((int64_t)1 << 36);   // (rows times a leading dimension stay 64-bit byte offsets)
    if (m > kOpMaxSize || n > kOpMaxSize || ldz > ((int64_t)1 << 31) || top > kMaxAlternatives || (top > 0 && ld_top > most))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    if (!aligned(Z, 16) || (ldz * elem_bytes(z_type)) % 16 || (logprob && !aligned(target, 8)) || !aligned(logprob, 4) ||
        !aligned(lse, 4) || !aligned(entropy, 4) || (top > 0 && (!aligned(top_index, 8) || !aligned(top_logprob, 4))))
        return MPGEMM_STATUS_NOT_SUPPORTED;
    return check_workspace(workspace, workspace_bytes, mpgemm_logprobs_workspace_size(m, n, z_type, top));
}

}  // extern "C"
