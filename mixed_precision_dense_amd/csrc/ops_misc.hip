// ops_misc.hip -- the small kernels beside the op products: sums of partial column sums, of
// partial products and of row statistics.  All of them are bound by what they read; every sum is
// taken in a fixed order, so that results do not change from call to call.
//
// A grid has at most kMostBlocks workgroups in x, which walk what lies past them: a launch holds
// less than 2^32 lanes, and rows times blocks of columns can be more.
#include "mpgemm_ops_epilogue.hpp"

namespace mpg {
namespace {

constexpr int64_t kMostBlocks = 65536;
constexpr int kSumCols = 64;   // columns per workgroup of colsum_kernel

// dbias[e][c] = sum over the partial rows of expert e's row tiles: 64 columns by 4 walkers over
// the rows, whose shares meet in the LDS.
__global__ __launch_bounds__(256) void colsum_kernel(OpParams p, int tile_rows, int rows_per_tile, float *dbias) {
    __shared__ float share[4][kSumCols];
    const int lane = threadIdx.x % 64, part = threadIdx.x / 64;
    const int e = blockIdx.y;
    const int64_t out = ((int64_t)e * gridDim.z + blockIdx.z) * p.n;
    int64_t first = 0;
    int tiles = p.tiles_m;
    if (p.groups_kind == GROUPS_ROWS) {
        int lo, hi;
        expert_tiles(p, tile_rows, e, lane, first, tiles, lo, hi);
        tiles = (int)min((int64_t)tiles, max((int64_t)0, p.tiles_m - first));   // (offsets outside the contract)
    }
    for (int64_t c0 = (int64_t)blockIdx.x * kSumCols; c0 < p.n; c0 += (int64_t)gridDim.x * kSumCols) {
        const int64_t col = c0 + lane;
        float s = 0.0f;
        if (col < p.n) {
            const float *at = p.colsum + blockIdx.z * p.stride_colsum + first * rows_per_tile * p.ld_colsum + col;
            for (int r = part; r < tiles * rows_per_tile; r += 4) s += at[(int64_t)r * p.ld_colsum];
        }
        share[part][lane] = s;
        __syncthreads();
        if (part == 0 && col < p.n)
            dbias[out + col] = (share[0][lane] + share[1][lane]) + (share[2][lane] + share[3][lane]);
        __syncthreads();   // share is written again
    }
}

// One workgroup per row: log-sum-exp from the parts' statistics, and the target's logit as a dot
// product of the row of X with the target's row of W (k * 4 bytes a row, where picking the logit
// out of the tiles would cost every tile's epilogue a comparison per element).  All four waves
// share a row, since with few rows the chain of one wave's loads is all there is to wait for (8 rows
// of 2000 parts, k = 4096: 15 us with one wave per row).
constexpr int kMergeThreads = 256;
template <int IN>
__global__ __launch_bounds__(kMergeThreads) void ce_merge_kernel(const CeStat *stats, int parts, int m, int n, int k, float alpha,
                                                                 const uint16_t *X, int64_t ldx, const uint16_t *W, int64_t ldw,
                                                                 const int64_t *target, float *loss, float *lse) {
    __shared__ float share[kMergeThreads / 64][3];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        const int64_t t = target[row];
        const bool counts = t >= 0 && t < n;
        const CeStat *st = stats + row * parts;
        float top = -__builtin_inff(), sum = 0.0f;
        auto join = [&](float o_top, float o_sum) {
            const float up = fmaxf(top, o_top), base = stat_base(up);
            sum = sum * fast_exp2(top - base) + o_sum * fast_exp2(o_top - base);
            top = up;
        };
        for (int i = threadIdx.x; i < parts; i += 4 * kMergeThreads) {
            CeStat s[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s[q] = CeStat{-__builtin_inff(), 0.0f};
                if (i + q * kMergeThreads < parts) s[q] = st[i + q * kMergeThreads];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) join(s[q].top, s[q].sum);
        }
        float dot = 0.0f;
        if (counts) {
            const uint16_t *x = X + row * ldx, *w = W + t * ldw;
            for (int c = 8 * threadIdx.x; c < k; c += 8 * kMergeThreads) {
                float a[8], b[8];
                widen8<IN>(*(const u32x4 *)(x + c), a);
                widen8<IN>(*(const u32x4 *)(w + c), b);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (c + q < k) dot = __builtin_fmaf(a[q], b[q], dot);
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            join(__shfl_xor(top, d, 64), __shfl_xor(sum, d, 64));
            dot += __shfl_xor(dot, d, 64);
        }
        if (lane == 0) {
            share[wave][0] = top;
            share[wave][1] = sum;
            share[wave][2] = dot;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kMergeThreads / 64; ++i) {
                join(share[i][0], share[i][1]);
                dot += share[i][2];
            }
            const float l = (top + __log2f(sum)) * 0.69314718055994531f;
            lse[row] = l;
            loss[row] = counts ? l - alpha * dot : 0.0f;
        }
        __syncthreads();   // share is written again
    }
}

// Row weights of the gradient: grad where the target counts, else 0, divided by the largest of them
// and, for FP16, brought to at most 2^13; scale[0] takes both back from the products.  FP16 gradients
// of logits are often below FP16's normal range (a probability times 1 / rows).  And with equal
// weights, a mean's, the largest entries of P, a target's p - 1, then start from a power of two:
// times 1 / rows they would all be rounded the same way, an error of up to half a step that no
// summation averages out (relative error of dX and dW in BF16 0.0034 where it is now 0.0017).
//
// With lists (rows.source), the rows that count are also numbered in their order, so that the products
// after this one take only them; their number stays on the device.  Nothing of a row that does not
// count may reach the gradients: an X of NaN there (padding) would, as 0 * NaN, through a P of 0.
constexpr int kRowThreads = 1024;
__global__ __launch_bounds__(kRowThreads) void ce_rows_kernel(int bf16, int m, int n, const int64_t *target, const float *mass,
                                                              const float *lse, const float *grad, CeRows rows) {
    __shared__ float most[kRowThreads / 64];
    __shared__ int found[kRowThreads / 64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    // the column that a row's target takes, or -1: the row does not count
    auto target_of = [&](int64_t r) -> int64_t {
        if (mass != nullptr) return mass[r] == 0.0f ? -1 : kNoColumn;
        const int64_t t = target[r];
        return t >= 0 && t < n ? t : -1;
    };
    float a = 0.0f;
    for (int64_t r = threadIdx.x; r < m; r += kRowThreads) {   // (m + kRowThreads may pass 31 bits)
        // (entries of P are at most the weight, or the mass times it)
        if (target_of(r) >= 0) a = fmaxf(a, __builtin_fabsf(grad[r]) * (mass != nullptr ? fmaxf(mass[r], 1.0f) : 1.0f));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) a = fmaxf(a, __shfl_xor(a, d, 64));
    if (lane == 0) most[wave] = a;
    __syncthreads();
    for (int i = 0; i < kRowThreads / 64; ++i) a = fmaxf(a, most[i]);
    const bool usable = a > 0.0f && a < __builtin_inff();   // (else the weights stay as they are)
    const float top = usable && !bf16 ? 8192.0f : 1.0f;
    if (threadIdx.x == 0) rows.scale[0] = usable ? a / top : 1.0f;
    int before = 0;                                         // entries of the rows before this turn's
    for (int64_t base = 0; base < m; base += kRowThreads) { // (the same number of turns for every wave)
        const int64_t r = base + threadIdx.x;
        const int64_t t = r < m ? target_of(r) : -1;
        const bool counts = t >= 0;
        const float g = counts ? grad[r] : 0.0f;
        const float weight = usable ? g / a * top : g;
        int64_t at = r;
        if (rows.source != nullptr) {
            const uint64_t mask = __ballot(counts);
            if (lane == 0) found[wave] = __popcll(mask);
            __syncthreads();
            int sum = 0, own = 0;
            for (int i = 0; i < kRowThreads / 64; ++i) {
                if (i == wave) own = sum;
                sum += found[i];
            }
            at = before + own + __popcll(mask & (((uint64_t)1 << lane) - 1));
            before += sum;
            __syncthreads();                                // found is written again in the next turn
            if (counts) rows.source[at] = (int)r;
        }
        if (r < m) rows.place[r] = counts ? (int)at : -1;
        if (r < m && (counts || rows.source == nullptr)) {
            rows.weight[at] = weight;
            rows.lse[at] = counts && mass != nullptr ? lse[r] - __logf(mass[r]) : lse[r];
            rows.target[at] = counts ? t : -1;
        }
    }
    if (threadIdx.x == 0) rows.count[0] = rows.source != nullptr ? before : m;
}

// One thread per 16-byte block of a listed row.
__global__ __launch_bounds__(256) void gather_rows_kernel(const uint16_t *in, int64_t ld_in, const int *source, const int *count,
                                                          int m, int blocks, uint16_t *out, int64_t ld_out) {
    const int64_t all = (int64_t)min(count[0], m) * blocks;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < all; t += (int64_t)gridDim.x * 256) {
        const int64_t j = t / blocks, at = (t - j * blocks) * 8;
        *(u32x4 *)(out + j * ld_out + at) = *(const u32x4 *)(in + source[j] * ld_in + at);
    }
}

template <int IN>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float *parts, int splits, int64_t stride, int64_t ld_part,
                                                        const int *place, int rows, int cols, float alpha, const float *scale, uint16_t *out,
                                                        int64_t ld_out) {
    const int64_t chunks = ((int64_t)cols + 7) / 8;
    const float f = alpha * scale[0];
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < rows * chunks; t += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = t / chunks;
        const int col = (int)(t - row * chunks) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        const int64_t from = place[row];
        const int own = from < 0 ? 0 : splits;
        const float *at = parts + from * ld_part + col;   // (rows of whole 8-column blocks)
        // eight parts on their way at a time (one after the other, 32 parts of 16 x 776 took 11 us)
        constexpr int kAhead = 8;
        for (int s = 0; s < own; s += kAhead, at += kAhead * stride) {
            f32x4 a[kAhead], b[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                a[i] = b[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (s + i < own) {
                    a[i] = *(const f32x4 *)(at + i * stride);
                    b[i] = *(const f32x4 *)(at + i * stride + 4);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[q] += a[i][q];
                    v[q + 4] += b[i][q];
                }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= f;
        uint16_t *to = out + row * ld_out + col;
        const u32x4 x = narrow8<IN>(v);
        if (col + 8 <= cols) {
            *(u32x4 *)to = x;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (col + q < cols) to[q] = (uint16_t)(q & 1 ? x[q / 2] >> 16 : x[q / 2]);
        }
    }
}

int launch_1d(const void *kernel, int64_t blocks, unsigned threads, void **args, void *stream) {
    if (blocks == 0) return (int)hipSuccess;
    return (int)hipLaunchKernel(kernel, dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(threads), args, 0,
                                (hipStream_t)stream);
}

}  // namespace

int launch_colsum(const OpParams &p, int tile_rows, int rows_per_tile, int halves, float *dbias, void *stream) {
    OpParams q = p;
    void *args[] = {&q, &tile_rows, &rows_per_tile, &dbias};
    const int64_t blocks = ((int64_t)p.n + kSumCols - 1) / kSumCols;
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&colsum_kernel),
                                dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks),
                                     p.groups_kind == GROUPS_ROWS ? (unsigned)p.groups : 1u, (unsigned)halves),
                                dim3(256), args, 0, (hipStream_t)stream);
}

int launch_ce_merge(bool bf16, const CeStat *stats, int parts, int m, int n, int k, float alpha, const void *X, int64_t ldx,
                    const void *W, int64_t ldw, const int64_t *target, float *loss, float *lse, void *stream) {
    const uint16_t *x = (const uint16_t *)X, *w = (const uint16_t *)W;
    void *args[] = {&stats, &parts, &m, &n, &k, &alpha, &x, &ldx, &w, &ldw, &target, &loss, &lse};
    return launch_1d(bf16 ? reinterpret_cast<const void *>(&ce_merge_kernel<IN_BF16>)
                          : reinterpret_cast<const void *>(&ce_merge_kernel<IN_F16>),
                     m, kMergeThreads, args, stream);
}

int launch_ce_rows(bool bf16, int m, int n, const int64_t *target, const float *mass, const float *lse, const float *grad,
                   const CeRows &rows, void *stream) {
    int b = bf16 ? 1 : 0;
    CeRows r = rows;
    void *args[] = {&b, &m, &n, &target, &mass, &lse, &grad, &r};
    return launch_1d(reinterpret_cast<const void *>(&ce_rows_kernel), 1, kRowThreads, args, stream);
}

int launch_gather_rows(const void *in, int64_t ld_in, const int *source, const int *count, int m, int k, void *out, int64_t ld_out,
                       void *stream) {
    const uint16_t *from = (const uint16_t *)in;
    uint16_t *to = (uint16_t *)out;
    int blocks = (k + 7) / 8;
    void *args[] = {&from, &ld_in, &source, &count, &m, &blocks, &to, &ld_out};
    return launch_1d(reinterpret_cast<const void *>(&gather_rows_kernel), ((int64_t)m * blocks + 255) / 256, 256, args, stream);
}

int launch_sum_parts(bool bf16, const float *parts, int splits, int64_t stride, int64_t ld_part, const int *place, int rows, int cols,
                     float alpha, const float *scale, void *out, int64_t ld_out, void *stream) {
    uint16_t *o = (uint16_t *)out;
    void *args[] = {&parts, &splits, &stride, &ld_part, &place, &rows, &cols, &alpha, &scale, &o, &ld_out};
    const int64_t lanes = (int64_t)rows * (((int64_t)cols + 7) / 8);
    const unsigned threads = lanes <= 65536 ? 64 : 256;   // (a wave per CU where there are few)
    return launch_1d(bf16 ? reinterpret_cast<const void *>(&sum_parts_kernel<IN_BF16>)
                          : reinterpret_cast<const void *>(&sum_parts_kernel<IN_F16>),
                     (lanes + threads - 1) / threads, threads, args, stream);
}

}  // namespace mpg
