// ops_distill.hip -- what the distillation loss of a linear head adds to its cross entropy: the logits
// at a teacher's top columns, the loss, and the entries of P at those columns.
//
// With y_j = scale t_j over the teacher's entries j of a row that count, L their log-sum-exp (or the
// teacher's own, over all columns) and q_j = exp(y_j - L), Q = sum of q_j:
//   loss = sum of q_j (y_j - L - z_j + lse),   P_v = weight (Q exp(z_v - lse) - sum of q_j at column v).
// The first term of P is the cross entropy's, with log Q taken from lse and no target; at the teacher's
// columns, where a trained student's two terms all but cancel, P is formed in FP32 from the logits that
// the forward call kept, and rounded once.
//
// P is held in the inputs' type: the matrix instructions take both factors in one type, and a second term of P
// (what its rounding left) would double both products.  No entry stands out as a target's p - 1 does in the cross
// entropy, where it is a power of two and exact, so that here the rounding of P is as much of the gradients'
// error as their own: dX and dW of 4096 x 128000 x 4096 in BF16 are 2.34e-3 and 2.35e-3 off in norm, 1.66e-3 with P in FP32,
// those of 517 x 50021 x 1000 in FP16 2.9e-4, 2.1e-4 with P in FP32.
#include "mpgemm_ops_epilogue.hpp"

namespace mpg {
namespace {

constexpr int kWaves = 4;             // per workgroup
constexpr int64_t kMostBlocks = 65536;
constexpr float kLn2 = 0.69314718055994531f;

// An entry of a teacher's row: its column, or -1 where it does not count.
__device__ __forceinline__ int entry_column(const Teacher &t, int64_t row, int j, int n) {
    if (j >= t.top) return -1;
    const int64_t v = t.index[row * t.ld + j];
    return v >= 0 && v < n ? (int)v : -1;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
// y in units of log 2; f = scale / log 2.  A logit of -infinity has no mass whatever the scale is: 0 times it would be
// NaN, and a negative number +infinity.
__device__ __forceinline__ float scaled(float f, float logit) { return logit == -__builtin_inff() ? logit : f * logit; }
// y - level in units of log 2, rounded once; -infinity for an entry without mass.
__device__ __forceinline__ float log_share(float f, float logit, float level2) {
    const float y2 = scaled(f, logit);
    return y2 == -__builtin_inff() ? y2 : __builtin_fmaf(f, logit, -level2);
}
// exp of it; an entry without mass is exactly 0.
__device__ __forceinline__ float share_of(float f, float logit, float level2) {
    const float d = log_share(f, logit, level2);
    return d == -__builtin_inff() ? 0.0f : fast_exp2(d);
}

// L (in units of log 2) and Q of a row, by a whole wave.  Q is 0 where no entry has mass: the row does
// not count.  Without the teacher's lse Q is 1, and not a sum that is 1 but for its rounding.
__device__ __forceinline__ void teacher_row(const Teacher &t, int64_t row, int n, int lane, float &level2, float &mass) {
    const float *logit = t.logit + row * t.ld;
    const float f = t.scale * kLog2e;
    float top = -__builtin_inff();
    bool nan = false;
    for (int j = lane; j < t.top; j += 64)
        if (entry_column(t, row, j, n) >= 0) {
            const float y = scaled(f, logit[j]);
            top = fmaxf(top, y);
            nan |= y != y;
        }
    top = wave_max(top);
    if (__any(nan)) top = __builtin_nanf("");
    const float base = t.lse != nullptr ? t.lse[row] * kLog2e : stat_base(top);
    float sum = 0.0f;
    for (int j = lane; j < t.top; j += 64)
        if (entry_column(t, row, j, n) >= 0) sum += share_of(f, logit[j], base);
    sum = wave_sum(sum);
    level2 = t.lse != nullptr ? base : base + __log2f(sum);
    mass = t.lse != nullptr || sum == 0.0f || sum != sum ? sum : 1.0f;
}

// picked[row][j] = alpha X(row) . W(index) for the row's entries j0 .. j0 + kEntries - 1, by a wave that reads
// their columns' rows of W side by side.  Those reads (top * k * 2 bytes a row, from beyond the L2 as a rule) bound
// it where there are many rows (4096 rows of 64 entries, k = 4096: 7 TB/s), the chain of a wave's turns where
// there are few.
constexpr int kEntries = 4;
template <int IN>
__device__ __forceinline__ void pick(const Teacher &t, int64_t row, int j0, int n, int k, float alpha, const uint16_t *X, int64_t ldx,
                                     const uint16_t *W, int64_t ldw, int lane, float (&out)[kEntries]) {
    const uint16_t *x = X + row * ldx;
    const uint16_t *w[kEntries];
    bool counts[kEntries];
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
        const int v = entry_column(t, row, j0 + e, n);
        counts[e] = v >= 0;
        w[e] = W + (int64_t)(counts[e] ? v : 0) * ldw;
        out[e] = 0.0f;
    }
#pragma unroll 2
    for (int c = 8 * lane; c < k; c += 512) {
        float a[8];
        u32x4 b[kEntries];
        const u32x4 xa = *(const u32x4 *)(x + c);
#pragma unroll
        for (int e = 0; e < kEntries; ++e) b[e] = *(const u32x4 *)(w[e] + c);
        widen8<IN>(xa, a);
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            float v[8];
            widen8<IN>(b[e], v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (c + q < k) out[e] = __builtin_fmaf(a[q], v[q], out[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
        const float s = wave_sum(out[e]);
        out[e] = counts[e] ? alpha * s : 0.0f;
    }
}

// All of a call's, a wave per kEntries of them.
template <int IN>
__global__ __launch_bounds__(64 * kWaves) void picked_kernel(Teacher t, int m, int n, int k, float alpha, const uint16_t *X,
                                                             int64_t ldx, const uint16_t *W, int64_t ldw, float *picked) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int groups = (t.top + kEntries - 1) / kEntries;
    const int64_t items = (int64_t)m * groups;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int64_t row = item / groups;
        const int j0 = (int)(item - row * groups) * kEntries;
        float z[kEntries];
        pick<IN>(t, row, j0, n, k, alpha, X, ldx, W, ldw, lane, z);
#pragma unroll
        for (int e = 0; e < kEntries; ++e)
            if (lane == 0 && j0 + e < t.top) picked[row * t.ld + j0 + e] = z[e];
    }
}

// One workgroup per row: lse from the parts' statistics, then the loss from the picked logits, which it
// forms itself (PICK) or finds formed.
constexpr int kMergeWaves = 8;
static_assert(kEntries * kMergeWaves == kMergePicks, "a turn of the merging kernel's waves, as the rule counts it");
template <int IN, bool PICK>
__global__ __launch_bounds__(64 * kMergeWaves) void distill_merge_kernel(Teacher t, const CeStat *stats, int parts, int m, int n, int k,
                                                                         float alpha, const uint16_t *X, int64_t ldx,
                                                                         const uint16_t *W, int64_t ldw, float *picked, float *loss,
                                                                         float *lse) {
    __shared__ float share[kMergeWaves][2];
    __shared__ float own_picked[PICK ? kMostTop : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        for (int j0 = kEntries * wave; PICK && j0 < t.top; j0 += kEntries * kMergeWaves) {
            float z[kEntries];
            pick<IN>(t, row, j0, n, k, alpha, X, ldx, W, ldw, lane, z);
#pragma unroll
            for (int e = 0; e < kEntries; ++e)
                if (lane == 0 && j0 + e < t.top) own_picked[j0 + e] = picked[row * t.ld + j0 + e] = z[e];
        }
        const CeStat *st = stats + row * parts;
        float top = -__builtin_inff(), sum = 0.0f;
        auto join = [&](float o_top, float o_sum) {
            const float up = fmaxf(top, o_top), base = stat_base(up);
            sum = sum * fast_exp2(top - base) + o_sum * fast_exp2(o_top - base);
            top = up;
        };
        for (int i = threadIdx.x; i < parts; i += 4 * 64 * kMergeWaves) {
            CeStat s[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s[q] = CeStat{-__builtin_inff(), 0.0f};
                if (i + q * 64 * kMergeWaves < parts) s[q] = st[i + q * 64 * kMergeWaves];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) join(s[q].top, s[q].sum);
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) join(__shfl_xor(top, d, 64), __shfl_xor(sum, d, 64));
        if (lane == 0) {
            share[wave][0] = top;
            share[wave][1] = sum;
        }
        __syncthreads();
        if (wave == 0) {
            for (int i = 1; i < kMergeWaves; ++i) join(share[i][0], share[i][1]);
            const float l2 = top + __log2f(sum);
            float level2, mass;
            teacher_row(t, row, n, lane, level2, mass);
            const float f = t.scale * kLog2e, own = l2 * kLn2;
            float s = 0.0f;
            for (int j = lane; j < t.top; j += 64) {
                if (entry_column(t, row, j, n) < 0) continue;
                const float d = log_share(f, t.logit[row * t.ld + j], level2), q = share_of(f, t.logit[row * t.ld + j], level2);
                if (q != 0.0f) s = __builtin_fmaf(q, d * kLn2 + (own - (PICK ? own_picked[j] : picked[row * t.ld + j])), s);
            }
            s = wave_sum(s);
            if (lane == 0) {
                lse[row] = own;
                loss[row] = mass == 0.0f ? 0.0f : s;
            }
        }
        __syncthreads();   // share and own_picked are written again
    }
}

// level[row] (in units of log 2) and mass[row], a wave a row.
__global__ __launch_bounds__(64 * kWaves) void mass_kernel(Teacher t, int m, int n, float *level, float *mass) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    for (int64_t row = (int64_t)blockIdx.x * kWaves + wave; row < m; row += (int64_t)gridDim.x * kWaves) {
        float l, q;
        teacher_row(t, row, n, lane, l, q);
        if (lane == 0) {
            level[row] = l;
            mass[row] = q;
        }
    }
}

// P at the teacher's columns of a piece of the vocabulary, written over the first term that the product
// left there: a wave a row, an entry a lane.  Entries of one column are all subtracted, and each of them
// writes the same value.
template <int IN>
__global__ __launch_bounds__(64 * kWaves) void scatter_kernel(Teacher t, int m, int n, int first, int have, const float *level,
                                                              const float *mass, const float *lse, const float *picked,
                                                              const int *place, const float *weight, uint16_t *P, int64_t ldp) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const float f = t.scale * kLog2e;
    for (int64_t row = (int64_t)blockIdx.x * kWaves + wave; row < m; row += (int64_t)gridDim.x * kWaves) {
        const int64_t at = place[row];
        if (at < 0) continue;
        const float w = weight[at], l2 = level[row];
        for (int j = lane; j - lane < t.top; j += 64) {       // (whole waves)
            const int v = entry_column(t, row, j, n);
            const bool in = v >= first && v - first < have;
            if (!__any(in)) continue;
            float q = 0.0f;
            for (int i0 = 0; i0 < t.top; i0 += 64) {
                const int o = i0 == j - lane ? v : entry_column(t, row, i0 + lane, n);
                const float s = o < 0 ? 0.0f : share_of(f, t.logit[row * t.ld + i0 + lane], l2);
                const int most = min(64, t.top - i0);
                for (int i = 0; i < most; ++i) {
                    const int other = __builtin_amdgcn_readlane(o, i);
                    const float so = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s), i));
                    q += other == v ? so : 0.0f;
                }
            }
            if (in) {
                const float p = mass[row] * fast_exp2((picked[row * t.ld + j] - lse[row]) * kLog2e);
                const float value = w == 0.0f ? 0.0f : w * (p - q);
                P[at * ldp + (v - first)] = (uint16_t)narrow2<IN>(value, 0.0f);
            }
        }
    }
}

int launch(const void *kernel, int64_t blocks, int waves, void **args, void *stream) {
    if (blocks == 0) return (int)hipSuccess;
    return (int)hipLaunchKernel(kernel, dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3((unsigned)(64 * waves)), args, 0,
                                (hipStream_t)stream);
}
int64_t by_waves(int64_t items) { return (items + kWaves - 1) / kWaves; }

template <int IN>
int launch_merge_type(const Teacher &t, const CeStat *stats, int parts, int m, int n, int k, float alpha, const uint16_t *x, int64_t ldx,
                      const uint16_t *w, int64_t ldw, float *picked, float *loss, float *lse, bool itself, void *stream) {
    if (!itself) {
        void *args[] = {const_cast<Teacher *>(&t), &m, &n, &k, &alpha, &x, &ldx, &w, &ldw, &picked};
        const int e = launch(reinterpret_cast<const void *>(&picked_kernel<IN>), by_waves((int64_t)m * ((t.top + kEntries - 1) / kEntries)),
                             kWaves, args, stream);
        if (e != 0) return e;
    }
    void *args[] = {const_cast<Teacher *>(&t), &stats, &parts, &m, &n, &k, &alpha, &x, &ldx, &w, &ldw, &picked, &loss, &lse};
    return launch(itself ? reinterpret_cast<const void *>(&distill_merge_kernel<IN, true>)
                         : reinterpret_cast<const void *>(&distill_merge_kernel<IN, false>),
                  m, kMergeWaves, args, stream);
}

}  // namespace

int launch_distill_merge(bool bf16, const Teacher &t, const CeStat *stats, int parts, int m, int n, int k, float alpha, const void *X,
                         int64_t ldx, const void *W, int64_t ldw, float *picked, float *loss, float *lse, bool itself, void *stream) {
    const auto f = bf16 ? launch_merge_type<IN_BF16> : launch_merge_type<IN_F16>;
    return f(t, stats, parts, m, n, k, alpha, (const uint16_t *)X, ldx, (const uint16_t *)W, ldw, picked, loss, lse, itself, stream);
}

int launch_mass(const Teacher &t, int m, int n, float *level, float *mass, void *stream) {
    void *args[] = {const_cast<Teacher *>(&t), &m, &n, &level, &mass};
    return launch(reinterpret_cast<const void *>(&mass_kernel), by_waves(m), kWaves, args, stream);
}

int launch_scatter(bool bf16, const Teacher &t, int m, int n, int first, int have, const float *level, const float *mass,
                   const float *lse, const float *picked, const int *place, const float *weight, void *P, int64_t ldp, void *stream) {
    uint16_t *p = (uint16_t *)P;
    void *args[] = {const_cast<Teacher *>(&t), &m, &n, &first, &have, &level, &mass, &lse, &picked, &place, &weight, &p, &ldp};
    return launch(bf16 ? reinterpret_cast<const void *>(&scatter_kernel<IN_BF16>) : reinterpret_cast<const void *>(&scatter_kernel<IN_F16>),
                  by_waves(m), kWaves, args, stream);
}

}  // namespace mpg
