// mpgemm_ops_epilogue.hpp -- what the op kernels do with a product's FP32 values: activations
// and their slopes, and the epilogue of eight consecutive columns of one row.
//
// Everything is computed in FP32; a result is rounded once, to nearest even, where it is stored.
#pragma once

#include "mpgemm_kernel.hpp"
#include "mpgemm_ops.hpp"

namespace mpg {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + exp(-x)) from the hardware's exp2 and reciprocal (1 ulp each): exp(-x) overflows to
// infinity for very negative x, whose reciprocal is the 0 that the sigmoid rounds to.
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp2(-kLog2e * x)); }

// Where a slope multiplies by z the factor beside it has reached 0 beyond +-30 in FP32: z is cut
// there, so that an infinite (or huge) value kept from the forward pass gives the slope's limit and
// no 0 * inf.  (NaN comes through the other factor.)
__device__ __forceinline__ float cut(float z) { return __builtin_amdgcn_fmed3f(z, -30.0f, 30.0f); }

// Phi(-|z|) of the normal distribution, and bell = exp(-z^2 / 2).  With x = |z| / sqrt(2) and
// t = 1 / (1 + 0.43 x), erfc(x) = exp(-x^2) t q(t), q a polynomial of degree 7 fitted to erfcx(x) in
// relative minimax over x in [0, 12] (2e-7, 5e-7 as evaluated in FP32); its coefficients are
// halved here.  The lower tail keeps its relative accuracy, as 1 + erf would not.
__device__ __forceinline__ float normal_tail(float z, float &bell) {
    const float t = fast_rcp(__builtin_fmaf(__builtin_fabsf(z), 0.43f * 0.70710678118654752f, 1.0f));
    bell = fast_exp2(z * (-0.5f * kLog2e) * z);
    float q = 0.5f * 0.07090955117377087f;
    q = __builtin_fmaf(q, t, -0.5f * 0.2990298556651683f);
    q = __builtin_fmaf(q, t, 0.5f * 0.36473237500049616f);
    q = __builtin_fmaf(q, t, -0.5f * 0.06881683436104556f);
    q = __builtin_fmaf(q, t, 0.5f * 0.2382076128012132f);
    q = __builtin_fmaf(q, t, 0.5f * 0.20746980043114047f);
    q = __builtin_fmaf(q, t, 0.5f * 0.24398845434153432f);
    q = __builtin_fmaf(q, t, 0.5f * 0.2425387182165695f);
    return bell * (q * t);
}

// The same without bell, for what is stored in 16 bits: exp2 of a polynomial of degree 7 fitted to
// log2 Phi(-a) over a in [0, kShortTail], 6.5e-6 relative there (an eightieth of half a step of FP16's);
// beyond, where Phi < 1e-9, it goes on falling, but to other values (0.6 % off at 8, 79 % at 12).  11
// instruction slots instead of 20 (a transcendental takes four).
constexpr float kShortTail = 6.0f;
__device__ __forceinline__ float normal_tail_short(float z) {
    const float a = __builtin_fabsf(z);
    float e = -1.8348151e-6f;
    e = __builtin_fmaf(e, a, 6.159837e-5f);
    e = __builtin_fmaf(e, a, -9.305254e-4f);
    e = __builtin_fmaf(e, a, 8.507893e-3f);
    e = __builtin_fmaf(e, a, -5.3960074e-2f);
    e = __builtin_fmaf(e, a, -4.5846438e-1f);
    e = __builtin_fmaf(e, a, -1.1512511f);
    e = __builtin_fmaf(e, a, -9.999953e-1f);
    return fast_exp2(e);
}

constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// SHORT: the value is stored in 16 bits and, for BF16, not below -kShortTail (see normal_tail_short).
template <int ACT, bool SHORT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z <= 0.0f ? 0.0f : z;   // NaN stays NaN
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|); |z| is cut where the tail is 0, for infinite z
    if constexpr (ACT == ACT_GELU) {
        float bell, tail;
        if constexpr (SHORT)
            tail = normal_tail_short(z);
        else
            tail = normal_tail(z, bell);
        return __builtin_fmaf(-__builtin_fminf(__builtin_fabsf(z), 30.0f), tail, __builtin_fmaxf(z, 0.0f));
    }
    // 0.5 z (1 + tanh u) = z / (1 + exp(-2u))
    if constexpr (ACT == ACT_GELU_TANH)
        return z * sigmoid(z * __builtin_fmaf(2.0f * kGeluC * kGeluA * z, z, 2.0f * kGeluC));
    if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == ACT_NONE) return 1.0f;
    if constexpr (ACT == ACT_GELU) {
        float bell;
        const float tail = normal_tail(z, bell);
        return __builtin_fmaf(cut(z) * 0.39894228040143268f, bell, z > 0.0f ? 1.0f - tail : tail);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float g = sigmoid(z * __builtin_fmaf(2.0f * kGeluC * kGeluA * z, z, 2.0f * kGeluC));
        // d(2u)/dz = 2 c (1 + 3 a z^2)
        const float c = cut(z);
        return __builtin_fmaf(__builtin_fmaf(-g, g, g) * c, __builtin_fmaf(6.0f * kGeluC * kGeluA * c, c, 2.0f * kGeluC), g);
    }
    const float g = sigmoid(z);   // ACT_SILU: g + z g (1 - g)
    return __builtin_fmaf(__builtin_fmaf(-g, g, g), cut(z), g);
}

// Both at once, from one exponential and one reciprocal.  z may have been kept in 16 bits, where a large
// negative value is -infinity: a factor that the sigmoid's 0 multiplies is cut, so that the value is 0 and
// no 0 * inf (NaN comes through the sigmoid).
template <int ACT>
__device__ __forceinline__ void act_both(float z, float &value, float &slope) {
    if constexpr (ACT == ACT_GELU) {
        float bell;
        const float tail = normal_tail(z, bell);
        value = __builtin_fmaf(-__builtin_fminf(__builtin_fabsf(z), 30.0f), tail, __builtin_fmaxf(z, 0.0f));
        slope = __builtin_fmaf(cut(z) * 0.39894228040143268f, bell, z > 0.0f ? 1.0f - tail : tail);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        const float g = sigmoid(z * __builtin_fmaf(2.0f * kGeluC * kGeluA * z, z, 2.0f * kGeluC));
        const float c = cut(z);
        value = __builtin_fmaxf(z, -1.0e4f) * g;
        slope = __builtin_fmaf(__builtin_fmaf(-g, g, g) * c, __builtin_fmaf(6.0f * kGeluC * kGeluA * c, c, 2.0f * kGeluC), g);
    } else if constexpr (ACT == ACT_SILU) {
        const float g = sigmoid(z);
        value = __builtin_fmaxf(z, -1.0e4f) * g;
        slope = __builtin_fmaf(__builtin_fmaf(-g, g, g), cut(z), g);
    } else {
        value = act_value<ACT, false>(z);
        slope = act_slope<ACT>(z);
    }
}

// Calls f(std::integral_constant<int, ACT>, std::bool_constant<SHORT>) for the activation named at
// run time and whether its long form is needed (both uniform).
template <typename F>
__device__ __forceinline__ void with_act(int act, bool wide, F &&f) {
    using Long = std::false_type;
    switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>{}, Long{}); break;
    case ACT_GELU:
        if (wide)
            f(std::integral_constant<int, ACT_GELU>{}, Long{});
        else
            f(std::integral_constant<int, ACT_GELU>{}, std::true_type{});
        break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>{}, Long{}); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>{}, Long{}); break;
    default: f(std::integral_constant<int, ACT_NONE>{}, Long{}); break;
    }
}

// ------------------------------------------------------------------------------- eight columns
template <int IN>
__device__ __forceinline__ float widen(uint32_t bits16) {
    if constexpr (IN == IN_F16)
        return (float)__builtin_bit_cast(_Float16, (unsigned short)bits16);
    else
        return __builtin_bit_cast(float, bits16 << 16);
}
// Two values as 16-bit ones, a in the low half: one conversion instruction for BF16 (converted one by
// one and joined they take four), two and a pack for FP16.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int IN>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (IN == IN_F16) {
        asm("" : "+v"(a), "+v"(b));   // the FP32 values first, then one rounding (no fused fma and conversion)
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    } else {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    }
}
template <int IN>
__device__ __forceinline__ void widen8(u32x4 x, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = widen<IN>(x[q] & 0xFFFFu);
        v[2 * q + 1] = widen<IN>(x[q] >> 16);
    }
}
template <int IN>
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
    u32x4 x;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x[q] = narrow2<IN>(v[2 * q], v[2 * q + 1]);
    return x;
}

// Where a workgroup's tile lies.
struct OpTile {
    int tm, tn;          // tile of its product
    int tile;            // GROUPS_ROWS: number of the row tile over all experts, else tm
    int expert, split;
    int row0;            // first row of A and D of its product
    int m, k;            // rows and summed length of its product
    int64_t d_off;       // element offset of its D
};

// What an epilogue reads besides the product: eight columns of C or of the kept Z, as stored (hi: the
// last four of FP32 values), or of a gated product's kept G and U (hi).
struct ChunkIn {
    u32x4 lo, hi;
};

// The eight columns col .. col + 7 of row `row` of D (ncol >= 1 of them exist).  C and aux are read
// in whole 16-byte blocks that hold a column that exists.
template <int MODE>
__device__ __forceinline__ void chunk_load(const OpParams &p, const OpTile &w, int64_t row, int col, int ncol,
                                           ChunkIn &in) {
    if (MODE == OP_FORWARD && p.C != nullptr) {
        const int64_t at = w.d_off + row * p.ldc + col;
        if (p.c_f32) {
            const float *c = (const float *)p.C + at;
            in.lo = *(const u32x4 *)c;
            if (ncol > 4) in.hi = *(const u32x4 *)(c + 4);
        } else {
            in.lo = *(const u32x4 *)((const uint16_t *)p.C + at);
        }
    }
    if (MODE == OP_SLOPE && p.aux != nullptr) in.lo = *(const u32x4 *)((const uint16_t *)p.aux + row * p.ld_aux + col);
}

// What OP_CE_PROBS takes from a row: its weight, its log-sum-exp in units of log 2 and where its target
// lies from the first of the eight columns (any other number: not among them).
struct RowScale {
    float weight, lse2;
    int target;
};

// A tile of D or aux: its first element and the bytes from one row to the next.
struct OpOut {
    __amdgpu_buffer_rsrc_t to;
    uint32_t ld;
};
__device__ __forceinline__ OpOut op_out(void *base, int64_t element, int64_t ld, int bytes) {
    return OpOut{make_rsrc((const char *)base + element * bytes), (uint32_t)(ld * bytes)};
}

// Stores eight values from column c of row `row` of a tile, ncol of which exist (whole: all).  What does
// not exist goes to an offset that the buffer drops, so that only a row's last, part-filled block
// takes a branch.  nt: past the caches (for whole 128-byte lines).
template <int POLICY>
__device__ __forceinline__ void store16(const OpOut &o, uint32_t off, u32x4 x) {
    __builtin_amdgcn_raw_buffer_store_b128(x, o.to, (int)off, 0, POLICY);
}
template <int IN>
__device__ __forceinline__ void store8(const OpOut &o, int f32, int row, int c, int ncol, bool whole, bool nt, const float (&v)[8]) {
    uint32_t off = (uint32_t)row * o.ld + (uint32_t)(f32 ? 4 * c : 2 * c);
    if (!whole && ncol <= 0) off = kOobOffset;
    if (f32) {
        const u32x4 lo = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
        const u32x4 hi = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
        if (!whole && ncol > 0 && ncol < 8) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                Out<OUT_F32>::store(o.to, q < ncol ? off + 4 * q : kOobOffset, v[q]);
        } else {
            // (two stores share each line: not past the caches, which would cost 273 us instead of 221 at
            // 8192 x 8192 x 2048)
            store16<0>(o, off, lo);
            store16<0>(o, off == kOobOffset ? off : off + 16, hi);
        }
    } else {
        const u32x4 x = narrow8<IN>(v);
        if (!whole && ncol > 0 && ncol < 8) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(q & 1 ? x[q / 2] >> 16 : x[q / 2]), o.to,
                                                      (int)(q < ncol ? off + 2 * q : kOobOffset), 0, 0);
        } else if (nt) {
            store16<kStreamPolicy>(o, off, x);
        } else {
            store16<0>(o, off, x);
        }
    }
}

// The bias of columns col .. col + 7 (zeros where there is none).
template <int IN>
__device__ __forceinline__ void bias_of(const OpParams &p, const void *bias, int expert, int col, float (&b)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) b[q] = 0.0f;
    if (bias == nullptr) return;
    const int64_t at = (int64_t)expert * p.bias_stride + col;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (col + q < p.n)
            b[q] = p.bias_f32 ? ((const float *)bias)[at + q] : widen<IN>(((const uint16_t *)bias)[at + q]);
}
template <int IN, int MODE>
__device__ __forceinline__ void bias_load(const OpParams &p, int expert, int col, float (&b)[8]) {
    bias_of<IN>(p, MODE == OP_FORWARD ? p.bias : nullptr, expert, col, b);
}

// alpha, times the device factor where there is one.
__device__ __forceinline__ float op_alpha(const OpParams &p) {
    return p.scale != nullptr ? p.alpha * p.scale[0] : p.alpha;
}

// Turns the products v of eight columns from column c of the tile in each of G rows into what is stored,
// and stores it to D's tile d (and Z's, aux); sums adds up what OP_SLOPE stores (before its rounding).
// row(i) is row i's place in the tile, ncol(i) how many of the columns exist there (at most 0: the row
// does not; whole: all do).  The arithmetic of two rows runs together, so that one element's
// latencies are covered by the others' (all rows at once would need more registers than a wave has).
template <int IN, int MODE, int G, typename Row, typename Cols>
__device__ __forceinline__ void rows_finish(const OpParams &p, float alpha, const OpOut &d, const OpOut &aux, int c, bool whole,
                                            bool nt, Row &&row, Cols &&ncol, const ChunkIn (&in)[G], const RowScale (&scale)[G],
                                            const float (&bias)[8], float (&v)[G][8], float (&sums)[8]) {
    if constexpr (MODE == OP_SLOPE) {
        float z[G][8];
#pragma unroll
        for (int i = 0; i < G; ++i) widen8<IN>(in[i].lo, z[i]);
        with_act(p.act, true, [&](auto a, auto) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[i][q] = alpha * v[i][q] * act_slope<decltype(a)::value>(z[i][q]);
                if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
        });
        if (p.colsum != nullptr) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 8; ++q) sums[q] += v[i][q];
            } else {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 8; ++q) sums[q] += ncol(i) > 0 ? v[i][q] : 0.0f;
            }
        }
    } else if constexpr (MODE == OP_CE_PROBS) {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float e = fast_exp2(__builtin_fmaf(alpha * kLog2e, v[i][q], -scale[i].lse2));
                // a row that does not count has weight 0: nothing of its product may reach D
                v[i][q] = scale[i].weight == 0.0f ? 0.0f : (e - (scale[i].target == q ? 1.0f : 0.0f)) * scale[i].weight;
            }
    } else {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = __builtin_fmaf(alpha, v[i][q], bias[q]);
        if (p.aux != nullptr) {
#pragma unroll
            for (int i = 0; i < G; ++i) store8<IN>(aux, 0, row(i), c, ncol(i), whole, nt, v[i]);
        }
        // z Phi(z) below the short tail's range: FP16 rounds it to 0 (|z| Phi < 6e-9), BF16 holds it, so that a wave
        // with such values takes the long form (above the range the tail is gone).  8192 x 8192 x 2048 with Z kept: 242 us
        // without the test, 244 where z has a deviation of 1, 255 where it has one of 4 and most groups are such.
        bool wide = p.d_f32;
        if (IN == IN_BF16 && p.act == ACT_GELU && !wide) {
            float low = 0.0f;
            if (whole) {
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 8; ++q) low = __builtin_fminf(low, v[i][q]);
            } else {   // (what lies past the rows' ends decides nothing)
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 8; ++q) low = __builtin_fminf(low, q < ncol(i) ? v[i][q] : 0.0f);
            }
            wide = __any(low < -kShortTail);
        }
        with_act(p.act, wide, [&](auto a, auto s) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[i][q] = act_value<decltype(a)::value, decltype(s)::value>(v[i][q]);
                if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
        });
        if (p.C != nullptr) {
            if (p.c_f32) {
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const f32x4 lo = __builtin_bit_cast(f32x4, in[i].lo), hi = __builtin_bit_cast(f32x4, in[i].hi);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[i][q] = __builtin_fmaf(p.beta, lo[q], v[i][q]);
                        v[i][q + 4] = __builtin_fmaf(p.beta, hi[q], v[i][q + 4]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    float old[8];
                    widen8<IN>(in[i].lo, old);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[i][q] = __builtin_fmaf(p.beta, old[q], v[i][q]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) store8<IN>(d, p.d_f32, row(i), c, ncol(i), whole, nt, v[i]);
}

// ------------------------------------------------------------------------------- gated products
// The outputs of a gated product's tile: D and both kept factors, or dG, dU and H.
struct GatedOut {
    OpOut d, g, u;
};

// rows_finish for a gated product: v holds the gate's products, x the up projection's.  D is stored to
// out.d, the factors (where p.aux is set) to out.g and out.u.
template <int IN, int G, typename Row, typename Cols>
__device__ __forceinline__ void gated_finish(const OpParams &p, const GatedOut &out, int c, bool whole, bool nt, Row &&row,
                                             Cols &&ncol, const float (&bias)[8], const float (&bias_up)[8], float (&v)[G][8],
                                             float (&x)[G][8]) {
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[i][q] = __builtin_fmaf(p.alpha, v[i][q], bias[q]);
            x[i][q] = __builtin_fmaf(p.alpha, x[i][q], bias_up[q]);
        }
    if (p.aux != nullptr) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            store8<IN>(out.g, 0, row(i), c, ncol(i), whole, nt, v[i]);
            store8<IN>(out.u, 0, row(i), c, ncol(i), whole, nt, x[i]);
        }
    }
    // (GELU in its long form throughout: the other factor may be large, so that a tail that 16 bits would
    // round to nothing by itself is not nothing in the product)
    with_act(p.act, true, [&](auto a, auto) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = act_value<decltype(a)::value, false>(v[i][q]) * x[i][q];
            if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
    });
#pragma unroll
    for (int i = 0; i < G; ++i) store8<IN>(out.d, p.d_f32, row(i), c, ncol(i), whole, nt, v[i]);
}

// The gradient: v holds the products E, in the kept G and U (lo, hi).  dG goes to out.d, dU to out.u and
// H (where p.H is set) to out.g; sums and sums_up add up dG and dU before their rounding.
template <int IN, int G, typename Row, typename Cols>
__device__ __forceinline__ void gated_grad_finish(const OpParams &p, const GatedOut &out, int c, bool whole, bool nt, Row &&row,
                                                  Cols &&ncol, const ChunkIn (&in)[G], float (&v)[G][8], float (&sums)[8],
                                                  float (&sums_up)[8]) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
        float g[8], u[8], du[8], h[8];
        widen8<IN>(in[i].lo, g);
        widen8<IN>(in[i].hi, u);
        with_act(p.act, true, [&](auto a, auto) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float value, slope;
                act_both<decltype(a)::value>(g[q], value, slope);
                const float e = p.alpha * v[i][q];
                du[q] = e * value;
                h[q] = value * u[q];
                v[i][q] = e * u[q] * slope;
            }
        });
        if (p.colsum != nullptr) {
            const bool live = whole || ncol(i) > 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                sums[q] += live ? v[i][q] : 0.0f;
                sums_up[q] += live ? du[q] : 0.0f;
            }
        }
        store8<IN>(out.d, p.d_f32, row(i), c, ncol(i), whole, nt, v[i]);
        store8<IN>(out.u, p.d_f32, row(i), c, ncol(i), whole, nt, du);
        if (p.H != nullptr) store8<IN>(out.g, 0, row(i), c, ncol(i), whole, nt, h);
    }
}

// ------------------------------------------------------------------------------- experts' rows
// Rows [lo, hi) of expert e.  Offsets outside 0 .. rows or decreasing ones are clamped, so that no
// value on the device makes a kernel touch memory outside the operands.
__device__ __forceinline__ void expert_rows(const int *offsets, int e, int rows, int &lo, int &hi) {
    lo = min(max(offsets[e], 0), rows);
    hi = max(lo, min(max(offsets[e + 1], 0), rows));
}

// A value that every lane of a wave holds alike, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v), hi = (uint32_t)uniform((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Inclusive prefix sum over a wave's 64 lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}

// Row tiles of `tile_rows` rows before expert e and of expert e itself, by one whole wave.
__device__ __forceinline__ void expert_tiles(const OpParams &p, int tile_rows, int expert, int lane, int64_t &before,
                                             int &own, int &lo, int &hi) {
    before = 0;
    for (int base = 0; base <= expert; base += 64) {
        int l = 0, h = 0;
        if (base + lane < p.groups) expert_rows(p.offsets, base + lane, p.m, l, h);
        const int t = (h - l + tile_rows - 1) / tile_rows;
        const int64_t incl = wave_scan(t, lane);
        if (expert < base + 64) {
            const int src = expert - base;
            before += __shfl(incl - t, src, 64);
            own = __shfl(t, src, 64);
            lo = __shfl(l, src, 64);
            hi = __shfl(h, src, 64);
        } else {
            before += __shfl(incl, 63, 64);
        }
    }
}

// tile_coords without a last group of one or two tile rows: of five tile rows (517 rows), in groups of four, the fifth
// would read op(B) once more with nothing beside it to share it (517 x 50021 x 1000, loss alone: 94 us so, 88
// together).  Of more than two rounds of tiles (65536 / BM a round) up to seven a group (its gradients, where dW has 391 x
// 8 tiles: 383 us with four, 363 with eight, 350 with seven), of 256-wide ones eight where that leaves none over, since an XCD
// has 32 at once (2047 x 50021 x 1000, loss alone: 236 us with four to seven, 232 with eight; but 31 x 20 tiles, 7868 x
// 5016 x 1880, 221 with six and seven, 240 with seven and eight), of fewer four (4925 x 1264 x 3411: 71.5 us, 77 with six to
// eight; 6160 rows of 350 gated outputs over 3618 in tiles of 64: 64.3, 70.8 with seven).
//
// wide: D's rows lie a multiple of 32 KB apart, over which the memory's channels (128 of 256 bytes) repeat: at the end of
// a round of equal tiles, the columns of 16 of them meet in a part of the channels, whatever the row.  There the regions
// of tile_coords become 8 x 32 tiles (gradient of a gated product, 4096 x 8192, D side by side: over 4096 268 -> 251 us,
// over 1024 140 -> 119; 4096 x 16384 x 4096, BF16 D 415 -> 404.  With other distances the two come to the same).  Only whole
// rounds are laid out so, 2048 rows by 8192 columns.
template <int BM>
__device__ __forceinline__ void op_tile_coords(bool wide, int wg, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int total = tiles_m * tiles_n, run = total / 8;
    const int id = wg < run * 8 ? (wg % 8) * run + wg / 8 : wg;
    if (tiles_m <= kGroupM + 2) {
        tn = tiles_m == 1 ? id : id / tiles_m;
        tm = id - tn * tiles_m;
        return;
    }
    if (BM == 256 && wide && tiles_m % 8 == 0 && tiles_n % 32 == 0) {
        const int xcd = wg % 8, i = wg / 8 % 32, round = wg / 256, regions = tiles_n / 32;
        const int ra = round / regions, rb = round % regions;
        tm = 8 * ra + 4 * (xcd % 2) + i % 4;
        tn = 32 * (ra % 2 == 0 ? rb : regions - 1 - rb) + 8 * (xcd / 2) + i / 4;
        return;
    }
    if (tiles_m % 16 == 0 && tiles_n % 16 == 0) return tile_coords(wg, tiles_m, tiles_n, tm, tn);
    int rows, cut, rows_after;   // tile rows of a group, and from tile row `cut` on
    if (total > 2 * (65536 / BM)) {
        const int groups = BM == 256 && tiles_m % 8 == 0 ? tiles_m / 8 : (tiles_m + 6) / 7;
        rows = tiles_m / groups;
        rows_after = rows + 1;
        cut = (groups - tiles_m % groups) * rows;
    } else {
        rows = kGroupM;
        cut = ((tiles_m + 1) / kGroupM - 1) * kGroupM;
        rows_after = tiles_m - cut;
    }
    const int before = id < cut * tiles_n ? 0 : cut;
    if (before > 0) rows = rows_after;
    const int group = (id - before * tiles_n) / (rows * tiles_n), in = id - (before + group * rows) * tiles_n;
    tm = before + group * rows + in % rows;
    tn = in / rows;
}

// The tile of workgroup `wg`; false: none is left for it.  Every wave of a workgroup finds it for
// itself.  The experts' tiles follow each other, an expert's own by columns of tiles (which share
// its weights); each XCD gets a contiguous run of them.
template <int BM>
__device__ __forceinline__ bool locate(const OpParams &p, int wg, int split, int lane, OpTile &w) {
    w.split = split;
    w.expert = 0;
    w.row0 = 0;
    w.m = p.m;
    w.k = p.k;
    w.d_off = 0;
    if (p.groups_kind == GROUPS_ROWS) {
        int64_t total = 0;
        for (int base = 0; base < p.groups; base += 64) {
            int lo = 0, hi = 0;
            if (base + lane < p.groups) expert_rows(p.offsets, base + lane, p.m, lo, hi);
            total += __shfl(wave_scan((hi - lo + BM - 1) / BM, lane), 63, 64);
        }
        total = uniform64(total) * p.tiles_n;
        if (wg >= total) return false;
        const int64_t run = min(total, (int64_t)p.tiles_m * p.tiles_n) / 8;
        const int64_t id = wg < run * 8 ? (wg % 8) * run + wg / 8 : wg;
        int64_t before = 0;
        for (int base = 0; base < p.groups; base += 64) {
            int lo = 0, hi = 0;
            if (base + lane < p.groups) expert_rows(p.offsets, base + lane, p.m, lo, hi);
            const int t = (hi - lo + BM - 1) / BM;
            const int64_t incl = before + wave_scan(t, lane);
            const uint64_t hit = (uint64_t)uniform64((int64_t)__ballot(t > 0 && id < incl * p.tiles_n && id >= (incl - t) * p.tiles_n));
            if (hit != 0) {
                const int src = __builtin_ctzll(hit);
                const int own = uniform(__shfl(t, src, 64));
                const int first = uniform((int)__shfl(incl - t, src, 64));
                w.expert = base + src;
                w.row0 = uniform(__shfl(lo, src, 64));
                w.m = uniform(__shfl(hi, src, 64)) - w.row0;
                const int local = uniform((int)(id - (int64_t)first * p.tiles_n));
                w.tm = local % own;
                w.tn = local / own;
                w.tile = first + w.tm;
                return true;
            }
            before = uniform64(__shfl(incl, 63, 64));
        }
        return false;
    }
    if (p.groups_kind == GROUPS_K) {
        const int per = p.tiles_m * p.tiles_n;
        const int total = per * p.groups, run = total / 8;
        const int id = wg < run * 8 ? (wg % 8) * run + wg / 8 : wg;
        w.expert = id / per;
        const int local = id - w.expert * per;
        w.tm = local % p.tiles_m;
        w.tn = local / p.tiles_m;
        w.tile = w.tm;
        int lo, hi;
        expert_rows(p.offsets, w.expert, p.k, lo, hi);
        w.row0 = 0;
        w.k = uniform(hi) - uniform(lo);
        w.d_off = (int64_t)w.expert * p.stride_d;
        return true;
    }
    // Only the tiles of rows that take part are laid out: the workgroups of the others leave from the end of the
    // grid and not from one XCD's run (2650 rows, half of them ignored, over 12305 columns, k = 2168, loss and gradients:
    // 564 us, 635 with them in).
    int tiles_m = p.tiles_m;
    if (p.count != nullptr) {
        const int count = max(uniform(p.count[0]), 0);
        if (p.count_k) {
            w.k = min(p.k, count);
        } else {
            w.m = min(p.m, count);
            tiles_m = (w.m + BM - 1) / BM;
        }
    }
    const int per = tiles_m * p.tiles_n;
    if (p.splits > 1) {
        // Ranges of k share nothing, the tiles of one range all of its rows and columns: each XCD gets a contiguous
        // run over (range, tile), so that a range's operands come to one or two L2s and not to all eight
        // (466 x 1000 over 50021 in 12 ranges of 32 tiles: 185 MB read, 66 us; tile by tile over the XCDs 541 MB, 102 us).
        const int total = per * p.splits, run = total / 8, l = split * p.tiles_m * p.tiles_n + wg;
        if (l >= total) return false;
        const int id = l < run * 8 ? (l % 8) * run + l / 8 : l;
        w.split = split = id / per;
        const int local = id - split * per;
        w.tm = local % tiles_m;
        w.tn = local / tiles_m;
    } else {
        if (wg >= per) return false;
        op_tile_coords<BM>(p.wide, wg, tiles_m, p.tiles_n, w.tm, w.tn);
    }
    w.tile = w.tm;
    if (p.splits > 1) {
        w.k = min(p.k_split, p.k - split * p.k_split);
        w.d_off = (int64_t)split * p.stride_split;
    }
    return true;
}

// The operands of a tile's product.
template <bool TA, bool TB>
__device__ __forceinline__ Params op_operands(const OpParams &p, const OpTile &w) {
    Params q = {};
    int64_t ka = 0, kb = 0;   // first summed index in A and in B
    if (p.groups_kind == GROUPS_K) {
        int lo, hi;
        expert_rows(p.offsets, w.expert, p.k, lo, hi);
        ka = kb = uniform(lo);
    } else if (p.splits > 1) {
        ka = kb = (int64_t)w.split * p.k_split;
    }
    const int64_t a = (int64_t)w.row0 * (TA ? 1 : p.lda) + ka * (TA ? p.lda : 1);
    const int64_t b = kb * (TB ? 1 : p.ldb) + (p.groups_kind == GROUPS_ROWS ? (int64_t)w.expert * p.stride_b : 0);
    q.A = (const char *)p.A + 2 * a;
    q.B = (const char *)p.B + 2 * b;
    q.lda = p.lda;
    q.ldb = p.ldb;
    q.m = w.m;
    q.n = p.n;
    q.k = w.k;
    return q;
}

// ------------------------------------------------------------------------------- row statistics
// Reductions over the 16 lanes of a DPP row (every lane gets the result).
template <int R>
__device__ __forceinline__ float row_rotate(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + R, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_max16(float v) {
    v = fmaxf(v, row_rotate<8>(v));
    v = fmaxf(v, row_rotate<4>(v));
    v = fmaxf(v, row_rotate<2>(v));
    return fmaxf(v, row_rotate<1>(v));
}
__device__ __forceinline__ float row_sum16(float v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
}
// What exponentials are taken from: the maximum, or 0 where there is no finite one below +inf
// (a range without columns, or of -inf alone, then sums to 0 and not to NaN).
__device__ __forceinline__ float stat_base(float top) { return top == -__builtin_inff() ? 0.0f : top; }

}  // namespace mpg
