// mpgemm_ops_kernel.hpp -- the tiled op kernel: the matrix product of mpgemm_kernel.hpp with the
// epilogues of mpgemm_ops.hpp, over one product, one product per expert or ranges of k.
//
// The K loop is tile_product's.  The epilogue takes the FP32 accumulators through the LDS, which
// the product has left free: each wave writes two block rows (32 rows of its sub-tile) at a time in
// row-major order to a region of its own (rows padded by 16 bytes, so that the four row groups an
// accumulator register holds fall on different banks) and reads them back eight columns a lane,
// so that C, aux and D move in 16-byte pieces of whole lines and a lane keeps its columns: the
// bias is read once per tile and the column sums of the gradient stay in registers until a
// tile's end.  Rows are taken in groups of up to four steps whose arithmetic runs together: with one
// wave per SIMD nothing else covers a step's latencies (8192 x 8192 x 2048 without an activation:
// 264 us step by step, 227 in groups, 207 with the present stores).
//
// What the epilogue reads (C, or the kept Z) comes by direct-to-LDS loads through a ring in the
// wave's region, up to four groups ahead of its use and without holding a register.
#pragma once

#include "mpgemm_ops_epilogue.hpp"

namespace mpg {

// Waits until at most n of the wave's vector-memory operations are in flight (n rounded down to a
// count that is built in; the tests are uniform).
__device__ __forceinline__ void wait_vmem_upto(int n) {
    if (n >= 24) wait_vmem<24>();
    else if (n >= 16) wait_vmem<16>();
    else if (n >= 12) wait_vmem<12>();
    else if (n >= 8) wait_vmem<8>();
    else if (n >= 4) wait_vmem<4>();
    else if (n >= 2) wait_vmem<2>();
    else wait_vmem<0>();
}

template <int IN, int MODE, int FM, int FN, int BM, int BN>
__device__ __forceinline__ void op_store_tile(const OpParams &p, const OpTile &w, f32x4 (&acc)[FM][FN], lds_char *smem,
                                              int wave, int lane) {
    constexpr int WR = BM / 2, WC = BN / 2;        // the wave's sub-tile
    constexpr int kBR = 2;                         // block rows per pass
    constexpr int RS = WC * 4 + 16;                // bytes of a staged row
    constexpr int CH = WC / 8;                     // lanes per row
    constexpr int RI = 64 / CH;                    // rows per step
    constexpr int kSteps = 16 * kBR / RI;          // steps per pass
    constexpr int G = BM == 256 ? 4 : 2;           // steps per group (fewer registers where two workgroups share a CU)
    constexpr int kGroups = WR / (RI * G);         // groups per tile
    constexpr int kDepth = kGroups < 4 ? kGroups : 4;   // groups of 16-bit values that the ring holds
    // (one group of FP32 values needs as much as two of 16 bits)
    constexpr int kStage = 16 * kBR * RS, kRing = (kDepth < 2 ? 2 : kDepth) * G * 1024;
    static_assert(4 * (kStage + kRing) <= tile_lds_bytes<IN, BM, BN>(), "staging and ring fit the stages");
    static_assert(kSteps % G == 0 && FM % kBR == 0, "whole groups and passes");
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

    const int wm = wave / 2, wn = wave % 2;
    lds_char *region = smem + wave * (kStage + kRing);
    lds_char *ring = region + kStage;
    const int g = lane / 16, u = lane % 16;
    lds_char *wr = region + (4 * g) * RS + u * 4;
    const int c = lane % CH, rr = lane / CH;
    const lds_char *rd = region + rr * RS + c * 32;
    const int col = w.tn * BN + wn * WC + 8 * c;
    const int ncol = p.n - col;                    // may be <= 0
    const int row_t = w.tm * BM + wm * WR;         // the wave's first row of its product
    // whole tiles (a uniform test) need no masks and move whole lines
    const bool full = (w.tm + 1) * BM <= w.m && (w.tn + 1) * BN <= p.n;
    const bool nt = full && p.lines;
    auto cols_of = [&](int row) { return full ? 8 : (row < w.m ? ncol : 0); };

    // The ring: a step's 16 bytes a lane (16-bit values) or twice that (FP32 C, half as many groups).
    const bool read_c = MODE == OP_FORWARD && p.C != nullptr, read_z = MODE == OP_SLOPE && p.aux != nullptr;
    const bool wide = read_c && p.c_f32;
    const int loads = read_c || read_z ? (wide ? 2 : 1) : 0;    // per step
    const int depth = wide ? (kDepth > 1 ? kDepth / 2 : 1) : kDepth;
    const int64_t src_ld = read_c ? p.ldc : p.ld_aux;
    const int src_bytes = wide ? 4 : 2;
    const char *src = (const char *)(read_c ? p.C : p.aux) +
                      ((read_c ? w.d_off : 0) + ((int64_t)w.row0 + row_t) * src_ld + w.tn * BN + wn * WC) * src_bytes;
    const i32x4 rs = make_rsrc_words(src);
    const uint32_t ring_addr = (uint32_t)(uintptr_t)ring;
    auto fetch = [&](int group) {                  // loads of a group into its place of the ring
        const uint32_t at = ring_addr + (uint32_t)(group % depth * G * loads) * 1024u;
#pragma unroll
        for (int q = 0; q < G; ++q) {
            const int row = (group * G + q) * RI + rr;
            const uint32_t off = (uint32_t)row * (uint32_t)(src_ld * src_bytes) + (uint32_t)(8 * c * src_bytes);
            const int nc = cols_of(row_t + row);
            dma16(rs, nc > 0 ? off : kOobOffset, 0u, at + (uint32_t)(q * loads) * 1024u);
            if (wide) dma16(rs, nc > 4 ? off + 16u : kOobOffset, 0u, at + (uint32_t)(q * loads + 1) * 1024u);
        }
    };
    // the wave's sub-tile of D and of the Z that is kept
    const int64_t row_d = (int64_t)w.row0 + row_t;
    const int col_d = w.tn * BN + wn * WC;
    const OpOut out_d = op_out(p.D, w.d_off + row_d * p.ldd + col_d, p.ldd, p.d_f32 ? 4 : 2);
    const OpOut out_z = op_out(p.aux, row_d * p.ld_aux + col_d, p.ld_aux, 2);
    const float alpha = op_alpha(p);
    float bias[8], sums[8];
    bias_load<IN, MODE>(p, w.expert, col, bias);
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[q] = 0.0f;
    // The loads below are counted: nothing the compiler has issued may be waited for later on.
    if (loads > 0) {
        wait_vmem<0>();
        for (int i = 0; i < depth; ++i) fetch(i);
    }
    // Row factors of the cross entropy's probabilities, read once per tile into the ring's place: weight,
    // log-sum-exp (in units of log 2) and the target's column.
    struct RowFactor {
        float weight, lse;
        int target, pad;
    };
    typedef __attribute__((address_space(3))) RowFactor lds_factor;
    static_assert(WR * (int)sizeof(RowFactor) <= kRing, "row factors fit the ring");
    if constexpr (MODE == OP_CE_PROBS) {
        for (int r = lane; r < WR; r += 64) {
            RowFactor f = {0.0f, 0.0f, -1, 0};
            if (row_t + r < w.m) {
                f.weight = p.weight[row_t + r];
                f.lse = p.lse[row_t + r] * kLog2e;
                const int64_t t = p.target[row_t + r] - p.col0;
                f.target = t >= 0 && t < p.n ? (int)t : -1;
            }
            lds_factor *to = (lds_factor *)(ring + r * (int)sizeof(RowFactor));
            to->weight = f.weight;
            to->lse = f.lse;
            to->target = f.target;
        }
    }
    // Operations that may be in flight when a group's loads have landed: the loads of the groups
    // after it and, in a whole tile (where none is masked off), the stores since.
    const int stores = full && loads > 0 ? G * ((p.d_f32 ? 2 : 1) + (MODE == OP_FORWARD && p.aux != nullptr ? 1 : 0)) : 0;

#pragma unroll 1
    for (int pass = 0; pass < FM / kBR; ++pass) {
        if (pass > 0) wait_lds<0>();               // the previous pass has been read back
        static_for<FM / kBR>([&](auto pass_c) {
            constexpr int at = decltype(pass_c)::value;
            if (pass == at) {
                // (a statement of its own in each branch: merged, they would index the accumulators at run time)
                asm volatile("; pass %0" : : "i"(at));
                static_for<kBR>([&](auto i_c) {
                    constexpr int i = decltype(i_c)::value;
                    static_for<FN>([&](auto j_c) {
                        constexpr int j = decltype(j_c)::value;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            *(lds_float *)(wr + (16 * i + r) * RS + 64 * j) = acc[at * kBR + i][j][r];
                    });
                });
                asm volatile("; staged %0" : : "i"(at));
            }
        });
#pragma unroll 1
        for (int s = 0; s < kSteps; s += G) {
            const int group = (pass * kSteps + s) / G;
            float v[G][8];
#pragma unroll
            for (int q = 0; q < G; ++q) {
                const lds_char *at = rd + (s + q) * RI * RS;
                const f32x4 a = *(const lds_f32x4 *)at, b = *(const lds_f32x4 *)(at + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[q][e] = a[e];
                    v[q][e + 4] = b[e];
                }
            }
            ChunkIn in[G];
            if (loads > 0) {
                const int after = min(depth - 1, kGroups - 1 - group);
                wait_vmem_upto(after * G * loads + min(depth - 1, group) * stores);
                const lds_char *at = ring + (group % depth * G * loads) * 1024 + 16 * lane;
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    in[q].lo = *(const lds_u32x4 *)(at + q * loads * 1024);
                    if (wide) in[q].hi = *(const lds_u32x4 *)(at + (q * loads + 1) * 1024);
                }
            }
            RowScale scale[G];
            if constexpr (MODE == OP_CE_PROBS) {
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    const lds_factor *f =
                        (const lds_factor *)(ring + ((pass * kSteps + s + q) * RI + rr) * (int)sizeof(RowFactor));
                    scale[q] = RowScale{f->weight, f->lse, f->target - col};
                }
            }
            const int row_s = (pass * kSteps + s) * RI + rr;
            rows_finish<IN, MODE, G>(
                p, alpha, out_d, out_z, 8 * c, full, nt, [&](int q) { return row_s + q * RI; },
                [&](int q) { return cols_of(row_t + row_s + q * RI); }, in, scale, bias, v, sums);
            if (loads > 0 && group + depth < kGroups) {
                wait_lds<0>();                     // the group's place has been read
                fetch(group + depth);
            }
        }
    }
    if (MODE == OP_SLOPE && p.colsum != nullptr && w.tile < p.tiles_m) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int d = CH; d < 64; d *= 2) sums[q] += __shfl_xor(sums[q], d, 64);
        if (rr == 0 && ncol > 0) {
            // (rows of whole 8-column blocks: the last one is written past n)
            float *to = p.colsum + (int64_t)(2 * w.tile + wm) * p.ld_colsum + col;
            *(f32x4 *)to = f32x4{sums[0], sums[1], sums[2], sums[3]};
            *(f32x4 *)(to + 4) = f32x4{sums[4], sums[5], sums[6], sums[7]};
        }
    }
}

// Maximum and sum of exponentials of each row over the wave's columns, straight from the
// accumulators: a row's columns lie in the 16 lanes of a DPP row and FN registers, so both
// reductions need no LDS.  Values are in units of log 2.  kPlain: a whole tile and scale > 0, where
// the maximum is taken of the products as they are and the scaling is part of the exponent's
// subtraction (3 instead of 6 operations around each exponential).
template <bool kPlain, int FM, int FN, int BM, int BN>
__device__ __forceinline__ void op_row_stats(const OpParams &p, const OpTile &w, f32x4 (&acc)[FM][FN], float scale, int wave, int lane) {
    const int wm = wave / 2, wn = wave % 2;
    const int g = lane / 16, u = lane % 16;
    const int col = w.tn * BN + wn * (BN / 2) + u;
    const int row0 = w.tm * BM + wm * (BM / 2) + 4 * g;
    CeStat *to = p.stats + (int64_t)row0 * p.parts + 2 * w.tn + wn;
    static_for<FM>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        float v[4][FN], top[4], sum[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            top[r] = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                v[r][j] = kPlain ? acc[i][j][r] : (col + 16 * j < p.n ? acc[i][j][r] * scale : -__builtin_inff());
                top[r] = fmaxf(top[r], v[r][j]);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) top[r] = row_max16(top[r]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (kPlain) top[r] *= scale;
            const float base = stat_base(top[r]);
            sum[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sum[r] += fast_exp2(kPlain ? __builtin_fmaf(v[r][j], scale, -base) : v[r][j] - base);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] = row_sum16(sum[r]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (u == 0 && row0 + 16 * i + r < w.m) to[(int64_t)(16 * i + r) * p.parts] = CeStat{top[r], sum[r]};
    });
}

// One instance per epilogue: with all of them in one kernel, chosen at run time, the accumulators no
// longer fit beside the epilogue's registers (60 spilled ones cost 10 % of 8192 x 8192 x 2048).
template <int IN, int MODE, bool TA, bool TB, int T>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(T == 256 ? 1 : 2, T == 256 ? 1 : 2)))
void op_kernel(OpParams p) {
    __shared__ __attribute__((aligned(16))) char smem_raw[tile_lds_bytes<IN, T, T>()];
    lds_char *smem = (lds_char *)smem_raw;
    constexpr int FM = T / 32, FN = T / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    OpTile w;
    if (!locate<T>(p, blockIdx.x, blockIdx.y, lane, w)) return;
    const Params q = op_operands<TA, TB>(p, w);
    f32x4 acc[FM][FN];
    tile_product<IN, TA, TB, T, T, 4>(q, w.tm * T, w.tn * T, smem, acc);
    int lane_e = lane;
    asm volatile("" : "+v"(lane_e));   // the epilogue's addresses are formed after the loop
    if constexpr (MODE == OP_CE_STATS) {
        const float scale = p.alpha * kLog2e;
        if ((w.tn + 1) * T <= p.n && scale > 0.0f)
            op_row_stats<true, FM, FN, T, T>(p, w, acc, scale, wave, lane_e);
        else
            op_row_stats<false, FM, FN, T, T>(p, w, acc, scale, wave, lane_e);
    } else {
        __syncthreads();               // every wave's fragment reads are done: the LDS is free
        op_store_tile<IN, MODE, FM, FN, T, T>(p, w, acc, smem, wave, lane_e);
    }
}

template <int IN, int MODE, bool TA, bool TB, int T>
int launch_op(const OpParams &p, hipStream_t stream) {
    const unsigned tiles = (unsigned)p.tiles_m * (unsigned)p.tiles_n * (p.groups_kind == GROUPS_K ? (unsigned)p.groups : 1u);
    void *args[] = {const_cast<OpParams *>(&p)};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&op_kernel<IN, MODE, TA, TB, T>),
                                dim3(tiles, (unsigned)p.splits), dim3(256), args, 0, stream);
}

template <int IN, int MODE, bool TA, bool TB>
int launch_op_tile(int tile, const OpParams &p, hipStream_t s) {
    switch (tile) {
    case 256: return launch_op<IN, MODE, TA, TB, 256>(p, s);
    case 128: return launch_op<IN, MODE, TA, TB, 128>(p, s);
    case 64: return launch_op<IN, MODE, TA, TB, 64>(p, s);
    default: return (int)hipErrorInvalidValue;
    }
}

}  // namespace mpg
