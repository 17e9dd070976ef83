// mpgemm_ops_kernel.hpp -- the tiled op kernel: the matrix product of mpgemm_kernel.hpp with the
// epilogues of mpgemm_ops.hpp, over one product, one product per expert or ranges of k.
//
// The K loop is tile_product's.  The epilogue takes the FP32 accumulators through the LDS, which
// the product has left free: each wave writes up to four block rows (64 rows of its sub-tile) in
// row-major order to a region of its own (rows padded by 16 bytes, so that the four row groups an
// accumulator register holds fall on different banks) and reads them back eight columns a lane,
// so that C, aux and D move in 16-byte pieces of whole lines and a lane keeps its columns: the
// bias is read once per tile and the column sums of the gradient stay in registers until a
// tile's end.  What the epilogue reads is asked for one group of rows ahead of its use.
#pragma once

#include "mpgemm_ops_epilogue.hpp"

namespace mpg {

template <int IN, int FM, int FN, int BM, int BN>
__device__ __forceinline__ void op_store_tile(const OpParams &p, const OpTile &w, f32x4 (&acc)[FM][FN], lds_char *smem,
                                              int wave, int lane) {
    constexpr int WR = BM / 2, WC = BN / 2;        // the wave's sub-tile
    constexpr int kBR = FM < 4 ? FM : 4;           // block rows per pass
    constexpr int RS = WC * 4 + 16;                // bytes of a staged row
    constexpr int CH = WC / 8;                     // lanes per row
    constexpr int RI = 64 / CH;                    // rows per step
    constexpr int kSteps = 16 * kBR / RI;          // steps per pass
    constexpr int G = kSteps < 4 ? kSteps : 4;     // steps per group
    static_assert(4 * 16 * kBR * RS <= tile_lds_bytes<IN, BM, BN>(), "staging fits the stages");
    static_assert(kSteps % G == 0, "whole groups");
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

    const int wm = wave / 2, wn = wave % 2;
    lds_char *region = smem + wave * (16 * kBR * RS);
    const int g = lane / 16, u = lane % 16;
    lds_char *wr = region + (4 * g) * RS + u * 4;
    const int c = lane % CH, rr = lane / CH;
    const lds_char *rd = region + rr * RS + c * 32;
    const int col = w.tn * BN + wn * WC + 8 * c;
    const int ncol = p.n - col;                    // may be <= 0
    const int row_t = w.tm * BM + wm * WR + rr;    // this lane's first row of its product
    const float alpha = op_alpha(p);
    float bias[8], sums[8];
    bias_load<IN>(p, w.expert, col, bias);
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[q] = 0.0f;
    auto live = [&](int row) { return (row < w.m) & (ncol > 0); };

    static_for<FM / kBR>([&](auto pass_c) {
        constexpr int pass = decltype(pass_c)::value;
        if constexpr (pass > 0) wait_lds<0>();     // the previous pass has been read back
        static_for<kBR>([&](auto i_c) {
            constexpr int i = decltype(i_c)::value;
            static_for<FN>([&](auto j_c) {
                constexpr int j = decltype(j_c)::value;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *(lds_float *)(wr + (16 * i + r) * RS + 64 * j) = acc[pass * kBR + i][j][r];
            });
        });
        const int row_p = row_t + 16 * kBR * pass;
        ChunkIn in[G], next[G];
        auto fetch = [&](int s, ChunkIn (&to)[G]) {
#pragma unroll
            for (int q = 0; q < G; ++q) {
                const int row = row_p + (s + q) * RI;
                if (live(row)) chunk_load(p, w, (int64_t)w.row0 + row, col, ncol, to[q]);
            }
        };
        fetch(0, in);
#pragma unroll 1
        for (int s = 0; s < kSteps; s += G) {
            if (s + G < kSteps) fetch(s + G, next);
#pragma unroll
            for (int q = 0; q < G; ++q) {
                const int row = row_p + (s + q) * RI;
                const lds_char *at = rd + (s + q) * RI * RS;
                const f32x4 a = *(const lds_f32x4 *)at, b = *(const lds_f32x4 *)(at + 16);
                float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                if (live(row))
                    chunk_finish<IN>(p, alpha, w, (int64_t)w.row0 + row, col, ncol, in[q], bias, v, sums);
            }
#pragma unroll
            for (int q = 0; q < G; ++q) in[q] = next[q];
        }
    });
    if (p.colsum != nullptr && w.tile < p.tiles_m) {
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
// reductions need no LDS.  Values are in units of log 2.
template <int FM, int FN, int BM, int BN>
__device__ __forceinline__ void op_row_stats(const OpParams &p, const OpTile &w, f32x4 (&acc)[FM][FN], int wave, int lane) {
    const int wm = wave / 2, wn = wave % 2;
    const int g = lane / 16, u = lane % 16;
    const int col = w.tn * BN + wn * (BN / 2) + u;
    const int row0 = w.tm * BM + wm * (BM / 2) + 4 * g;
    const int part = 2 * w.tn + wn;
    const float scale = p.alpha * kLog2e;
    static_for<FM>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v[FN], top = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                v[j] = col + 16 * j < p.n ? acc[i][j][r] * scale : -__builtin_inff();
                top = fmaxf(top, v[j]);
            }
            top = row_max16(top);
            const float base = stat_base(top);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < FN; ++j) sum += fast_exp2(v[j] - base);
            sum = row_sum16(sum);
            const int row = row0 + 16 * i + r;
            if (u == 0 && row < w.m) p.stats[(int64_t)row * p.parts + part] = CeStat{top, sum};
        }
    });
}

template <int IN, bool TA, bool TB, int T>
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
    if constexpr (!TA && TB) {
        if (p.mode == OP_CE_STATS) {
            op_row_stats<FM, FN, T, T>(p, w, acc, wave, lane_e);
            return;
        }
    }
    __syncthreads();                   // every wave's fragment reads are done: the LDS is free
    op_store_tile<IN, FM, FN, T, T>(p, w, acc, smem, wave, lane_e);
}

template <int IN, bool TA, bool TB, int T>
int launch_op(const OpParams &p, hipStream_t stream) {
    const unsigned tiles = (unsigned)p.tiles_m * (unsigned)p.tiles_n * (p.groups_kind == GROUPS_K ? (unsigned)p.groups : 1u);
    void *args[] = {const_cast<OpParams *>(&p)};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&op_kernel<IN, TA, TB, T>), dim3(tiles, (unsigned)p.splits),
                                dim3(256), args, 0, stream);
}

}  // namespace mpg
