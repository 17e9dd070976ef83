// mpgemm_skinny_kernel.hpp -- the op kernel for few rows: D of 16 FM rows by 16 W columns per
// workgroup, with the same epilogues as the tiled kernel.
//
// With few rows a product is bound by reading B once, and a tile of 64 or more columns per
// workgroup leaves most CUs without work.  Here a workgroup of four or eight waves takes 16, 32 or
// 64 columns and its waves share k: each reads blocks of B (and the rows of A, which the L2 holds) straight
// into MFMA fragments, a block ahead of the one it multiplies, and the partial sums meet in the LDS
// at the end, in a fixed order.  No barrier stands inside the loop, so the loads of all waves keep
// flowing.
//
// Fragments of a K-contiguous operand are its 16-byte chunks.  An operand that is contiguous the
// other way is read W (or FM) neighbouring elements of a row per lane, for the lane's eight k, and
// transposed within the lane by byte permutes: lane u then holds columns W u .. W u + W - 1 as
// column u of W different MFMA blocks.
#pragma once

#include "mpgemm_ops_epilogue.hpp"

namespace mpg {

template <int IN>
__device__ __forceinline__ f32x4 mfma32(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (IN == IN_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// NB blocks of 16 rows (or columns) of one operand over one MFMA step of 32 k, in registers.
template <bool KC, int NB>
struct Strip {
    static constexpr int kLoads = KC ? NB : 8;
    static constexpr int kDwords = KC ? 4 : (NB + 1) / 2;   // per load
    uint32_t raw[kLoads][kDwords];

    // Lane's offset from the strip's first element at the block's first k.  left: rows (columns)
    // that exist from the strip's first one; those past it are read as zeros.
    static __device__ __forceinline__ uint32_t offset(int lane, uint32_t ld_bytes, int i) {
        const int u = lane % 16, g = lane / 16;
        if constexpr (KC)
            return (uint32_t)(16 * i + u) * ld_bytes + 16u * g;
        else
            return (uint32_t)(8 * g + i) * ld_bytes + (uint32_t)(2 * NB * u);
    }
    // Reads the step that starts at k index k0 of k; r addresses that index.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int lane, uint32_t ld_bytes, int left, int k0, int k) {
        const int u = lane % 16, g = lane / 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool in = KC ? (16 * i + u < left) & (k0 + 8 * g < k) : (NB * u < left) & (k0 + 8 * g + i < k);
            const int off = (int)(in ? offset(lane, ld_bytes, i) : kOobOffset);
            if constexpr (kDwords == 4) {
                const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
                raw[i][0] = x[0]; raw[i][1] = x[1]; raw[i][2] = x[2]; raw[i][3] = x[3];
            } else if constexpr (kDwords == 2) {
                const i32x2 x = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
                raw[i][0] = (uint32_t)x[0]; raw[i][1] = (uint32_t)x[1];
            } else if constexpr (NB == 2) {
                raw[i][0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
            } else {
                raw[i][0] = (uint32_t)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
            }
        }
    }
    // Fragment of block j; elements at and past k are zeroed where k ends inside the step.
    __device__ __forceinline__ u32x4 frag(int j, int lane, int k0, int k) const {
        u32x4 x;
        if constexpr (KC) {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = raw[j][q];
            const int left = k - k0 - 8 * (lane / 16);
            if (k - k0 < 32 && left > 0 && left < 8) x = keep_first_bytes(x, 2 * left);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[q] = __builtin_amdgcn_perm(raw[2 * q + 1][j / 2], raw[2 * q][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
        }
        return x;
    }
    // Row (or column) of the strip that index u of block j's MFMA operand stands for.
    static __device__ __forceinline__ int place(int j, int u) { return KC ? 16 * j + u : NB * u + j; }
};

template <int IN, bool TA, bool TB, int FM, int W, int NWV>
__global__ __launch_bounds__(64 * NWV)
void skinny_kernel(OpParams p) {
    constexpr int BM = 16 * FM, BN = 16 * W;
    constexpr int RS = BN + 4;                     // floats of a staged row
    constexpr int UN = FM * W >= 8 ? 2 : 4;        // MFMA steps per block
    __shared__ __attribute__((aligned(16))) float part[NWV][BM][RS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    OpTile w;
    if (!locate<BM>(p, blockIdx.x, blockIdx.y, lane, w)) return;
    const Params o = op_operands<TA, TB>(p, w);
    const int m_left = w.m - w.tm * BM, n_left = p.n - w.tn * BN;
    const uint32_t lda_b = (uint32_t)(2 * p.lda), ldb_b = (uint32_t)(2 * p.ldb);
    const char *a0 = (const char *)o.A + (int64_t)w.tm * BM * (TA ? 2 : 2 * p.lda);
    const char *b0 = (const char *)o.B + (int64_t)w.tn * BN * (TB ? 2 * p.ldb : 2);

    using SA = Strip<!TA, FM>;
    using SB = Strip<TB, W>;
    struct Block {
        SA a[UN];
        SB b[UN];
    } blk[2];
    auto load = [&](Block &to, int b) {
#pragma unroll
        for (int s = 0; s < UN; ++s) {
            const int64_t k0 = (int64_t)b * (32 * UN) + 32 * s;
            to.a[s].load(make_rsrc(a0 + k0 * (TA ? 2 * p.lda : 2)), lane, lda_b, m_left, (int)min(k0, (int64_t)w.k), w.k);
            to.b[s].load(make_rsrc(b0 + k0 * (TB ? 2 : 2 * p.ldb)), lane, ldb_b, n_left, (int)min(k0, (int64_t)w.k), w.k);
        }
    };
    f32x4 acc[FM][W];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Block &x, int b) {
#pragma unroll
        for (int s = 0; s < UN; ++s) {
            const int k0 = b * (32 * UN) + 32 * s;
            u32x4 fa[FM], fb[W];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = x.a[s].frag(i, lane, k0, w.k);
#pragma unroll
            for (int j = 0; j < W; ++j) fb[j] = x.b[s].frag(j, lane, k0, w.k);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) acc[i][j] = mfma32<IN>(fa[i], fb[j], acc[i][j]);
        }
    };
    // Blocks wave, wave + NWV, ... of an order that starts at another block in every column tile: one
    // is multiplied while the next is on its way.  (Where the columns' rows lie a power of two apart,
    // workgroups that all read the same k at a time would crowd the same memory channels: 8 x 32000 x
    // 4096 in 60 us from block 0, 57 so.)
    const int nb = (w.k + 32 * UN - 1) / (32 * UN);
    const int first = TB && nb > 0 ? (int)((unsigned)w.tn * 37u % (unsigned)nb) : 0;
    auto block = [&](int b) { return b + first < nb ? b + first : b + first - nb; };
    int b = wave;
    if (b < nb) load(blk[0], block(b));
    for (; b < nb; b += 2 * NWV) {
        if (b + NWV < nb) load(blk[1], block(b + NWV));
        multiply(blk[0], block(b));
        if (b + 2 * NWV < nb) load(blk[0], block(b + 2 * NWV));
        if (b + NWV < nb) multiply(blk[1], block(b + NWV));
    }

    const int g = lane / 16, u = lane % 16;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[wave][SA::place(i, 4 * g + r)][SB::place(j, u)] = acc[i][j][r];
    __syncthreads();

    // eight columns a thread; all threads of a row are neighbours in one wave
    constexpr int CH = BN / 8;
    const float alpha = op_alpha(p);
    const int c = threadIdx.x % CH, row = threadIdx.x / CH;
    const bool mine = row < BM;
    static_assert(BM * CH <= 64 * NWV, "one chunk per thread");
    const int col = w.tn * BN + 8 * c, ncol = p.n - col;
    float v[1][8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[0][q] = 0.0f;
    if (mine) {
#pragma unroll
        for (int x = 0; x < NWV; ++x) {
            const f32x4 lo = *(const f32x4 *)&part[x][row][8 * c], hi = *(const f32x4 *)&part[x][row][8 * c + 4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[0][q] += lo[q];
                v[0][q + 4] += hi[q];
            }
        }
    }
    const bool live = mine & (row < m_left) & (ncol > 0);
    if (!TA && TB && p.mode == OP_CE_STATS) {
        float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[0][q] = q < ncol ? v[0][q] * (alpha * kLog2e) : -__builtin_inff();
            top = fmaxf(top, v[0][q]);
        }
#pragma unroll
        for (int d = 1; d < CH; d *= 2) top = fmaxf(top, __shfl_xor(top, d, 64));
#pragma unroll
        for (int q = 0; q < 8; ++q) sum += fast_exp2(v[0][q] - stat_base(top));
#pragma unroll
        for (int d = 1; d < CH; d *= 2) sum += __shfl_xor(sum, d, 64);
        if (c == 0 && mine && row < m_left) p.stats[(int64_t)(w.tm * BM + row) * p.parts + w.tn] = CeStat{top, sum};
        return;
    }
    float sums[8], bias[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[q] = 0.0f;
    const int64_t tile_row = (int64_t)w.row0 + w.tm * BM, drow = tile_row + row;
    const OpOut out_d = op_out(p.D, w.d_off + tile_row * p.ldd + w.tn * BN, p.ldd, p.d_f32 ? 4 : 2);
    const OpOut out_z = op_out(p.aux, tile_row * p.ld_aux + w.tn * BN, p.ld_aux, 2);
    if (live) {
        auto finish = [&](auto mode) {
            constexpr int MODE = decltype(mode)::value;
            ChunkIn in[1];
            chunk_load<MODE>(p, w, drow, col, ncol, in[0]);
            bias_load<IN, MODE>(p, w.expert, col, bias);
            RowScale scale[1];
            if constexpr (MODE == OP_CE_PROBS) {
                const int64_t t = p.target[drow] - p.col0 - col;
                scale[0] = RowScale{p.weight[drow], p.lse[drow] * kLog2e, t >= 0 && t < 8 ? (int)t : -1};
            }
            rows_finish<IN, MODE, 1>(p, alpha, out_d, out_z, 8 * c, false, false, [&](int) { return row; },
                                     [&](int) { return ncol; }, in, scale, bias, v, sums);
        };
        if (p.mode == OP_SLOPE)
            finish(std::integral_constant<int, OP_SLOPE>{});
        else if (!TA && TB && p.mode == OP_CE_PROBS)
            finish(std::integral_constant<int, OP_CE_PROBS>{});
        else
            finish(std::integral_constant<int, OP_FORWARD>{});
    }
    if (p.colsum != nullptr) {
        // the rows of a wave by lane exchanges, the waves through the LDS (its partial sums have been read)
#pragma unroll
        for (int d = CH; d < 64; d *= 2)
#pragma unroll
            for (int q = 0; q < 8; ++q) sums[q] += __shfl_xor(sums[q], d, 64);
        constexpr int kRowWaves = (BM * CH + 63) / 64;
        float *stage = &part[0][0][0];
        __syncthreads();
        if (wave < kRowWaves && lane < CH)
#pragma unroll
            for (int q = 0; q < 8; ++q) stage[wave * BN + 8 * c + q] = sums[q];
        __syncthreads();
        const int at = w.tn * BN + (int)threadIdx.x;
        if (threadIdx.x < BN && at < p.n && w.tile < p.tiles_m) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < kRowWaves; ++r) s += stage[r * BN + threadIdx.x];
            p.colsum[(int64_t)w.tile * p.ld_colsum + at] = s;
        }
    }
}

template <int IN, bool TA, bool TB, int FM, int W, int NWV>
int launch_skinny_shape(const OpParams &p, hipStream_t stream) {
    const unsigned tiles = (unsigned)p.tiles_m * (unsigned)p.tiles_n;
    void *args[] = {const_cast<OpParams *>(&p)};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&skinny_kernel<IN, TA, TB, FM, W, NWV>),
                                dim3(tiles, (unsigned)p.splits), dim3(64 * NWV), args, 0, stream);
}

template <int IN, bool TA, bool TB, int FM, int W>
int launch_skinny(int waves, const OpParams &p, hipStream_t s) {
    return waves == 8 ? launch_skinny_shape<IN, TA, TB, FM, W, 8>(p, s) : launch_skinny_shape<IN, TA, TB, FM, W, 4>(p, s);
}

}  // namespace mpg
