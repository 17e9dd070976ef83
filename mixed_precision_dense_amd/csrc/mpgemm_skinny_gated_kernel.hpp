// mpgemm_skinny_gated_kernel.hpp -- the gated product for few rows: 16 FM rows by 16 W outputs per
// workgroup, D = act(alpha A op(Bg) + bg) * (alpha A op(Bu) + bu).
//
// Both weights are read once and everything else is small, so that the bytes of the weights bound it.
// As in the op kernel for few rows the waves of a workgroup share k and read both operands straight into
// MFMA fragments, a block ahead of the one that is multiplied; here a block holds the same columns of
// both weights, so that a fragment of A serves two products and the two factors of an output meet in
// the LDS when the waves' partial sums do.  One row of 8192 outputs over 4096: 134 MB in 27 us, 5.0 TB/s; 64 rows of 32
// experts, 1408 outputs over 2048: 298 MB in 57-60 us, 5.0 TB/s.  (A copy of 4 GiB moves 4.8 on the same device.)
#pragma once

#include "mpgemm_skinny_kernel.hpp"

namespace mpg {

template <int IN, bool TB, int FM, int W, int NWV>
__global__ __launch_bounds__(64 * NWV)
void gated_skinny_kernel(OpParams p) {
    constexpr int BM = 16 * FM, BN = 16 * W;
    constexpr int RS = 2 * BN + 4;                 // floats of a staged row: the gate's, the up projection's
    constexpr int UN = FM * W >= 4 ? 2 : 4;        // MFMA steps per block
    __shared__ __attribute__((aligned(16))) float part[NWV][BM][RS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    OpTile w;
    if (!locate<BM>(p, blockIdx.x, 0, lane, w)) return;
    const Params o = op_operands<false, TB>(p, w);
    const int m_left = w.m - w.tm * BM, n_left = p.n - w.tn * BN;
    const uint32_t lda_b = (uint32_t)(2 * p.lda), ldb_b = (uint32_t)(2 * p.ldb);
    const char *a0 = (const char *)o.A + (int64_t)w.tm * BM * 2 * p.lda;
    const char *g0 = (const char *)o.B + (int64_t)w.tn * BN * (TB ? 2 * p.ldb : 2);
    const char *u0 = g0 + 2 * p.stride_up;

    using SA = Strip<true, FM>;
    using SB = Strip<TB, W>;
    struct Block {
        SA a[UN];
        SB g[UN], u[UN];
    } blk[2];
    auto load = [&](Block &to, int b) {
#pragma unroll
        for (int s = 0; s < UN; ++s) {
            const int64_t k0 = (int64_t)b * (32 * UN) + 32 * s, bk = k0 * (TB ? 2 : 2 * p.ldb);
            const int at = (int)min(k0, (int64_t)w.k);
            to.a[s].load(make_rsrc(a0 + k0 * 2), lane, lda_b, m_left, at, w.k);
            to.g[s].load(make_rsrc(g0 + bk), lane, ldb_b, n_left, at, w.k);
            to.u[s].load(make_rsrc(u0 + bk), lane, ldb_b, n_left, at, w.k);
        }
    };
    f32x4 gate[FM][W], up[FM][W];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) gate[i][j] = up[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Block &x, int b) {
#pragma unroll
        for (int s = 0; s < UN; ++s) {
            const int k0 = b * (32 * UN) + 32 * s;
            u32x4 fa[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = x.a[s].frag(i, lane, k0, w.k);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const u32x4 fg = x.g[s].frag(j, lane, k0, w.k), fu = x.u[s].frag(j, lane, k0, w.k);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    gate[i][j] = mfma32<IN>(fa[i], fg, gate[i][j]);
                    up[i][j] = mfma32<IN>(fa[i], fu, up[i][j]);
                }
            }
        }
    };
    // (the order of blocks starts at another one in every column tile, as in the op kernel for few rows)
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
            for (int r = 0; r < 4; ++r) {
                float *to = &part[wave][SA::place(i, 4 * g + r)][SB::place(j, u)];
                to[0] = gate[i][j][r];
                to[BN] = up[i][j][r];
            }
    __syncthreads();

    // eight outputs a thread
    constexpr int CH = BN / 8;
    static_assert(BM * CH <= 64 * NWV, "one chunk per thread");
    const int c = threadIdx.x % CH, row = threadIdx.x / CH;
    const int col = w.tn * BN + 8 * c, ncol = p.n - col;
    if (row >= BM || row >= m_left || ncol <= 0) return;
    float v[1][8], x[1][8], bias[8], bias_up[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[0][q] = x[0][q] = 0.0f;
#pragma unroll
    for (int i = 0; i < NWV; ++i) {
        const float *at = &part[i][row][8 * c];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 a = *(const f32x4 *)(at + 4 * h), d = *(const f32x4 *)(at + BN + 4 * h);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[0][4 * h + q] += a[q];
                x[0][4 * h + q] += d[q];
            }
        }
    }
    bias_of<IN>(p, p.bias, w.expert, col, bias);
    bias_of<IN>(p, p.bias_up, w.expert, col, bias_up);
    const int64_t tile_row = (int64_t)w.row0 + w.tm * BM;
    const GatedOut out = {op_out(p.D, tile_row * p.ldd + w.tn * BN, p.ldd, p.d_f32 ? 4 : 2),
                          op_out(p.aux, tile_row * p.ld_aux + w.tn * BN, p.ld_aux, 2),
                          op_out(p.aux, p.stride_aux + tile_row * p.ld_aux + w.tn * BN, p.ld_aux, 2)};
    gated_finish<IN, 1>(p, out, 8 * c, false, false, [&](int) { return row; }, [&](int) { return ncol; }, bias, bias_up, v, x);
}

template <int IN, bool TB, int FM, int W, int NWV>
int launch_gated_skinny_shape(const OpParams &p, hipStream_t stream) {
    void *args[] = {const_cast<OpParams *>(&p)};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&gated_skinny_kernel<IN, TB, FM, W, NWV>),
                                dim3((unsigned)p.tiles_m * (unsigned)p.tiles_n), dim3(64 * NWV), args, 0, stream);
}

}  // namespace mpg
