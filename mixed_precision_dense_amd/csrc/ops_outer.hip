// ops_outer.hip -- D = alpha A^T B for few summed rows (A: k x m, B: k x n, both row-major, k <= 128):
// the weights' gradient of a head over few tokens.  D has up to a hundred times the operands'
// elements, so that writing it is all that counts: 4.7 TB/s for 16 x 100112 x 2048 and 2.7 - 3.6 for 128
// to 64 rows of 32000 x 4096, where tiles that pass through the LDS write 2.2 - 2.3.  Rows of D that are not
// whole 128-byte lines cost a third (24 x 100112 x 1781: 3.3 TB/s).
//
// A wave keeps 64 columns of B in registers, as fragments over all of k, and walks down D 32 rows
// at a time with the next rows of A on their way.  B takes the first operand's place in the matrix
// instruction, whose result holds four consecutive indexes of that operand in a lane; with the
// columns dealt out as Strip does (index 4 g + r of block j is column 8 g + 2 r + j), a lane holds eight
// consecutive columns of a row of D in two blocks, and the four lanes of a row 64 bytes: nothing goes
// through the LDS and nothing waits for another wave.
#include "mpgemm_skinny_kernel.hpp"

namespace mpg {
namespace {

constexpr int kStrip = 64;      // columns of D of a wave
constexpr int kRows = 32;       // rows per step (with 64, a second wave per SIMD finds no registers: 128 x 32000 x 4096 110 us, not 96)
constexpr int kOuterWaves = 4;  // neighbouring column strips share their rows of A in the caches

// A fragment with the elements of rows that do not take part zeroed (row i of the lane's eight: bit i).
__device__ __forceinline__ u32x4 keep_rows(u32x4 x, uint32_t live) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x[q] &= (live >> (2 * q) & 1 ? 0xFFFFu : 0u) | (live >> (2 * q + 1) & 1 ? 0xFFFF0000u : 0u);
    return x;
}

template <int IN, int KS>   // KS: MFMA steps of 32 summed rows
__global__ __launch_bounds__(64 * kOuterWaves)
void outer_kernel(OpParams p, int steps, int strips) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    // Workgroups go to the XCDs in turn: the strips of the same rows go to one of them, one after the
    // other, so that its cache joins the lines that two strips share where rows are not whole lines.
    const int xcd = (int)blockIdx.x % 8, turn = (int)blockIdx.x / 8;
    const int part = turn / strips * 8 + xcd;
    const int col0 = (turn % strips * kOuterWaves + wave) * kStrip;
    if (col0 >= p.n) return;
    const uint32_t lda_b = (uint32_t)(2 * p.lda), ldb_b = (uint32_t)(2 * p.ldb);
    using S = Strip<false, kRows / 16>;
    using SB = Strip<false, 2>;
    // rows that take part, a bit each
    uint64_t live[(KS + 1) / 2];
#pragma unroll
    for (int h = 0; h < (KS + 1) / 2; ++h) live[h] = __ballot(64 * h + lane < p.k && p.target[64 * h + lane] >= 0);
    u32x4 fb[KS][4];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            SB x;
            x.load(make_rsrc((const char *)p.B + 2 * ((int64_t)32 * s * p.ldb + col0 + 32 * h)), lane, ldb_b, p.n - col0 - 32 * h,
                   32 * s, p.k);
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[s][2 * h + j] = keep_rows(x.frag(j, lane, 32 * s, p.k), (uint32_t)(live[s / 2] >> (32 * (s % 2) + 8 * (lane / 16))));
        }
    const float alpha = op_alpha(p);
    const int first = part * steps;
    const int last = min(first + steps, (p.m + kRows - 1) / kRows);
    S a[2][KS];
    auto load = [&](S (&to)[KS], int b) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
            to[s].load(make_rsrc((const char *)p.A + 2 * ((int64_t)32 * s * p.lda + (int64_t)b * kRows)), lane, lda_b,
                       p.m - b * kRows, 32 * s, p.k);
    };
    const int g = lane / 16, u = lane % 16;
    const int c = 8 * g, ncol = p.n - col0 - c;   // the lane's columns, and 32 further
    auto step = [&](const S (&x)[KS], int b) {
        const OpOut out = op_out(p.D, (int64_t)b * kRows * p.ldd + col0, p.ldd, 2);
#pragma unroll
        for (int j = 0; j < kRows / 16; ++j) {
            f32x4 acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const u32x4 fa = x[s].frag(j, lane, 32 * s, p.k);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = mfma32<IN>(fb[s][i], fa, acc[i]);
            }
            const int row = S::place(j, u);
            const bool in = b * kRows + row < p.m;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = alpha * acc[2 * h + q % 2][q / 2];
                store8<IN>(out, 0, row, c + 32 * h, in ? ncol - 32 * h : 0, false, false, v);
            }
        }
    };
    if (first < last) load(a[0], first);
    for (int b = first; b < last; b += 2) {
        if (b + 1 < last) load(a[1], b + 1);
        step(a[0], b);
        if (b + 2 < last) load(a[0], b + 2);
        if (b + 1 < last) step(a[1], b + 1);
    }
}

// (instantiated explicitly: host code that only reaches a kernel through an inlined launcher does not
// reliably emit its launch stub)
template __global__ void outer_kernel<IN_F16, 1>(OpParams, int, int);
template __global__ void outer_kernel<IN_F16, 2>(OpParams, int, int);
template __global__ void outer_kernel<IN_F16, 3>(OpParams, int, int);
template __global__ void outer_kernel<IN_F16, 4>(OpParams, int, int);
template __global__ void outer_kernel<IN_BF16, 1>(OpParams, int, int);
template __global__ void outer_kernel<IN_BF16, 2>(OpParams, int, int);
template __global__ void outer_kernel<IN_BF16, 3>(OpParams, int, int);
template __global__ void outer_kernel<IN_BF16, 4>(OpParams, int, int);

template <int IN, int KS>
int launch_steps(const OpParams &p, hipStream_t stream) {
    const int strips = (p.n + kStrip * kOuterWaves - 1) / (kStrip * kOuterWaves), rows = (p.m + kRows - 1) / kRows;
    // about eight workgroups for each CU (a wave's columns of B are loaded once per workgroup)
    int parts = (8 * 256 + strips - 1) / strips;
    parts = parts < 1 ? 1 : (parts > rows ? rows : parts);
    const int steps = (rows + parts - 1) / parts;
    parts = ((rows + steps - 1) / steps + 7) / 8 * 8;   // (whole turns over the XCDs; surplus parts have no rows)
    // (its own status: an error that the caller left pending on the thread is neither reported nor cleared)
    void *args[] = {const_cast<OpParams *>(&p), const_cast<int *>(&steps), const_cast<int *>(&strips)};
    return (int)hipLaunchKernel(reinterpret_cast<const void *>(&outer_kernel<IN, KS>), dim3((unsigned)(strips * parts)),
                                dim3(64 * kOuterWaves), args, 0, stream);
}

template <int IN>
int launch_type(const OpParams &p, hipStream_t stream) {
    if (p.k <= 32) return launch_steps<IN, 1>(p, stream);
    if (p.k <= 64) return launch_steps<IN, 2>(p, stream);
    if (p.k <= 96) return launch_steps<IN, 3>(p, stream);
    return p.k <= 128 ? launch_steps<IN, 4>(p, stream) : (int)hipErrorInvalidValue;
}

}  // namespace

int launch_outer(bool bf16, const OpParams &p, void *stream) {
    return bf16 ? launch_type<IN_BF16>(p, (hipStream_t)stream) : launch_type<IN_F16>(p, (hipStream_t)stream);
}

}  // namespace mpg
