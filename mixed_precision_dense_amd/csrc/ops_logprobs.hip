// ops_logprobs.hip -- log probabilities of given tokens, entropy and the largest alternatives of rows of
// stored logits, in one pass over them.
//
// With z = alpha x, m = max x, u = (x - m) alpha / log 2 over a row: s = sum of 2^u, t = sum of u 2^u, and
//   lse = alpha m + log s,   log p_v = alpha (x_v - m) - log s,   entropy = log s - log 2 t / s.
// Every lane keeps (m, s, t) of what it has read and rescales s and t where its maximum grows; lanes,
// waves and parts of a row are joined by the same rule in a fixed order.  Differences of the logits are
// taken before the scaling, so that rows of a type's lowest value alone (a mask that leaves nothing) come out
// as the equal values that they are.
//
// The largest: a wave holds a sorted list of 64, one a lane, of keys that order values first and lower
// indexes second (no two are alike, so that the result does not depend on the order of reading), and lets
// in only what is above the list's last needed one.  Of a random row of n that is about top (1 + log(n /
// 512)) elements a wave; a vector without any costs a comparison.  A few are inserted one by one; more than
// kFew are sorted across the lanes and merged, so that rows in rising order stay within a constant
// factor too.
#include "mpgemm_ops_epilogue.hpp"

namespace mpg {
namespace {

constexpr int kWaves = 4;
constexpr int kFew = 6;
constexpr int64_t kMostBlocks = 65536;
constexpr float kLn2 = 0.69314718055994531f;

// ------------------------------------------------------------------------------- the largest
// Order of a float as an unsigned number: above 0; both zeros alike; NaN below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return x != x ? 1u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 1u ? __builtin_nanf("") : __builtin_bit_cast(float, o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t xor_lane(uint64_t v, int d) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, d, 64), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), d, 64);
    return (uint64_t)hi << 32 | lo;
}
// One step of a bitonic network: the pair (lane, lane ^ d) keeps its larger key in the lower lane, or in the
// upper one where `up`.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int d, bool up, int lane) {
    const uint64_t o = xor_lane(v, d);
    const bool larger = ((lane & d) == 0) != up;
    return (v > o) == larger ? v : o;
}

struct TopList {
    uint64_t key;     // lane i: the i-th largest, 0 where there is none
    uint64_t last;    // the one at place top - 1 (uniform)
    int top;

    __device__ __forceinline__ void init(int n) {
        key = last = 0;
        top = n;
    }
    // A sorted list of another wave or part (64 keys, falling).
    __device__ __forceinline__ void merge(uint64_t other, int lane) {
        const uint64_t o = xor_lane(other, 63);        // the larger of the list and the other one reversed
        key = key > o ? key : o;                       // is bitonic and holds the 64 largest
#pragma unroll
        for (int d = 32; d > 0; d /= 2) key = exchange(key, d, false, lane);
        last = lane_value(key, top - 1);
    }
    // One candidate a lane (0: none); all lanes call it.
    __device__ __forceinline__ void offer(uint64_t cand, int lane) {
        uint64_t in = __ballot(cand > last);
        if (__popcll(in) > kFew) {
            uint64_t v = cand > last ? cand : 0;
#pragma unroll
            for (int size = 2; size <= 64; size *= 2)
#pragma unroll
                for (int d = size / 2; d > 0; d /= 2) v = exchange(v, d, (lane & size) != 0 && size < 64, lane);
            merge(v, lane);
            return;
        }
        while (in != 0) {
            const int from = __builtin_ctzll(in);
            in &= in - 1;
            const uint64_t k = lane_value(cand, from);
            const int place = __popcll(__ballot(key > k));   // (a prefix of the lanes)
            const uint32_t lo = (uint32_t)__shfl_up((int)(uint32_t)key, 1, 64), hi = (uint32_t)__shfl_up((int)(uint32_t)(key >> 32), 1, 64);
            key = lane < place ? key : (lane == place ? k : (uint64_t)hi << 32 | lo);
            last = lane_value(key, top - 1);
        }
    }
};

// ------------------------------------------------------------------------------- statistics
struct Stat {
    float m, s, t;
    __device__ __forceinline__ void init() {
        m = -__builtin_inff();
        s = t = 0.0f;
    }
    // Takes s and t to a maximum `to`, at least m; c = alpha / log 2.
    __device__ __forceinline__ void rescale(float to, float c) {
        const float d = (m - stat_base(to)) * c, f = fast_exp2(d);
        // (nothing has been summed below a maximum of -inf, and 0 * inf must not be formed)
        t = f * __builtin_fmaf(fmaxf(d, -1.0e4f), s, t);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(Stat o, float c) {
        const float to = fmaxf(m, o.m);
        rescale(to, c);
        o.rescale(to, c);
        s += o.s;
        t += o.t;
    }
    __device__ __forceinline__ void join_wave(float c) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const Stat o = {__shfl_xor(m, d, 64), __shfl_xor(s, d, 64), __shfl_xor(t, d, 64)};
            // (the lower lane's first, so that both halves of a pair come to the same bits)
            Stat a = threadIdx.x & d ? o : *this, b = threadIdx.x & d ? *this : o;
            a.join(b, c);
            *this = a;
        }
    }
};

template <int T>
struct Logits {
    static constexpr int E = T == LOGITS_F32 ? 4 : 8;   // of a 16-byte vector
    static __device__ __forceinline__ void widen(u32x4 raw, float (&x)[E]) {
        if constexpr (T == LOGITS_F32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = __builtin_bit_cast(float, (uint32_t)raw[q]);
        } else {
            widen8<T == LOGITS_F16 ? IN_F16 : IN_BF16>(raw, x);
        }
    }
    static __device__ __forceinline__ float at(const void *z, int64_t i) {
        if constexpr (T == LOGITS_F32)
            return ((const float *)z)[i];
        else
            return mpg::widen<T == LOGITS_F16 ? IN_F16 : IN_BF16>(((const uint16_t *)z)[i]);
    }
};

// What a row comes to, by one wave.
template <int T>
__device__ __forceinline__ void finish_row(const LogprobParams &p, int64_t row, Stat st, const TopList &list, int lane) {
    const bool none = st.m == -__builtin_inff() && st.s == 0.0f;   // nothing but -inf: no distribution
    const float log_s = none ? 0.0f : kLn2 * __log2f(st.s);
    auto log_p = [&](float x) { return none ? -__builtin_inff() : __builtin_fmaf(x - st.m, p.alpha, -log_s); };
    if (lane == 0) {
        if (p.lse != nullptr) p.lse[row] = none ? st.m : __builtin_fmaf(p.alpha, st.m, log_s);
        if (p.entropy != nullptr) p.entropy[row] = none ? 0.0f : log_s - kLn2 * st.t / st.s;
        if (p.logprob != nullptr) {
            const int64_t v = p.target[row];
            const int bytes = T == LOGITS_F32 ? 4 : 2;
            p.logprob[row] = v >= 0 && v < p.n ? log_p(Logits<T>::at((const char *)p.Z + row * p.ldz * bytes, v)) : 0.0f;
        }
    }
    if (lane < p.top) {
        const bool some = list.key != 0;
        p.top_index[row * p.ld_top + lane] = some ? (int64_t)(0xFFFFFFFFu - (uint32_t)list.key) : -1;
        p.top_logprob[row * p.ld_top + lane] = some ? log_p(value_of((uint32_t)(list.key >> 32))) : -__builtin_inff();
    }
}

// The waves' statistics and lists to wave 0's, through the LDS.
struct Share {
    Stat stat[kWaves];
    uint64_t key[kWaves][64];
};
template <bool TOP>
__device__ __forceinline__ void join_waves(Share &share, Stat &st, TopList &list, float c, int wave, int lane) {
    st.join_wave(c);
    if (lane == 0) share.stat[wave] = st;
    if (TOP) share.key[wave][lane] = list.key;
    __syncthreads();
    if (wave == 0) {
        for (int i = 1; i < kWaves; ++i) {
            st.join(share.stat[i], c);
            if (TOP) list.merge(share.key[i][lane], lane);
        }
    }
}

// A workgroup takes a part of a row: its waves take 64 vectors of 16 bytes in turn, UN at a time.
template <int T, bool ENT, bool TOP>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobParams p) {
    constexpr int E = Logits<T>::E, UN = 4;
    __shared__ Share share;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const float c = p.alpha * kLog2e;
    const int vectors = (p.n + E - 1) / E;
    const int64_t items = (int64_t)p.m * p.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / p.parts;
        const int part = (int)(item - row * p.parts);
        const char *z = (const char *)p.Z + row * p.ldz * (16 / E);
        const int first = part * p.part_vectors, end = min(vectors, first + p.part_vectors);
        Stat st;
        st.init();
        TopList list;
        list.init(TOP ? p.top : 1);
        for (int base = first + 64 * UN * wave; base < end; base += 64 * UN * kWaves) {
            u32x4 raw[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int v = base + 64 * i + lane;
                raw[i] = *(const u32x4 *)(z + 16 * (int64_t)min(v, end - 1));
            }
            float x[UN][E], most[UN], up = st.m;
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int v = base + 64 * i + lane;
                Logits<T>::widen(raw[i], x[i]);
                if (base + 64 * (i + 1) >= end || base + 64 * (i + 1) >= vectors) {   // (uniform) what is not there
                    const int left = v < end ? p.n - v * E : 0;
#pragma unroll
                    for (int e = 0; e < E; ++e) x[i][e] = e < left ? x[i][e] : -__builtin_inff();
                }
                most[i] = x[i][0];
#pragma unroll
                for (int e = 1; e < E; ++e) most[i] = fmaxf(most[i], x[i][e]);
                up = fmaxf(up, most[i]);
            }
            if (__any(up > st.m)) st.rescale(up, c);
            const float m = stat_base(st.m);
#pragma unroll
            for (int i = 0; i < UN; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = (x[i][e] - m) * c, w = fast_exp2(u);
                    st.s += w;
                    if (ENT) st.t = __builtin_fmaf(fmaxf(u, -1.0e4f), w, st.t);
                }
            if (TOP) {
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    const int v = base + 64 * i + lane;
                    // (equal to the last one at a higher index is not above it)
                    if (base + 64 * i >= end || !__any(order_of(most[i]) > (uint32_t)(list.last >> 32))) continue;
                    uint32_t key[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) key[e] = v < end && v * E + e < p.n ? order_of(x[i][e]) : 0u;
                    while (true) {
                        uint32_t best = 0;
                        int at = 0;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (key[e] > best) {
                                best = key[e];
                                at = e;
                            }
                        const uint64_t cand = best == 0 ? 0 : (uint64_t)best << 32 | (0xFFFFFFFFu - (uint32_t)(v * E + at));
                        const bool in = cand > list.last;
                        if (!__any(in)) break;
                        list.offer(cand, lane);
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (in && e == at) key[e] = 0;
                    }
                }
            }
        }
        join_waves<TOP>(share, st, list, c, wave, lane);
        if (wave == 0) {
            if (p.parts == 1) {
                finish_row<T>(p, row, st, list, lane);
            } else {
                if (lane == 0) {
                    float *to = p.stats + item * 4;
                    to[0] = st.m;
                    to[1] = st.s;
                    to[2] = st.t;
                }
                if (TOP && lane < p.top) p.keys[item * p.top + lane] = list.key;
            }
        }
        __syncthreads();   // share is written again
    }
}

// A workgroup joins the parts of a row.
template <int T>
__global__ __launch_bounds__(64 * kWaves) void logprobs_join_kernel(LogprobParams p) {
    __shared__ Share share;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const float c = p.alpha * kLog2e;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        Stat st;
        st.init();
        for (int i = threadIdx.x; i < p.parts; i += 64 * kWaves) {
            const float *from = p.stats + (row * p.parts + i) * 4;
            st.join(Stat{from[0], from[1], from[2]}, c);
        }
        TopList list;
        list.init(p.top > 0 ? p.top : 1);
        const int keys = p.parts * p.top;
        for (int i = 64 * wave; i < keys; i += 64 * kWaves)
            list.offer(i + lane < keys ? p.keys[row * keys + i + lane] : 0, lane);
        join_waves<true>(share, st, list, c, wave, lane);
        if (wave == 0) finish_row<T>(p, row, st, list, lane);
        __syncthreads();   // share is written again
    }
}

// (instantiated explicitly: host code that only reaches a kernel through an inlined launcher does not
// reliably emit its launch stub)
template __global__ void logprobs_kernel<LOGITS_F16, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, true, true>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_F16>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_BF16>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_F32>(LogprobParams);

int launch(const void *kernel, int64_t blocks, const LogprobParams &p, hipStream_t stream) {
    void *args[] = {const_cast<LogprobParams *>(&p)};
    return (int)hipLaunchKernel(kernel, dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(64 * kWaves), args, 0, stream);
}

template <int T>
int launch_type(const LogprobParams &p, hipStream_t stream) {
    const bool ent = p.entropy != nullptr, top = p.top > 0;
    const void *first = ent ? (top ? reinterpret_cast<const void *>(&logprobs_kernel<T, true, true>)
                                   : reinterpret_cast<const void *>(&logprobs_kernel<T, true, false>))
                            : (top ? reinterpret_cast<const void *>(&logprobs_kernel<T, false, true>)
                                   : reinterpret_cast<const void *>(&logprobs_kernel<T, false, false>));
    const int e = launch(first, (int64_t)p.m * p.parts, p, stream);
    if (e != 0 || p.parts == 1) return e;
    return launch(reinterpret_cast<const void *>(&logprobs_join_kernel<T>), p.m, p, stream);
}

}  // namespace

int launch_logprobs(int type, const LogprobParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (type == LOGITS_F16) return launch_type<LOGITS_F16>(p, s);
    return type == LOGITS_BF16 ? launch_type<LOGITS_BF16>(p, s) : launch_type<LOGITS_F32>(p, s);
}

}  // namespace mpg
