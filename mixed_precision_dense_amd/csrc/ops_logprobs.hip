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
// The largest.  Keys order values first and lower indexes second, so that no two are alike and the result
// does not depend on the order of reading.  While the logits stream by, only the maximum of every 32 elements
// of a lane is kept (in the LDS).  The top-th largest of the workgroup's lanes' maxima (256, or 64 where a wave has
// a row) is then a bound T that at least `top` elements reach; few of the kept maxima do, and only their elements are read once more
// (4095 x 128000 BF16 with 8: about 9 of 4096 maxima a row).  What reaches T is put
// in order by one wave.  Where too many do, as equal values, those above T are taken and then the first that
// equal it; where even these are too many or a NaN hides the maxima, the workgroup goes through its part again with
// lists that let in what is above their last place.  That is the way of rising rows, and of random ones with so
// many alternatives that T is near the least of the lanes' maxima: beyond about 48 below 2560 columns (4096 x 2048 BF16 23 us with
// 48, 40 with 64), elsewhere such rows get four waves.  (4095 x 128000 BF16: constant rows and
// rows masked but for ten as random ones; rising rows so with 20, but 4.1 ms with 64, where random ones take 0.22; 4096 x
// 32000 1.1 ms and 0.075; 4096 x 4096 with 20 0.12 and 0.018.)  With such lists alone,
// kept while streaming, 4095 x 128000 BF16 took 340 us with 8 alternatives and 640 with 64; so 198 and 211
// (5.3 and 5.0 TB/s), against 188 without any: the row's bytes bound it.  Of a short row most of the time
// is the chain of dependent lane exchanges (16 x 4096: 8.3 us, an empty launch 4).
#include "mpgemm_ops_epilogue.hpp"

namespace mpg {
namespace {

constexpr int kGroup = 32;                          // elements of a lane whose maximum is kept
constexpr int kGroups = kLogprobPart / (kGroup * 64 * 4);   // of a lane, in a part (a part of one wave has a fourth)
constexpr int kFound = 128;                         // elements of a wave that reach T, kept in the LDS
constexpr int kFew = 10;                            // inserted one by one; more are sorted (28 steps)
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
// The value of lane ^ D, by moves within rows of 16 lanes and swaps between them (the LDS's permutation, ten
// times as long, would be most of the time that a short row takes).
template <int CTRL>
__device__ __forceinline__ uint32_t row_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int D>
__device__ __forceinline__ uint32_t xor_lane(uint32_t v, int lane) {
    if constexpr (D == 1) return row_move<0xB1>(v);                      // within quads: 1 0 3 2
    if constexpr (D == 2) return row_move<0x4E>(v);                      // 2 3 0 1
    if constexpr (D == 4) return row_move<0x1B>(row_move<0x141>(v));     // half rows reversed (^ 7), quads reversed (^ 3)
    if constexpr (D == 8) return row_move<0x128>(v);                     // rows rotated by 8
    if constexpr (D == 16) {   // both results hold rows 0, 0, 2, 2 and 1, 1, 3, 3
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return lane & 16 ? r[0] : r[1];
    }
    if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return lane & 32 ? r[0] : r[1];
    }
    if constexpr (D == 63) return xor_lane<32>(xor_lane<16>(row_move<0x140>(v), lane), lane);   // rows reversed (^ 15)
}
template <int D>
__device__ __forceinline__ uint64_t xor_lane(uint64_t v, int lane) {
    return (uint64_t)xor_lane<D>((uint32_t)(v >> 32), lane) << 32 | xor_lane<D>((uint32_t)v, lane);
}
// One step of a bitonic network: the pair (lane, lane ^ D) keeps its larger key in the lower lane, or in the
// upper one where `up`.
template <int D, typename K>
__device__ __forceinline__ K exchange(K v, bool up, int lane) {
    const K o = xor_lane<D>(v, lane);
    const bool larger = ((lane & D) == 0) != up;
    return (v > o) == larger ? v : o;
}
template <int D, typename K>
__device__ __forceinline__ K exchange_down(K v, bool up, int lane) {
    v = exchange<D>(v, up, lane);
    if constexpr (D > 1) v = exchange_down<D / 2>(v, up, lane);
    return v;
}

// The keys of the lanes, falling from lane 0.
template <typename K>
__device__ __forceinline__ K sort_lanes(K v, int lane) {
    v = exchange_down<1>(v, (lane & 2) != 0, lane);
    v = exchange_down<2>(v, (lane & 4) != 0, lane);
    v = exchange_down<4>(v, (lane & 8) != 0, lane);
    v = exchange_down<8>(v, (lane & 16) != 0, lane);
    v = exchange_down<16>(v, (lane & 32) != 0, lane);
    return exchange_down<32>(v, false, lane);
}
// The 64 largest of two falling sequences, falling: the larger of the one and the other reversed is
// bitonic and holds them.
template <typename K>
__device__ __forceinline__ K merge_lanes(K v, K other, int lane) {
    const K o = xor_lane<63>(other, lane);
    return exchange_down<32>(v > o ? v : o, false, lane);
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
        key = merge_lanes(key, other, lane);
        last = lane_value(key, top - 1);
    }
    // One candidate a lane (0: none); all lanes call it.
    __device__ __forceinline__ void offer(uint64_t cand, int lane) {
        uint64_t in = __ballot(cand > last);
        if (__popcll(in) > kFew) {
            merge(sort_lanes(cand > last ? cand : 0, lane), lane);
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
    // The wave's in every lane: the maximum first, so that a lane rescales once.
    __device__ __forceinline__ void join_wave(float c, int lane) {
        float to = m;
        over_lanes(lane, [&](auto d) { to = fmaxf(to, other_lane<decltype(d)::value>(to, lane)); });
        rescale(to, c);
        over_lanes(lane, [&](auto d) {
            s += other_lane<decltype(d)::value>(s, lane);
            t += other_lane<decltype(d)::value>(t, lane);
        });
    }
    template <int D>
    static __device__ __forceinline__ float other_lane(float v, int lane) {
        return __builtin_bit_cast(float, xor_lane<D>(__builtin_bit_cast(uint32_t, v), lane));
    }
    template <typename F>
    static __device__ __forceinline__ void over_lanes(int lane, F &&f) {
        f(std::integral_constant<int, 1>{});
        f(std::integral_constant<int, 2>{});
        f(std::integral_constant<int, 4>{});
        f(std::integral_constant<int, 8>{});
        f(std::integral_constant<int, 16>{});
        f(std::integral_constant<int, 32>{});
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

// What the NW waves of a workgroup share.
template <int NW>
struct Share {
    Stat stat[NW];
    int count[NW];
    uint32_t sorted[NW][64];
    uint16_t ids[NW][64];
    uint64_t found[NW][kFound];   // (or a list of 64)

    __device__ __forceinline__ void join_stats(Stat &st, float c, int wave, int lane) {
        st.join_wave(c, lane);
        if (lane == 0) stat[wave] = st;
        __syncthreads();
        if (wave == 0)
            for (int i = 1; i < NW; ++i) st.join(stat[i], c);
    }
    // The list of all waves' found keys, by wave 0.  Up to 64 of them (as a rule little more than `top`) are put
    // in order by how many are above each; more are offered to the list.
    __device__ __forceinline__ void order_found(TopList &list, int lane) {
        int all = 0, from = 0, at = lane;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if (lane >= all) {
                from = i;
                at = lane - all;
            }
            all += __builtin_amdgcn_readfirstlane(count[i]);
        }
        if (all <= 64) {
            const uint64_t k = lane < all ? found[from][at] : 0;
            int above = 0;
            for (int j = 0; j < all; ++j) above += lane_value(k, j) > k ? 1 : 0;
            // (every key has been read: found is free)
            if (lane < all) found[0][above] = k;
            __builtin_amdgcn_wave_barrier();
            list.key = lane < all ? found[0][lane] : 0;
            list.last = lane_value(list.key, list.top - 1);
            return;
        }
        for (int i = 0; i < NW; ++i)
            for (int b = 0; b < count[i]; b += 64) list.offer(b + lane < count[i] ? found[i][b + lane] : 0, lane);
    }
    __device__ __forceinline__ void join_lists(TopList &list, int wave, int lane) {
        __syncthreads();
        found[wave][lane] = list.key;
        __syncthreads();
        if (wave == 0)
            for (int i = 1; i < NW; ++i) list.merge(found[i][lane], lane);
    }
};

// A part of a row: vectors first .. end - 1, of which each of NW waves takes 64 UN in turn.
template <int T, int NW>
struct Part {
    static constexpr int E = Logits<T>::E, UN = kGroup / E;
    const char *z;
    int first, end, n, lane;

    // Vector i of the lane's in a turn that starts at `base`, and its elements; what is not there is -inf.
    __device__ __forceinline__ int vector(int base, int i) const { return base + 64 * i + lane; }
    __device__ __forceinline__ u32x4 load(int v) const { return *(const u32x4 *)(z + 16 * (int64_t)min(v, end - 1)); }
    __device__ __forceinline__ void widen(u32x4 raw, int v, bool whole, float (&x)[E]) const {
        Logits<T>::widen(raw, x);
        if (!whole) {
            const int left = v < end ? n - v * E : 0;
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = e < left ? x[e] : -__builtin_inff();
        }
    }
    // (the last vector of a row may be part-filled)
    __device__ __forceinline__ bool whole(int base, int i) const { return base + 64 * (i + 1) < end; }
    __device__ __forceinline__ uint64_t key(float x, int v, int e) const {
        return v < end && v * E + e < n ? (uint64_t)order_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)(v * E + e)) : 0;
    }

    // Offers the elements of 64 vectors, or those of one order.
    __device__ __forceinline__ void offer_vectors(TopList &list, int v, uint32_t only) const {
        float x[E];
        Logits<T>::widen(load(v), x);
        uint32_t left = (1u << E) - 1;     // bit e: element e has not been offered
        while (true) {
            uint64_t best = 0;
            int at = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint64_t k = left >> e & 1 ? key(x[e], v, e) : 0;
                if (k > best && (only == 0 || (uint32_t)(k >> 32) == only)) {
                    best = k;
                    at = e;
                }
            }
            const bool in = best > list.last;
            if (!__any(in)) return;
            list.offer(best, lane);
            if (in) left &= ~(1u << at);
        }
    }
    // The wave's largest by its list alone, whatever the part holds.
    __device__ __forceinline__ void list_all(TopList &list, int wave) const {
        for (int base = first + 64 * UN * wave; base < end; base += 64 * UN * NW)
#pragma unroll 1
            for (int i = 0; i < UN && base + 64 * i < end; ++i) offer_vectors(list, vector(base, i), 0);
    }
    // Fills a list that holds all above `bound` with the first elements that equal it (there are enough: the
    // maxima that make the bound).
    __device__ __forceinline__ void list_equal(TopList &list, uint32_t bound) const {
        for (int base = first; base < end && list.last == 0; base += 64) offer_vectors(list, vector(base, 0), bound);
    }
    // The wave's elements of order `least` and more, found by the maxima of its turns; returns how many, or
    // more than kFound where there is no room for them.
    __device__ __forceinline__ int find(const float (*group_max)[64], int turns, uint32_t least, uint16_t *ids, uint64_t *found, int wave) const {
        // the lanes' turns that reach it, packed
        int groups = 0;
        for (int g = 0; g < turns; ++g) {
            const bool in = order_of(group_max[g][lane]) >= least;
            const uint64_t mask = __ballot(in);
            const int at = groups + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
            if (in && at < 64) ids[at] = (uint16_t)(g * 64 + lane);
            groups += __popcll(mask);
        }
        if (groups > 64) return kFound + 1;
        // their elements that reach it
        int count = 0;
        for (int i = lane; i - lane < groups * UN && count <= kFound; i += 64) {
            uint64_t k[E];
#pragma unroll
            for (int e = 0; e < E; ++e) k[e] = 0;
            if (i < groups * UN) {
                const int id = ids[i / UN];
                const int v = first + 64 * UN * (wave + NW * (id / 64)) + 64 * (i % UN) + id % 64;
                float x[E];
                Logits<T>::widen(load(v), x);
#pragma unroll
                for (int e = 0; e < E; ++e) k[e] = key(x[e], v, e);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = k[e] != 0 && (uint32_t)(k[e] >> 32) >= least;
                const uint64_t mask = __ballot(in);
                if (mask == 0) continue;
                const int at = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
                if (in && at < kFound) found[at] = k[e];
                count += __popcll(mask);
            }
        }
        return count;
    }
};

// A workgroup of NW waves takes a part of a row.
template <int T, int NW, bool ENT, bool TOP>
__global__ __launch_bounds__(64 * NW) void logprobs_kernel(LogprobParams p) {
    constexpr int E = Part<T, NW>::E, UN = Part<T, NW>::UN;
    __shared__ Share<NW> share;
    __shared__ float group_max[TOP ? NW : 1][TOP ? kGroups : 1][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const float c = p.alpha * kLog2e;
    const int vectors = (p.n + E - 1) / E;
    const int64_t items = (int64_t)p.m * p.parts;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / p.parts;
        const int first = (int)(item - row * p.parts) * p.part_vectors;
        const Part<T, NW> part = {(const char *)p.Z + row * p.ldz * (16 / E), first, min(vectors, first + p.part_vectors), p.n, lane};
        Stat st;
        st.init();
        int turns = 0;
        for (int base = first + 64 * UN * wave; base < part.end; base += 64 * UN * NW, ++turns) {
            u32x4 raw[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i) raw[i] = part.load(part.vector(base, i));
            float x[UN][E], most = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                part.widen(raw[i], part.vector(base, i), part.whole(base, i), x[i]);
#pragma unroll
                for (int e = 0; e < E; ++e) most = fmaxf(most, x[i][e]);
            }
            if (TOP) group_max[wave][turns][lane] = most;
            if (__any(most > st.m)) st.rescale(fmaxf(st.m, most), c);
            const float m = stat_base(st.m);
#pragma unroll
            for (int i = 0; i < UN; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = (x[i][e] - m) * c, w = fast_exp2(u);
                    st.s += w;
                    if (ENT) st.t = __builtin_fmaf(fmaxf(u, -1.0e4f), w, st.t);
                }
        }
        TopList list;
        list.init(TOP ? p.top : 1);
        if (TOP) {
            // T: the top-th of all lanes' maxima (0: fewer lanes have elements)
            const uint32_t own = part.vector(first + 64 * UN * wave, 0) < part.end ? order_of(st.m) : 0u;
            share.sorted[wave][lane] = sort_lanes(own, lane);
            const bool nan = __any(st.s != st.s);
            __syncthreads();
            uint32_t best = share.sorted[0][lane];
#pragma unroll
            for (int i = 1; i < NW; ++i) best = merge_lanes(best, share.sorted[i][lane], lane);
            const uint32_t bound = (uint32_t)__builtin_amdgcn_readlane((int)best, p.top - 1);
            // All that reach T; or, where too many do, those above it, and then the first ones that equal it (masks and
            // other equal values); or everything again (rising values: the maxima say too little; NaN).
            bool listed = false;
            for (int turn = 0; turn < 2 && !listed; ++turn) {
                const int found = nan ? kFound + 1 : part.find(group_max[wave], turns, bound + turn, share.ids[wave], share.found[wave], wave);
                if (lane == 0) share.count[wave] = found;
                __syncthreads();
                listed = true;
                for (int i = 0; i < NW; ++i) listed &= share.count[i] <= kFound;
                if (listed && wave == 0) {
                    share.order_found(list, lane);
                    if (turn == 1 && list.last == 0) part.list_equal(list, bound);
                }
                __syncthreads();   // share is written again
            }
            if (!listed) {
                part.list_all(list, wave);
                share.join_lists(list, wave, lane);
            }
        }
        share.join_stats(st, c, wave, lane);
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

// A workgroup joins the parts of a row.  A wave takes 64 parts at a time and their lists rank by rank: once
// no part's key of a rank enters, none of a later one does.
constexpr int kWaves = 4;
template <int T>
__global__ __launch_bounds__(64 * kWaves) void logprobs_join_kernel(LogprobParams p) {
    __shared__ Share<kWaves> share;
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
        for (int i = 64 * wave; p.top > 0 && i < p.parts; i += 64 * kWaves) {
            const bool in = i + lane < p.parts;
            const uint64_t *keys = p.keys + (row * p.parts + min(i + lane, p.parts - 1)) * p.top;
            uint64_t next = keys[0];
            for (int j = 0; j < p.top; ++j) {
                const uint64_t k = in ? next : 0;
                next = keys[min(j + 1, p.top - 1)];
                if (!__any(k > list.last)) break;
                list.offer(k, lane);
            }
        }
        if (p.parts > 64) share.join_lists(list, wave, lane);   // (else the first wave has them all)
        share.join_stats(st, c, wave, lane);
        if (wave == 0) finish_row<T>(p, row, st, list, lane);
        __syncthreads();   // share is written again
    }
}

// (instantiated explicitly: host code that only reaches a kernel through an inlined launcher does not
// reliably emit its launch stub)
template __global__ void logprobs_kernel<LOGITS_F16, 1, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 1, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 1, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 1, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 4, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 4, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 4, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F16, 4, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 1, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 1, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 1, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 1, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 4, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 4, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 4, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_BF16, 4, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 1, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 1, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 1, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 1, true, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 4, false, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 4, false, true>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 4, true, false>(LogprobParams);
template __global__ void logprobs_kernel<LOGITS_F32, 4, true, true>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_F16>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_BF16>(LogprobParams);
template __global__ void logprobs_join_kernel<LOGITS_F32>(LogprobParams);

int launch(const void *kernel, int64_t blocks, int waves, const LogprobParams &p, hipStream_t stream) {
    void *args[] = {const_cast<LogprobParams *>(&p)};
    return (int)hipLaunchKernel(kernel, dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3((unsigned)(64 * waves)), args, 0,
                                stream);
}

template <int T, int NW>
const void *kernel_of(const LogprobParams &p) {
    if (p.entropy != nullptr)
        return p.top > 0 ? reinterpret_cast<const void *>(&logprobs_kernel<T, NW, true, true>)
                         : reinterpret_cast<const void *>(&logprobs_kernel<T, NW, true, false>);
    return p.top > 0 ? reinterpret_cast<const void *>(&logprobs_kernel<T, NW, false, true>)
                     : reinterpret_cast<const void *>(&logprobs_kernel<T, NW, false, false>);
}

template <int T>
int launch_type(int waves, const LogprobParams &p, hipStream_t stream) {
    const int e = launch(waves == 1 ? kernel_of<T, 1>(p) : kernel_of<T, 4>(p), (int64_t)p.m * p.parts, waves, p, stream);
    if (e != 0 || p.parts == 1) return e;
    return launch(reinterpret_cast<const void *>(&logprobs_join_kernel<T>), p.m, kWaves, p, stream);
}

}  // namespace

int launch_logprobs(int type, int waves, const LogprobParams &p, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    if (type == LOGITS_F16) return launch_type<LOGITS_F16>(waves, p, s);
    return type == LOGITS_BF16 ? launch_type<LOGITS_BF16>(waves, p, s) : launch_type<LOGITS_F32>(waves, p, s);
}

}  // namespace mpg
