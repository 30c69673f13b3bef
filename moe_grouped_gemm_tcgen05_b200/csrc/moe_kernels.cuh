// Kernels around the experts' products: routing (with its gradient), the rows
// of each expert, the tokens' copies in those rows cast to E4M3, and the sum of
// the experts' rows back into tokens (with its gradients).
//
// All of them move bytes: a few operations per value read. Every sum has one
// fixed order, so repeated calls give identical bits; no kernel uses atomics
// whose order could change a result.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace dg {

constexpr int MOE_MAX_EXPERTS = 1024;
constexpr int MOE_MAX_TOPK = 32;       // one lane of a warp per chosen expert
constexpr int MOE_MAX_EXPERT_GROUPS = 32;
constexpr float ROUTE_EPS = 1e-20f;    // added to the sum that weights are divided by

// ---------------------------------------------------------------- routing ----
//
// Per token: s = sigmoid(x) or softmax(x); key = s + bias; the groups of
// experts are ranked by the sum of their group_top best keys and the
// top_groups best stay; ids are the k largest keys left, ties to the lowest
// index; weights are scale * s[ids], divided by their sum when renormalised.
//
// One warp per token, expert e = lane * V + i in register i of its lane, so a
// group is a run of lanes whenever its size is V times a power of two.
//
// What bounds it: the chain that a token's instructions form, and their number. A
// token of 256 experts is 1 KB of fp32 logits, and its choice ~900 warp instructions
// with the following representation (1824 with keys and indices apart). 16384 such
// tokens take 30 us (45 with the indices apart; the memory alone needs 2.7): 60% of
// the issue slots are used, and the warps wait for the round before (a reduction, a
// ballot and a shift each). 64 tokens take 4.3 us, nearly all of it latency;
// bf16 logits under softmax take 18.5 us. A key is an unsigned integer that orders like the fp32 value, with
// the complement of the register's index in its lowest bits; a lane's keys are
// sorted once, a round takes the largest first key of all lanes (one reduction),
// and its lane moves up.
//
// Two keys can lie closer than that resolves, or than fp32 does (16384 tokens of
// 256 experts hold a few such pairs), and the choice must not depend on the
// rounding of a fast exponential. So a token where two neighbours of the sorted
// choice, or the last group that stays and the first that does not, lie within a
// tolerance (keys: twice the error of the fp32 score, below 1e-6 of the row's
// best score, and the bits that the index took) is ranked again in fp64. Without a bias the
// logits themselves rank like the scores; bf16 logits leave 16 bits free, which
// hold the whole index, so that no two keys are equal.

struct RouteParams {
    const void* logits;   // [T, E]
    const float* bias;    // [E] or null
    int32_t* ids;         // [T, k]
    float* weights;       // [T, k]
    int tokens, experts, k;
    int groups, top_groups, group_top;
    int softmax, renorm;
    float scale;
};

template <bool F32>
__device__ __forceinline__ float load_logit(const void* x, size_t i) {
    if constexpr (F32) return __ldg(static_cast<const float*>(x) + i);
    else return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(x) + i)) << 16);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Keys rank as themselves with NaN below every number and -0 equal to +0.
template <typename Key>
__device__ __forceinline__ Key rank_key(Key v) {
    return v != v ? static_cast<Key>(-INFINITY) : v + static_cast<Key>(0);
}

// fp32 keys as unsigned integers of the same order (never 0, which marks "none left").
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float from_ordered_bits(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}

// Bits of a key that hold its register's index.
template <int V>
__host__ __device__ constexpr int route_index_bits() {
    int b = 0;
    while ((1 << b) < V) ++b;
    return b;
}
// The value of a key whose lowest bits hold an index, which counts as nothing. Without
// them the key of -inf (0x007fffff), and 0 ("none left"), would read as a NaN.
template <int V>
__device__ __forceinline__ float key_value(uint32_t key) {
    constexpr uint32_t kIndexMask = (1u << route_index_bits<V>()) - 1u;
    const uint32_t u = key & ~kIndexMask;
    return u <= 0x007fffffu ? -INFINITY : from_ordered_bits(u);
}

// Relative difference (to the row's best score, for keys below it) under which two fp32 keys may be in the wrong order.
template <int V>
__device__ constexpr float route_tolerance() { return 4e-6f + 2.4e-7f * (1 << route_index_bits<V>()); }

// A sorting network (Knuth, The Art of Computer Programming 3, algorithm 5.2.2M:
// merge exchange) for n keys as a list of compare-exchange pairs.
struct SortNetwork {
    int a[192], b[192], n;
};
__host__ __device__ constexpr SortNetwork sort_network(int n) {
    SortNetwork net{};
    int t = 0;
    while ((1 << t) < n) ++t;
    for (int p = t > 0 ? 1 << (t - 1) : 0; p > 0; p /= 2) {
        int q = 1 << (t - 1), r = 0, d = p;
        while (true) {
            for (int i = 0; i + d < n; ++i)
                if ((i & p) == r) {
                    net.a[net.n] = i;
                    net.b[net.n] = i + d;
                    ++net.n;
                }
            if (q == p) break;
            d = q - p;
            q /= 2;
            r = p;
        }
    }
    return net;
}

// The lane's keys in falling order.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V]) {
    constexpr SortNetwork net = sort_network(V);
#pragma unroll
    for (int i = 0; i < net.n; ++i) {
        const uint32_t hi = max(key[net.a[i]], key[net.b[i]]), lo = min(key[net.a[i]], key[net.b[i]]);
        key[net.a[i]] = hi;
        key[net.b[i]] = lo;
    }
}

// The groups that stay, as a bit mask over groups: those of the top_groups best
// scores (lane g holds the score of group g).
template <typename Key>
__device__ __forceinline__ uint32_t route_rank_groups(const RouteParams& p, Key score, int lane) {
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
        const Key other = __shfl_sync(0xffffffffu, score, h);
        rank += (other > score || (other == score && h < lane)) ? 1 : 0;
    }
    return __ballot_sync(0xffffffffu, lane < p.groups && rank < p.top_groups);
}

// A group's score from its best two keys (half their sum: it cannot overflow), and the
// larger of their sizes (the sum of keys of both signs can be far smaller than its error).
template <typename Key>
struct GroupScore {
    Key score, size;
    __device__ __forceinline__ GroupScore(const RouteParams& p, Key b1, Key b2)
        : score(rank_key(p.group_top == 2 ? b1 / 2 + b2 / 2 : b1)), size(p.group_top == 2 ? fmax(fabs(b1), fabs(b2)) : fabs(b1)) {}
    __device__ __forceinline__ GroupScore from_lane(int l) const {
        GroupScore g = *this;
        g.score = __shfl_sync(0xffffffffu, score, l);
        g.size = __shfl_sync(0xffffffffu, size, l);
        return g;
    }
};

// Score of group `lane` (in lanes below p.groups) from keys in registers in any order.
template <int V, typename Key>
__device__ __forceinline__ GroupScore<Key> route_group_score(const RouteParams& p, const Key (&key)[V], int lane) {
    const int size = p.experts / p.groups;
    const int run = size / V;
    if (size % V == 0 && (run & (run - 1)) == 0) {
        // a group is a run of lanes
        Key b1 = key[0], b2 = static_cast<Key>(-INFINITY);
#pragma unroll
        for (int i = 1; i < V; ++i) {
            b2 = fmax(b2, fmin(b1, key[i]));
            b1 = fmax(b1, key[i]);
        }
        for (int o = 1; o < run; o <<= 1) {
            const Key c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = fmax(fmin(b1, c1), fmax(b2, c2));
            b1 = fmax(b1, c1);
        }
        return GroupScore<Key>(p, b1, b2).from_lane((lane * run) & 31);
    }
    GroupScore<Key> mine(p, static_cast<Key>(-INFINITY), static_cast<Key>(-INFINITY));
    for (int g = 0; g < p.groups; ++g) {
        Key b1 = static_cast<Key>(-INFINITY), b2 = b1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            if (e >= g * size && e < (g + 1) * size) {
                b2 = fmax(b2, fmin(b1, key[i]));
                b1 = fmax(b1, key[i]);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Key c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = fmax(fmin(b1, c1), fmax(b2, c2));
            b1 = fmax(b1, c1);
        }
        if (lane == g) mine = GroupScore<Key>(p, b1, b2);
    }
    return mine;
}

// Experts of this lane that may be chosen, as a bit mask over its registers.
template <int V>
__device__ __forceinline__ uint32_t route_alive(const RouteParams& p, uint32_t kept, int lane) {
    const int size = p.experts / p.groups;
    uint32_t alive = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e < p.experts && (p.top_groups == p.groups || (kept >> (e / size)) & 1u)) alive |= 1u << i;
    }
    return alive;
}

// Unrolling of the fp64 loops: whole while the arrays stay in registers.
template <int V>
__host__ __device__ constexpr int route_unroll64() { return V <= 8 ? V : 1; }

// Maximum and 1 / sum of a softmax row in fp64 (0 where every logit is -inf).
template <int V, bool F32>
__device__ __forceinline__ void route_softmax64(const RouteParams& p, size_t row, int lane, double& top, double& inv) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < p.experts) m = fmaxf(m, load_logit<F32>(p.logits, row + lane * V + i));
    m = warp_max(m);
    top = m == -INFINITY ? 0.0 : static_cast<double>(m);
    double sum = 0.0;
#pragma unroll route_unroll64<V>()
    for (int i = 0; i < V; ++i)
        if (lane * V + i < p.experts) sum += exp(static_cast<double>(load_logit<F32>(p.logits, row + lane * V + i)) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
}

__device__ __forceinline__ double route_score64(const RouteParams& p, float x, double top, double inv) {
    const double v = static_cast<double>(x);
    return p.softmax ? exp(v - top) * inv : 1.0 / (1.0 + exp(-v));
}

// Candidate `expert` of every lane below n, ranked by fp64 keys: lane j < n
// returns the j-th. Candidates are in falling order of their fp32 keys, and all
// experts that these leave undecided are among them.
template <int V, bool F32>
__device__ __noinline__ int route_order64(const RouteParams& p, size_t row, int lane, int expert, int n) {
    double top = 0.0, inv = 0.0;
    if (p.bias != nullptr && p.softmax) route_softmax64<V, F32>(p, row, lane, top, inv);
    double key = -INFINITY;
    if (lane < n) {
        const float x = load_logit<F32>(p.logits, row + expert);
        // without a bias the experts are ranked by their logits
        key = rank_key(p.bias == nullptr ? static_cast<double>(x)
                                         : route_score64(p, x, top, inv) + static_cast<double>(__ldg(p.bias + expert)));
    }
    int rank = 0;
    for (int l = 0; l < n; ++l) {
        const double k = __shfl_sync(0xffffffffu, key, l);
        const int e = __shfl_sync(0xffffffffu, expert, l);
        rank += (k > key || (k == key && e < expert)) ? 1 : 0;
    }
    int mine = 0;
    for (int l = 0; l < n; ++l) {
        const int r = __shfl_sync(0xffffffffu, rank, l), e = __shfl_sync(0xffffffffu, expert, l);
        if (r == lane) mine = e;
    }
    return mine;
}

// The whole choice again with fp64 keys (groups too close, or more candidates
// than lanes): lane j < k returns its expert.
template <int V, bool F32>
__device__ __noinline__ int route_choose64(const RouteParams& p, size_t row, int lane) {
    double top = 0.0, inv = 0.0;
    if (p.softmax) route_softmax64<V, F32>(p, row, lane, top, inv);
    double s[V], key[V];
#pragma unroll route_unroll64<V>()
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        s[i] = key[i] = -INFINITY;
        if (e < p.experts) {
            const float x = load_logit<F32>(p.logits, row + e);
            s[i] = rank_key(route_score64(p, x, top, inv) + (p.bias != nullptr ? static_cast<double>(__ldg(p.bias + e)) : 0.0));
            // without a bias the experts are ranked by their logits
            key[i] = p.bias != nullptr ? s[i] : rank_key(static_cast<double>(x));
        }
    }
    uint32_t kept = 0;
    if (p.top_groups < p.groups) kept = route_rank_groups(p, route_group_score<V, double>(p, s, lane).score, lane);
    uint32_t alive = route_alive<V>(p, kept, lane);
    int mine = 0;
    for (int j = 0; j < p.k; ++j) {
        double best = -INFINITY;
        int e = MOE_MAX_EXPERTS;
#pragma unroll route_unroll64<V>()
        for (int i = 0; i < V; ++i)
            if (((alive >> i) & 1u) && (e == MOE_MAX_EXPERTS || key[i] > best)) {
                best = key[i];
                e = lane * V + i;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double b = __shfl_xor_sync(0xffffffffu, best, o);
            const int f = __shfl_xor_sync(0xffffffffu, e, o);
            if (f != MOE_MAX_EXPERTS && (e == MOE_MAX_EXPERTS || b > best || (b == best && f < e))) {
                best = b;
                e = f;
            }
        }
        if (lane == j) mine = e;
        if (e / V == lane) alive &= ~(1u << (e % V));
    }
    return mine;
}

constexpr int ROUTE_THREADS = 256;

// A lane's V logits of one row: 16-byte loads when the rows allow (`vec`).
template <int V, bool F32>
__device__ __forceinline__ void load_logits(const RouteParams& p, size_t row, int lane, bool vec, float (&x)[V]) {
    constexpr int kPer = F32 ? 4 : 8;  // values in 16 bytes
    if (V % kPer == 0 && vec) {
        if (lane * V >= p.experts) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
            return;
        }
        const char* src = static_cast<const char*>(p.logits) + (row + lane * V) * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < V / kPer; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (F32) {
                    x[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    x[(8 * i + 2 * j) % V] = __uint_as_float(w[j] << 16);
                    x[(8 * i + 2 * j + 1) % V] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        x[i] = e < p.experts ? load_logit<F32>(p.logits, row + e) : -INFINITY;
    }
}

template <int V, bool F32>
__global__ void __launch_bounds__(ROUTE_THREADS, V <= 8 ? 4 : 1) moe_route_kernel(const RouteParams p) {
    constexpr uint32_t kIndexMask = (1u << route_index_bits<V>()) - 1u;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = static_cast<int>(threadIdx.x & 31u);
    const int warps = static_cast<int>(gridDim.x * (ROUTE_THREADS / 32));
    const bool by_score = p.bias != nullptr;
    const bool grouped = p.top_groups < p.groups;
    // the groups' scores need the scores themselves when they are sums
    const bool need_scores = by_score || (grouped && p.group_top == 2);
    // bf16 logits ranked as they are: the whole index fits below them
    const bool whole_index = !F32 && !by_score;
    const int size = p.experts / p.groups;
    const int run = size / V;  // lanes of a group, when its experts fill whole lanes
    const bool runs = size % V == 0 && (run & (run - 1)) == 0;
    const int my_group = runs ? min(lane / run, 31) : 0;
    const bool partial = 32 * V != p.experts;  // lanes or registers without an expert
    const bool vec = p.experts % V == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 &&
                     (static_cast<size_t>(p.experts) * (F32 ? 4 : 2)) % 16 == 0;
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = by_score && lane * V + i < p.experts ? __ldg(p.bias + lane * V + i) : 0.f;

    for (int t = static_cast<int>(blockIdx.x) * (ROUTE_THREADS / 32) + static_cast<int>(threadIdx.x >> 5); t < p.tokens;
         t += warps) {
        const size_t row = static_cast<size_t>(t) * p.experts;
        float x[V];
        load_logits<V, F32>(p, row, lane, vec, x);
        // softmax: the row's maximum (0 where every logit is -inf) and 1 / sum (0 then)
        float top = 0.f, inv = 1.f;
        if (p.softmax) {
            top = x[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.f;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += lane * V + i < p.experts ? expf(x[i] - top) : 0.f;
            sum = warp_sum(sum);
            inv = sum == 0.f ? 0.f : 1.f / sum;
        }
        // no score is larger: its error bounds those of the others, and the sum's error
        // moves all scores by the same factor
        const float best_score = p.softmax ? inv : 1.f;
        // scores plus bias in fp32
        float s[V];
        if (need_scores) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (p.softmax) {
                    s[i] = fmaf(__expf(x[i] - top), inv, bias[i]);
                } else {
                    float r;  // (an infinite 1 + exp gives 0)
                    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x[i])));
                    s[i] = r + bias[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = x[i];
        }
        // the keys (fmaxf: a NaN ranks as -inf)
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = fmaxf(s[i], -INFINITY);
            const uint32_t u = ordered_bits((by_score ? s[i] : fmaxf(x[i], -INFINITY)) + 0.f);
            key[i] = whole_index ? (u & ~1023u) | (1023u - static_cast<uint32_t>(lane * V + i))
                                 : (u & ~kIndexMask) | static_cast<uint32_t>(V - 1 - i);
        }
        if (partial) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i >= p.experts) {
                    s[i] = -INFINITY;
                    key[i] = 0u;
                }
        }
        bool close = false;
        if (grouped) {
            GroupScore<float> group(p, 0.f, 0.f);
            if (runs && by_score) {
                // each lane's two best, from its sorted keys
                sort_keys<V>(key);
                float b1 = key_value<V>(key[0]), b2 = V > 1 ? key_value<V>(key[V > 1 ? 1 : 0]) : -INFINITY;
                for (int o = 1; o < run; o <<= 1) {
                    const float c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
                    b2 = fmaxf(fminf(b1, c1), fmaxf(b2, c2));
                    b1 = fmaxf(b1, c1);
                }
                group = GroupScore<float>(p, b1, b2).from_lane((lane * run) & 31);
            } else {
                group = route_group_score<V, float>(p, s, lane);
            }
            const uint32_t kept = route_rank_groups(p, group.score, lane);
            if (need_scores) {
                // the least that a group that stays may score against the most that another
                // may (the best logits of groups are exact, sums and biased scores are not;
                // infinite scores are, too: their order goes by the index)
                const float off = isinf(group.score) ? 0.f : 0.5f * route_tolerance<V>() * fmaxf(best_score, group.size);
                const bool stays = (kept >> lane) & 1u;
                const uint32_t lo = __reduce_min_sync(0xffffffffu, stays ? ordered_bits(group.score - off) : 0xffffffffu);
                const uint32_t hi = __reduce_max_sync(
                    0xffffffffu, !stays && lane < p.groups ? ordered_bits(group.score + off) : 0u);
                close = lo <= hi && from_ordered_bits(lo) != -INFINITY;
            }
            if (runs) {
                if (!((kept >> my_group) & 1u)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = 0u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!((kept >> min((lane * V + i) / size, 31)) & 1u)) key[i] = 0u;
            }
        }
        int mine = 0;
        if (close) {
            mine = route_choose64<V, F32>(p, row, lane);
        } else {
            if (!(grouped && runs && by_score)) sort_keys<V>(key);
            uint32_t my_key = 0, last = 0;
            int my_src = 0;
            // the j-th largest key, kept by lane j (0: nothing is left)
            auto take = [&](int j) {
                last = __reduce_max_sync(0xffffffffu, key[0]);
                const int src = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, key[0] == last))) - 1;
                if (lane == j) {
                    my_key = last;
                    my_src = src;
                }
                const bool up = lane == src;
#pragma unroll
                for (int i = 0; i + 1 < V; ++i) key[i] = up ? key[i + 1] : key[i];
                key[V - 1] = up ? 0u : key[V - 1];
            };
            // one more than k: the last choice may be a close one
            for (int j = 0; j <= p.k; ++j) take(j);
            // equal but for the index's bits, infinite keys too (equal ones go by the whole
            // index); scores: also within the tolerance, which no infinite key has
            auto near = [&](uint32_t above, uint32_t below) {
                if (whole_index || below == 0u) return false;
                if (((above ^ below) & ~kIndexMask) == 0u) return true;
                if (!by_score) return false;
                const float a = key_value<V>(above), b = key_value<V>(below);
                const float size = fmaxf(best_score, fmaxf(fabsf(a), fabsf(b)));
                return size < INFINITY && a - b <= route_tolerance<V>() * size;
            };
            uint32_t next = __shfl_down_sync(0xffffffffu, my_key, 1);
            if (lane == p.k - 1) next = last;
            const bool redo = __any_sync(0xffffffffu, lane < p.k && near(my_key, next)) != 0;
            // further candidates while they are close to the one before
            int n = p.k + 1;
            if (redo) {
                uint32_t above = __shfl_sync(0xffffffffu, my_key, p.k - 1);
                while (n < 32 && near(above, last)) {
                    above = last;
                    take(n++);
                }
            }
            mine = whole_index ? 1023 - static_cast<int>(my_key & 1023u)
                               : my_src * V + V - 1 - static_cast<int>(my_key & kIndexMask);
            if (redo) {
                if (n >= 32) mine = route_choose64<V, F32>(p, row, lane);
                else mine = route_order64<V, F32>(p, row, lane, mine, __popc(__ballot_sync(0xffffffffu, lane < n && my_key != 0u)));
            }
        }
        // weights, from the chosen experts' logits
        float w = 0.f;
        if (lane < p.k) {
            const float v = load_logit<F32>(p.logits, row + mine);
            w = p.softmax ? expf(v - top) * inv : 1.f / (1.f + expf(-v));
        }
        float out = p.scale * w;
        if (p.renorm) out /= warp_sum(w) + ROUTE_EPS;
        if (lane < p.k) {
            p.ids[static_cast<size_t>(t) * p.k + lane] = mine;
            p.weights[static_cast<size_t>(t) * p.k + lane] = out;
        }
    }
}

// Gradient of the weights with respect to the logits, for given ids:
//   renormalised  ds_j = scale / S^2 * (sum_l (g_j - g_l) s_l + g_j eps),  S = sum s_l + eps
//   otherwise     ds_j = scale * g_j
//   sigmoid       dx_j = ds_j s_j (1 - s_j), 0 elsewhere
//   softmax       dx_i = s_i (ds_i - c),  c = sum_j ds_j s_j (scale * mean(g) * eps / S when renormalised)
// The differences g_j - g_l keep the digits that g_j - mean(g) would cancel. So do, for a
// chosen expert of a softmax that is not renormalised, those in
//   ds_i - c = sum over the chosen j of s_j (ds_i - ds_j) + ds_i * (sum of s over the others)
// when little is left to the others (ds the sum of an expert's slots).
// One warp per token; lane j < k holds choice j. Ids outside [0, E) count as
// not chosen; an expert named twice gets both slots' gradients. 16384 tokens of
// 256 experts take 7.0 us (33.6 MB: L2 holds them), 8191 of 32 in bf16 4.3 us; not
// renormalised, a softmax takes 9.0 us for the former, 12.6 where every row is peaked.
struct RouteBackwardParams {
    const void* logits;      // [T, E]
    const int32_t* ids;      // [T, k]
    const float* d_weights;  // [T, k]
    void* d_logits;          // [T, E], the logits' type
    int tokens, experts, k;
    int softmax, renorm;
    float scale;
};

template <bool F32>
__device__ __forceinline__ void store_logit(void* x, size_t i, float v) {
    if constexpr (F32) static_cast<float*>(x)[i] = v;
    else static_cast<__nv_bfloat16*>(x)[i] = __float2bfloat16_rn(v);
}

// EXACT_REST: a softmax that is not renormalised. (In one instance with the others its
// registers cost them 3 to 4%; eight blocks per SM: 32 registers, which V <= 8 holds.)
template <int V, bool F32, bool EXACT_REST>
__global__ void __launch_bounds__(ROUTE_THREADS, EXACT_REST && V <= 8 ? 8 : 1) moe_route_backward_kernel(const RouteBackwardParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = static_cast<int>(threadIdx.x & 31u);
    const int t = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
    if (t >= p.tokens) return;
    const size_t row = static_cast<size_t>(t) * p.experts;
    // expert e = 32 i + lane: a row is read and written in whole lines
    float s[V];
    float top = 0.f, inv = 0.f;
    if (p.softmax) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 32 * i + lane;
            s[i] = e < p.experts ? load_logit<F32>(p.logits, row + e) : -INFINITY;
            top = fmaxf(top, s[i]);
        }
        top = warp_max(top);
        if (top == -INFINITY) top = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = 32 * i + lane < p.experts ? expf(s[i] - top) : 0.f;
            sum += s[i];
        }
        sum = warp_sum(sum);
        inv = sum == 0.f ? 0.f : 1.f / sum;
    }
    int id = -1;
    float g = 0.f, sj = 0.f, not_sj = 0.f;
    if (lane < p.k) {
        id = __ldg(p.ids + static_cast<size_t>(t) * p.k + lane);
        if (id < 0 || id >= p.experts) id = -1;
    }
    if (id >= 0) {
        g = __ldg(p.d_weights + static_cast<size_t>(t) * p.k + lane);
        const float x = load_logit<F32>(p.logits, row + id);
        if (p.softmax) {
            sj = expf(x - top) * inv;
        } else {
            sj = 1.f / (1.f + expf(-x));
            not_sj = 1.f / (1.f + expf(x));
        }
    }
    float ds = p.scale * g, c;
    if (p.renorm) {
        const float total = warp_sum(sj) + ROUTE_EPS;
        float diff = 0.f;
        for (int l = 0; l < p.k; ++l) {
            const float gl = __shfl_sync(0xffffffffu, g, l), sl = __shfl_sync(0xffffffffu, sj, l);
            diff += (g - gl) * sl;
        }
        ds = id >= 0 ? p.scale * ((diff + g * ROUTE_EPS) / total) / total : 0.f;
        c = p.scale * (warp_sum(g * sj) / total) * (ROUTE_EPS / total);
    } else {
        c = warp_sum(ds * sj);
    }
    float both = 0.f;  // every slot that names this lane's expert
    for (int l = 0; l < p.k; ++l) {
        const float dl = __shfl_sync(0xffffffffu, ds, l);
        const int il = __shfl_sync(0xffffffffu, id, l);
        if (il == id) both += dl;
    }
    float diff = both - c;
    if constexpr (EXACT_REST) {
        // (scores that leave a quarter to the others: |ds_i| and |c| are within 4 times the
        // sum of the terms' sizes, and nothing cancels)
        if (warp_sum(sj) > 0.75f) {
            uint32_t chosen = 0;   // which of this lane's entries of the row are chosen
            bool first = id >= 0;  // no earlier slot names this lane's expert
            for (int l = 0; l < p.k; ++l) {
                const int il = __shfl_sync(0xffffffffu, id, l);
                if (il == id && l < lane) first = false;
                if (il >= 0 && (il & 31) == lane) chosen |= 1u << (il >> 5);
            }
            float rest = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) rest += (chosen >> i) & 1u ? 0.f : s[i];
            diff = both * (warp_sum(rest) * inv);
            const float sf = first ? sj : 0.f;
            for (int l = 0; l < p.k; ++l) {
                const float bl = __shfl_sync(0xffffffffu, both, l), sl = __shfl_sync(0xffffffffu, sf, l);
                diff += sl * (both - bl);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = 32 * i + lane;
        if (e < p.experts) store_logit<F32>(p.d_logits, row + e, p.softmax ? -c * (s[i] * inv) : 0.f);
    }
    __syncwarp();  // the chosen experts' entries are written again, after the row
    if (id >= 0) store_logit<F32>(p.d_logits, row + id, p.softmax ? sj * diff : both * sj * not_sj);
}

// ------------------------------------------------------- rows of the experts ----
//
// A stable counting sort of the T*k choices by expert: choice i = t*k + j gets
// row base[e] + (choices of expert e before i), where base[e] is the sum of
// the earlier experts' rows rounded up to whole 128-row blocks (contiguous
// form), or e * max_m (masked form; ranks at or past max_m get row -1).
//
// One cluster of up to 16 CTAs does it in one launch, with no workspace: every
// warp owns a run of choices and a row of counters in shared memory, counts
// it, the counters are turned into first rows by a scan over warps, CTAs
// (through distributed shared memory) and experts, and the run is walked a
// second time to hand the rows out. Ranks inside 32 choices come from ballots
// over the expert's bits (match_any takes a step per distinct expert: 65536
// choices of 256 experts 16 us against 13, with 8 CTAs).
//
// Bound by the steps of 32 choices, each of which waits for the counters that the
// last one left; four steps' loads and ballots overlap. 512 choices of 32 experts
// take 6 us, 65536 of 256 experts 9.4 us, 524288 of them 31 us: next to the
// dispatch that follows (99 us for those 65536, of 7168 values) a second launch
// and a workspace would not pay.

constexpr int ROWS_THREADS = 1024;
constexpr int ROWS_WARPS = ROWS_THREADS / 32;
constexpr int ROWS_MAX_CLUSTER = 16;  // CTAs, where the device has a place for them
constexpr int ROWS_BATCH = 4;         // steps of 32 choices that overlap

struct RowsParams {
    const int32_t* ids;   // [n]; outside [0, G): no row
    int32_t* row_of;      // [n]
    int32_t* meta;        // m_indices [m_cap] (contiguous) or masked_m [G] (masked)
    int32_t* counts;      // [G]
    int n, groups;
    int m_cap;            // contiguous: rows of m_indices
    int max_m;            // masked: rows of an expert; 0 = contiguous
};

// dynamic shared memory: [ROWS_WARPS][G] counters, [G] this CTA's choices, [G] all choices, [G + 1] first rows
__host__ __device__ constexpr int rows_smem_bytes(int groups) { return (ROWS_WARPS * groups + 3 * groups + 1) * 4; }

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Rows of the N * 32 choices from i0 on, in order; `next` holds the warp's next row of every expert.
template <int N>
__device__ __forceinline__ void rows_hand_out(const RowsParams& p, int* next, int i0, int end, int bits, int lane) {
    int expert[N], row[N];
    uint32_t same[N];  // lanes of the step whose choice is this lane's expert
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int i = i0 + 32 * s + lane;
        expert[s] = i < end ? __ldg(p.ids + i) : -1;
        if (expert[s] < 0 || expert[s] >= p.groups) expert[s] = -1;  // (differs from every expert in bit `bits`)
        same[s] = 0xffffffffu;
    }
    for (int b = 0; b <= bits; ++b) {
#pragma unroll
        for (int s = 0; s < N; ++s) {
            const uint32_t mine = 0u - ((static_cast<uint32_t>(expert[s]) >> b) & 1u);  // the bit, in every lane's place
            same[s] &= ~(__ballot_sync(0xffffffffu, mine) ^ mine);
        }
    }
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int e = expert[s];
        const int at = e >= 0 ? next[e] : 0;
        __syncwarp();
        row[s] = at + __popc(same[s] & ((1u << lane) - 1u));
        if (e >= 0 && lane == 31 - __clz(static_cast<int>(same[s]))) next[e] = row[s] + 1;
        __syncwarp();
    }
#pragma unroll
    for (int s = 0; s < N; ++s) {
        const int i = i0 + 32 * s + lane, e = expert[s];
        if (i >= end) continue;
        const bool fits = e >= 0 && (p.max_m == 0 || row[s] - e * p.max_m < p.max_m);
        p.row_of[i] = fits ? row[s] : -1;
    }
}

__global__ void __launch_bounds__(ROWS_THREADS, 1) moe_rows_kernel(const RowsParams p) {
    extern __shared__ int rows_smem[];
    __shared__ int warp_totals[ROWS_WARPS];
    griddep_launch_dependents();
    griddep_wait();
    const int G = p.groups;
    int* hist = rows_smem;                    // [warp][G]
    int* cta_total = hist + ROWS_WARPS * G;   // [G], read by the other CTAs too
    int* all_total = cta_total + G;           // [G]
    int* first = all_total + G;               // [G + 1]
    const int tid = static_cast<int>(threadIdx.x);
    const int lane = tid & 31, warp = tid >> 5;
    const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);  // one cluster
    for (int i = tid; i < ROWS_WARPS * G; i += ROWS_THREADS) hist[i] = 0;
    __syncthreads();

    // this warp's run of choices, in whole steps of 32
    const int warps = ctas * ROWS_WARPS;
    const int64_t steps = (static_cast<int64_t>(p.n) + 31) / 32;
    const int64_t me = rank * ROWS_WARPS + warp;
    const int begin = static_cast<int>(steps * me / warps * 32);
    const int end = static_cast<int>(min(static_cast<int64_t>(p.n), steps * (me + 1) / warps * 32));
    int* mine = hist + warp * G;
    for (int i0 = begin; i0 < end; i0 += 32 * ROWS_BATCH) {
        int e[ROWS_BATCH];
#pragma unroll
        for (int b = 0; b < ROWS_BATCH; ++b) e[b] = i0 + 32 * b + lane < end ? __ldg(p.ids + i0 + 32 * b + lane) : -1;
#pragma unroll
        for (int b = 0; b < ROWS_BATCH; ++b)
            if (e[b] >= 0 && e[b] < G) atomicAdd(mine + e[b], 1);  // whole numbers: any order gives the same count
    }
    __syncthreads();

    // counters -> choices of the expert in earlier warps of this CTA; thread e owns expert e
    if (tid < G) {
        int run = 0;
#pragma unroll 8
        for (int w = 0; w < ROWS_WARPS; ++w) {
            const int c = hist[w * G + tid];
            hist[w * G + tid] = run;
            run += c;
        }
        cta_total[tid] = run;
    }
    cluster_sync();
    int before = 0, total = 0;
    if (tid < G) {
        const uint32_t at = smem_u32(cta_total + tid);
        for (int r = 0; r < ctas; ++r) {
            const int c = ld_cluster_s32(mapa_shared(at, static_cast<uint32_t>(r)));
            if (r < rank) before += c;
            total += c;
        }
    }
    // first rows: an exclusive scan of the experts' whole blocks
    const int rows = (tid < G && p.max_m == 0) ? (total + 127) / 128 * 128 : 0;
    int incl = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_totals[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = warp_totals[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        warp_totals[lane] = v;
    }
    __syncthreads();
    if (tid < G) {
        const int base = p.max_m ? tid * p.max_m : (warp ? warp_totals[warp - 1] : 0) + incl - rows;
        first[tid] = base;
        if (tid == G - 1) first[G] = base + rows;
#pragma unroll 8
        for (int w = 0; w < ROWS_WARPS; ++w) hist[w * G + tid] += base + before;
        if (rank == 0) {
            p.counts[tid] = total;
            if (p.max_m) p.meta[tid] = min(total, p.max_m);
        }
        all_total[tid] = total;
    }
    __syncthreads();
    const int bits = 32 - __clz((G - 1) | 1);
    int i0 = begin;
    for (; i0 + 32 * ROWS_BATCH <= end; i0 += 32 * ROWS_BATCH) rows_hand_out<ROWS_BATCH>(p, mine, i0, end, bits, lane);
    for (; i0 < end; i0 += 32) rows_hand_out<1>(p, mine, i0, end, bits, lane);
    if (p.max_m == 0) {
        // the expert of every row of every 128-row block; -1 on padding rows and past the last block
        const int blocks = (p.m_cap + 127) / 128;
        for (int b = rank * ROWS_WARPS + warp; b < blocks; b += warps) {
            const int r0 = b * 128;
            int e = -1, filled = 0;
            if (r0 < first[G]) {
                int lo = 0, hi = G - 1;  // the last expert whose first row is at or before r0
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (first[mid] <= r0) lo = mid;
                    else hi = mid - 1;
                }
                e = lo;
                filled = first[e] + all_total[e];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + 32 * j + lane;
                if (r < p.m_cap) p.meta[r] = r < filled ? e : -1;
            }
        }
    }
    cluster_sync();  // no CTA leaves while a peer may read its totals
}

// ---------------------------------------------------------------- dispatch ----
//
// q[row_of[t, j]] = E4M3(x[t] / s), with one scale s per 128 values: a power of
// two, packed as UE8M0 (the rule of quantize_fp8_1x128), or amax / 448 in
// fp32. A token is read and cast once and its codes are written k times, so
// the traffic is the floor: T*H values in, T*k*H codes out.
//
// A warp handles four 128-value blocks of a token (one packed scale word):
// lane l takes 16 values of block l / 8, whose amax is a maximum over 8 lanes.
//
// Bound by memory, its writes above all (80% of the bytes): 8192 tokens of 7168
// bf16 values in 8 copies each move 602 MB in 99 us (6.1 TB/s), as a plain quantiser
// (one copy) 4096 x 7168 take 18 us. A warp does one word and ends: eight CTAs per
// SM that loop over words took 115 and 20.6 us (a warp's next load was issued
// behind all its stores).

constexpr int DISPATCH_THREADS = 256;

struct DispatchParams {
    const void* x;          // [T, H] bf16 or fp32
    const int32_t* row_of;  // [T, k], or null: row t (k = 1)
    uint4* q;               // [rows, H] E4M3
    void* sf;               // [rows, ceil(H/512)] int32 (UE8M0) or [rows, H/128] fp32
    int64_t rows;
    int tokens, k;
    int kb, kp;             // H / 128, ceil(H / 512)
};

template <bool IN_F32>
__device__ __forceinline__ void load16(const void* x, int64_t at, float (&v)[16]) {
    if constexpr (IN_F32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = __ldg(src + i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 u = __ldg(src + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    }
}

template <bool IN_F32, bool SF_F32>
__global__ void __launch_bounds__(DISPATCH_THREADS) moe_dispatch_fp8_kernel(const DispatchParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = static_cast<int>(threadIdx.x & 31u);
    const uint32_t i = blockIdx.x * (DISPATCH_THREADS / 32) + (threadIdx.x >> 5);  // (T * kp < 2^32 - 2^28)
    const uint32_t t = i / static_cast<uint32_t>(p.kp);
    if (t >= static_cast<uint32_t>(p.tokens)) return;
    const int word = static_cast<int>(i - t * static_cast<uint32_t>(p.kp));
    const int block = 4 * word + (lane >> 3);
    const bool there = block < p.kb;
    // the token's rows, one per lane (k <= 32), loaded beside its values
    int64_t my_row = p.row_of != nullptr ? int64_t{-1} : static_cast<int64_t>(t);
    if (p.row_of != nullptr && lane < p.k) my_row = __ldg(p.row_of + static_cast<int64_t>(t) * p.k + lane);
    float v[16];
    if (there) {
        load16<IN_F32>(p.x, (static_cast<int64_t>(t) * p.kb + block) * 128 + 16 * (lane & 7), v);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
    uint32_t m = __float_as_uint(1e-4f);
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale, inv;
    uint32_t byte = 0;
    if constexpr (SF_F32) {
        scale = __uint_as_float(m) / 448.f;
        inv = 448.f / __uint_as_float(m);
    } else {
        const int e = static_cast<int>((m >> 23) & 0xFFu) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        byte = there ? static_cast<uint32_t>(127 + e) : 0u;
        scale = 0.f;
        inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = e4m3x2_rn(v[4 * j + 1] * inv, v[4 * j] * inv) |
               (e4m3x2_rn(v[4 * j + 3] * inv, v[4 * j + 2] * inv) << 16);
    const uint4 codes = make_uint4(c[0], c[1], c[2], c[3]);
    // the four blocks' bytes meet in lane 0's word
    uint32_t packed = 0;
    if constexpr (!SF_F32) {
        packed = byte << (8 * (lane >> 3));
        packed |= __shfl_xor_sync(0xffffffffu, packed, 8);
        packed |= __shfl_xor_sync(0xffffffffu, packed, 16);
    }
    for (int j = 0; j < p.k; ++j) {
        const int64_t r = __shfl_sync(0xffffffffu, my_row, j);
        if (r < 0 || r >= p.rows) continue;  // the same in every lane
        if (there) p.q[(r * p.kb + block) * 8 + (lane & 7)] = codes;
        if constexpr (SF_F32) {
            if (there && (lane & 7) == 0) static_cast<float*>(p.sf)[r * p.kb + block] = scale;
        } else {
            if (lane == 0) static_cast<uint32_t*>(p.sf)[r * p.kp + word] = packed;
        }
    }
}

// ----------------------------------------------------------------- combine ----
//
// out[t] = sum_j w[t, j] y[row_of[t, j]], in fp32 in the order of j, rounded to
// bf16 once. Slots without a row (outside [0, rows)) are not read and add
// nothing. One thread per eight columns of a token, up to eight rows' loads in
// flight. Bound by memory: 4096 tokens of 8 rows of 7168 values move 528 MB in
// 83 us (6.4 TB/s; 87.5 with a grid that stays and loops).

constexpr int COMBINE_THREADS = 256;
constexpr int COMBINE_BATCH = 8;

struct CombineParams {
    const uint4* y;         // [rows, H] bf16
    const int32_t* row_of;  // [T, k]
    const float* w;         // [T, k], or null: ones
    uint4* out;             // [T, H] bf16
    int64_t rows;
    int tokens, k;
    int vecs;               // H / 8
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_kernel(const CombineParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * COMBINE_THREADS + threadIdx.x;
    if (i >= static_cast<int64_t>(p.tokens) * p.vecs) return;
    const int t = static_cast<int>(i / p.vecs);
    const int c = static_cast<int>(i - static_cast<int64_t>(t) * p.vecs);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += COMBINE_BATCH) {
        uint4 u[COMBINE_BATCH];
        float w[COMBINE_BATCH];
        bool live[COMBINE_BATCH];
#pragma unroll
        for (int j = 0; j < COMBINE_BATCH; ++j) {
            live[j] = false;
            if (j0 + j >= p.k) continue;
            const int64_t at = static_cast<int64_t>(t) * p.k + j0 + j;
            const int64_t r = __ldg(p.row_of + at);
            live[j] = r >= 0 && r < p.rows;
            if (!live[j]) continue;
            w[j] = p.w != nullptr ? __ldg(p.w + at) : 1.f;
            u[j] = __ldg(p.y + r * p.vecs + c);
        }
#pragma unroll
        for (int j = 0; j < COMBINE_BATCH; ++j) {
            if (!live[j]) continue;
            float v[8];
            bf16x8_to_f32(u[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], v[e], acc[e]);
        }
    }
    p.out[i] = f32_to_bf16x8(acc);
}

// Gradients of combine: d_y[row_of[t, j]] = w[t, j] d_out[t] (bf16) and
// d_w[t, j] = <y[row_of[t, j]], d_out[t]> (fp32). Slots without a row get
// d_w = 0; rows that no slot names are left as they were.
// One CTA per token: its threads cover the columns and add up eight slots at a
// time; the sums over threads go by warps and then in warp order. Bound by memory:
// 4096 tokens of 8 rows of 7168 values move 998 MB in 161-164 us (6.1 TB/s);
// d_w is why y is read at all, and both gradients come out of one pass over it.

struct CombineBackwardParams {
    const uint4* y;         // [rows, H] bf16
    const int32_t* row_of;  // [T, k]
    const float* w;         // [T, k], or null: ones
    const uint4* d_out;     // [T, H] bf16
    uint4* d_y;             // [rows, H] bf16
    float* d_w;             // [T, k]
    int64_t rows;
    int tokens, k;
    int vecs;
};

__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_backward_kernel(const CombineBackwardParams p) {
    __shared__ float part[COMBINE_THREADS / 32][COMBINE_BATCH];
    griddep_launch_dependents();
    griddep_wait();
    const int t = static_cast<int>(blockIdx.x);
    const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
    const int warps = static_cast<int>(blockDim.x >> 5);
    const int64_t slot0 = static_cast<int64_t>(t) * p.k;
    for (int j0 = 0; j0 < p.k; j0 += COMBINE_BATCH) {
        int64_t r[COMBINE_BATCH];
        float w[COMBINE_BATCH], dot[COMBINE_BATCH];
#pragma unroll
        for (int j = 0; j < COMBINE_BATCH; ++j) {
            dot[j] = 0.f;
            r[j] = -1;
            w[j] = 0.f;
            if (j0 + j >= p.k) continue;
            r[j] = __ldg(p.row_of + slot0 + j0 + j);
            if (r[j] >= p.rows) r[j] = -1;
            if (r[j] >= 0) w[j] = p.w != nullptr ? __ldg(p.w + slot0 + j0 + j) : 1.f;
        }
        for (int c = static_cast<int>(threadIdx.x); c < p.vecs; c += static_cast<int>(blockDim.x)) {
            uint4 u[COMBINE_BATCH];
#pragma unroll
            for (int j = 0; j < COMBINE_BATCH; ++j)
                if (r[j] >= 0) u[j] = __ldg(p.y + r[j] * p.vecs + c);
            float d[8];
            bf16x8_to_f32(__ldg(p.d_out + static_cast<int64_t>(t) * p.vecs + c), d);
#pragma unroll
            for (int j = 0; j < COMBINE_BATCH; ++j) {
                if (r[j] < 0) continue;
                float v[8], o[8];
                bf16x8_to_f32(u[j], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[j] = fmaf(v[e], d[e], dot[j]);
                    o[e] = w[j] * d[e];
                }
                p.d_y[r[j] * p.vecs + c] = f32_to_bf16x8(o);
            }
        }
#pragma unroll
        for (int j = 0; j < COMBINE_BATCH; ++j) {
            const float s = warp_sum(dot[j]);
            if (lane == 0) part[warp][j] = s;
        }
        __syncthreads();
        const int j = static_cast<int>(threadIdx.x);
        if (j < COMBINE_BATCH && j0 + j < p.k) {
            float s = 0.f;
            for (int i = 0; i < warps; ++i) s += part[i][j];
            p.d_w[slot0 + j0 + j] = s;
        }
        __syncthreads();
    }
}

}  // namespace dg
