// The router of a layer of experts: k experts and their weights for each token, and
// the gradient of the weights with respect to the logits.
//
//   p = softmax(l) or sigmoid(l);  chosen by v = p + bias (within the best groups);
//   w_j = scale p_j (/ sum of the chosen p).
//
// A warp has one token.  The experts of a group lie next to each other in a run of
// lanes, V to a lane, so that expert indices rise with the lane and, within it, with
// the register: the lowest lane that holds the largest value holds the lowest index
// of a tie.
//
// Without a bias experts are chosen by the logits themselves, which order as their scores
// do.  Otherwise (and for sums of two scores of a group) v is computed in FP32 with an
// error bound, and experts or groups whose order hangs on values closer than that are
// compared in FP64: about one token in a thousand.  Values that FP64 makes equal (sigmoids
// past 37 are 1) are ties.
//
// The k-th largest of the lanes' largest values bounds the k-th largest of all from below:
// the experts above it, a few more than k, are brought together in shared memory and
// ranked by comparing each with each.  Where they are more than a warp's lanes (many
// equal values), the choice takes a round of maxima for each expert.
//
// Renormalised weights need no sum over all experts: the largest chosen logit is
// taken out of the quotient, so that scores that FP32 cannot hold cancel.
//
// The logits are read once and are a microsecond or two of bandwidth: what bounds the
// kernels is instructions (60 % of the issue slots at 20 to 27 warps an SM) and the latency
// of warp-wide steps, which do not get fewer with the experts.  8192 x 256 FP32, sigmoid, bias,
// four of eight groups, k = 8: 13.7 us (1170 instructions a token; with a round of maxima for
// each expert 29 us), 10.9 without a bias, 7.0 without groups either (590); 16384 x 122 BF16,
// softmax, k = 6: 9.8 us (500), its backward 5.0 over all experts and 4.8 renormalised.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "tile_sched.cuh"

namespace tmagemm {

namespace {

constexpr int kWarps = 8;               // tokens of a CTA
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (TYPE == kLogitsF32) return static_cast<const float*>(p)[i];
    if constexpr (TYPE == kLogitsBf16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

template <int TYPE>
__device__ __forceinline__ void store_logit(void* p, int64_t i, float v) {
    if constexpr (TYPE == kLogitsF32)
        static_cast<float*>(p)[i] = v;
    else if constexpr (TYPE == kLogitsBf16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// V logits from `i`, in 16- or 8-byte loads where they are aligned to their size.
template <int TYPE, int V>
__device__ __forceinline__ void load_logits(const void* p, int64_t i, int count, bool aligned,
                                            float (&l)[V]) {
    constexpr int kBytes = V * (TYPE == kLogitsF32 ? 4 : 2);
    if constexpr (kBytes >= 8) {
        if (aligned) {
            constexpr int kWords = kBytes / 4;
            uint32_t w[kWords];
            const char* from = static_cast<const char*>(p) + i * (TYPE == kLogitsF32 ? 4 : 2);
            if constexpr (kBytes >= 16) {
#pragma unroll
                for (int k = 0; k < kWords; k += 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(from + 4 * k);
                    w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
                }
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                w[0] = v.x, w[1] = v.y;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (TYPE == kLogitsF32)
                    l[j] = __uint_as_float(w[j]);
                else if constexpr (TYPE == kLogitsBf16)
                    l[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
                else
                    l[j] = __half2float(__ushort_as_half(
                        static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)))));
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = j < count ? load_logit<TYPE>(p, i + j) : -kInf;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// part / sum: exactly 1 for all of it, so that one choice has its scale and no gradient
// (a division rounded right does that too, and makes the backward of 16384 x 122 5.3 us
// instead of 4.8).
__device__ __forceinline__ float share(float part, float sum) {
    return part == sum ? 1.0f : __fdividef(part, sum);
}

// Unsigned keys that order as the numbers do: 0 for a closed expert, zeros of both
// signs alike, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t key = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return v != v ? 0xffffffffu : key;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    const uint64_t key = (b >> 63) ? ~b : b | (1ull << 63);
    return v != v ? ~0ull : key;
}
__device__ __forceinline__ double key_value(uint64_t key) {
    return __longlong_as_double(static_cast<int64_t>((key >> 63) ? key & ~(1ull << 63) : ~key));
}
__device__ __forceinline__ uint32_t warp_key_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_key_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(
        kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Where a lane's experts are: V from `first`, of which `count` exist.
struct LaneExperts {
    int32_t first, count;
    int group, lanes;   // of `lanes` lanes each
};
template <int V>
__device__ __forceinline__ LaneExperts lane_experts(const RouteArgs& a, int lane) {
    const int group = lane >> a.lanes_shift, part = lane & ((1 << a.lanes_shift) - 1);
    const int32_t left = group < a.groups ? a.group_size - part * V : 0;
    return {group * a.group_size + part * V, left < 0 ? 0 : left < V ? left : V, group,
            1 << a.lanes_shift};
}

// The two largest keys of a group, each with ties.
template <int V, class K>
__device__ __forceinline__ void group_best(const LaneExperts& at, const K (&key)[V], K& best,
                                           K& second) {
    best = second = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        second = max(second, min(best, key[j]));
        best = max(best, key[j]);
    }
    for (int d = 1; d < at.lanes; d <<= 1) {
        const K b = __shfl_xor_sync(kAll, best, d), s = __shfl_xor_sync(kAll, second, d);
        second = max(max(second, s), min(best, b));
        best = max(best, b);
    }
}

// Closes the groups that are not among the top_groups of largest `value` (a key; 0: no
// expert is open), ties to the lowest: keys of their experts become 0.  Returns the
// smallest value kept and the largest closed (0: none).
template <int V, class K>
__device__ __forceinline__ void close_groups(const RouteArgs& a, const LaneExperts& at, K value,
                                             K (&key)[V], K& worst, K& out) {
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
        const K other = __shfl_sync(kAll, value, g * at.lanes);
        ahead += other > value || (other == value && g < at.group);
    }
    const bool keep = ahead < a.top_groups;
    if (!keep) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 0;
    }
    worst = ~warp_key_max(keep && at.group < a.groups ? static_cast<K>(~value) : K(0));
    out = warp_key_max(keep || at.group >= a.groups ? K(0) : value);
}

// A lane's two best keys, its lowest index first among equals.
template <int V, class K>
struct Best {
    K first, second;
    int j1, j2;
    bool two;            // `second` is known
    uint32_t taken;
    __device__ __forceinline__ void look(const K (&key)[V]) {
        first = second = 0;
        j1 = j2 = 0;
        two = true;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const K k = (taken >> j) & 1u ? K(0) : key[j];
            if (k > first) {
                second = first, j2 = j1;
                first = k, j1 = j;
            } else if (k > second) {
                second = k, j2 = j;
            }
        }
    }
    // The largest key of the warp is taken out (0: there is none), of equal ones the lowest
    // lane's; its lane leaves the expert in *out.
    __device__ __forceinline__ K take(const K (&key)[V], int lane, int32_t first_expert,
                                      int32_t* out) {
        const K largest = warp_key_max(first);
        const uint32_t equal = __ballot_sync(kAll, first == largest);
        if (first == largest && (equal & ((1u << lane) - 1u)) == 0u) {
            *out = first_expert + j1;
            taken |= 1u << j1;
            if (two) {
                first = second, j1 = j2;
                two = false;
            } else {
                look(key);
            }
        }
        return largest;
    }
};

// A token's sum of exponentials in FP64 (for softmax), of all lanes.
template <int TYPE>
__device__ __noinline__ double sum64(const RouteArgs& a, int64_t row, int lane, float m) {
    double sum = 0.0;
#pragma unroll 1
    for (int32_t e = lane; e < a.E; e += 32)
        sum += exp(static_cast<double>(load_logit<TYPE>(a.logits, row + e)) - m);
    return warp_sum(sum);
}
// The value that experts are chosen by, in FP64 (softmax of a token with a NaN: its logits).
template <int TYPE>
__device__ __noinline__ double value64(const RouteArgs& a, int64_t row, int32_t e, float m,
                                       double sum) {
    const double l = load_logit<TYPE>(a.logits, row + e);
    if (sum != sum) return l;
    const bool softmax = a.score == kScoreSoftmax;
    const double x = exp(softmax ? l - m : -l);
    const double p = softmax ? x / sum : 1.0 / (1.0 + x);
    return a.bias ? p + a.bias[e] : p;
}

// The whole choice of one token in FP64, where FP32 cannot tell which experts' order is in
// doubt: lane j gets the id of choice j (-1: no expert is left).
template <int TYPE, int V>
__device__ __noinline__ int32_t choose64(const RouteArgs& a, int64_t row, int lane, float m,
                                         int32_t* chosen) {
    const LaneExperts at = lane_experts<V>(a, lane);
    const double sum = a.score == kScoreSoftmax ? sum64<TYPE>(a, row, lane, m) : 1.0;
    uint64_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        key[j] = 0;
        if (j < at.count && load_logit<TYPE>(a.logits, row + at.first + j) != -kInf)
            key[j] = order_key(value64<TYPE>(a, row, at.first + j, m, sum));
    }
    if (a.groups > 1) {
        uint64_t best, second, worst, out;
        group_best<V>(at, key, best, second);
        const double v = key_value(best) +
                         (a.group_sum == 2 && second != 0 ? key_value(second) : 0.0);
        close_groups<V>(a, at, best == 0 ? 0 : order_key(v), key, worst, out);
    }
    Best<V, uint64_t> best{};
    best.look(key);
    int c = 0;
    while (c < a.k && best.take(key, lane, at.first, chosen + c) != 0) ++c;
    __syncwarp();
    const int32_t id = lane < c ? chosen[lane] : -1;
    __syncwarp();
    return id;
}

// The ids of the first `count` lanes in the order of their values in FP64.
template <int TYPE>
__device__ __noinline__ int32_t order64(const RouteArgs& a, int64_t row, int lane, float m,
                                        int32_t id, int count) {
    const double sum = a.score == kScoreSoftmax ? sum64<TYPE>(a, row, lane, m) : 1.0;
    const uint64_t exact = id >= 0 ? order_key(value64<TYPE>(a, row, id, m, sum)) : 0ull;
    int rank = 0;
    for (int i = 0; i < count; ++i) {
        const uint64_t other = __shfl_sync(kAll, exact, i);
        const int32_t oid = __shfl_sync(kAll, id, i);
        rank += other > exact || (other == exact && oid < id);
    }
    int32_t placed = -1;
    for (int i = 0; i < count; ++i) {
        const int r = __shfl_sync(kAll, rank, i);
        const int32_t oid = __shfl_sync(kAll, id, i);
        if (r == lane) placed = oid;
    }
    return placed;
}

// The exact value of a lane's group from its two best experts (by their keys), or false where
// a third is too close to them to say which the two are (keys of logits always say so).
template <int TYPE, int V>
__device__ __noinline__ bool group_value64(const RouteArgs& a, const LaneExperts& at, int64_t row,
                                           int lane, float m, const uint32_t (&key)[V],
                                           uint32_t best, uint32_t second, float near,
                                           uint64_t& value) {
    int32_t i1 = 0x7fffffff, i2 = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (key[j] == best) i1 = min(i1, at.first + j);
    for (int d = 1; d < at.lanes; d <<= 1) i1 = min(i1, __shfl_xor_sync(kAll, i1, d));
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (key[j] == second && at.first + j != i1) i2 = min(i2, at.first + j);
    for (int d = 1; d < at.lanes; d <<= 1) i2 = min(i2, __shfl_xor_sync(kAll, i2, d));
    const double sum = a.score == kScoreSoftmax ? sum64<TYPE>(a, row, lane, m) : 1.0;
    // Those left out are below the last of those counted, or equal to it (as in 16 bits they
    // often are) where the other one counted is above or equal too.
    const int32_t last = a.group_sum == 2 ? i2 : i1;
    const uint32_t in = a.group_sum == 2 ? second : best;
    const auto below = [&](uint32_t lower, uint32_t upper) {
        const float x = key_value(upper), y = key_value(lower);
        return x - y > near + 0x1p-22f * (fabsf(x) + fabsf(y));
    };
    const auto equal = [&](int32_t e) {
        return load_logit<TYPE>(a.logits, row + e) == load_logit<TYPE>(a.logits, row + last) &&
               (!a.bias || a.bias[e] == a.bias[last]);
    };
    uint32_t others = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (a.bias && key[j] != 0 && in != 0 && at.first + j != i1 && at.first + j != last &&
            !below(key[j], in))
            others |= 1u << j;
    bool clear = true;
    for (; others != 0; others &= others - 1)
        clear = clear && equal(at.first + __ffs(others) - 1) &&
                (i1 == last || below(in, best) || equal(i1));
    __syncwarp();
    value = 0;
    if (best != 0 && at.group < a.groups) {
        double v = value64<TYPE>(a, row, i1, m, sum);
        if (a.group_sum == 2 && second != 0) v += value64<TYPE>(a, row, i2, m, sum);
        value = order_key(v);
    }
    return __all_sync(kAll, clear || at.group >= a.groups);
}

// The experts of a token that are in question, in the order of their indices, and in the
// order of their values.
struct alignas(16) Candidates {
    uint32_t key[kMaxChoices + 4];    // (read four at a time: each warp's at 16 bytes)
    uint32_t sorted_key[kMaxChoices];
    int32_t id[kMaxChoices], sorted_id[kMaxChoices + 2];
};

static_assert(sizeof(Candidates) % 16 == 0, "each warp's keys are read as vectors");

// The choice in rounds: `k` of them, and up to 32 as long as the next value is within the
// error (`near`, and a part of the values) of the k-th.  Returns how many; 33: more.
template <int V>
__device__ __noinline__ int choose_rounds(const uint32_t (&key)[V], int32_t first_expert, int k,
                                          bool by_logits, float near, Candidates& m, int lane) {
    Best<V, uint32_t> best{};
    best.look(key);
    uint32_t last = 0;
    int count = 0;
    for (; count <= 32; ++count) {
        if (by_logits && count == k) break;
        const uint32_t largest = best.take(key, lane, first_expert, m.sorted_id + count);
        if (largest == 0) break;
        if (count < k) {
            last = largest;
        } else {
            const float x = key_value(last), y = key_value(largest);
            if (x - y > near + 0x1p-22f * (fabsf(x) + fabsf(y))) break;
        }
        if (lane == 0 && count < 32) m.sorted_key[count] = largest;
    }
    return count;
}

// A bitonic sort of one key a lane, largest first.
__device__ __forceinline__ uint32_t sort_lanes(uint32_t key, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d > 0; d /= 2) {
            const uint32_t other = __shfl_xor_sync(kAll, key, d);
            const bool larger = ((lane & size) == 0) == ((lane & d) == 0);
            key = larger ? max(key, other) : min(key, other);
        }
    return key;
}

template <int TYPE, int V>
__global__ void __launch_bounds__(kWarps * 32, 4) route_kernel(const __grid_constant__ RouteArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const LaneExperts at = lane_experts<V>(a, lane);
    __shared__ Candidates all[kWarps];
    Candidates& c = all[threadIdx.x >> 5];
    // (T k < 2^31, so that tokens and choices are counted in 32 bits.)
#pragma unroll 1
    for (uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < static_cast<uint32_t>(a.T);
         t += gridDim.x * kWarps) {
        const int64_t row = static_cast<int64_t>(t) * a.E;
        float l[V];
        load_logits<TYPE, V>(a.logits, row + at.first, at.count, a.aligned, l);
        float m = -kInf;
        const bool softmax = a.score == kScoreSoftmax;
        // Scores order as logits do; sums of two of them do not.
        const bool by_logits = !a.bias, sums = a.groups > 1 && a.group_sum == 2;
        float inverse = 1.0f;   // of the sum over all experts
        if (softmax && (!by_logits || sums || !a.renormalize)) {
#pragma unroll
            for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);
            m = warp_max(m);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(l[j] - m);   // (no experts: NaN, not used)
            inverse = __fdividef(1.0f, warp_sum(sum));
        }
        const auto score = [&](float x) {
            // (A quotient by more than 2^126 would be 0 or NaN.)
            return softmax ? expf(x - m) * inverse
                           : x < -80.0f ? 0.0f : __fdividef(1.0f, 1.0f + expf(-x));
        };
        uint32_t key[V];
        if (by_logits) {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = l[j] == -kInf ? 0u : order_key(l[j]);
        } else {
            float b[V] = {};
            load_logits<kLogitsF32, V>(a.bias, at.first, at.count, a.bias_aligned, b);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = score(l[j]) + b[j];
                // (All scores are NaN: the logits, so that the one that made them so is chosen.)
                if (inverse != inverse) v = l[j];
                key[j] = l[j] == -kInf ? 0u : order_key(v);
            }
        }
        // How far two values of v may be off together: a score of at most p by 2^-19 p
        // (its exponent's argument, expf, a sum of up to 512 terms in a tree of 16 and 5
        // levels, the quotient: 25 roundings; sigmoid: expf's 2 places, a sum, a quotient of one
        // place: under 2^-21), the addition of the bias by 2^-24 of v.
        const float near = softmax ? 0x1p-18f * inverse : 0x1p-20f;
        bool whole = false;        // the choice has to be made again, all of it in FP64
        if (a.groups > 1) {
            uint32_t best, second, worst, out;
            group_best<V>(at, key, best, second);
            float v1 = key_value(best), v2 = sums && second != 0 ? key_value(second) : 0.0f;
            if (by_logits && sums) {
                v1 = score(v1);
                if (second != 0) v2 = score(v2);
            }
            const uint32_t value = best == 0 ? 0u : order_key(v1 + v2);
            uint32_t open[V];
#pragma unroll
            for (int j = 0; j < V; ++j) open[j] = key[j];
            close_groups<V>(a, at, value, key, worst, out);
            // Each value is rounded by 2^-24 of itself and of the one or two that it adds up,
            // which may cancel out: by 2^-22 of the largest of all groups, twice for a
            // difference.  (Infinite ones are not rounded.)
            const uint32_t size1 = best != 0 && fabsf(v1) < kInf ? __float_as_uint(fabsf(v1)) : 0u;
            const uint32_t size2 = fabsf(v2) < kInf ? __float_as_uint(fabsf(v2)) : 0u;
            const float most = __uint_as_float(warp_key_max(max(size1, size2)));
            const float x = key_value(worst), y = key_value(out);
            if ((sums || !by_logits) && out != 0 && !(x - y > 2.0f * near + 0x1p-20f * most)) {
                uint64_t exact, w, o;
                whole = !group_value64<TYPE, V>(a, at, row, lane, m, open, best, second, near, exact);
                uint64_t kept[V];
#pragma unroll
                for (int j = 0; j < V; ++j) kept[j] = open[j];
                close_groups<V>(a, at, exact, kept, w, o);
#pragma unroll
                for (int j = 0; j < V; ++j) key[j] = static_cast<uint32_t>(kept[j]);
            }
        }
        // The experts that may be chosen: those not below the k-th largest of the lanes' largest,
        // by more than values may be off.
        uint32_t bound = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) bound = max(bound, key[j]);
        bound = __shfl_sync(kAll, sort_lanes(bound, lane), a.k - 1);
        if (!by_logits && bound != 0) {
            const float v = key_value(bound);
            // (An infinite one is what it is.)
            if (fabsf(v) < kInf) bound = order_key(v - (near + 0x1p-20f * fabsf(v)));
            whole |= near != near;       // (a softmax with a NaN)
        }
        bound = max(bound, 1u);
        int n = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) n += key[j] >= bound;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, upto, d);
            if (lane >= d) upto += o;
        }
        int count = __shfl_sync(kAll, upto, 31);
        if (count <= 32) {
            int place = upto - n;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] >= bound) {
                    c.key[place] = key[j];
                    c.id[place] = at.first + j;
                    ++place;
                }
            if (lane < 4) c.key[count + lane] = 0;
            __syncwarp();
            const uint32_t mine = lane < count ? c.key[lane] : 0u;
            int rank = 0;
#pragma unroll 1
            for (int i = 0; i < count; i += 4) {
                const uint4 q = *reinterpret_cast<const uint4*>(c.key + i);
                rank += (q.x > mine) + (q.x == mine && i < lane);
                rank += (q.y > mine) + (q.y == mine && i + 1 < lane);
                rank += (q.z > mine) + (q.z == mine && i + 2 < lane);
                rank += (q.w > mine) + (q.w == mine && i + 3 < lane);
            }
            if (lane < count) {
                c.sorted_key[rank] = mine;
                c.sorted_id[rank] = c.id[lane];
            }
        } else {
            count = choose_rounds<V>(key, at.first, a.k, by_logits, near, c, lane);
            whole |= count > 32;
        }
        __syncwarp();
        const uint32_t mine = lane < count ? c.sorted_key[lane] : 0u;
        int32_t id = lane < count ? c.sorted_id[lane] : -1;    // of this lane's choice
        __syncwarp();
        float logit = -kInf;
        if (id >= 0) logit = load_logit<TYPE>(a.logits, row + id);
        if (!by_logits) {
            // Neighbours too close to order, the first of them a choice, or a tie of the last
            // choice (experts with the same logit and bias are ties, in order as they are).
            const float x = key_value(mine), y = __shfl_down_sync(kAll, x, 1);
            const float b = id >= 0 && a.bias ? a.bias[id] : 0.0f;
            const float next_logit = __shfl_down_sync(kAll, logit, 1);
            const float next_b = __shfl_down_sync(kAll, b, 1);
            const bool pair = lane + 1 < count, same = next_logit == logit && next_b == b;
            const bool doubt = pair && !same && !(x - y > near + 0x1p-22f * (fabsf(x) + fabsf(y)));
            // (Lane 31 is no tie: there is one that is not.)
            const int last_tie =
                a.k - 2 + __ffs(~__ballot_sync(kAll, pair && same) >> (a.k - 1));
            if (whole) {
                id = choose64<TYPE, V>(a, row, lane, m, c.sorted_id);
            } else if (__any_sync(kAll, doubt && lane <= last_tie)) {
                id = order64<TYPE>(a, row, lane, m, id, count);
            }
            if (id >= 0) logit = load_logit<TYPE>(a.logits, row + id);
        }
        if (lane >= a.k) id = -1;
        if (id < 0) logit = -kInf;
        float w = 0.0f;
        if (a.renormalize) {
            const float top = warp_max(logit);
            if (softmax) {
                w = id >= 0 ? expf(logit - top) : 0.0f;
            } else if (id >= 0) {
                // sigmoid(l) / e^low with low <= 0: neither factor overflows.
                const float low = fminf(top, 0.0f);
                w = logit <= 0.0f ? expf(logit - low) / (1.0f + expf(logit))
                                  : 1.0f / (1.0f + expf(-logit));
            }
            const float sum = warp_sum(w);
            w = id >= 0 ? a.scale * share(w, sum) : 0.0f;
        } else if (id >= 0) {
            w = a.scale * (softmax ? expf(logit - m) * inverse : 1.0f / (1.0f + expf(-logit)));
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.weights[t * a.k + lane] = w;
        }
    }
}

// dl_i = sum_j dw_j dw_j/dl_i.  With c_j the chosen scores and s_j = c_j / sum c:
//   softmax             d w_j / d l_i = w_j ([i = j] - p_i)     over all experts
//   softmax, normalised d w_j / d l_i = w_j ([i = j] - s_i)     over the chosen
//   sigmoid             d w_j / d l_i = w_j (1 - p_i) [i = j]
//   sigmoid, normalised d w_j / d l_i = w_j (1 - p_i) ([i = j] - s_i)
// A warp has one token: its lanes the chosen experts, whose gradients are stored over
// those that all experts have alike.
template <int TYPE, int V>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_kernel(const __grid_constant__ RouteArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const bool softmax = a.score == kScoreSoftmax;
#pragma unroll 1
    for (uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < static_cast<uint32_t>(a.T);
         t += gridDim.x * kWarps) {
        const int64_t row = static_cast<int64_t>(t) * a.E;
        int32_t id = lane < a.k ? a.ids[t * a.k + lane] : -1;
        float logit = -kInf, dw = 0.0f;
        if (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.E)) {
            logit = load_logit<TYPE>(a.logits, row + id);
            dw = a.scale * a.dweights[t * a.k + lane];
        }
        if (logit == -kInf) id = -1;
        float d = 0.0f;
        if (softmax && !a.renormalize) {
            float l[V], m = -kInf, sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                l[j] = lane + 32 * j < a.E ? load_logit<TYPE>(a.logits, row + lane + 32 * j) : -kInf;
                m = fmaxf(m, l[j]);
            }
            m = warp_max(m);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                l[j] = expf(l[j] - m);
                sum += l[j];
            }
            const float inverse = __fdividef(1.0f, warp_sum(sum));
            const float p = id >= 0 ? expf(logit - m) * inverse : 0.0f;
            d = p * dw;
            const float all = warp_sum(d);
            d -= p * all;
            const float f = m == -kInf ? 0.0f : -all * inverse;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (lane + 32 * j < a.E)
                    store_logit<TYPE>(a.dlogits, row + lane + 32 * j, m == -kInf ? 0.0f : l[j] * f);
        } else {
            for (int32_t e = lane; e < a.E; e += 32) store_logit<TYPE>(a.dlogits, row + e, 0.0f);
            const float p1 = 1.0f / (1.0f + expf(logit));    // 1 - sigmoid
            if (a.renormalize) {
                const float top = warp_max(id >= 0 ? logit : -kInf);
                float s = 0.0f;
                if (softmax) {
                    s = id >= 0 ? expf(logit - top) : 0.0f;
                } else if (id >= 0) {
                    const float low = fminf(top, 0.0f);
                    s = logit <= 0.0f ? expf(logit - low) * p1 : 1.0f / (1.0f + expf(-logit));
                }
                const float sum = warp_sum(s);
                s = id >= 0 ? share(s, sum) : 0.0f;
                const float mean = warp_sum(dw * s);
                d = s * (dw - mean);
                if (!softmax) d *= p1;
            } else {
                d = id >= 0 ? dw * p1 / (1.0f + expf(-logit)) : 0.0f;
            }
        }
        __syncwarp();      // the stores above come first
        if (id >= 0) store_logit<TYPE>(a.dlogits, row + id, d);
    }
}

// CTAs, whose warps take tokens in turn: two waves of four to an SM (8192 x 256 in groups 13.7
// us, one wave 15.1, a CTA for each eight tokens 13.7; 16384 x 122 9.8, 10.2 and 10.4); the
// backward two of eight (5.0 us, one 5.7).
unsigned route_grid(int64_t T, int sms) {
    const int64_t ctas = ceil_div(T, kWarps);
    return static_cast<unsigned>(ctas < 8ll * sms ? ctas : 8ll * sms);
}

template <int TYPE>
cudaError_t launch_typed(const RouteArgs& a, int sms, bool pdl, cudaStream_t stream) {
    const dim3 grid(route_grid(a.T, sms)), block(kWarps * 32);
    const int64_t need = ceil_div(a.group_size, 1 << a.lanes_shift);   // experts of a lane
    auto kernel = need <= 1   ? route_kernel<TYPE, 1>
                  : need <= 2 ? route_kernel<TYPE, 2>
                  : need <= 4 ? route_kernel<TYPE, 4>
                  : need <= 8 ? route_kernel<TYPE, 8>
                  : need <= 16 ? route_kernel<TYPE, 16>
                               : route_kernel<TYPE, 32>;
    return launch_kernel(kernel, grid, block, 0, stream, 1u, pdl, a);
}

template <int TYPE>
cudaError_t launch_backward_typed(const RouteArgs& a, int sms, bool pdl, cudaStream_t stream) {
    const dim3 grid(route_grid(a.T, 2 * sms)), block(kWarps * 32);
    auto kernel = a.E <= 64    ? route_backward_kernel<TYPE, 2>
                  : a.E <= 128 ? route_backward_kernel<TYPE, 4>
                  : a.E <= 256 ? route_backward_kernel<TYPE, 8>
                               : route_backward_kernel<TYPE, 16>;
    return launch_kernel(kernel, grid, block, 0, stream, 1u, pdl, a);
}

}  // namespace

cudaError_t launch_route(RouteArgs a, int type, int sms, bool pdl, cudaStream_t stream) {
    int runs = 1;   // groups, rounded up to a power of two
    a.lanes_shift = 5;
    while (runs < a.groups) {
        runs *= 2;
        --a.lanes_shift;
    }
    a.group_size = a.E / a.groups;
    // Whole lanes of experts in every group, and rows that start at 16 bytes: vector loads.
    const int64_t lanes = 1 << a.lanes_shift, need = ceil_div(a.group_size, lanes);
    int64_t v = 1;
    while (v < need) v *= 2;
    const int64_t bytes = v * (type == kLogitsF32 ? 4 : 2), unit = bytes < 16 ? bytes : 16;
    const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    const bool even = a.group_size == v * lanes && runs == a.groups;
    a.aligned = even && at(a.logits) % unit == 0 && a.E * (bytes / v) % unit == 0;
    a.bias_aligned = even && at(a.bias) % 16 == 0;
    return type == kLogitsF32    ? launch_typed<kLogitsF32>(a, sms, pdl, stream)
           : type == kLogitsBf16 ? launch_typed<kLogitsBf16>(a, sms, pdl, stream)
                                 : launch_typed<kLogitsF16>(a, sms, pdl, stream);
}

cudaError_t launch_route_backward(const RouteArgs& a, int type, int sms, bool pdl,
                                  cudaStream_t stream) {
    return type == kLogitsF32    ? launch_backward_typed<kLogitsF32>(a, sms, pdl, stream)
           : type == kLogitsBf16 ? launch_backward_typed<kLogitsBf16>(a, sms, pdl, stream)
                                 : launch_backward_typed<kLogitsF16>(a, sms, pdl, stream);
}

}  // namespace tmagemm
