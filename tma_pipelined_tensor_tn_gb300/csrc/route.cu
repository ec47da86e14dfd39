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
// The choice follows exact arithmetic.  Without a bias (and with groups valued by one
// expert) it is made on the logits themselves, which order as their scores do.
// Otherwise v is computed in FP32 with the error bound below, and a token whose
// choice hangs on two values closer than that is decided again in FP64.
//
// Renormalised weights need no sum over all experts: the largest chosen logit is
// taken out of the quotient, so that scores that FP32 cannot hold cancel.
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
    const int32_t size = a.E / a.groups;
    const int group = lane / a.group_lanes, part = lane % a.group_lanes;
    const int32_t left = group < a.groups ? size - part * V : 0;
    return {group * size + part * V, left < 0 ? 0 : left < V ? left : V, group, a.group_lanes};
}

// Closes the groups that are not among the top_groups best ones: keys of their experts
// become 0.  `key` of type K orders like the values of type F.  Returns the distance of
// the worst group kept from the best one closed.
template <int V, class K, class F>
__device__ __forceinline__ F close_groups(const RouteArgs& a, const LaneExperts& at, K (&key)[V]) {
    // The two best of the lane, then of the group's lanes.
    K best = 0, second = 0;
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
    F value = key_value(best);
    if (a.group_sum == 2 && second != 0) value += key_value(second);
    K mine = best == 0 ? 0 : order_key(value);
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
        const K other = __shfl_sync(kAll, mine, g * at.lanes);
        ahead += other > mine || (other == mine && g < at.group);
    }
    const bool keep = ahead < a.top_groups;
    if (!keep) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 0;
    }
    const K worst = ~warp_key_max(keep && at.group < a.groups ? static_cast<K>(~mine) : K(0));
    const K out = warp_key_max(keep || at.group >= a.groups ? K(0) : mine);
    return out == 0 ? static_cast<F>(kInf) : key_value(worst) - key_value(out);
}

// The largest key of the warp, taken out of its lane: the lane that held it (and, there,
// the register in `at`).
template <int V, class K>
__device__ __forceinline__ int take_largest(K (&key)[V], K& mine, K& largest, int lane, int& at) {
    largest = warp_key_max(mine);
    const int winner = __ffs(__ballot_sync(kAll, mine == largest)) - 1;
    if (lane == winner) {
        bool found = false;
        K next = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!found && key[j] == largest) {
                found = true;
                at = j;
                key[j] = 0;
            }
            next = max(next, key[j]);
        }
        mine = next;
    }
    return winner;
}

// The choice of one token in FP64, for the few that FP32 cannot decide: lane j gets
// the id of choice j (-1: no expert is left).
template <int TYPE, int V>
__device__ __noinline__ int32_t choose64(const RouteArgs& a, int64_t row, int lane) {
    const LaneExperts at = lane_experts<V>(a, lane);
    double v[V];
    float m = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float l = j < at.count ? load_logit<TYPE>(a.logits, row + at.first + j) : -kInf;
        v[j] = l;
        m = fmaxf(m, l);
    }
    m = warp_max(m);
    uint64_t key[V];
    double sum = 0.0;
    if (a.score == kScoreSoftmax) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum += exp(v[j] - m);
        sum = warp_sum(sum);
    }
    uint64_t mine = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool open = j < at.count && v[j] != -kInf;
        double p = a.score == kScoreSoftmax ? exp(v[j] - m) / sum : 1.0 / (1.0 + exp(-v[j]));
        if (a.bias && j < at.count) p += a.bias[at.first + j];
        if (sum != sum) p = v[j];
        key[j] = open ? order_key(p) : 0;
    }
    if (a.groups > 1) close_groups<V, uint64_t, double>(a, at, key);
#pragma unroll
    for (int j = 0; j < V; ++j) mine = max(mine, key[j]);
    int32_t id = -1;
    for (int c = 0; c < a.k; ++c) {
        uint64_t largest;
        int j = 0;
        const int winner = take_largest<V>(key, mine, largest, lane, j);
        const int32_t who = __shfl_sync(kAll, at.first + j, winner);
        if (lane == c && largest != 0) id = who;
    }
    return id;
}

template <int TYPE, int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int64_t row = t * a.E;
    const LaneExperts at = lane_experts<V>(a, lane);
    float l[V];
    float m = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        l[j] = j < at.count ? load_logit<TYPE>(a.logits, row + at.first + j) : -kInf;
        m = fmaxf(m, l[j]);
    }
    const bool softmax = a.score == kScoreSoftmax;
    // Scores order as logits do.
    const bool by_logits = !a.bias && (a.groups == 1 || a.group_sum == 1);
    float inverse = 1.0f;   // of the sum over all experts
    if (softmax && (!by_logits || !a.renormalize)) {
        m = warp_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += expf(l[j] - m);   // (no experts: NaN, not used)
        inverse = 1.0f / warp_sum(sum);
    }
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float v = l[j];
        if (!by_logits) {
            v = softmax ? expf(l[j] - m) * inverse : 1.0f / (1.0f + expf(-l[j]));
            if (a.bias && j < at.count) v += a.bias[at.first + j];
            // (All scores are NaN: the logits, so that the one that made them so is chosen.)
            if (inverse != inverse) v = l[j];
        }
        key[j] = l[j] == -kInf ? 0u : order_key(v);
    }
    // How far two values of v may be off together: a score of at most p by 2^-19 p
    // (its exponent's argument, expf, a sum of up to 512 terms in a tree of 16 and 5
    // levels, the quotient: 25 roundings; sigmoid: 4, 2^-21), the addition of the bias by
    // 2^-24 of v.
    const float near = softmax ? 0x1p-18f * inverse : 0x1p-20f;
    bool decided = true;
    if (a.groups > 1) {
        const float gap = close_groups<V, uint32_t, float>(a, at, key);
        if (!by_logits) {
            float big = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] != 0) big = fmaxf(big, fabsf(key_value(key[j])));
            decided = gap > 2.0f * near + 0x1p-20f * warp_max(big);
        }
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) mine = max(mine, key[j]);
    int32_t id = -1;         // of this lane's choice
    float logit = -kInf;
    uint32_t before = 0;
    int32_t who_before = 0;
    // (One more than k where the last has to be told from the first that is not chosen.)
    const int rounds = by_logits ? a.k : a.k + 1;
    for (int c = 0; c < rounds; ++c) {
        uint32_t largest;
        int j = 0;
        const int winner = take_largest<V>(key, mine, largest, lane, j);
        const int32_t who = __shfl_sync(kAll, at.first + j, winner);
        if (lane == c && largest != 0) id = who;
        if (!by_logits && c > 0 && largest != 0) {
            const float x = key_value(before), y = key_value(largest);
            if (!(x - y > near + 0x1p-22f * (fabsf(x) + fabsf(y)))) {
                // Experts with the same logit and bias have the same value: a tie.
                const float u = load_logit<TYPE>(a.logits, row + who_before);
                const float w = load_logit<TYPE>(a.logits, row + who);
                if (!(u == w && (!a.bias || a.bias[who_before] == a.bias[who]))) decided = false;
            }
        }
        before = largest;
        who_before = who;
    }
    if (lane >= a.k) id = -1;
    if (!decided) id = choose64<TYPE, V>(a, row, lane);
    if (id >= 0) logit = load_logit<TYPE>(a.logits, row + id);
    float w = 0.0f;
    if (a.renormalize) {
        float top = id >= 0 ? logit : -kInf;
        top = warp_max(top);
        if (softmax) {
            w = id >= 0 ? expf(logit - top) : 0.0f;
        } else if (id >= 0) {
            // sigmoid(l) / e^low with low <= 0: neither factor overflows.
            const float low = fminf(top, 0.0f);
            w = logit <= 0.0f ? expf(logit - low) / (1.0f + expf(logit))
                              : 1.0f / (1.0f + expf(-logit));
        }
        const float sum = warp_sum(w);
        w = id >= 0 ? a.scale * (w / sum) : 0.0f;
    } else if (id >= 0) {
        w = a.scale * (softmax ? expf(logit - m) * inverse : 1.0f / (1.0f + expf(-logit)));
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = w;
    }
}

// dl_i = sum_j dw_j dw_j/dl_i.  With c_j the chosen scores and s_j = c_j / sum c:
//   softmax             d w_j / d l_i = w_j ([i = j] - p_i)     over all experts
//   softmax, normalised d w_j / d l_i = w_j ([i = j] - s_i)     over the chosen
//   sigmoid             d w_j / d l_i = w_j (1 - p_i) [i = j]
//   sigmoid, normalised d w_j / d l_i = w_j (1 - p_i) ([i = j] - s_i)
// A warp has one token: its lanes the chosen experts, whose gradients go through a row
// in shared memory to their places.
template <int TYPE>
__global__ void __launch_bounds__(kWarps * 32)
route_backward_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ float rows[];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.E;
    float* out = rows + warp * a.E;
    const bool softmax = a.score == kScoreSoftmax;
    int32_t id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    float logit = -kInf, dw = 0.0f;
    if (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.E)) {
        logit = load_logit<TYPE>(a.logits, row + id);
        dw = a.scale * a.dweights[t * a.k + lane];
    }
    if (logit == -kInf) id = -1;
    float d = 0.0f;
    if (softmax && !a.renormalize) {
        float m = -kInf, sum = 0.0f;
        for (int32_t e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit<TYPE>(a.logits, row + e));
        m = warp_max(m);
        for (int32_t e = lane; e < a.E; e += 32) {
            out[e] = expf(load_logit<TYPE>(a.logits, row + e) - m);
            sum += out[e];
        }
        sum = warp_sum(sum);
        d = id >= 0 ? dw * (expf(logit - m) / sum) : 0.0f;
        const float all = warp_sum(d);
        const float f = m == -kInf ? 0.0f : all / sum;
        for (int32_t e = lane; e < a.E; e += 32) out[e] = m == -kInf ? 0.0f : -out[e] * f;
    } else {
        for (int32_t e = lane; e < a.E; e += 32) out[e] = 0.0f;
        const float p1 = 1.0f / (1.0f + expf(logit));    // 1 - sigmoid
        if (a.renormalize) {
            const float top = warp_max(logit);
            float s = 0.0f;
            if (softmax) {
                s = id >= 0 ? expf(logit - top) : 0.0f;
            } else if (id >= 0) {
                const float low = fminf(top, 0.0f);
                s = logit <= 0.0f ? expf(logit - low) * p1 : 1.0f / (1.0f + expf(-logit));
            }
            const float sum = warp_sum(s);
            s = id >= 0 ? s / sum : 0.0f;
            const float mean = warp_sum(dw * s);
            d = s * (dw - mean);
            if (!softmax) d *= p1;
        } else {
            d = id >= 0 ? dw * p1 / (1.0f + expf(-logit)) : 0.0f;
        }
    }
    __syncwarp();
    if (id >= 0) atomicAdd(out + id, d);
    __syncwarp();
    for (int32_t e = lane; e < a.E; e += 32) store_logit<TYPE>(a.dlogits, row + e, out[e]);
}

template <int TYPE>
cudaError_t launch_typed(const RouteArgs& a, bool pdl, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.T, kWarps))), block(kWarps * 32);
    const int64_t need = ceil_div(a.E / a.groups, a.group_lanes);   // experts of a lane
    auto kernel = need <= 1   ? route_kernel<TYPE, 1>
                  : need <= 2 ? route_kernel<TYPE, 2>
                  : need <= 4 ? route_kernel<TYPE, 4>
                  : need <= 8 ? route_kernel<TYPE, 8>
                  : need <= 16 ? route_kernel<TYPE, 16>
                               : route_kernel<TYPE, 32>;
    return launch_kernel(kernel, grid, block, 0, stream, 1u, pdl, a);
}

template <int TYPE>
cudaError_t launch_backward_typed(const RouteArgs& a, bool pdl, cudaStream_t stream) {
    return launch_kernel(route_backward_kernel<TYPE>,
                         dim3(static_cast<unsigned>(ceil_div(a.T, kWarps))), dim3(kWarps * 32),
                         static_cast<size_t>(kWarps) * a.E * sizeof(float), stream, 1u, pdl, a);
}

}  // namespace

cudaError_t launch_route(RouteArgs a, int type, bool pdl, cudaStream_t stream) {
    int runs = 1;   // groups, rounded up to a power of two
    while (runs < a.groups) runs *= 2;
    a.group_lanes = 32 / runs;
    return type == kLogitsF32    ? launch_typed<kLogitsF32>(a, pdl, stream)
           : type == kLogitsBf16 ? launch_typed<kLogitsBf16>(a, pdl, stream)
                                 : launch_typed<kLogitsF16>(a, pdl, stream);
}

cudaError_t launch_route_backward(const RouteArgs& a, int type, bool pdl, cudaStream_t stream) {
    return type == kLogitsF32    ? launch_backward_typed<kLogitsF32>(a, pdl, stream)
           : type == kLogitsBf16 ? launch_backward_typed<kLogitsBf16>(a, pdl, stream)
                                 : launch_backward_typed<kLogitsF16>(a, pdl, stream);
}

}  // namespace tmagemm
