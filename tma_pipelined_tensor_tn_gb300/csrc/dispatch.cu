// Rows of tokens by expert, and back: dispatch_rows, combine_rows and its gradients.
//
// Slot t k + j (choice j of token t) gets the row  offsets[expert] + slots of the same
// expert before it: a counting sort, stable and without atomics whose order could
// change it.  The slots are cut into chunks, a CTA each: count_kernel counts each
// chunk's slots by expert, place_kernel adds up the chunks before its own and ranks
// its slots warp by warp.  The rows themselves are copied token by token: each token
// is read once and written to all of its rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"
#include "tile_sched.cuh"

namespace tmagemm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------------ places ----

__global__ void __launch_bounds__(kThreads)
count_kernel(const int32_t* ids, int32_t* counts, int64_t slots, int32_t chunk, int32_t E) {
    __shared__ int32_t n[kMaxExperts];
    grid_launch_dependents();
    for (int e = threadIdx.x; e < E; e += kThreads) n[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t s1 = min(s0 + chunk, slots);
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kThreads) {
        const int32_t e = ids[s];
        if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&n[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads)
        counts[static_cast<int64_t>(blockIdx.x) * E + e] = n[e];
}

__global__ void __launch_bounds__(kThreads)
place_kernel(const int32_t* ids, const int32_t* counts, int32_t* offsets, int32_t* row_of,
             int64_t slots, int32_t chunk, int32_t chunks, int32_t E) {
    __shared__ int32_t first[kMaxExperts];           // row of the chunk's first slot of each
    __shared__ int32_t next[kWarps][kMaxExperts];    // and of each warp's next
    __shared__ int32_t warp_total[kWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    // Two experts of each thread: what all chunks have of them, and those before.
    constexpr int kMine = kMaxExperts / kThreads;
    int32_t total[kMine] = {}, before[kMine] = {};
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int e = static_cast<int>(threadIdx.x) * kMine + i;
        if (e >= E) continue;
        for (int32_t c = 0; c < chunks; ++c) {
            const int32_t n = counts[static_cast<int64_t>(c) * E + e];
            total[i] += n;
            if (c < static_cast<int32_t>(blockIdx.x)) before[i] += n;
        }
    }
    // Sums over the experts before.
    int32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) mine += total[i];
    int32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) warp_total[warp] = upto;
    for (int e = threadIdx.x; e < kWarps * kMaxExperts; e += kThreads) (&next[0][0])[e] = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += warp_total[w];
    int32_t at = upto - mine;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int e = static_cast<int>(threadIdx.x) * kMine + i;
        if (e < E) {
            first[e] = at + before[i];
            if (blockIdx.x == 0) offsets[e] = at;
        }
        at += total[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) offsets[E] = upto;
    // Each warp's slots by expert, then the places.
    const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk + warp * (chunk / kWarps);
    const int64_t s1 = min(s0 + chunk / kWarps, slots);
    auto walk = [&](bool store) {
        for (int64_t s = s0; s < s1; s += 32) {
            const int32_t e = s + lane < s1 ? ids[s + lane] : -1;
            const bool have = static_cast<uint32_t>(e) < static_cast<uint32_t>(E);
            const uint32_t same = __match_any_sync(kAll, have ? e : -1);
            int32_t row = -1;
            if (have) row = next[warp][e] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (have && lane == __ffs(same) - 1) next[warp][e] += __popc(same);
            __syncwarp();
            if (store && s + lane < s1) row_of[s + lane] = row;
        }
    };
    walk(false);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int32_t row = first[e];
        for (int w = 0; w < kWarps; ++w) {
            const int32_t n = next[w][e];
            next[w][e] = row;
            row += n;
        }
    }
    __syncthreads();
    walk(true);
}

// ------------------------------------------------------------------- rows ----
// A warp takes 256 columns (16 bytes a lane) of one token.

struct Piece {
    int64_t t;
    int32_t c;      // this lane's chunk of eight columns
    bool inside;
};
__device__ __forceinline__ Piece piece(int64_t item, int32_t per_token, int32_t C8, int lane) {
    Piece p;
    p.t = item / per_token;
    p.c = static_cast<int32_t>(item % per_token) * 32 + lane;
    p.inside = p.c < C8;
    return p;
}

template <bool BF16, bool QUANTIZE>
__global__ void __launch_bounds__(kThreads)
spread_rows_kernel(const uint4* x, const int32_t* row_of, void* rows, float* scales, int64_t T,
                   int32_t k, int32_t C8, int64_t s_row, int64_t s_blk) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int32_t per_token = (C8 + 31) / 32;
    const int64_t items = T * per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += step) {
        const Piece p = piece(i, per_token, C8, lane);
        const uint4 v = p.inside ? x[p.t * C8 + p.c] : make_uint4(0u, 0u, 0u, 0u);
        const int32_t mine = lane < k ? row_of[p.t * k + lane] : -1;
        if constexpr (QUANTIZE) {
            float f[8];
            unpack8<BF16>(v, f);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, magnitude_bits(f[j]));
            const BlockScale b = block_scale(__uint_as_float(half_warp_max(m)));
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], b.inverse);
            const uint2 q = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]),
                                       e4m3x4(f[4], f[5], f[6], f[7]));
            for (int j = 0; j < k; ++j) {
                const int64_t r = __shfl_sync(kAll, mine, j);
                if (r >= 0 && p.inside) {
                    static_cast<uint2*>(rows)[r * C8 + p.c] = q;
                    if ((lane & 15) == 0) scales[r * s_row + p.c / 16 * s_blk] = b.scale;
                }
            }
        } else {
            for (int j = 0; j < k; ++j) {
                const int64_t r = __shfl_sync(kAll, mine, j);
                if (r >= 0 && p.inside) static_cast<uint4*>(rows)[r * C8 + p.c] = v;
            }
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
combine_kernel(const uint4* rows, const int32_t* row_of, const float* weights, uint4* y, int64_t T,
               int32_t k, int32_t C8, int64_t R) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int32_t per_token = (C8 + 31) / 32;
    const int64_t items = T * per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += step) {
        const Piece p = piece(i, per_token, C8, lane);
        int32_t mine = -1;
        float w = 1.0f;
        if (lane < k) {
            mine = row_of[p.t * k + lane];
            if (mine >= R) mine = -1;
            if (weights) w = weights[p.t * k + lane];
        }
        f32x2 sum[4] = {};
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(kAll, mine, j);
            const float wj = __shfl_sync(kAll, w, j);
            if (r >= 0 && p.inside) {
                f32x2 v[4];
                unpack8<BF16>(rows[r * C8 + p.c], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = fma2(v[e], pack_f32x2(wj, wj), sum[e]);
            }
        }
        if (p.inside) y[p.t * C8 + p.c] = pack8<BF16>(sum);
    }
}

// A warp has one slot: the row of it gets w dy, and the sum of dy times the row is the
// gradient of w.  (dy comes from L1 for all but the first of a token's slots.)
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const uint4* dy, const uint4* rows, const int32_t* row_of,
                        const float* weights, uint4* drows, float* dweights, int64_t slots,
                        int32_t k, int32_t C8, int64_t R) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); s < slots;
         s += step) {
        const int64_t t = s / k, r = row_of[s];
        const bool have = r >= 0 && r < R;
        const float w = weights[s];
        f32x2 dot = 0;
        if (have) {
            for (int32_t c = lane; c < C8; c += 32) {
                f32x2 d[4], v[4];
                unpack8<BF16>(dy[t * C8 + c], d);
                unpack8<BF16>(rows[r * C8 + c], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dot = fma2(d[e], v[e], dot);
                    d[e] = mul2(d[e], pack_f32x2(w, w));
                }
                drows[r * C8 + c] = pack8<BF16>(d);
            }
        }
        float sum = sum2(dot);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        if (lane == 0) dweights[s] = sum;
    }
}

__global__ void no_slots_kernel(int32_t* offsets, int32_t E) {
    grid_launch_dependents();
    grid_dependency_wait();
    for (int e = threadIdx.x; e <= E; e += kThreads) offsets[e] = 0;
}

// Slots of a chunk: 1024, or more where that would be more than 512 chunks (each
// CTA reads the counts of all).
int32_t chunk_slots(int64_t slots) {
    const int64_t n = ceil_div(slots, 512 * 1024) * 1024;
    return static_cast<int32_t>(n < 1024 ? 1024 : n);
}

unsigned grid_for(int64_t items) {
    const int64_t ctas = ceil_div(items, kWarps);
    return static_cast<unsigned>(ctas < (1 << 30) ? ctas : (1 << 30));
}

}  // namespace

int64_t dispatch_workspace(int64_t slots, int64_t E) {
    if (slots == 0) return 0;
    return ceil_div(ceil_div(slots, chunk_slots(slots)) * E * 4, 16) * 16;
}

cudaError_t launch_dispatch(const DispatchArgs& a, bool bf16, bool pdl, cudaStream_t stream) {
    const int64_t slots = a.T * a.k;
    if (slots == 0)
        return launch_kernel(no_slots_kernel, dim3(1), dim3(kThreads), 0, stream, 1u, pdl,
                             a.offsets, a.E);
    const int32_t chunk = chunk_slots(slots);
    const int32_t chunks = static_cast<int32_t>(ceil_div(slots, chunk));
    cudaError_t e = launch_kernel(count_kernel, dim3(chunks), dim3(kThreads), 0, stream, 1u, pdl,
                                  a.ids, a.counts, slots, chunk, a.E);
    if (e != cudaSuccess) return e;
    e = launch_kernel(place_kernel, dim3(chunks), dim3(kThreads), 0, stream, 1u, pdl, a.ids,
                      static_cast<const int32_t*>(a.counts), a.offsets, a.row_of, slots, chunk,
                      chunks, a.E);
    if (e != cudaSuccess) return e;
    auto kernel = a.scales ? (bf16 ? spread_rows_kernel<true, true> : spread_rows_kernel<false, true>)
                           : (bf16 ? spread_rows_kernel<true, false>
                                   : spread_rows_kernel<false, false>);
    return launch_kernel(kernel, dim3(grid_for(a.T * ceil_div(a.C8, 32))), dim3(kThreads), 0,
                         stream, 1u, pdl, a.x, static_cast<const int32_t*>(a.row_of), a.rows,
                         a.scales, a.T, a.k, a.C8, a.s_row, a.s_blk);
}

cudaError_t launch_combine(const CombineArgs& a, bool bf16, bool pdl, cudaStream_t stream) {
    return launch_kernel(bf16 ? combine_kernel<true> : combine_kernel<false>,
                         dim3(grid_for(a.T * ceil_div(a.C8, 32))), dim3(kThreads), 0, stream, 1u,
                         pdl, a.rows, a.row_of, a.weights, a.y, a.T, a.k, a.C8, a.R);
}

cudaError_t launch_combine_backward(const CombineArgs& a, bool bf16, bool pdl,
                                    cudaStream_t stream) {
    return launch_kernel(bf16 ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                         dim3(grid_for(a.T * a.k)), dim3(kThreads), 0, stream, 1u, pdl, a.dy,
                         a.rows, a.row_of, a.weights, a.drows, a.dweights, a.T * a.k, a.k, a.C8,
                         a.R);
}

}  // namespace tmagemm
