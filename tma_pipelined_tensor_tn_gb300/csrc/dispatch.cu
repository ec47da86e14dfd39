// Rows of tokens by expert, and back: dispatch_rows, combine_rows and its gradients.
//
// Slot t k + j (choice j of token t) gets the row  offsets[expert] + slots of the same
// expert before it: a counting sort, stable and without atomics whose order could
// change it.  Up to 256 slots every CTA sorts them all for itself and copies its tokens:
// one launch, whose first loads travel while it sorts.  Up to 131072 slots are sorted by one
// cluster, which holds them in registers; more are cut into chunks, a CTA each: count_kernel
// counts each chunk's slots by expert, place_kernel adds up the chunks before its own and
// ranks its slots warp by warp.  Then the rows are copied by another kernel.  Each token is
// read once and written to all of its rows.
//
// The copies and sums are bound by memory: 4099 x 4096 FP16 tokens to 8 rows of codes each
// 31 us (172 MB), and 5 us before them to place the slots; the sums of 8 rows of 8192 x 2048 BF16
// 46.7 us (6.5 TB/s), their gradients 87 (6.5 TB/s).  Writes alone run slower than copies, at
// 3.8 to 5 TB/s.  16 tokens of 4096 columns to 4 rows each take 3.2 us, their sums 1.8.
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

// Shared memory of the placing of a chunk's slots.
struct Places {
    int32_t total[kMaxExperts], before[kMaxExperts];   // slots of all chunks, of those before
    int32_t next[kWarps][kMaxExperts];                 // row of each warp's next slot
    int32_t warp_total[kWarps];
};

// The lanes of the same expert, N times, a bit of the ids at a time (a match instruction
// takes several times as long); ids outside the experts become E.
template <int N>
__device__ __forceinline__ void same_expert(int32_t (&e)[N], uint32_t (&same)[N], int32_t E) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (static_cast<uint32_t>(e[u]) >= static_cast<uint32_t>(E)) e[u] = E;
        same[u] = kAll;
    }
#pragma unroll 1
    for (int i = 0; E >> i != 0; ++i)
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const bool bit = (e[u] >> i & 1) != 0;
            const uint32_t set = __ballot_sync(kAll, bit);
            same[u] &= bit ? set : ~set;
        }
}

// From totals (and slots in the chunks before) by expert: offsets, and the row of each slot
// of this chunk, slots s0 .. s1 - 1, left in rows[slot].  All threads; `len` is the slots of
// a warp, a multiple of 32.
__device__ __forceinline__ void place(Places& m, const int32_t* ids, int32_t* offsets,
                                      int32_t* rows, int64_t s0, int64_t s1, int32_t len,
                                      int32_t E) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    // First rows: sums over the experts before, of two experts a thread.
    constexpr int kMine = kMaxExperts / kThreads;
    const int e0 = static_cast<int>(threadIdx.x) * kMine;
    int32_t n[kMine], mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        n[i] = e0 + i < E ? m.total[e0 + i] : 0;
        mine += n[i];
    }
    int32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) m.warp_total[warp] = upto;
    for (int e = lane; e < E; e += 32) m.next[warp][e] = 0;
    __syncwarp();
    // Each slot's place among its warp's slots of the same expert, four times 32 slots whose
    // ids are read together.
    const int64_t w0 = s0 + static_cast<int64_t>(warp) * len, w1 = min(w0 + len, s1);
    constexpr int kAhead = 4;
    const auto expert = [&](int64_t s) { return s < w1 ? ids[s] : -1; };
#pragma unroll 1
    for (int64_t s = w0 + lane; s - lane < w1; s += 32 * kAhead) {
        int32_t e[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) e[u] = expert(s + 32 * u);
        uint32_t same[kAhead];
        same_expert(e, same, E);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s - lane + 32 * u >= w1) break;
            const bool have = e[u] < E;
            int32_t row = 0;
            if (have) row = m.next[warp][e[u]] + __popc(same[u] & ((1u << lane) - 1u));
            __syncwarp();
            if (have && lane == __ffs(same[u]) - 1) m.next[warp][e[u]] = row + __popc(same[u]);
            __syncwarp();
            if (s + 32 * u < w1) rows[s + 32 * u] = row;
        }
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += m.warp_total[w];
    int32_t at = upto - mine;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (e0 + i < E) {
            if (offsets) offsets[e0 + i] = at;
            // The first rows of the expert's slots of each warp.
            int32_t row = at + m.before[e0 + i];
            for (int w = 0; w < kWarps; ++w) {
                const int32_t c = m.next[w][e0 + i];
                m.next[w][e0 + i] = row;
                row += c;
            }
        }
        at += n[i];
    }
    if (offsets && threadIdx.x == kThreads - 1) offsets[E] = upto;
    __syncthreads();
#pragma unroll 4
    for (int64_t s = w0 + lane; s < w1; s += 32) {
        const int32_t e = ids[s];
        const bool have = static_cast<uint32_t>(e) < static_cast<uint32_t>(E);
        rows[s] = have ? rows[s] + m.next[warp][e] : -1;
    }
}

__global__ void __launch_bounds__(kThreads)
place_kernel(const int32_t* ids, const int32_t* counts, int32_t* offsets, int32_t* row_of,
             int64_t slots, int32_t chunk, int32_t chunks, int32_t E) {
    __shared__ Places m;
    grid_launch_dependents();
    for (int e = threadIdx.x; e < E; e += kThreads) m.total[e] = m.before[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    const int32_t all = chunks * E, mine = static_cast<int32_t>(blockIdx.x) * E;
#pragma unroll 4
    for (int32_t i = threadIdx.x; i < all; i += kThreads) {
        const int32_t n = counts[i];
        if (n != 0) {
            atomicAdd(&m.total[i % E], n);
            if (i < mine) atomicAdd(&m.before[i % E], n);
        }
    }
    __syncthreads();
    const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
    place(m, ids, blockIdx.x == 0 ? offsets : nullptr, row_of, s0, min(s0 + chunk, slots),
          chunk / kWarps, E);
}

// All of it in one launch of one cluster: a warp has BATCHES times 32 slots, ranked in
// registers; the counts of the CTAs meet through distributed shared memory.  Every batch
// costs its ballots whether it has slots or not (0.5 to 0.7 us), so that each number of
// slots runs the form with the fewest that hold it.
// (64 columns, with the copies: 8192 slots 4.7 us, in chunks 6.9; 32792 8.1 and 11.4; 131072
// 17.0 and 18.9.)
// (64 experts: 8192 slots in one batch 4.6 us, in two 5.2; 16384 in two 5.4, in three 5.9; 24576
// in three 6.6, in five 7.8; 32768 and 40960 in five 8.0, in eight 10.0; 49152 in eight 10.0,
// in sixteen 14.0; 65536 10.6 and 14.7.)
constexpr int kClusterSlots = 131072;
constexpr int kClusterCtas = 8, kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;
template <int BATCHES>
__global__ void __launch_bounds__(kClusterThreads)
place_cluster_kernel(const int32_t* ids, int32_t* offsets, int32_t* row_of, int32_t slots,
                     int32_t E) {
    __shared__ uint16_t next[kClusterWarps][kMaxExperts];   // slots of each warp, then before it
    __shared__ int32_t count[kMaxExperts], first[kMaxExperts], warp_total[kMaxExperts / 32];
    grid_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    for (int e = lane; e < E; e += 32) next[warp][e] = 0;
    __syncwarp();
    grid_dependency_wait();
    const int32_t s0 =
        (static_cast<int32_t>(rank) * kClusterWarps + warp) * (32 * BATCHES) + lane;
    int32_t e[BATCHES];
#pragma unroll
    for (int b = 0; b < BATCHES; ++b) e[b] = s0 + 32 * b < slots ? ids[s0 + 32 * b] : -1;
    // The expert and the slots of this warp before it with the same, in the two halves.
    uint32_t place[BATCHES];
    uint32_t same[BATCHES];
    same_expert(e, same, E);
#pragma unroll
    for (int b = 0; b < BATCHES; ++b) {
        const bool have = e[b] < E;
        uint32_t before = 0;
        if (have) before = next[warp][e[b]] + __popc(same[b] & ((1u << lane) - 1u));
        __syncwarp();
        if (have && lane == __ffs(same[b]) - 1)
            next[warp][e[b]] = static_cast<uint16_t>(before + __popc(same[b]));
        __syncwarp();
        place[b] = have ? static_cast<uint32_t>(e[b]) << 16 | before : ~0u;
    }
    __syncthreads();
    if (tid < E) {
        uint32_t sum = 0;
#pragma unroll 16
        for (int w = 0; w < kClusterWarps; ++w) {
            const uint32_t n = next[w][tid];
            next[w][tid] = static_cast<uint16_t>(sum);
            sum += n;
        }
        count[tid] = static_cast<int32_t>(sum);
    }
    __syncwarp();
    cluster_sync();
    int32_t total = 0, before = 0;
    if (tid < E) {
#pragma unroll
        for (uint32_t q = 0; q < kClusterCtas; ++q) {
            int32_t n;
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(n)
                         : "r"(map_to_rank(smem_u32(&count[tid]), q))
                         : "memory");
            total += n;
            if (q < rank) before += n;
        }
    }
    __syncwarp();
    cluster_arrive_release();             // this CTA has read its peers' counts
    int32_t upto = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31 && warp < kMaxExperts / 32) warp_total[warp] = upto;
    __syncthreads();
    if (tid < E) {
        for (int w = 0; w < warp; ++w) upto += warp_total[w];
        first[tid] = upto - total + before;
        if (rank == 0) {
            offsets[tid] = upto - total;
            if (tid == E - 1) offsets[E] = upto;
        }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < BATCHES; ++b) {
        const int32_t at = static_cast<int32_t>(place[b] >> 16);
        if (s0 + 32 * b < slots)
            row_of[s0 + 32 * b] =
                place[b] == ~0u ? -1
                                : first[at] + next[warp][at] + static_cast<int32_t>(place[b] & 0xffffu);
    }
    __syncwarp();
    cluster_wait_acquire();
}

// ------------------------------------------------------------------- rows ----
// A warp takes 256 VECS columns (16 bytes a lane, VECS times) of one token.

// A row's part, which nothing reads again.
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

struct Piece {
    int64_t t;
    int32_t c;      // this lane's first chunk of eight columns; the next are 32 further on
};
template <int VECS>
__device__ __forceinline__ Piece piece(int64_t item, int32_t per_token, int lane) {
    Piece p;
    p.t = item / per_token;
    p.c = static_cast<int32_t>(item - p.t * per_token) * (32 * VECS) + lane;
    return p;
}

template <int VECS>
__device__ __forceinline__ void load_piece(const uint4* x, const Piece& p, int32_t C8,
                                           uint4 (&v)[VECS]) {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
        v[i] = p.c + 32 * i < C8 ? x[p.t * C8 + p.c + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
}

struct Spread {
    void* rows;
    float* scales;
    int64_t s_row, s_blk;
};

// A piece to the rows of its token: lane j's `mine` is the row of choice j, or -1.
template <bool BF16, bool QUANTIZE, int VECS>
__device__ __forceinline__ void spread(const Spread& to, const Piece& p, int32_t C8, int32_t k,
                                       int lane, int32_t mine, const uint4 (&v)[VECS]) {
    if constexpr (QUANTIZE) {
        uint2 q[VECS];
        float scale[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            float f[8];
            unpack8<BF16>(v[i], f);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, magnitude_bits(f[j]));
            const BlockScale b = block_scale(__uint_as_float(half_warp_max(m)));
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], b.inverse);
            q[i] = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
            scale[i] = b.scale;
        }
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(kAll, mine, j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int32_t c = p.c + 32 * i;
                if (c < C8) {
                    static_cast<uint2*>(to.rows)[r * C8 + c] = q[i];
                    if ((lane & 15) == 0) to.scales[r * to.s_row + c / 16 * to.s_blk] = scale[i];
                }
            }
        }
    } else {
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(kAll, mine, j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                if (p.c + 32 * i < C8) static_cast<uint4*>(to.rows)[r * C8 + p.c + 32 * i] = v[i];
        }
    }
}

// All of it for up to kSmallSlots slots.
// (4096 columns, 64 experts: 64 slots 3.6 us, placed by a launch before 4.1; 256 slots 4.2 and
// 4.1, 768 7.3 and 4.8.)
constexpr int kSmallSlots = 256;
template <bool BF16, bool QUANTIZE>
__global__ void __launch_bounds__(kThreads)
small_dispatch_kernel(const uint4* x, const int32_t* ids, int32_t* offsets, int32_t* row_of,
                      const Spread to, int32_t T, int32_t k, int32_t E, int32_t C8) {
    __shared__ Places m;
    __shared__ int32_t row[kSmallSlots];
    grid_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int32_t per_token = (C8 + 31) / 32, items = T * per_token, slots = T * k;
    for (int e = threadIdx.x; e < E; e += kThreads) m.total[e] = m.before[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    int32_t i = static_cast<int32_t>(blockIdx.x) * kWarps + static_cast<int32_t>(threadIdx.x >> 5);
    uint4 v[1] = {};
    if (i < items) load_piece<1>(x, piece<1>(i, per_token, lane), C8, v);
    for (int32_t s = threadIdx.x; s < slots; s += kThreads) {
        const int32_t e = ids[s];
        if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&m.total[e], 1);
    }
    __syncthreads();
    place(m, ids, blockIdx.x == 0 ? offsets : nullptr, row, 0, slots,
          (slots + kThreads - 1) / kThreads * 32, E);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int32_t s = threadIdx.x; s < slots; s += kThreads) row_of[s] = row[s];
    const int32_t step = static_cast<int32_t>(gridDim.x) * kWarps;
    while (i < items) {
        const Piece p = piece<1>(i, per_token, lane);
        spread<BF16, QUANTIZE, 1>(to, p, C8, k, lane, lane < k ? row[p.t * k + lane] : -1, v);
        i += step;
        if (i < items) load_piece<1>(x, piece<1>(i, per_token, lane), C8, v);
    }
}

template <bool BF16, bool QUANTIZE, int VECS>
__global__ void __launch_bounds__(kThreads)
spread_rows_kernel(const uint4* x, const int32_t* row_of, const Spread to, int64_t T, int32_t k,
                   int32_t C8) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int32_t per_token = (C8 + 32 * VECS - 1) / (32 * VECS);
    const int64_t items = T * per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < items;
         i += step) {
        const Piece p = piece<VECS>(i, per_token, lane);
        uint4 v[VECS];
        load_piece<VECS>(x, p, C8, v);
        const int32_t mine = lane < k ? row_of[p.t * k + lane] : -1;
        spread<BF16, QUANTIZE, VECS>(to, p, C8, k, lane, mine, v);
    }
}

// Sums in the order of the choices; the loads of four choices, or of two with more columns,
// are in flight at once.
template <bool BF16, int VECS>
__global__ void __launch_bounds__(kThreads, 4)
combine_kernel(const uint4* rows, const int32_t* row_of, const float* weights, uint4* y, int64_t T,
               int32_t k, int32_t C8, int64_t R) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int kAhead = VECS == 1 ? 4 : 2;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int32_t per_token = (C8 + 32 * VECS - 1) / (32 * VECS);
    const int64_t items = T * per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    // The rows and weights of a token are read while the item before it is added up.
    int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    Piece next{};
    int32_t next_row = -1;
    float next_w = 1.0f;
    auto fetch = [&](int64_t item) {
        next = piece<VECS>(item, per_token, lane);
        if (lane < k) {
            next_row = row_of[next.t * k + lane];
            if (weights) next_w = weights[next.t * k + lane];
        }
    };
    if (i < items) fetch(i);
#pragma unroll 1
    for (; i < items; i += step) {
        const Piece p = next;
        const int32_t mine = next_row < R ? next_row : -1;
        const float w = next_w;
        if (i + step < items) fetch(i + step);
        f32x2 sum[VECS][4] = {};
#pragma unroll 1
        for (int j0 = 0; j0 < k; j0 += kAhead) {
            uint4 v[kAhead][VECS];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                // (Past k: a lane without a row.)
                const int32_t r = __shfl_sync(kAll, mine, (j0 + u) & 31);
                const bool have = j0 + u < k && r >= 0;
                const uint4* from = rows + static_cast<int64_t>(r) * C8 + p.c;
#pragma unroll
                for (int q = 0; q < VECS; ++q)
                    v[u][q] = have && p.c + 32 * q < C8 ? ld_row(from + 32 * q) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int j = (j0 + u) & 31;
                const float wj = __shfl_sync(kAll, w, j);
                // (Choices without a row add nothing, whatever their weight.)
                if (j0 + u >= k || __shfl_sync(kAll, mine, j) < 0) continue;
#pragma unroll
                for (int q = 0; q < VECS; ++q) {
                    f32x2 f[4];
                    unpack8<BF16>(v[u][q], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[q][e] = fma2(f[e], pack_f32x2(wj, wj), sum[q][e]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < VECS; ++q)
            if (p.c + 32 * q < C8) y[p.t * C8 + p.c + 32 * q] = pack8<BF16>(sum[q]);
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
            const uint4 *from = rows + r * C8, *grad = dy + t * C8;
            uint4* to = drows + r * C8;
            constexpr int kAhead = 4;
            for (int32_t c0 = lane; c0 < C8; c0 += 32 * kAhead) {
                uint4 d[kAhead], v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (c0 + 32 * u < C8) {
                        v[u] = from[c0 + 32 * u];
                        d[u] = grad[c0 + 32 * u];
                    }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (c0 + 32 * u < C8) {
                        f32x2 g[4], f[4];
                        unpack8<BF16>(d[u], g);
                        unpack8<BF16>(v[u], f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dot = fma2(g[e], f[e], dot);
                            g[e] = mul2(g[e], pack_f32x2(w, w));
                        }
                        to[c0 + 32 * u] = pack8<BF16>(g);
                    }
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

cudaError_t launch_places(const DispatchArgs& a, int64_t slots, bool pdl, cudaStream_t stream) {
    if (slots <= kClusterSlots) {
        const int32_t batches =
            static_cast<int32_t>(ceil_div(slots, kClusterCtas * kClusterThreads));
        auto kernel = batches <= 1   ? place_cluster_kernel<1>
                      : batches <= 2 ? place_cluster_kernel<2>
                      : batches <= 3 ? place_cluster_kernel<3>
                      : batches <= 5 ? place_cluster_kernel<5>
                      : batches <= 8 ? place_cluster_kernel<8>
                                     : place_cluster_kernel<16>;
        return launch_kernel(kernel, dim3(kClusterCtas), dim3(kClusterThreads), 0, stream,
                             static_cast<unsigned>(kClusterCtas), pdl, a.ids, a.offsets, a.row_of,
                             static_cast<int32_t>(slots), a.E);
    }
    const int32_t chunk = chunk_slots(slots);
    const int32_t chunks = static_cast<int32_t>(ceil_div(slots, chunk));
    if (cudaError_t e = launch_kernel(count_kernel, dim3(chunks), dim3(kThreads), 0, stream, 1u,
                                      pdl, a.ids, a.counts, slots, chunk, a.E))
        return e;
    return launch_kernel(place_kernel, dim3(chunks), dim3(kThreads), 0, stream, 1u, pdl, a.ids,
                         static_cast<const int32_t*>(a.counts), a.offsets, a.row_of, slots, chunk,
                         chunks, a.E);
}

template <bool BF16, bool QUANTIZE>
cudaError_t launch_dispatch_typed(const DispatchArgs& a, int sms, bool pdl, cudaStream_t stream) {
    const int64_t slots = a.T * a.k;
    const Spread to{a.rows, a.scales, a.s_row, a.s_blk};
    if (slots <= kSmallSlots) {
        const int64_t ctas = ceil_div(a.T * ceil_div(a.C8, 32), kWarps);
        return launch_kernel(small_dispatch_kernel<BF16, QUANTIZE>,
                             dim3(static_cast<unsigned>(ctas < 2ll * sms ? ctas : 2ll * sms)),
                             dim3(kThreads), 0, stream, 1u, pdl, a.x, a.ids, a.offsets, a.row_of,
                             to, static_cast<int32_t>(a.T), a.k, a.E, a.C8);
    }
    if (cudaError_t e = launch_places(a, slots, pdl, stream)) return e;
    constexpr int kVecs = 4;
    const bool wide = a.T * ceil_div(a.C8, 32 * kVecs) >= 16ll * sms;
    auto kernel = wide ? spread_rows_kernel<BF16, QUANTIZE, kVecs>
                       : spread_rows_kernel<BF16, QUANTIZE, 1>;
    return launch_kernel(kernel, dim3(grid_for(a.T * ceil_div(a.C8, wide ? 32 * kVecs : 32))),
                         dim3(kThreads), 0, stream, 1u, pdl, a.x,
                         static_cast<const int32_t*>(a.row_of), to, a.T, a.k, a.C8);
}

}  // namespace

int64_t dispatch_workspace(int64_t slots, int64_t E) {
    if (slots <= kClusterSlots) return 0;
    return ceil_div(ceil_div(slots, chunk_slots(slots)) * E * 4, 16) * 16;
}

cudaError_t launch_dispatch(const DispatchArgs& a, bool bf16, int sms, bool pdl,
                            cudaStream_t stream) {
    if (a.T == 0)
        return launch_kernel(no_slots_kernel, dim3(1), dim3(kThreads), 0, stream, 1u, pdl,
                             a.offsets, a.E);
    if (a.scales)
        return bf16 ? launch_dispatch_typed<true, true>(a, sms, pdl, stream)
                    : launch_dispatch_typed<false, true>(a, sms, pdl, stream);
    return bf16 ? launch_dispatch_typed<true, false>(a, sms, pdl, stream)
                : launch_dispatch_typed<false, false>(a, sms, pdl, stream);
}

cudaError_t launch_combine(const CombineArgs& a, bool bf16, int sms, bool pdl,
                           cudaStream_t stream) {
    // Four loads of a lane: of four choices, or of two to twice the columns (where that leaves
    // no SMs idle).
    const bool few = a.T * ceil_div(a.C8, 64) < 32ll * sms;
    const int vecs = few || a.k > 2 ? 1 : 2;
    auto kernel = vecs == 1 ? (bf16 ? combine_kernel<true, 1> : combine_kernel<false, 1>)
                            : (bf16 ? combine_kernel<true, 2> : combine_kernel<false, 2>);
    const int64_t ctas = ceil_div(a.T * ceil_div(a.C8, 32 * vecs), kWarps);
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas < 16ll * sms ? ctas : 16ll * sms)),
                         dim3(kThreads), 0, stream, 1u, pdl, a.rows, a.row_of, a.weights, a.y, a.T,
                         a.k, a.C8, a.R);
}

cudaError_t launch_combine_backward(const CombineArgs& a, bool bf16, bool pdl,
                                    cudaStream_t stream) {
    return launch_kernel(bf16 ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                         dim3(grid_for(a.T * a.k)), dim3(kThreads), 0, stream, 1u, pdl, a.dy,
                         a.rows, a.row_of, a.weights, a.drows, a.dweights, a.T * a.k, a.k, a.C8,
                         a.R);
}

}  // namespace tmagemm
