// gemm_fp8 for a few rows of activations (1 <= M <= 16): the decode step, bound
// by reading the weights once.  As in the 16-bit few-row kernel, the weights go
// from HBM straight into register fragments of mma.sync (here m16n8k32 on e4m3
// operands, FP32 sums), 16 bytes per load, with no shared-memory staging; the
// CTAs of a cluster split K and add their FP32 partial tiles in slice order
// through distributed shared memory.  No workspace, one launch, deterministic.
//
// Fragment layout.  In m16n8k32 a thread with g = lane / 4 and t = lane % 4
// holds A(row g and g + 8; k slots 4t .. 4t+3 and 16+4t .. 16+4t+3) and B(the
// same k slots; column g).  Any map from slots to physical k that is the same
// for A and B gives the same sum: a step of two MMAs covers 64 physical k, and
// thread (g, t) takes the 16 consecutive k from 16 t of weight rows g and
// g + 8 and of token row g (bytes 0..7 for the first MMA, 8..15 for the
// second): one 16-byte load each, the four threads of a group reading 64
// contiguous bytes of each row.
//
// Scales.  A 128-k block is two steps; its product is made in accumulators of
// its own and added to the running sums times SA[token] * SB: two products and
// four multiply-adds per block and 8 tokens.
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"
#include "tile_sched.cuh"

namespace tmagemm {

namespace {

constexpr int kWarps = 4;              // warps per CTA, 16 weight rows each
constexpr int kRows = 16 * kWarps;     // weight rows per CTA and per cluster
constexpr int kMaxM = 16;

__device__ __forceinline__ uint4 ld_weights(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// c += A * B for one m16n8k32 tile of e4m3 operands.
__device__ __forceinline__ void mma_m16n8k32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// What a thread holds of U consecutive 128-k blocks: weights, tokens, scales.
template <int NT, int U>
struct Group {
    uint4 wa[U][2], wb[U][2], x[U][2][NT];
    float sa[U][NT][2], sb[U];
};

// A thread's rows and scales; null rows (past N or M) read as zero.
template <int NT>
struct Rows {
    const uint4 *wa, *wb, *x[NT];
    const float *sa[NT][2], *sb;
    int64_t sa_blk;
};

template <int NT, int U>
__device__ __forceinline__ void load_group(Group<NT, U>& G, const Rows<NT>& r, int32_t t,
                                           int32_t kb0, int32_t kb_end, int32_t K16) {
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int32_t kb = kb0 + u;
        const bool in = kb < kb_end;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t c = kb * 8 + s * 4 + t;   // 16-byte chunk of the rows
            const bool ok = in && c < K16;
            G.wa[u][s] = ok && r.wa ? ld_weights(r.wa + c) : z;
            G.wb[u][s] = ok && r.wb ? ld_weights(r.wb + c) : z;
#pragma unroll
            for (int j = 0; j < NT; ++j) G.x[u][s][j] = ok && r.x[j] ? r.x[j][c] : z;
        }
        G.sb[u] = in ? r.sb[kb] : 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                G.sa[u][j][e] = in && r.sa[j][e] ? r.sa[j][e][kb * r.sa_blk] : 0.0f;
    }
}

template <int NT, int U>
__device__ __forceinline__ void mma_group(const Group<NT, U>& G, float (&acc)[NT][4]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float c[4] = {};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint4 &a = G.wa[u][s], &b = G.wb[u][s], &x = G.x[u][s][j];
                mma_m16n8k32(c, a.x, b.x, a.y, b.y, x.x, x.y);
                mma_m16n8k32(c, a.z, b.z, a.w, b.w, x.z, x.w);
            }
            const float f0 = G.sa[u][j][0] * G.sb[u], f1 = G.sa[u][j][1] * G.sb[u];
            acc[j][0] = fmaf(c[0], f0, acc[j][0]);
            acc[j][1] = fmaf(c[1], f1, acc[j][1]);
            acc[j][2] = fmaf(c[2], f0, acc[j][2]);
            acc[j][3] = fmaf(c[3], f1, acc[j][3]);
        }
    }
}

struct Args {
    const uint4 *X, *W;
    const float *sa, *sb;
    int64_t sa_row, sa_blk;
    uint16_t* D;
    int32_t M, N, K16, k_blocks, slice;   // slice: 128-k blocks per CTA of a cluster
};

template <int NT, int U, int S, bool BF16>
__global__ void __launch_bounds__(kWarps * 32)
small_m_fp8_kernel(const Args p, uint32_t* __restrict__ err) {
    constexpr int kMp = 8 * NT;
    __shared__ float part[kRows][kMp];

    grid_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t rank = cluster_ctarank();
    const int32_t row0 = static_cast<int32_t>(blockIdx.x / S) * kRows;
    const int32_t ra = row0 + warp * 16 + g, rb = ra + 8;
    const int32_t kb_begin = static_cast<int32_t>(rank) * p.slice;
    const int32_t kb_end = min(p.k_blocks, kb_begin + p.slice);

    Rows<NT> r;
    r.wa = ra < p.N ? p.W + static_cast<int64_t>(ra) * p.K16 : nullptr;
    r.wb = rb < p.N ? p.W + static_cast<int64_t>(rb) * p.K16 : nullptr;
    // A warp's 16 rows lie in one 128-row block of weight scales.
    r.sb = p.sb + static_cast<int64_t>(min(row0 + warp * 16, p.N - 1) / kFp8Block) * p.k_blocks;
    r.sa_blk = p.sa_blk;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        r.x[j] = g + 8 * j < p.M ? p.X + static_cast<int64_t>(g + 8 * j) * p.K16 : nullptr;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int32_t m = 8 * j + 2 * t + e;   // this thread's accumulator columns
            r.sa[j][e] = m < p.M ? p.sa + m * p.sa_row : nullptr;
        }
    }

    // While the previous grid finishes, pull the first eighth of this CTA's K
    // slice of its weight rows into L2 (a prefetch cannot see stale data: L2
    // is where global memory is coherent).
    if (t == 0 && kb_end > kb_begin) {
        const int32_t c0 = kb_begin * 8, n = min(kb_end * 8, p.K16) - c0;
        const uint32_t bytes = static_cast<uint32_t>(max(1, n / 8)) * 16u;
        if (r.wa) prefetch_l2_bytes(r.wa + c0, bytes);
        if (r.wb) prefetch_l2_bytes(r.wb + c0, bytes);
    }
    grid_dependency_wait();

    // Groups of U blocks; group i + 1 is loaded before group i is multiplied.
    float acc[NT][4] = {};
    Group<NT, U> ga, gb;
    if (kb_begin < kb_end) load_group(ga, r, t, kb_begin, kb_end, p.K16);
    for (int32_t kb = kb_begin; kb < kb_end; kb += 2 * U) {
        if (kb + U < kb_end) load_group(gb, r, t, kb + U, kb_end, p.K16);
        mma_group(ga, acc);
        if (kb + 2 * U < kb_end) load_group(ga, r, t, kb + 2 * U, kb_end, p.K16);
        if (kb + U < kb_end) mma_group(gb, acc);
    }

    // This slice's partial tile: rows g, g + 8 of the warp's 16 weight rows,
    // columns (tokens) 8 j + 2 t + {0, 1}.
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        part[warp * 16 + g][8 * j + 2 * t] = acc[j][0];
        part[warp * 16 + g][8 * j + 2 * t + 1] = acc[j][1];
        part[warp * 16 + g + 8][8 * j + 2 * t] = acc[j][2];
        part[warp * 16 + g + 8][8 * j + 2 * t + 1] = acc[j][3];
    }
    cluster_sync();   // every slice's partial tile is visible cluster-wide

    // CTA `rank` finishes weight rows [64 rank / S, 64 (rank + 1) / S).
    constexpr int kShare = kRows / S;
    for (int o = static_cast<int>(threadIdx.x); o < kShare * p.M; o += kWarps * 32) {
        const int rl = static_cast<int>(rank) * kShare + o % kShare;
        const int m = o / kShare;
        const uint32_t local = smem_u32(&part[rl][m]);
        float v[S];
#pragma unroll
        for (int q = 0; q < S; ++q) v[q] = ld_shared_cluster_f32(map_to_rank(local, q));
        float sum = v[0];
#pragma unroll
        for (int q = 1; q < S; ++q) sum += v[q];
        const int32_t n = row0 + rl;
        if (n < p.N)
            p.D[static_cast<int64_t>(m) * p.N + n] = cvt16_rn<BF16>(__float_as_uint(sum));
    }
    cluster_sync();   // peers' shared memory stays alive until every CTA has read it
    if (threadIdx.x == 0) check_count_unit(err, static_cast<int32_t>(blockIdx.x));
}

template <int NT, int U, int S, bool BF16>
cudaError_t launch_variant(Args p, const Fp8Device& dev, cudaStream_t stream) {
    p.slice = static_cast<int32_t>(ceil_div(p.k_blocks, S));
    const int64_t clusters = ceil_div(p.N, kRows);
    return launch_kernel(small_m_fp8_kernel<NT, U, S, BF16>,
                         dim3(static_cast<unsigned>(clusters * S)), dim3(kWarps * 32), 0, stream,
                         static_cast<unsigned>(S), dev.pdl, p, dev.err_word);
}

// Slices per cluster: as many as keep the grid one wave of 4 CTAs per SM.
template <int NT, int U, bool BF16>
cudaError_t launch_sliced(const Args& p, const Fp8Device& dev, cudaStream_t stream) {
    const int64_t clusters = ceil_div(p.N, kRows), wave = 4ll * dev.sms;
    if (clusters * 8 <= wave) return launch_variant<NT, U, 8, BF16>(p, dev, stream);
    if (clusters * 4 <= wave) return launch_variant<NT, U, 4, BF16>(p, dev, stream);
    if (clusters * 2 <= wave) return launch_variant<NT, U, 2, BF16>(p, dev, stream);
    return launch_variant<NT, U, 1, BF16>(p, dev, stream);
}

template <bool BF16>
cudaError_t launch_typed(const Args& p, const Fp8Device& dev, cudaStream_t stream) {
    return p.M <= 8 ? launch_sliced<1, 2, BF16>(p, dev, stream)
                    : launch_sliced<2, 1, BF16>(p, dev, stream);
}

}  // namespace

int64_t small_m_fp8_max_m() { return kMaxM; }

cudaError_t launch_small_m_fp8(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    Args p{};
    p.X = static_cast<const uint4*>(g.A);
    p.W = static_cast<const uint4*>(g.B);
    p.sa = g.SA;
    p.sb = g.SB;
    p.sa_row = g.sa_row;
    p.sa_blk = g.sa_blk;
    p.D = static_cast<uint16_t*>(g.D);
    p.M = static_cast<int32_t>(g.M);
    p.N = static_cast<int32_t>(g.N);
    p.K16 = static_cast<int32_t>(g.K / 16);
    p.k_blocks = static_cast<int32_t>(ceil_div(g.K, kFp8Block));
    return g.bf16 ? launch_typed<true>(p, dev, stream) : launch_typed<false>(p, dev, stream);
}

}  // namespace tmagemm
