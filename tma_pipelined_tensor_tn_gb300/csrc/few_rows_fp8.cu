// gemm_fp8 for few rows of activations on tcgen05.  Up to 64 tokens the operands'
// roles are swapped: the weights are the 128-row MMA operand and the activations
// the narrow one, in blocks of NP = 16, 32 or 64 tokens (rows past M zero), so the
// work follows the number of tokens and all 128 accumulator lanes hold weight rows.
// Blocks of NP = 128 tokens keep the rows themselves.  Bound by streaming the
// weights; K is split over the CTAs of a cluster so that enough of them stream at
// once.
//
// As in the tile kernel each 128-k block's product has a TMEM accumulator of its
// own (four of them), added as acc += t * scale.  Swapped, a lane is a weight row
// and a column a token, so a block's scale varies along the columns: the epilogue
// threads keep SA[token] * SB (the tile's 128 weight rows share one SB per block) of
// four blocks in shared memory, read as broadcasts.  Otherwise a lane is a token
// and its scale one register (100 x 14336 x 4096, each call by itself: 15.1 us,
// swapped 16.4: the broadcast reads of 128 columns took longer than their MMAs).
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, then four scaling warps (eight
// for 128 tokens, half of the columns each).  The CTAs of a cluster leave their
// FP32 partial tiles [token][weight row] in shared memory (over the ring) and
// each adds and stores a share of the outputs, in slice order: no workspace,
// one launch, deterministic.
//
// Up to 64 tokens two CTAs share an SM (half the ring and at most 256 TMEM
// columns each): while one sets up or reduces, the other streams.
//
// Measured on GB300 (calls in a graph, weights colder than L2): 1 x 4096 x 14336
// 11.2 us (5.2 TB/s of weights), 32 x 14336 x 4096 12.1 us, 12 x 9664 x 5584
// 11.9 us; 100 x 14336 x 4096, 112 tiles undivided, 12.8 us (each call by itself
// 15.1, and with two CTAs an SM, half the accumulators and registers each, 22.3).
// There 40 of 152 SMs have no tile, and a CTA takes in 0.9 MB.  A kernel that streamed the
// weights into mma.sync fragments, as the 16-bit few-row kernel does, took 12.6 us
// at one token and 19.7 us at 16.
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"
#include "tile_sched.cuh"

namespace tmagemm {

namespace {

template <int NP_, int STAGES_, int EPI_WARPS_, int CTAS_PER_SM_, bool BF16_>
struct FewCfg {
    static constexpr int NP = NP_, STAGES = STAGES_, BN = 128, BK = kFp8Block;
    static constexpr int kCtasPerSm = CTAS_PER_SM_;
    static constexpr bool kBF16 = BF16_;
    static constexpr int kEpiThreads = 32 * EPI_WARPS_;
    static constexpr int kThreads = 64 + kEpiThreads, kAccs = 4;
    // 128 tokens are as good an MMA operand as 128 weight rows: they keep their role,
    // so that a lane is a token and its scale one register.
    static constexpr bool kSwap = NP_ < 128;
    static constexpr int kCols = NP_ / (EPI_WARPS_ / 4);   // columns of one epilogue warp
    static constexpr uint32_t kTmemCols = kAccs * NP;
    static constexpr uint32_t kWBytes = BN * BK, kXBytes = NP * BK;
    static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
    static constexpr uint32_t kPartStride = BN + 4;   // floats; rows stay 16-byte aligned
    static constexpr uint32_t kOffScale = STAGES * kStageBytes;   // [2][4][NP] floats (kSwap)
    static constexpr uint32_t kOffBar = kOffScale + (kSwap ? 2 * 4 * NP * 4 : 0);
    static constexpr uint32_t kNumBars = 2 * STAGES + 2 * kAccs + 1;
    static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
    static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kTmemCols * CTAS_PER_SM_ <= 512, "resident CTAs share TMEM");
    static_assert((kSmemBytes + 1024) * CTAS_PER_SM_ <= 233472, "and shared memory");
    static_assert(NP * kPartStride * 4 <= STAGES * kStageBytes, "partial tile over the ring");
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms stay aligned");
};

struct FewProblem {
    CUtensorMap tmW;   // B {K, N}, box {128, 128}
    CUtensorMap tmX;   // A {K, M}, box {128, NP}
    // blockIdx.x = (token block * n_tiles + weight tile) * splits + K slice
    const float *sa, *sb;
    int64_t sa_row, sa_blk;
    uint16_t* d;
    int32_t M, N, k_blocks, n_tiles, splits;   // splits: CTAs of a cluster
};

// Tokens first, first + warps, ... below `end` of the tile at (m0, n0): the
// partial sums of the cluster's CTAs (at most MOST), in slice order, rounded
// once and stored.  ROWS tokens at a time, whose loads are in flight together (one
// by one, the store of a 128 x 128 tile took 2 us).
template <class C, int ROWS, int MOST>
__device__ __forceinline__ void add_and_store(const FewProblem& prob, const float* part,
                                              int32_t m0, int32_t n0, int first, int end,
                                              uint32_t* err) {
    constexpr int kWarps = C::kThreads / 32;
    const int n = n0 + 4 * (static_cast<int>(threadIdx.x) % 32);
    if (n >= prob.N) return;
    for (int m = first; m < end; m += ROWS * kWarps) {
        float v[ROWS][MOST][4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int row = m + r * kWarps;
            if (row >= end) break;
            const uint32_t at = smem_u32(part) + (row * C::kPartStride + (n - n0)) * 4u;
#pragma unroll
            for (int q = 0; q < MOST; ++q) {
                if constexpr (MOST == 1)
                    *reinterpret_cast<float4*>(v[r][0]) = *reinterpret_cast<const float4*>(
                        part + row * C::kPartStride + (n - n0));
                else if (q < prob.splits)
                    ld_shared_cluster_v4(map_to_rank(at, q), v[r][q]);
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int row = m + r * kWarps;
            if (row >= end) break;
            float s[4] = {v[r][0][0], v[r][0][1], v[r][0][2], v[r][0][3]};
#pragma unroll
            for (int q = 1; q < MOST; ++q)
                if (q < prob.splits)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] += v[r][q][e];
            uint2 out;
            out.x = pack2_rn<C::kBF16>(__float_as_uint(s[0]), __float_as_uint(s[1]));
            out.y = pack2_rn<C::kBF16>(__float_as_uint(s[2]), __float_as_uint(s[3]));
            if (check_ok(m0 + row < prob.M && n + 4 <= prob.N, err, kSiteCheckBounds))
                *reinterpret_cast<uint2*>(prob.d + static_cast<int64_t>(m0 + row) * prob.N + n) =
                    out;
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm)
few_rows_fp8_kernel(const __grid_constant__ FewProblem prob, const uint64_t limit_ns,
                    uint32_t* __restrict__ err) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (C::STAGES + s); };
    auto acc_full_bar = [&](uint32_t a) { return bar0 + 8u * (2 * C::STAGES + a); };
    auto acc_empty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * C::STAGES + C::kAccs + a); };
    const uint32_t mma_done_bar = bar0 + 8u * (2 * C::STAGES + 2 * C::kAccs);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const uint32_t rank = cluster_ctarank();
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / prob.splits;
    const int32_t n0 = tile % prob.n_tiles * C::BN, m0 = tile / prob.n_tiles * C::NP;
    const int32_t tokens = min(C::NP, prob.M - m0);
    // This CTA's k-blocks [kb0, kb1); may be none.
    const int32_t kb0 = static_cast<int32_t>(rank) * prob.k_blocks / prob.splits;
    const int32_t kb1 = (static_cast<int32_t>(rank) + 1) * prob.k_blocks / prob.splits;

    grid_launch_dependents();
    if (warp == 0) {
        if (elect_one()) {
            for (uint32_t s = 0; s < (uint32_t)C::STAGES; ++s) {
                mbar_init(full_bar(s), 1);
                mbar_init(empty_bar(s), 1);
            }
            for (uint32_t a = 0; a < (uint32_t)C::kAccs; ++a) {
                mbar_init(acc_full_bar(a), 1);
                mbar_init(acc_empty_bar(a), C::kEpiThreads / 32);
            }
            mbar_init(mma_done_bar, 1);
            *abort_flag = 0;
            fence_mbarrier_init();
            tma_prefetch_desc(&prob.tmW);
            tma_prefetch_desc(&prob.tmX);
            // Weights of the first k-blocks into L2 while the previous grid
            // finishes (a prefetch cannot see stale data).
            for (int32_t kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb)
                tma_prefetch_l2_2d(&prob.tmW, kb * C::BK, n0);
        }
        __syncwarp();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dependency_wait();

    // Both role warps walk their loops whole (the control flow and addresses are
    // the same in every lane); one lane issues.
    if (warp == 0) {
        const bool lead = elect_one();
        uint32_t s = 0, phase = 0, it = 0;
        for (int32_t kb = kb0; kb < kb1; ++kb, ++it) {
            if (!__all_sync(0xffffffffu, wait_many(empty_bar(s), phase ^ 1u, abort_flag, err,
                                                   kSiteProducerEmpty, limit_ns)) ||
                !check_ok(n0 >= 0 && n0 < prob.N && m0 >= 0 && m0 < prob.M, err, kSiteCheckTma)) {
                *abort_flag = 1;
                break;
            }
            if (lead) {
                mbar_arrive_expect_tx(full_bar(s), C::kStageBytes);
                const uint32_t w = sbase + s * C::kStageBytes;
                tma_load_2d(w, &prob.tmW, kb * C::BK, n0, full_bar(s));
                tma_load_2d(w + C::kWBytes, &prob.tmX, kb * C::BK, m0, full_bar(s));
            }
            __syncwarp();
            if (++s == (uint32_t)C::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        // The last stages issued must have landed before shared memory is reused.
        if (lead) {
            const uint32_t first = it > (uint32_t)C::STAGES ? it - C::STAGES : 0u;
            for (uint32_t j = first; j < it; ++j)
                wait_bounded(full_bar(ring_stage(j, C::STAGES)), ring_phase(j, C::STAGES), err,
                             kSiteDrainFull, limit_ns);
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t kIdesc = idesc_e4m3(C::BN, C::NP);
        const bool lead = elect_one();
        const uint64_t w_desc0 = umma_desc_sw128_kmajor(sbase);
        const uint64_t x_desc0 = umma_desc_sw128_kmajor(sbase + C::kWBytes);
        uint32_t s = 0, phase = 0, a = 0, a_phase = 1;
        for (int32_t kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu,
                            wait_many(acc_empty_bar(a), a_phase, abort_flag, err,
                                      kSiteMmaAccEmpty, limit_ns) &&
                                wait_many(full_bar(s), phase, abort_flag, err, kSiteMmaFull,
                                          limit_ns)))
                break;
            tc_fence_after();
            if (lead) {
                const uint64_t w_desc = w_desc0 + s * (C::kStageBytes / 16);
                const uint64_t x_desc = x_desc0 + s * (C::kStageBytes / 16);
#pragma unroll
                for (int j = 0; j < C::BK / 32; ++j)   // 32 k = 32 bytes = 2 address units
                    mma_e4m3<false>(tmem_base + a * C::NP, (C::kSwap ? w_desc : x_desc) + 2 * j,
                                    (C::kSwap ? x_desc : w_desc) + 2 * j, kIdesc,
                                    j != 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
                mma_commit(acc_full_bar(a));
            }
            __syncwarp();
            if (++s == (uint32_t)C::STAGES) {
                s = 0;
                phase ^= 1u;
            }
            if (++a == (uint32_t)C::kAccs) {
                a = 0;
                a_phase ^= 1u;
            }
        }
        if (lead) {
            mma_commit(mma_done_bar);
            wait_bounded(mma_done_bar, 0, err, kSiteDrainMma, limit_ns);
        }
        __syncwarp();
    } else {
        const uint32_t quarter = static_cast<uint32_t>(warp) & 3u;
        const int tid = static_cast<int>(threadIdx.x) - 64;
        const int col0 = ((warp - 2) >> 2) * C::kCols;   // this warp's first column
        const uint32_t t_base = tmem_base + ((quarter * 32u) << 16) + col0;
        const int row = static_cast<int>(quarter) * 32 + lane;   // this lane's accumulator row
        float* scale = reinterpret_cast<float*>(smem + C::kOffScale);
        // A token's scales (times the tile's weight scales) of four blocks at a time,
        // read while the four before them are used: of the lane's token, or of token
        // `tid`, which every lane then reads from shared memory.
        const int mine = C::kSwap ? tid : row;
        const bool token = mine < tokens;
        const float* sa = prob.sa + (token ? (m0 + mine) * prob.sa_row : 0);
        const float* sb = prob.sb + static_cast<int64_t>(n0 / kFp8Block) * prob.k_blocks;
        float next[4];
        auto fetch = [&](int32_t kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                next[j] = token && kb + j < kb1 ? sa[(kb + j) * prob.sa_blk] * sb[kb + j] : 0.0f;
        };
        fetch(kb0);
        f32x2 acc[C::kCols / 2] = {};
        bool ok = true;
        uint32_t it = 0;
        for (int32_t kb = kb0; kb < kb1; kb += 4) {
            float* sc = scale + ((kb - kb0) & 4) * C::NP;   // the two buffers in turn
            float now[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) now[j] = next[j];
            if constexpr (C::kSwap) {
                if (tid < C::NP) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[j * C::NP + tid] = now[j];
                }
                __syncwarp();   // (the barrier is an aligned one)
                // Also ends the loop in every warp once a wait has failed in one.
                if (!named_bar_and(1, C::kEpiThreads, ok)) break;
            } else if (!ok) {
                break;
            }
            fetch(kb + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (kb + j >= kb1 || !ok) break;
                const uint32_t a = ring_stage(it, C::kAccs);
                ok = __all_sync(0xffffffffu,
                                wait_many(acc_full_bar(a), ring_phase(it, C::kAccs), abort_flag,
                                          err, kSiteEpiAccFull, limit_ns));
                if (!ok) break;
                ++it;
                tc_fence_after();
                constexpr int kPart = C::kCols < 32 ? C::kCols : 32;
#pragma unroll
                for (int c = 0; c < C::kCols; c += kPart) {
                    uint32_t v[kPart];
                    if constexpr (kPart == 16)
                        tmem_ld_32x32b_x16(t_base + a * C::NP + c, v);
                    else
                        tmem_ld_32x32b_x32(t_base + a * C::NP + c, v);
                    tmem_ld_wait();
                    if (c + kPart == C::kCols) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_empty_bar(a));
                    }
#pragma unroll
                    for (int i = 0; i < kPart; i += 4) {
                        float4 f = make_float4(now[j], now[j], now[j], now[j]);
                        if constexpr (C::kSwap)
                            f = *reinterpret_cast<const float4*>(sc + j * C::NP + col0 + c + i);
                        scale_add(acc[(c + i) / 2], v[i], v[i + 1], pack_f32x2(f.x, f.y));
                        scale_add(acc[(c + i) / 2 + 1], v[i + 2], v[i + 3], pack_f32x2(f.z, f.w));
                    }
                }
            }
        }
        // Every block has been multiplied, so every stage has been read: the
        // partial tile goes over the ring, a column (token) per row of it.
        // (After a failed wait stages may still be written: leave them alone.)
        __syncwarp();
        if (named_bar_and(1, C::kEpiThreads, ok)) {
            float* part = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int c = 0; c < C::kCols; c += 4) {
                float v[4];
                unpack_f32x2(acc[c / 2], v[0], v[1]);
                unpack_f32x2(acc[c / 2 + 1], v[2], v[3]);
                if constexpr (C::kSwap) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col0 + c + i < tokens)
                            part[(col0 + c + i) * C::kPartStride + row] = v[i];
                } else if (token) {
                    *reinterpret_cast<float4*>(part + row * C::kPartStride + col0 + c) =
                        make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
    }

    // The cluster barriers are aligned ones: all lanes of a warp arrive together.
    __syncwarp();
    tc_fence_before();
    if (prob.splits > 1) cluster_sync(); else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
    // Each CTA of the cluster adds and stores a share of the tokens, a warp a
    // token and a lane four outputs (N is a multiple of 8: they are all inside
    // or all outside).
    const int first = static_cast<int>(rank) * tokens / prob.splits + warp;
    const int end = (static_cast<int>(rank) + 1) * tokens / prob.splits;
    const float* part = reinterpret_cast<const float*>(smem);
    if (prob.splits == 1)
        add_and_store<C, 4, 1>(prob, part, m0, n0, first, end, err);
    else if (prob.splits <= 4)
        add_and_store<C, 4, 4>(prob, part, m0, n0, first, end, err);
    else
        add_and_store<C, 2, 8>(prob, part, m0, n0, first, end, err);
    if (threadIdx.x == 0 && !*abort_flag)
        check_count_unit(err, static_cast<int32_t>(blockIdx.x));
    __syncwarp();   // (lanes past N left add_and_store early)
    // Peers' shared memory stays alive until every CTA has read it.
    if (prob.splits > 1) cluster_sync();
}

// Never launched: CTAs of the size of C's, to ask how many clusters fit the device.
// (Of a kernel that allocates TMEM the occupancy query counts one CTA per SM, whatever
// it allocates: 36 clusters of 4 for 16 tokens, where 74 are resident.)
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm) few_rows_size_kernel() {}

// Clusters of 2 to 8 CTAs of C's kernel that the current device holds at once, asked
// once per context.  (A cluster lies within a GPC, whose SMs differ from device to
// device.)  `into` has kMaxFewSlices + 1 entries; a size that cannot be asked for is 0.
template <class C>
void resident_clusters(int64_t* into) {
    static ContextMarks known, attr_done;
    static std::atomic<int> held[64][kMaxFewSlices + 1];
    auto kernel = few_rows_size_kernel<C>;
    int dev = 0;
    const uint64_t ctx = current_context_id();
    const bool tracked = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && ctx != 0;
    const bool asked = tracked && known[dev].load(std::memory_order_acquire) == ctx;
    for (int size = 2; size <= kMaxFewSlices; ++size) {
        int n = 0;
        if (asked) {
            n = held[dev][size].load(std::memory_order_relaxed);
        } else {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(size));
            cfg.blockDim = dim3(C::kThreads);
            cfg.dynamicSmemBytes = C::kSmemBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(size);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (smem_opt_in(kernel, static_cast<int>(C::kSmemBytes), attr_done) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            if (tracked) held[dev][size].store(n, std::memory_order_relaxed);
        }
        into[size] = n;
    }
    if (tracked && !asked) known[dev].store(ctx, std::memory_order_release);
}

template <class C>
cudaError_t launch_cfg(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    FewProblem p;
    if (encode_fp8_operand(dev.encode, &p.tmW, g.B, g.K, g.N, 0, C::BN) ||
        encode_fp8_operand(dev.encode, &p.tmX, g.A, g.K, g.M, 0, C::NP))
        return cudaErrorInvalidValue;
    p.sa = g.SA;
    p.sb = g.SB;
    p.sa_row = g.sa_row;
    p.sa_blk = g.sa_blk;
    p.d = static_cast<uint16_t*>(g.D);
    p.M = static_cast<int32_t>(g.M);
    p.N = static_cast<int32_t>(g.N);
    p.k_blocks = static_cast<int32_t>(ceil_div(g.K, C::BK));
    p.n_tiles = static_cast<int32_t>(ceil_div(g.N, C::BN));
    const int64_t tiles = p.n_tiles * ceil_div(g.M, C::NP);
    static ContextMarks attr_done;
    auto kernel = few_rows_fp8_kernel<C>;
    if (cudaError_t e = smem_opt_in(kernel, static_cast<int>(C::kSmemBytes), attr_done)) return e;
    int64_t resident[kMaxFewSlices + 1];
    resident_clusters<C>(resident);
    p.splits = few_rows_slices(tiles, p.k_blocks, resident);
    const int splits = p.splits;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(tiles * splits)), dim3(C::kThreads),
                         C::kSmemBytes, stream, static_cast<unsigned>(splits), dev.pdl, p,
                         dev.limit_ns, dev.err_word);
}

template <bool T>
cudaError_t launch_typed(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    switch (few_rows_tokens(g.M)) {
        case 16: return launch_cfg<FewCfg<16, 6, 4, 2, T>>(g, dev, stream);
        case 32: return launch_cfg<FewCfg<32, 5, 4, 2, T>>(g, dev, stream);
        case 64: return launch_cfg<FewCfg<64, 4, 4, 2, T>>(g, dev, stream);
        default: return launch_cfg<FewCfg<128, 6, 8, 1, T>>(g, dev, stream);
    }
}

}  // namespace

// One block of tokens, or more where the 128 x 128 tiles leave room to split a
// long enough K: 256 x 4096 x 4096 (64 tiles) 10.1 us (9.1 in a graph of calls)
// against 12.2 us for the tile kernel and 512 x 4096 x 4096 (128 tiles, no split)
// 12.7 against 12.5; 256 x 4096 x 2048 7.5 against 8.0 and 256 x 4096 x 1536 6.8
// against 6.8.
bool few_rows_fp8(int64_t M, int64_t N, int64_t K, int sms) {
    return M <= 128 || (K >= 2048 && 2 * ceil_div(M, 128) * ceil_div(N, 128) <= sms);
}

// Tokens of a block.
int few_rows_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// K slices (CTAs of a cluster): the most with which all clusters are resident at
// once and each CTA has four k-blocks (3 x 2360 x 432, four blocks: 3.0 us
// undivided, 3.2 in two; 40 x 512 x 2048, sixteen: 4.2 us in four, 4.4 in five).
// With clusters left over a second round begins: 12 x 9728 x 5632 (76 tiles, 74
// clusters of four) takes 11.2 us in 3 slices and 15.1 in 4, 5 x 5088 x 2656 (40, 38
// of seven) 5.5 in 6 and 8.6 in 7.  Where they just fit: 1 x 12160 x 8192 (95 tiles)
// 17.2 us in 3 and 19.6 in 2, 1 x 4864 x 14336 (38) 12.9 in 7 and 13.0 in 6, and with
// four or five k-blocks a slice 40 x 4608 x 4096 (36) 8.3 in 8 and 7.8 in 7.
int few_rows_slices(int64_t tiles, int64_t k_blocks, const int64_t* resident) {
    for (int slices = kMaxFewSlices; slices > 1; --slices)
        if (tiles <= resident[slices] && k_blocks >= 4 * slices) return slices;
    return 1;
}

cudaError_t launch_few_rows_fp8(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    return g.bf16 ? launch_typed<true>(g, dev, stream) : launch_typed<false>(g, dev, stream);
}

}  // namespace tmagemm
