// Block-scaled 8-bit products on tcgen05, dense and grouped by expert:
//   D[m, n] = sum_b SA[m, b] SB[n / 128, b] sum_{k in block b} A[m, k] B[n, k]
// with e4m3 A (M x K) and B (N x K), one FP32 scale per 128 values of a row of
// A and per 128 x 128 values of B, FP32 sums and one rounding to fp16 or bf16.
//
// The scales change every 128 k, so the tensor cores cannot add over all of
// K: each 128-k block's product (four K = 32 MMAs) goes to a TMEM accumulator
// of its own, and the epilogue warps read it, multiply it by SA * SB (one
// scalar per row and 128 columns) and add it to FP32 accumulators in their
// registers, while the next block's MMAs fill another TMEM accumulator.
//
// Roles (one CTA per SM):
//   warp 0      TMA producer: A and B k-blocks (128 bytes a row, 128B swizzle)
//               into a ring of stages;
//   warps 1, 2  MMA issuers, one per part (half the columns of a pair's tile;
//               a CTA's own tile is one part): per k-block four
//               tcgen05.mma.kind::f8f6f4 into the part's next TMEM accumulator,
//               then commits onto the stage's `empty` barrier and the
//               accumulator's `acc_full` barrier;
//   warps 4..11 scaling and epilogue: two warps per 32 rows, each half of the
//               tile's columns.  Their FP32 sums (128 per thread for 256
//               columns) take the registers that warps 0..3 (3, and 2 for one
//               part, idle) give up.
// What bounds it.  Per k-block of a pair's 256 x 256 tile each SM has 512 cycles
// of MMAs (128 x 256 x 128 at 8192 multiply-adds a cycle: 0.25 us), 256 of TMEM
// reads (128 lanes x 256 columns, at 32 lanes x 4 bytes per cycle and quarter) and
// 64 packed multiply-adds in each of the two warps of a scheduler (256 cycles of
// its FP32 lanes, more or less under the reads), and takes in 32 KB of operands.
// A single call of 8192^3 takes 368 to 376 us (2.9 to 3.0 PFLOP/s, 0.41 us per
// k-block; 415 to 424 back to back, at the power limit's clock): without the
// multiply-adds the same kernel takes 306 us, without the operand loads 343 and
// without both 261, and with sums left to the tensor cores over all of K (no
// scales) 306.  All SMs together take in about 13.4 TB/s through
// TMA (128 x 128 tiles: 0.36 us per k-block of 32 KB on 152 SMs, 0.25 on 32),
// which bounds those tiles and makes 0.36 us per k-block the pair tile's bound
// too; the multiply-adds are not quite hidden under it.
// Sixteen epilogue warps of 64 columns (104 registers each) took 621 us.
//
// CTA pairs (PAIR): cta_group::2 MMAs on 256 x 256 tiles, each CTA holding 128
// rows of A and half of B, as in the 16-bit kernel.
//
// Grouped: the rows of group g are [off[g], off[g + 1]) with the offsets in
// device memory; every CTA derives the tile schedule from them, so a router's
// result is used without a copy to the host.  A row tile may read rows of the
// next group; they only reach accumulator rows that are not stored.
//
// Every mbarrier wait is bounded (ptx.cuh).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"
#include "tile_sched.cuh"

namespace tmagemm {

namespace {

template <int BN_, int ACC_COLS_, int COLS_, int STAGES_, bool PAIR_, bool GROUPED_, bool BF16_>
struct Fp8Cfg {
    static constexpr int BM = 128, BN = BN_, BK = kFp8Block, STAGES = STAGES_;
    static constexpr bool kPair = PAIR_, kGrouped = GROUPED_, kBF16 = BF16_;
    static constexpr int kTileM = PAIR_ ? 256 : 128;
    // A k-block's product is made in parts of kAccCols columns, each in a TMEM
    // accumulator of its own: the MMAs of one part run while the parts before
    // it are scaled.
    static constexpr int kAccCols = ACC_COLS_, kAccs = 4, kParts = BN_ / ACC_COLS_;
    // Rows of B in this CTA; a pair's CTAs each hold half of every part.
    static constexpr int kBRows = PAIR_ ? BN_ / 2 : BN_;
    static constexpr int kBBoxRows = PAIR_ ? ACC_COLS_ / 2 : ACC_COLS_;
    static constexpr int kCols = COLS_;                    // columns of one epilogue warp
    static constexpr int kEpiWarps = 4 * BN_ / kCols;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    // A warp's columns are 32-column pieces; each lies in one 128-column block
    // of weight scales, and all of them in at most two.
    static constexpr int kPieces = COLS_ / 32;
    static constexpr int kBatch = kPieces % 2 ? kPieces : 2;   // pieces read from TMEM at once
    static constexpr bool kTwoBlocks = BN_ % kFp8Block != 0;
    // Registers: the role warps give up what the epilogue warps take.
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kRoleRegs = 56;
    static constexpr int kEpiRegs =
        (kThreads * kLaunchRegs - 128 * kRoleRegs) / (32 * kEpiWarps) / 8 * 8;
    static_assert(128 * kRoleRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs,
                  "the shares fit what the block was launched with");
    // A comes in boxes of 32 rows for grouped problems, where a tile may have
    // few rows (a box without any is not loaded), else in one of 128.
    static constexpr int kABoxRows = GROUPED_ ? 32 : 128;
    static constexpr uint32_t kABytes = BM * BK;
    static constexpr uint32_t kBBytes = kBRows * BK;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes;
    // Staging of D: per epilogue warp 32 rows x kCols, as store boxes of one
    // swizzle span (64 columns in 128 bytes, or 32 in 64).
    static constexpr int kBoxCols = COLS_ % 64 == 0 ? 64 : 32;
    static constexpr int kBoxes = COLS_ / kBoxCols;
    static constexpr uint32_t kBoxRowBytes = kBoxCols * 2, kBoxChunks = kBoxRowBytes / 16;
    static constexpr uint32_t kBoxBytes = 32 * kBoxRowBytes;
    static constexpr uint32_t kOffD = STAGES * kStageBytes;
    // Byte offset in a box of 16-byte chunk c of row r: the swizzle XORs the
    // chunk with the address bits from 7 up.
    static __device__ __forceinline__ uint32_t box_at(uint32_t r, uint32_t c) {
        return r * kBoxRowBytes + ((c ^ ((r * kBoxRowBytes / 128) % kBoxChunks)) << 4);
    }
    static constexpr uint32_t kOffBar = kOffD + kEpiWarps * kBoxes * kBoxBytes;
    static constexpr uint32_t kNumBars = 2 * STAGES + 2 * kAccs + kParts;
    static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
    static constexpr uint32_t kOffStart = kOffMisc + 32;   // grouped: tile starts, a flag before
    static constexpr uint32_t kSmemBytes =
        kOffStart + (GROUPED_ ? (kMaxFp8Groups + 1) * 4 : 0) + 1024;
    static_assert(kSmemBytes <= 232448, "fits the 227 KB opt-in shared memory");
    static_assert((kParts == 1 || kParts == 2) && kAccs % kParts == 0,
                  "an MMA issuer (warp 1 or 2) and accumulators of its own per part");
    static_assert(kAccs * kAccCols <= 512, "TMEM columns");
    static_assert(BN_ % ACC_COLS_ == 0 && ACC_COLS_ % COLS_ == 0 && COLS_ % 32 == 0 &&
                      ACC_COLS_ % 16 == 0 && kBBoxRows % 8 == 0,
                  "whole parts, epilogue warps, pieces and swizzle atoms");
    static_assert(kStageBytes % 1024 == 0 && kBoxBytes % 1024 == 0, "atoms stay aligned");
};

// One arrival on an mbarrier at a shared::cluster address by the threads whose
// `p` is not 0; predicated rather than branched around, and relaxed (what it
// hands over is a TMEM accumulator that has been read, behind a tcgen05 fence;
// a release would wait for the loads of later scales in flight).
__device__ __forceinline__ void mbar_arrive_if(uint32_t p, uint32_t cluster_addr) {
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "setp.ne.u32 P, %0, 0;\n\t"
        "@P mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%1];\n\t}"
        ::"r"(p), "r"(cluster_addr)
        : "memory");
}

// Registers of this warp's group of four, lowered or raised within what the
// block was launched with.
template <int N>
__device__ __forceinline__ void set_max_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

struct Fp8Problem {
    CUtensorMap tmA;   // A {K, rows}, box {128, kABoxRows}
    CUtensorMap tmB;   // B {K, N, G}, box {128, kBBoxRows, 1}
    CUtensorMap tmD;   // D {N, rows}, box {kBoxCols, 32}
    const float* sa;   // scale of row m, block b: sa[m * sa_row + b * sa_blk]
    int64_t sa_row, sa_blk;
    const float* sb;   // [G][n_blocks][k_blocks]
    uint16_t* d;
    const int32_t* offsets;   // grouped: device array of groups + 1 row offsets
    int32_t rows, N, k_blocks, n_blocks, groups, grid_n, group_m, num_tiles;
};

// A work unit: one output tile.
struct Fp8Unit {
    int32_t row0, row_end;   // the tile's rows are [row0, min(row0 + kTileM, row_end))
    int32_t n0, group;
};

// Rows [lo, hi) of group g.  `ordered`: no offset is outside [0, rows] or below the
// one before it.  Otherwise each counts as the largest so far, within [0, rows], so
// that groups neither overlap nor lead outside the operands.
struct RowRange {
    int32_t lo, hi;
};
__device__ __forceinline__ RowRange group_rows(const Fp8Problem& p, int32_t g, bool ordered) {
    RowRange r = {p.offsets[g], p.offsets[g + 1]};
    if (!ordered) {
#pragma unroll 1
        for (int32_t i = 0; i < g; ++i) r.lo = max(r.lo, p.offsets[i]);
        r.lo = min(max(r.lo, 0), p.rows);
        r.hi = min(max(r.hi, r.lo), p.rows);
    }
    return r;
}

template <class C>
__device__ __forceinline__ Fp8Unit unit_of(const Fp8Problem& p, const int32_t* start, int32_t u) {
    Fp8Unit t;
    if constexpr (C::kGrouped) {
        int32_t lo = 0, hi = p.groups;   // the last group whose first tile is <= u
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (start[mid] <= u) lo = mid; else hi = mid;
        }
        const RowRange r = group_rows(p, lo, start[-1] == 0);
        const TileCoord tc = tile_coord(u - start[lo], (r.hi - r.lo + C::kTileM - 1) / C::kTileM,
                                        p.grid_n, p.group_m);
        t.row0 = r.lo + tc.m_blk * C::kTileM;
        t.row_end = r.hi;
        t.n0 = tc.n_blk * C::BN;
        t.group = lo;
    } else {
        const TileCoord tc = tile_coord(u, ceil_div(p.rows, C::kTileM), p.grid_n, p.group_m);
        t.row0 = tc.m_blk * C::kTileM;
        t.row_end = p.rows;
        t.n0 = tc.n_blk * C::BN;
        t.group = 0;
    }
    return t;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
gemm_fp8_kernel(const __grid_constant__ Fp8Problem prob, const uint64_t limit_ns,
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
    auto mma_done_bar = [&](uint32_t h) {
        return bar0 + 8u * (2 * C::STAGES + 2 * C::kAccs + h);
    };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile uint32_t* ring_count = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);
    int32_t* start = reinterpret_cast<int32_t*>(smem + C::kOffStart);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const uint32_t rank = C::kPair ? cluster_ctarank() : 0u;
    const int32_t unit0 = static_cast<int32_t>(blockIdx.x) / (C::kPair ? 2 : 1);
    const int32_t unit_step = static_cast<int32_t>(gridDim.x) / (C::kPair ? 2 : 1);

    grid_launch_dependents();

    if (warp == 0) {
        if (elect_one()) {
            for (uint32_t s = 0; s < (uint32_t)C::STAGES; ++s) {
                mbar_init(full_bar(s), 1);
                mbar_init(empty_bar(s), C::kParts);   // one commit per MMA issuer
            }
            for (uint32_t a = 0; a < (uint32_t)C::kAccs; ++a) {
                mbar_init(acc_full_bar(a), 1);
                // The leader's acc_empty collects the epilogue warps of both CTAs.
                mbar_init(acc_empty_bar(a), (C::kPair ? 2 : 1) * (C::kEpiWarps / C::kParts));
            }
            for (uint32_t h = 0; h < (uint32_t)C::kParts; ++h) mbar_init(mma_done_bar(h), 1);
            *abort_flag = 0;
            if constexpr (kChecked) {
                for (int i = 0; i <= C::kParts; ++i) ring_count[i] = 0;
            }
            fence_mbarrier_init();
            tma_prefetch_desc(&prob.tmA);
            tma_prefetch_desc(&prob.tmB);
            tma_prefetch_desc(&prob.tmD);
        }
        __syncwarp();
    }
    if (warp == 1) {
        if constexpr (C::kPair) {
            tmem_alloc_pair(smem_u32(tmem_holder), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_holder), 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (C::kPair) cluster_sync_after_init();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_dependency_wait();

    int32_t num_units = prob.num_tiles;
    if constexpr (C::kGrouped) {
        // Tiles of each group, then their running sum by one warp.
        auto count_tiles = [&](int32_t g, RowRange r) {
            start[g + 1] = (r.hi - r.lo + C::kTileM - 1) / C::kTileM * prob.grid_n;
        };
        bool ordered = true;
        for (int32_t g = static_cast<int32_t>(threadIdx.x); g < prob.groups; g += C::kThreads) {
            const RowRange r = group_rows(prob, g, true);
            const bool good = 0 <= r.lo && r.lo <= r.hi && r.hi <= prob.rows;
            if (good) count_tiles(g, r);
            ordered = ordered && good;
        }
        ordered = __syncthreads_and(ordered);
        if (!ordered) {
            for (int32_t g = static_cast<int32_t>(threadIdx.x); g < prob.groups; g += C::kThreads)
                count_tiles(g, group_rows(prob, g, false));
            __syncthreads();
        }
        if (warp == 0) {
            int32_t carry = 0;
            for (int32_t g0 = 0; g0 < prob.groups; g0 += 32) {
                int32_t v = g0 + lane < prob.groups ? start[g0 + lane + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += o;
                }
                if (g0 + lane < prob.groups) start[g0 + lane + 1] = carry + v;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) {
                start[0] = 0;
                start[-1] = !ordered;   // (a word of shared memory: no register to spare)
            }
        }
        __syncthreads();
        num_units = start[prob.groups];
    }

    if (warp < 4) {
        set_max_regs_dec<C::kRoleRegs>();
    if (warp == 0) {
        // ================= TMA producer =================
        // The whole warp walks the loop (its control flow and addresses are the
        // same in every lane); one lane issues.
        const bool lead = elect_one();
        uint32_t s = 0, phase = 0, it = 0;
        bool ok = true;
        for (int32_t u = unit0; ok && u < num_units; u += unit_step) {
            const Fp8Unit t = unit_of<C>(prob, start, u);
            // Boxes of A with at least one row, in this CTA and in all.
            int32_t boxes = 1, all_boxes = C::kPair ? 2 : 1;
            if constexpr (C::kGrouped) {
                constexpr int32_t kMost = C::BM / C::kABoxRows;
                auto count = [&](int32_t r) {
                    const int32_t left = t.row_end - (t.row0 + r * C::BM);
                    return min(max((left + C::kABoxRows - 1) / C::kABoxRows, 0), kMost);
                };
                boxes = count(static_cast<int32_t>(rank));
                all_boxes = C::kPair ? count(0) + count(1) : boxes;
            }
            const uint32_t bytes = static_cast<uint32_t>(all_boxes) * (C::kABoxRows * C::BK) +
                                   (C::kPair ? 2u : 1u) * C::kBBytes;
            const int32_t a_row = t.row0 + static_cast<int32_t>(rank) * C::BM;
            const int32_t b_row = t.n0 + static_cast<int32_t>(rank) * C::kBBoxRows;
            for (int32_t kb = 0; kb < prob.k_blocks; ++kb, ++it) {
                ok = __all_sync(0xffffffffu, wait_many(empty_bar(s), phase ^ 1u, abort_flag, err,
                                                       kSiteProducerEmpty, limit_ns)) &&
                     check_ok(a_row >= 0 && b_row >= 0, err, kSiteCheckTma);
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                if (lead) {
                    const uint32_t a_dst = sbase + s * C::kStageBytes;
                    const uint32_t b_dst = a_dst + C::kABytes;
                    if constexpr (C::kPair) {
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(s), bytes);
                        const uint32_t bar = map_to_rank(full_bar(s), 0);
                        for (int32_t i = 0; i < boxes; ++i)
                            tma_load_2d_pair(a_dst + i * (C::kABoxRows * C::BK), &prob.tmA,
                                             kb * C::BK, a_row + i * C::kABoxRows, bar);
#pragma unroll
                        for (int h = 0; h < C::kParts; ++h)
                            tma_load_3d_pair(b_dst + h * (C::kBBoxRows * C::BK), &prob.tmB,
                                             kb * C::BK, b_row + h * C::kAccCols, t.group, bar);
                    } else {
                        mbar_arrive_expect_tx(full_bar(s), bytes);
                        for (int32_t i = 0; i < boxes; ++i)
                            tma_load_2d(a_dst + i * (C::kABoxRows * C::BK), &prob.tmA, kb * C::BK,
                                        a_row + i * C::kABoxRows, full_bar(s));
                        tma_load_3d(b_dst, &prob.tmB, kb * C::BK, b_row, t.group, full_bar(s));
                    }
                }
                __syncwarp();
                if (++s == (uint32_t)C::STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        if constexpr (kChecked) ring_count[0] = it;
        // The last stages issued must have landed before shared memory is
        // released (a pair: the leader's barriers count both CTAs' loads, and
        // the peer stays until the final cluster barrier).
        if (rank == 0 && lead) {
            const uint32_t first = it > (uint32_t)C::STAGES ? it - C::STAGES : 0u;
            for (uint32_t j = first; j < it; ++j)
                wait_bounded(full_bar(ring_stage(j, C::STAGES)), ring_phase(j, C::STAGES), err,
                             kSiteDrainFull, limit_ns);
        }
        __syncwarp();
    } else if (warp <= C::kParts) {
        // ===== MMA issuers (the leader's, for a pair): warp 1 + h part h =====
        if (rank == 0) {
            constexpr uint32_t kIdesc = idesc_e4m3(C::kTileM, C::kAccCols);
            // B rows (in this CTA) of one part.
            constexpr uint32_t kPartBytes = (C::kBRows / C::kParts) * C::BK;
            const bool lead = elect_one();
            const uint32_t h = static_cast<uint32_t>(warp - 1);
            const uint64_t a_desc0 = umma_desc_sw128_kmajor(sbase);
            const uint64_t b_desc0 = umma_desc_sw128_kmajor(sbase + C::kABytes + h * kPartBytes);
            // The stage and its phase; the accumulator (parts h, h + kParts, ...
            // of the running count go round the kAccs) and the phase in which
            // its use before this one is read (the first time: at once).
            uint32_t s = 0, phase = 0, a = h, a_phase = 1, it = 0;
            bool ok = true;
            for (int32_t u = unit0; ok && u < num_units; u += unit_step) {
                for (int32_t kb = 0; kb < prob.k_blocks; ++kb, ++it) {
                    ok = __all_sync(0xffffffffu,
                                    wait_many(acc_empty_bar(a), a_phase, abort_flag, err,
                                              kSiteMmaAccEmpty, limit_ns) &&
                                        wait_many(full_bar(s), phase, abort_flag, err,
                                                  kSiteMmaFull, limit_ns));
                    if (!ok) break;
                    tc_fence_after();
                    if (lead) {
                        // Each step of 32 k is 32 bytes further along the rows (the
                        // descriptors' address field counts 16 bytes).
                        const uint64_t a_desc = a_desc0 + s * (C::kStageBytes / 16);
                        const uint64_t b_desc = b_desc0 + s * (C::kStageBytes / 16);
                        const uint32_t d_tmem = tmem_base + a * C::kAccCols;
#pragma unroll
                        for (int j = 0; j < C::BK / 32; ++j)
                            mma_e4m3<C::kPair>(d_tmem, a_desc + 2 * j, b_desc + 2 * j, kIdesc,
                                               j != 0 ? 1u : 0u);
                        // The accumulator is full, and this part done with stage
                        // s (in both CTAs of a pair), once these MMAs finish.
                        if constexpr (C::kPair) {
                            mma_commit_pair(acc_full_bar(a), 0x3u);
                            mma_commit_pair(empty_bar(s), 0x3u);
                        } else {
                            mma_commit(acc_full_bar(a));
                            mma_commit(empty_bar(s));
                        }
                    }
                    __syncwarp();
                    if (++s == (uint32_t)C::STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                    a += C::kParts;
                    if (a >= (uint32_t)C::kAccs) {
                        a = h;
                        a_phase ^= 1u;
                    }
                }
            }
            if constexpr (kChecked) ring_count[1 + h] = it;
            // All issued MMAs must finish before TMEM is released.
            if (lead) {
                if constexpr (C::kPair)
                    mma_commit_pair(mma_done_bar(h), 0x1u);
                else
                    mma_commit(mma_done_bar(h));
                wait_bounded(mma_done_bar(h), 0, err, kSiteDrainMma, limit_ns);
            }
            __syncwarp();
        }
    }
    } else {
        set_max_regs_inc<C::kEpiRegs>();
        // ================= scaling and epilogue (warps 4..11) =================
        const uint32_t quarter = static_cast<uint32_t>(warp) & 3u;      // TMEM lane quarter
        // Columns [kCols * group, + kCols) of the tile: part h, from column c0 of
        // its accumulator.
        const uint32_t col = (static_cast<uint32_t>(warp - 4) >> 2) * C::kCols;
        const uint32_t h = col / C::kAccCols;
        const uint32_t t_base = tmem_base + ((quarter * 32u) << 16) + col % C::kAccCols;
        const uint32_t buf = sbase + C::kOffD +
                             static_cast<uint32_t>(warp - 4) * (C::kBoxes * C::kBoxBytes);
        // The accumulator of this warp's next part: parts h, h + kParts, ... of
        // the running count go round the kAccs accumulators.
        uint32_t slot = h, parity = 0;
        const uint32_t full0 = acc_full_bar(0);
        const uint32_t empty0 = C::kPair ? map_to_rank(acc_empty_bar(0), 0) : acc_empty_bar(0);
        uint32_t full_at = full0 + 8u * slot, empty_at = empty0 + 8u * slot;
        uint32_t t_acc = t_base + slot * C::kAccCols;
        auto next_acc = [&]() {
            slot += C::kParts;
            if (slot >= static_cast<uint32_t>(C::kAccs)) {
                slot = h;
                parity ^= 1u;
            }
            full_at = full0 + 8u * slot;
            empty_at = empty0 + 8u * slot;
            t_acc = t_base + slot * C::kAccCols;
        };
        // The tile that is being scaled, or about to be: this warp's 32 rows from
        // y and kCols columns from x of D.
        const int32_t last = prob.k_blocks - 1;
        int32_t y = 0, x = 0, row_end = 0;
        // Its scales: the row's for four k-blocks at a time, read while the four
        // before them are used (loads issued one by one as they are used would
        // make every use wait for the newest: a warp waits for all loads it has
        // in flight), and the weights' for 32, one per lane.  Lanes past the
        // last row read that row's (their sums are not stored), and blocks past
        // the last read the last.  A warp's columns lie in two blocks of weight
        // scales at most.
        const float *sa = prob.sa, *sb = prob.sb, *sb2 = prob.sb;
        float sa_next[4], sb_next[2] = {};
        auto fetch = [&](int32_t kb0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) sa_next[j] = sa[min(kb0 + j, last) * prob.sa_blk];
        };
        auto fetch_sb = [&](int32_t kb) {
            sb_next[0] = sb[min(kb + lane, last)];
            if constexpr (C::kTwoBlocks) sb_next[1] = sb2[min(kb + lane, last)];
        };
        // Moves on to tile u and starts on its first scales, which so travel while
        // the tile before it is stored.
        auto begin_tile = [&](int32_t u) {
            if (u >= num_units) return;
            const Fp8Unit t = unit_of<C>(prob, start, u);
            y = t.row0 + static_cast<int32_t>(rank * C::BM + quarter * 32u);
            x = t.n0 + static_cast<int32_t>(col);
            row_end = t.row_end;
            if (y >= row_end) return;
            sa = prob.sa + min(y + lane, row_end - 1) * prob.sa_row;
            const int32_t nb = min(x / kFp8Block, prob.n_blocks - 1);
            sb = prob.sb +
                 (static_cast<int64_t>(t.group) * prob.n_blocks + nb) * prob.k_blocks;
            sb2 = nb + 1 < prob.n_blocks ? sb + prob.k_blocks : sb;
            fetch_sb(0);
            fetch(0);
        };
        begin_tile(unit0);
        for (int32_t u = unit0; u < num_units; u += unit_step) {
            if (y >= row_end) {
                // No row of this warp exists: it only hands the accumulators back.
                for (int32_t kb = 0; kb <= last; ++kb) {
                    if (!__all_sync(0xffffffffu,
                                    wait_many(full_at, parity, abort_flag, err,
                                                   kSiteEpiAccFull, limit_ns)))
                        goto stop;
                    mbar_arrive_if(lane == 0, empty_at);
                    next_acc();
                }
                begin_tile(u + unit_step);
                continue;
            }
            // The first piece in the second block of weight scales.
            const int32_t second = (kFp8Block - x % kFp8Block) / 32;
            float sb_lane[2] = {};
            f32x2 acc[C::kCols / 2];
#pragma unroll
            for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
            // The pieces go through kBatch register buffers.  Where they take
            // them all at once, a part is read whole and its accumulator goes back
            // to the MMA warp before the first multiply-add.  Where a part takes
            // more than one round of the buffers, a buffer is refilled as soon as
            // its piece has been scaled, with a piece of the next round (of this
            // part, or of the next k-block's): TMEM is read under the
            // multiply-adds, and the accumulator goes back after its last round
            // (at 8192^3 371 against 390 us; for one-round parts this order hands
            // them back later and costs more than it hides, 444 against 396 us).
            constexpr int kRounds = C::kPieces / C::kBatch;
            uint32_t v[C::kBatch][32];
            auto part_ready = [&]() {
                const bool ready = __all_sync(
                    0xffffffffu, wait_many(full_at, parity, abort_flag, err, kSiteEpiAccFull,
                                           limit_ns));
                tc_fence_after();
                return ready;
            };
            // (Read by every lane: the wait is collective.)
            auto round_read = [&](bool last_round) {
                tmem_ld_wait();
                if (last_round) {
                    tc_fence_before();
                    mbar_arrive_if(lane == 0, empty_at);
                    next_acc();
                }
            };
            auto first_round = [&]() {
                if (!part_ready()) return false;
#pragma unroll
                for (int c = 0; c < C::kBatch; ++c) tmem_ld_32x32b_x32(t_acc + 32 * c, v[c]);
                round_read(kRounds == 1);
                return true;
            };
            if (kRounds > 1 && !first_round()) goto stop;
            for (int32_t kb0 = 0; kb0 <= last; kb0 += 4) {
                if ((kb0 & 31) == 0) {
                    sb_lane[0] = sb_next[0];
                    sb_lane[1] = sb_next[1];
                }
                float sa_now[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) sa_now[j] = sa_next[j];
                fetch(kb0 + 4);
                if ((kb0 & 31) == 0) fetch_sb(kb0 + 32);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kb0 + j > last) break;
                    float scale[2];
                    scale[0] = sa_now[j] * __shfl_sync(0xffffffffu, sb_lane[0], (kb0 & 31) + j);
                    if constexpr (C::kTwoBlocks)
                        scale[1] =
                            sa_now[j] * __shfl_sync(0xffffffffu, sb_lane[1], (kb0 & 31) + j);
                    if (kRounds == 1 && !first_round()) goto stop;
#pragma unroll
                    for (int r = 0; r < kRounds; ++r) {
                        // The round to read after this one, if there is one.
                        constexpr int kLast = kRounds - 1;
                        const int next_r = r == kLast ? 0 : r + 1;
                        const bool more = kRounds > 1 && (r < kLast || kb0 + j < last);
#pragma unroll
                        for (int c = 0; c < C::kBatch; ++c) {
                            const int piece = r * C::kBatch + c;
                            const float f = C::kTwoBlocks && piece >= second ? scale[1] : scale[0];
                            const f32x2 f2 = pack_f32x2(f, f);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                scale_add(acc[16 * piece + i], v[c][2 * i], v[c][2 * i + 1], f2);
                            if (more) {
                                if (c == 0 && next_r == 0 && !part_ready()) goto stop;
                                tmem_ld_32x32b_x32(t_acc + 32 * (next_r * C::kBatch + c), v[c]);
                            }
                        }
                        if (more) round_read(next_r == kLast);
                    }
                }
            }
            // ---- round, stage in shared memory, store ----
            const int32_t y0 = y, x0 = x;
            const int32_t left = row_end - y;   // rows of this warp that exist
            begin_tile(u + unit_step);
            if (lane == 0) bulk_wait_group_read<0>();   // the last tile's stores have left
            __syncwarp();
#pragma unroll
            for (int c = 0; c < C::kCols / 8; ++c) {
                constexpr int kChunks = C::kBoxChunks;
                const uint32_t at = buf + (c / kChunks) * C::kBoxBytes +
                                    C::box_at(static_cast<uint32_t>(lane), c % kChunks);
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    unpack_f32x2(acc[4 * c + i], lo, hi);
                    p[i] = pack2_rn<C::kBF16>(__float_as_uint(lo), __float_as_uint(hi));
                }
                st_shared_v4(at, p[0], p[1], p[2], p[3]);
            }
            const bool whole = !C::kGrouped || left >= 32;
            if (whole) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && left > 0) {
#pragma unroll
                    for (int b = 0; b < C::kBoxes; ++b)
                        if (x0 + C::kBoxCols * b < prob.N &&
                            check_ok((x0 & 7) == 0 && x0 >= 0 && y0 >= 0, err, kSiteCheckTma))
                            tma_store_2d(&prob.tmD, buf + b * C::kBoxBytes, x0 + C::kBoxCols * b,
                                         y0);
                    bulk_commit_group();
                }
                __syncwarp();
            } else {
                // The group ends inside these 32 rows: plain stores of the rows
                // that exist, a lane per 16-byte chunk (the next rows are another
                // group's).
                __syncwarp();
                constexpr int32_t kLanes = C::kBoxChunks;   // lanes of a row
                const int32_t chunk = lane % kLanes;
                for (int32_t r = lane / kLanes; r < left; r += 32 / kLanes) {
#pragma unroll
                    for (int b = 0; b < C::kBoxes; ++b) {
                        const int32_t n = x0 + C::kBoxCols * b + 8 * chunk;
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            smem + (buf - sbase) + b * C::kBoxBytes + C::box_at(r, chunk));
                        if (n < prob.N && check_ok(y0 + r < prob.rows && n + 8 <= prob.N, err,
                                                   kSiteCheckBounds))
                            *reinterpret_cast<uint4*>(
                                prob.d + static_cast<int64_t>(y0 + r) * prob.N + n) = v;
                    }
                }
                __syncwarp();
            }
            if constexpr (kChecked) {
                if (warp == 4 && lane == 0 && rank == 0) check_count_unit(err, u);
                __syncwarp();
            }
        }
    stop:
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if constexpr (kChecked) {
        if (threadIdx.x == 0 && rank == 0 && !*abort_flag)
            for (int h = 0; h < C::kParts; ++h)
                check_ok(ring_count[0] == ring_count[1 + h], err, kSiteCheckRing);
        __syncwarp();
    }
    if constexpr (C::kPair) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (C::kPair)
            tmem_dealloc_pair(tmem_base, 512);
        else
            tmem_dealloc(tmem_base, 512);
    }
}

// The tiles: 256 x 256 and 256 x 192 in CTA pairs, 128 x 128.
template <bool G, bool T> using FpPair256 = Fp8Cfg<256, 128, 128, 5, true, G, T>;
template <bool G, bool T> using FpPair192 = Fp8Cfg<192, 96, 96, 6, true, G, T>;
template <bool G, bool T> using FpTile = Fp8Cfg<128, 128, 64, 6, false, G, T>;

// D {N, rows} in store boxes of 64 or 32 columns x 32 rows.
int encode_output(EncodeTiled encode, CUtensorMap* map, void* base, uint64_t N, uint64_t rows,
                  bool bf16, uint32_t box_cols) {
    cuuint64_t dims[2] = {N, rows};
    cuuint64_t strides[1] = {N * 2};
    cuuint32_t box[2] = {box_cols, 32};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? 0
               : -1;
}

template <class C>
cudaError_t launch_cfg(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    Fp8Problem p;
    const int64_t G = C::kGrouped ? g.groups : 1;
    if (encode_fp8_operand(dev.encode, &p.tmA, g.A, g.K, g.M, 0, C::kABoxRows) ||
        encode_fp8_operand(dev.encode, &p.tmB, g.B, g.K, g.N, G, C::kBBoxRows) ||
        encode_output(dev.encode, &p.tmD, g.D, g.N, g.M, C::kBF16, C::kBoxCols))
        return cudaErrorInvalidValue;
    p.sa = g.SA;
    p.sa_row = g.sa_row;
    p.sa_blk = g.sa_blk;
    p.sb = g.SB;
    p.d = static_cast<uint16_t*>(g.D);
    p.offsets = g.offsets;
    p.rows = static_cast<int32_t>(g.M);
    p.N = static_cast<int32_t>(g.N);
    p.k_blocks = static_cast<int32_t>(ceil_div(g.K, C::BK));
    p.n_blocks = static_cast<int32_t>(ceil_div(g.N, kFp8Block));
    p.groups = static_cast<int32_t>(G);
    p.grid_n = static_cast<int32_t>(ceil_div(g.N, C::BN));
    p.group_m = 8;
    const int64_t grid_m = ceil_div(g.M, C::kTileM);
    // Grouped: the most tiles the groups can have (each adds at most one
    // partly filled row of tiles); the real number is read on the device.
    int64_t tiles = grid_m * p.grid_n;
    if (C::kGrouped) tiles = (g.M / C::kTileM + (G < g.M ? G : g.M)) * p.grid_n;
    p.num_tiles = static_cast<int32_t>(tiles);
    const int64_t slots = C::kPair ? dev.pairs : dev.sms;
    const int64_t ctas = (tiles < slots ? tiles : slots) * (C::kPair ? 2 : 1);
    static ContextMarks attr_done;
    auto kernel = gemm_fp8_kernel<C>;
    if (cudaError_t e = smem_opt_in(kernel, static_cast<int>(C::kSmemBytes), attr_done)) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)), dim3(C::kThreads),
                         C::kSmemBytes, stream, C::kPair ? 2 : 1, dev.pdl, p, dev.limit_ns,
                         dev.err_word);
}

// Which pair tile: the one whose rounds of tiles over the pairs take less.  A
// round of 256 x 192 tiles takes about 0.76 of one of 256 x 256 (4096^3: 10.3
// against 13.8 us), so 1237 x 5000 x 2064 (135 tiles in 2 rounds against 100 in 2)
// runs in 17.4 against 19.5 us and 4096^3 (352 in 5 against 256 in 4) in 51.7
// against 55.1, but 2048 x 4096 x 4096 (176 in 3 against 128 in 2) in 31.8
// against 29.4 us.  At 8192^3 (19 rounds against 14) both take 368 us.
bool narrow_pairs(int64_t tile_rows, int64_t N, int pairs) {
    const int64_t wide = ceil_div(tile_rows * ceil_div(N, 256), pairs) * 100;
    const int64_t narrow = ceil_div(tile_rows * ceil_div(N, 192), pairs) * 76;
    return narrow < wide;
}

template <bool G, bool T>
cudaError_t launch_pairs(const Fp8Gemm& g, int64_t tile_rows, const Fp8Device& dev,
                         cudaStream_t stream) {
    return narrow_pairs(tile_rows, g.N, dev.pairs) ? launch_cfg<FpPair192<G, T>>(g, dev, stream)
                                                   : launch_cfg<FpPair256<G, T>>(g, dev, stream);
}

template <bool T>
cudaError_t launch_typed(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    const int64_t rows256 = ceil_div(g.M, 256);
    if (g.offsets) {
        // Whole 256-row tiles pay when the groups fill most of them and there are
        // enough of them.  (How the rows fall into groups is only known on the
        // device: half a tile row is added for each group's last, partly filled one.)
        // 4 groups, 2000 x 512 x 1024: 6.2 us in 128 x 128 tiles, 7.0 in pairs.
        const int64_t tile_rows = rows256 + g.groups / 2;
        if (dev.pairs > 0 && g.M >= 192 * g.groups &&
            2 * tile_rows * ceil_div(g.N, 256) > dev.pairs)
            return launch_pairs<true, T>(g, tile_rows, dev, stream);
        return launch_cfg<FpTile<true, T>>(g, dev, stream);
    }
    if (dev.pairs > 0 && 2 * rows256 * ceil_div(g.N, 256) > dev.pairs)
        return launch_pairs<false, T>(g, rows256, dev, stream);
    return launch_cfg<FpTile<false, T>>(g, dev, stream);
}

}  // namespace

int encode_fp8_operand(EncodeTiled encode, CUtensorMap* map, const void* base, uint64_t K,
                       uint64_t rows, uint64_t mats, uint32_t box_rows) {
    cuuint64_t dims[3] = {K, rows, mats};
    cuuint64_t strides[2] = {K, K * rows};
    cuuint32_t box[3] = {kFp8Block, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, mats == 0 ? 2 : 3, const_cast<void*>(base),
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? 0
               : -1;
}

cudaError_t launch_gemm_fp8(const Fp8Gemm& g, const Fp8Device& dev, cudaStream_t stream) {
    return g.bf16 ? launch_typed<true>(g, dev, stream) : launch_typed<false>(g, dev, stream);
}

}  // namespace tmagemm
