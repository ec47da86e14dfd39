// Products of more than a few tokens with 4-bit weights and group scales, on tcgen05:
//   D[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] (q[n][k] - z[n][g]).
//
// The weights are the left operand, 128 rows of them by up to 32 tokens.  A thread owns a
// row: it takes its codes out of shared memory, makes exact 16-bit numbers of q - z and
// stores those into its lane of TMEM, from where tcgen05.mma reads them, so that the widened
// weights, four times the bytes that are read, never pass through shared memory.  Each scale
// group's sum is in an accumulator of its own; the thread reads it back and adds it, times
// the row's scale, to its FP32 sums in registers.
//
// Sixteen warps are four warpgroups with a part of TMEM and a ring of stages each: while one
// waits for its products the others widen.  With units for all of them each has units of its
// own; otherwise they take every fourth 128 k of one.  Each has one more
// warp that copies by TMA and issues the products: done by a widening warp those took
// a third of its time, 0.5 us of 1.5 a step.
// At the end of a unit that they share the warpgroups' sums meet in shared memory and are
// added in a fixed order; with a cluster its CTAs split K, and each adds up a part of their
// sums.
//
// A step of 128 rows by 512 k takes 0.85 us as measured.  Widening is 10 instructions for
// eight codes, six of them on the ALU, which takes one in two cycles: 0.4 us of that.  The
// rest is latency that 20 warps an SM do not cover: the wait for a stage, the hand-over to
// the products and back, the read-back of their sums (47 to 58 % of the issue slots, 29 to
// 41 % of the ALU and 9 to 12 % of the tensor pipe are in use).
// 64 groups with 128 rows, 35 of them with any, N x K = 4096 x 2048: 42.5 us (3.5 TB/s of
// codes; 52 with shared units).
// 27 x 14336 x 4096 takes 13.5 us with groups of 128 (2.2 TB/s of codes; 16.2 with the warps that
// widen issuing), 15.8 with 64 and 23.3 with 32, whose sums are read back more often.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"
#include "tile_sched.cuh"
#include "w4.cuh"

namespace tmagemm {

namespace {

constexpr int kRows = 128;                  // of a unit: TMEM's lanes
constexpr int kParts = 4;                   // warpgroups
constexpr int kWorkers = 128 * kParts;      // threads that compute
constexpr int kThreads = kWorkers + 32 * kParts;       // and a warp that copies and issues for each part
// Registers of a worker and of an issuer (of the 96 that each thread starts with).
constexpr int kWorkerRegs = 112, kIssuerRegs = 32;
static_assert(kWorkers * kWorkerRegs + (kThreads - kWorkers) * kIssuerRegs <= kThreads * 96);
constexpr uint32_t kCodeBytes = kRows * 64; // of a stage: 128 k
constexpr uint32_t kPartCols = 512 / kParts;           // of TMEM: 64 for weights, 64 for sums

template <bool BF16_, int GB_, bool GROUPED_, bool ALONE_>
struct ManyCfg {
    static constexpr int NT = 32, kTokens = NT;
    static constexpr int GB = GB_;          // blocks of 32 k of a scale
    static constexpr bool kBF16 = BF16_, kGrouped = GROUPED_;
    static constexpr bool kAlone = ALONE_;  // a warpgroup has a unit of its own
    static constexpr int kSplit = ALONE_ ? 1 : kParts;      // warpgroups that split K
    // A step: blocks of 32 k whose sums, one per scale, are in TMEM at a time.
    static constexpr int kStep = 64 / NT * GB < 4 ? 64 / NT * GB : 4;
    static constexpr int kAccs = kStep / GB, kScales = 4 / GB;
    static constexpr uint32_t kSumBytes = kAlone ? 0 : kParts * 16 * kRows * 4;
    static_assert(kAccs >= 1 && kAccs * NT <= 64 && kStep % GB == 0 && 4 % kStep == 0);
};

struct ManyProblem {
    CUtensorMap tm_codes;    // {K / 2, rows of all groups}, box {64, 128}
    CUtensorMap tm_tokens;   // A {K, M}, box {64, tokens}
    W4Args a;
    int32_t box, row_blocks; // rows of a unit; units of rows of a group
    int32_t cluster, depth;  // CTAs that split K, stages of a ring
    int32_t tokens;          // of a stage, a multiple of 16
    uint32_t stage_bytes;    // codes and tokens
    uint32_t off_sums, off_misc;
};

struct ManyMisc {
    uint64_t full[kParts][kMaxDepth], ready[kParts], done[kParts], sum_full, sum_empty;
    int abort_flag;
    uint32_t tmem;
    W4Groups groups;
};

// Eight codes as four pairs of neighbours, exactly.  The bytes of a word with the lower or the
// upper codes alone (16 times as large) are put, with zeros above them, into the halves of a
// word: the 16-bit subnormals q 2^-24 and 16 q 2^-24 (fp16) or 2^-133 (bf16; those past 127
// are its smallest normal numbers, which go on in the same steps).  One multiply-add makes
// (q - z) 2^-9 or (q - z) 2^-6 of them.
template <bool BF16>
struct WidenPairs {
    static constexpr float kScale = BF16 ? 64.0f : 512.0f;   // what the products are multiplied with
    uint32_t add;
    __device__ __forceinline__ explicit WidenPairs(uint32_t z) {
        add = fma16x2<BF16>(z * 0x10001u, BF16 ? 0xff00ff00u : 0xf800f800u, 0x80008000u);
    }
    template <int BYTE>
    __device__ __forceinline__ uint32_t pair(uint32_t lower, uint32_t upper) const {
        // (Selectors with bit 3 set copy the sign of a lower code's byte: zeros.)
        uint32_t v;
        asm("prmt.b32 %0, %1, %2, %3;"
            : "=r"(v)
            : "r"(lower), "r"(upper), "n"(0x8480 + 0x101 * BYTE));
        return fma16x2<BF16>(v, BF16 ? 0x7d007f00u : 0x68007800u, add);
    }
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t* out) const {
        const uint32_t lower = w & 0x0f0f0f0fu, upper = w & 0xf0f0f0f0u;
        out[0] = pair<0>(lower, upper);
        out[1] = pair<1>(lower, upper);
        out[2] = pair<2>(lower, upper);
        out[3] = pair<3>(lower, upper);
    }
};

// 16 consecutive columns of the warp's 32 lanes of TMEM.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
          "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
          "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D(tmem) (+)= A(tmem) B(smem)^T, one CTA.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// wait_or_abort for a barrier that other CTAs of the cluster arrive on, whose writes
// are read after it.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, uint32_t* err,
                                             uint64_t limit_ns) {
    const uint64_t t0 = clock64(), lim = limit_cycles(limit_ns);
    for (uint32_t spin = 0;; ++spin) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred P;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, P;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if ((spin & 15u) == 15u && static_cast<uint64_t>(clock64()) - t0 > lim) {
            *abort_flag = 1;
            record_error(err, kSiteEpiAccFull);
            return false;
        }
    }
}

// A worker: its place, and its sums.
template <class C>
struct Worker {
    int wg, row;
    uint32_t lanes;                      // its warp's, in TMEM
    float acc[C::NT];
};

// Adds a step's sums, times its scales.
template <class C>
__device__ __forceinline__ void add_sums(Worker<C>& w, uint32_t at, const float (&scale)[C::kAccs],
                                         int tokens) {
#pragma unroll
    for (int j = 0; j < C::kAccs; ++j) {
        uint32_t lo[16], hi[16];
        tmem_ld_32x32b_x16(at + j * C::NT, lo);
        if (tokens > 16) tmem_ld_32x32b_x16(at + j * C::NT + 16, hi);
        tmem_ld_wait();
        // (Nothing that uses them comes earlier.)
#pragma unroll
        for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(lo[e]), "+r"(hi[e]));
#pragma unroll
        for (int e = 0; e < 16; ++e)
            w.acc[e] = fmaf(__uint_as_float(lo[e]), scale[j], w.acc[e]);
        if (tokens > 16)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                w.acc[16 + e] = fmaf(__uint_as_float(hi[e]), scale[j], w.acc[16 + e]);
    }
}

// The results of a warpgroup's own unit.
template <class C>
__device__ __forceinline__ void store_rows(const W4Args& a, const Worker<C>& w, const Unit& t,
                                           uint32_t* err) {
    if (w.row < t.rows && check_ok(t.n + w.row < a.N && t.m + t.tokens <= a.M, err,
                                   kSiteCheckBounds)) {
        uint16_t* to = a.D + static_cast<int64_t>(t.m) * a.N + t.n + w.row;
#pragma unroll
        for (int tok = 0; tok < C::NT; ++tok)
            if (tok < t.tokens)
                to[static_cast<int64_t>(tok) * a.N] = cvt16_rn<C::kBF16>(
                    __float_as_uint(w.acc[tok] * WidenPairs<C::kBF16>::kScale));
    }
    __syncwarp();
}

// The end of a unit that warpgroups share (see above).  False after a wait that failed, in this warp or another.
template <class C>
__device__ __forceinline__ bool finish(const ManyProblem& p, ManyMisc& misc, float* sums,
                                       Worker<C>& w, const Unit& t, int32_t rank, uint32_t unit,
                                       bool ok, uint64_t limit_ns, uint32_t* err) {
    const W4Args& a = p.a;
    const bool clusters = p.cluster > 1;
    volatile int* abort_flag = &misc.abort_flag;
    const int tid = static_cast<int>(threadIdx.x);
    auto store = [&](int tok, int row, float sum) {
        if (row < t.rows && check_ok(t.n + row < a.N && t.m + tok < a.M, err, kSiteCheckBounds))
            a.D[static_cast<int64_t>(t.m + tok) * a.N + t.n + row] =
                cvt16_rn<C::kBF16>(__float_as_uint(sum));
    };
    if (clusters && unit > 0)     // the cluster has read the sums of the unit before
        ok = __all_sync(kAll, wait_cluster(smem_u32(&misc.sum_empty), (unit - 1) & 1u, abort_flag,
                                           err, limit_ns)) &&
             ok;
    // Sixteen tokens at a time: each warpgroup adds up four of them.
    float sum[C::NT / 4];
#pragma unroll
    for (int n = 0; n < C::NT; n += 16) {
        if (n > 0 && n >= t.tokens) break;
        __syncwarp();
        if (!named_bar_and(1, kWorkers, ok)) return false;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[(w.wg * 16 + i) * kRows + w.row] = w.acc[n + i] * WidenPairs<C::kBF16>::kScale;
        __syncwarp();
        named_bar_sync(1, kWorkers);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float* at = sums + (w.wg * 4 + e) * kRows + w.row;
            float v = at[0];
#pragma unroll
            for (int q = 1; q < kParts; ++q) v += at[q * 16 * kRows];
            sum[n / 4 + e] = v;
            const int tok = n + w.wg * 4 + e;
            if (!clusters && tok < t.tokens) store(tok, w.row, v);
        }
    }
    if (clusters) {
        __syncwarp();
        named_bar_sync(1, kWorkers);
#pragma unroll
        for (int n = 0; n < C::NT; n += 16)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n == 0 || n < t.tokens)
                    sums[(n + w.wg * 4 + e) * kRows + w.row] = sum[n / 4 + e];
        __syncwarp();
        named_bar_sync(1, kWorkers);
        if (tid < p.cluster) mbar_arrive_cluster(map_to_rank(smem_u32(&misc.sum_full), tid));
        ok = __all_sync(kAll, wait_cluster(smem_u32(&misc.sum_full), unit & 1u, abort_flag, err,
                                           limit_ns));
        if (ok) {
            const int all = t.tokens * kRows, v1 = all * (rank + 1) / p.cluster;
#pragma unroll 1
            for (int v = all * rank / p.cluster + tid; v < v1; v += kWorkers) {
                float sum = 0.0f;
                for (int q = 0; q < p.cluster; ++q) {
                    float other;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(other)
                                 : "r"(map_to_rank(smem_u32(sums + v), q))
                                 : "memory");
                    sum += other;
                }
                store(v / kRows, v % kRows, sum);
            }
        }
        __syncwarp();
        if (!named_bar_and(1, kWorkers, ok)) return false;
        if (tid < p.cluster) mbar_arrive_cluster(map_to_rank(smem_u32(&misc.sum_empty), tid));
    }
    return true;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
gemm_w4_many_kernel(const __grid_constant__ ManyProblem p, const uint64_t limit_ns,
                    uint32_t* __restrict__ err) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
    ManyMisc& misc = *reinterpret_cast<ManyMisc*>(smem + p.off_misc);
    volatile int* abort_flag = &misc.abort_flag;
    const W4Args& a = p.a;
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = __shfl_sync(kAll, tid / 32, 0), lane = tid % 32;
    const bool clusters = !C::kAlone && p.cluster > 1;
    const int32_t rank = clusters ? static_cast<int32_t>(cluster_ctarank()) : 0;

    if (tid == 0) {
        for (int i = 0; i < kParts; ++i) {
            for (int s = 0; s < p.depth; ++s) mbar_init(smem_u32(&misc.full[i][s]), 1);
            mbar_init(smem_u32(&misc.ready[i]), 4);
            mbar_init(smem_u32(&misc.done[i]), 1);
        }
        mbar_init(smem_u32(&misc.sum_full), p.cluster);
        mbar_init(smem_u32(&misc.sum_empty), p.cluster);
        misc.abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&misc.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (Only now: a grid that starts here next must not hold the TMEM this one waits for.)
    grid_launch_dependents();
    grid_dependency_wait();
    if (C::kGrouped) {
        if (warp == 0) find_groups<C>(a, misc.groups, lane);
        __syncthreads();
    }
    __syncwarp();
    if (clusters) cluster_sync_after_init();

    // This part's units, and its blocks of 128 k of one: c0, c0 + parts, ...
    const int wg = warp < kWorkers / 32 ? warp / 4 : warp - kWorkers / 32;
    const int32_t k128 = (a.K + 127) / 128;
    const int32_t c0 = k128 * rank / p.cluster + (C::kAlone ? 0 : wg);
    const int32_t c1 = k128 * (rank + 1) / p.cluster;
    const int32_t per_unit = max((c1 - c0 + C::kSplit - 1) / C::kSplit, 0);
    const int32_t block = static_cast<int32_t>(blockIdx.x), grid = static_cast<int32_t>(gridDim.x);
    const int32_t unit0 = C::kAlone ? block * kParts + wg : block / p.cluster;
    const int32_t unit_step = C::kAlone ? grid * kParts : grid / p.cluster;
    Units<C, ManyProblem> units(p, misc.groups, unit0, unit_step);
    const uint32_t ring = sbase + wg * p.depth * p.stage_bytes;
    const uint32_t full = smem_u32(&misc.full[wg][0]);
    const uint32_t ready = smem_u32(&misc.ready[wg]), done = smem_u32(&misc.done[wg]);
    const uint32_t t_a = misc.tmem + wg * kPartCols, t_acc = t_a + 64;
    uint32_t steps = 0;                  // of products

    if (warp >= kWorkers / 32) {
        // ---- copies and products' issue, by one elected lane each time (a branch on the lane's
        // number instead makes both several times slower) ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
        Units<C, ManyProblem> ahead = units;
        Unit at{};
        int32_t copied = 0;
        uint32_t fills = 0, copy_slot = 0;
        // The next stage into the slot of the oldest, which is done with.
        auto copy_next = [&]() {
            if (copied == 0) {
                if (per_unit == 0 || ahead.left == 0) return;
                at = ahead.next(p, misc.groups);
            }
            const uint32_t bar = full + 8 * copy_slot, dst = ring + copy_slot * p.stage_bytes;
            const int32_t c = c0 + copied * C::kSplit;
            if (++copied == per_unit) copied = 0;
            if (++copy_slot == static_cast<uint32_t>(p.depth)) copy_slot = 0;
            ++fills;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, p.stage_bytes);
                tma_load_2d(dst, &p.tm_codes, c * 64, at.g * a.N + at.n, bar);
                tma_load_2d(dst + kCodeBytes, &p.tm_tokens, c * 128, at.m, bar);
                tma_load_2d(dst + kCodeBytes + p.tokens * 128, &p.tm_tokens, c * 128 + 64, at.m,
                            bar);
            }
            __syncwarp();
        };
        for (int i = 0; i < p.depth; ++i) copy_next();
        const uint64_t desc0 = umma_desc_sw128_kmajor(ring + kCodeBytes);
        int slot = 0;
        bool ok = true;
#pragma unroll 1
        while (ok && units.left > 0) {
            const Unit t = units.next(p, misc.groups);
            // Columns of the products: the tokens there are, in sixteens.
            const uint32_t idesc =
                umma_idesc_16bit_f32(kRows, (t.tokens + 15) / 16 * 16, C::kBF16);
#pragma unroll 1
            for (int32_t st = 0; ok && st < per_unit; ++st) {
                const uint64_t desc = desc0 + (slot * p.stage_bytes >> 4);
                if (++slot == p.depth) slot = 0;
#pragma unroll
                for (int b = 0; b < 4; b += C::kStep) {
                    ok = ok && __all_sync(kAll, wait_or_abort(ready, steps & 1u, abort_flag, err,
                                                              kSiteMmaAccEmpty, limit_ns));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 2 * C::kStep; ++i)     // 16 k each
                            mma_f16_ts(
                                t_acc + i / (2 * C::GB) * C::NT, t_a + i * 8,
                                desc + ((2 * b + i) / 4 * p.tokens * 8 + (2 * b + i) % 4 * 2),
                                idesc, i % (2 * C::GB) != 0);
                        mma_commit(done);
                    }
                    __syncwarp();
                    // The products before these have ended: the stage before this one is free.
                    if (b == 0 && steps > 0) copy_next();
                    ++steps;
                }
            }
        }
        // After a failed wait: the copies and products under way must have ended before this
        // CTA does.
        if (*abort_flag && lane == 0) {
            const uint32_t depth = static_cast<uint32_t>(p.depth);
            for (uint32_t f = fills > depth ? fills - depth : 0; f < fills; ++f)
                wait_bounded(full + 8 * (f % depth), (f / depth) & 1u, err, kSiteDrainFull,
                             limit_ns);
            if (steps > 0) wait_bounded(done, (steps - 1) & 1u, err, kSiteDrainMma, limit_ns);
        }
        __syncwarp();
    } else {
        // ---- widening and sums ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWorkerRegs));
        Worker<C> w;
        w.wg = wg;
        w.lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        w.row = tid % 128;
        const uint32_t t_st = t_a + w.lanes, t_ld = t_acc + w.lanes;
        float* sums = reinterpret_cast<float*>(smem + p.off_sums);
        // This row's codes in a stage: 64 bytes, whose 16-byte pieces are swizzled.
        const uint32_t codes = ring + w.row * 64, swizzle = (w.row >> 1) & 3;
        // Scales and zero points of the next stage.
        uint32_t s_next[C::kScales], z_next[C::kScales];
        int64_t s_row = 0;
        auto read_scales = [&](int32_t c) {      // of block c of 128 k
#pragma unroll
            for (int j = 0; j < C::kScales; ++j) {
                const int32_t g = c * C::kScales + j;
                const bool in = g < a.scale_groups;   // (past K the tokens are zeros)
                s_next[j] = in ? a.S[s_row + g] : 0;
                z_next[j] = in && a.Z ? a.Z[s_row + g] : 8;
            }
        };
        auto scales_of = [&](const Unit& u) {
            s_row = (static_cast<int64_t>(u.g) * a.N + u.n + min(w.row, u.rows - 1)) *
                    a.scale_groups;
            read_scales(c0);
        };
        Unit t{}, next{};
        uint32_t unit = 0, phase = 0;
        int slot = 0;
        bool ok = true, more = units.left > 0;
        if (more) {
            next = units.next(p, misc.groups);
            scales_of(next);
        }
        float scale[C::kAccs] = {};          // of the step under way
        auto collect = [&]() {
            ok = __all_sync(kAll, wait_many(done, (steps - 1) & 1u, abort_flag, err,
                                            kSiteEpiAccFull, limit_ns)) &&
                 ok;
            tc_fence_after();
            add_sums<C>(w, t_ld, scale, t.tokens);
        };
#pragma unroll 1
        while (ok && more) {
            t = next;
            more = units.left > 0;
            if (more) next = units.next(p, misc.groups);
#pragma unroll
            for (int i = 0; i < C::NT; ++i) w.acc[i] = 0.0f;
            int32_t c = c0;
            bool pending = false;
#pragma unroll 1
            for (int32_t st = 0; ok && st < per_unit; ++st, c += C::kSplit) {
                ok = __all_sync(kAll, wait_many(full + 8 * slot, phase, abort_flag, err,
                                                kSiteMmaFull, limit_ns));
                uint32_t s_now[C::kScales], z_now[C::kScales];
#pragma unroll
                for (int j = 0; j < C::kScales; ++j) {
                    s_now[j] = s_next[j];
                    z_now[j] = z_next[j];
                }
                if (st + 1 < per_unit)
                    read_scales(c + C::kSplit);
                else if (more)
                    scales_of(next);
                const uint32_t stage = slot * p.stage_bytes;
#pragma unroll
                for (int b = 0; b < 4; b += C::kStep) {
                    // The step before this one has read its weights and made its sums.
                    if (pending) collect();
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < C::kStep; ++i) {
                        const WidenPairs<C::kBF16> widen(z_now[(b + i) / C::GB]);
                        const uint4 v = ld_shared_v4(codes + stage + (((b + i) ^ swizzle) * 16));
                        uint32_t out[16];
                        widen(v.x, out);
                        widen(v.y, out + 4);
                        widen(v.z, out + 8);
                        widen(v.w, out + 12);
                        tmem_st_32x32b_x16(t_st + i * 16, out);
                    }
#pragma unroll
                    for (int j = 0; j < C::kAccs; ++j)
                        scale[j] = scale_value<C::kBF16>(s_now[b / C::GB + j]);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ready);
                    ++steps;
                    pending = true;
                }
                if (++slot == p.depth) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            if (ok && pending) collect();
            if constexpr (!C::kAlone)
                ok = finish<C>(p, misc, sums, w, t, rank, unit, ok, limit_ns, err);
            else if (ok)
                store_rows<C>(a, w, t, err);
            if (ok && (C::kAlone ? tid % 128 : tid) == 0 && rank == 0)
                check_count_unit(err, unit0 + static_cast<int32_t>(unit) * unit_step);
            ++unit;
        }
    }
    tc_fence_before();
    __syncthreads();
    // Peers' shared memory stays alive until every CTA is done with it.
    if (clusters) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(misc.tmem, 512);
    }
}

// Clusters of `size` (1, 2 or 4) CTAs with all of an SM's shared memory that the current
// device holds at once, asked once per context.
int resident_clusters(int size, int sms) {
    if (size == 1) return sms;
    static ContextMarks known[5], attr_done;
    static std::atomic<int> held[64][5];
    auto kernel = gemm_w4_many_kernel<ManyCfg<false, 4, false, false>>;
    int dev = 0;
    const uint64_t ctx = current_context_id();
    const bool tracked = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && ctx != 0;
    if (tracked && known[size][dev].load(std::memory_order_acquire) == ctx)
        return held[dev][size].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemLimit;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (smem_opt_in(kernel, static_cast<int>(kSmemLimit), attr_done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (tracked) {
        held[dev][size].store(n, std::memory_order_relaxed);
        known[size][dev].store(ctx, std::memory_order_release);
    }
    return n;
}

// The CTAs that split K, and the time that is expected to take.
struct ManyShape {
    int cluster, depth, tokens;
    uint32_t stage_bytes;
    int64_t clusters;
    double time;
};

template <class C>
bool shape_of(const W4Args& a, int cluster, int sms, ManyShape* s) {
    s->cluster = cluster;
    s->clusters = resident_clusters(cluster, sms);
    const uint32_t rest = C::kSumBytes + static_cast<uint32_t>(sizeof(ManyMisc)) + 1024;
    s->tokens = a.M >= C::NT ? C::NT : static_cast<int32_t>(ceil_div(a.M, 16) * 16);
    s->stage_bytes = kCodeBytes + s->tokens * 256u;
    const uint32_t depth = (kSmemLimit - rest) / (kParts * s->stage_bytes);
    s->depth = static_cast<int>(depth < kMaxDepth ? depth : kMaxDepth);
    if (s->clusters < 1 || depth < 2) return false;
    // Units: of the groups, those that can have rows; dense, all blocks of tokens.
    const int64_t chunks =
        a.offsets ? (a.groups < a.M ? a.groups : a.M) : ceil_div(a.M, C::kTokens);
    const int64_t rounds = ceil_div(chunks * ceil_div(a.N, kRows),
                                    s->clusters * (C::kAlone ? kParts : 1));
    const int64_t stages = ceil_div(ceil_div(ceil_div(a.K, 128), cluster), C::kSplit);
    // In stages of 0.85 us; the end of a unit takes a few more.
    s->time = rounds * (stages + (cluster > 1 ? 3.2 : C::kAlone ? 1.0 : 1.9));
    return true;
}

template <class C>
cudaError_t launch_cfg(const W4Args& a, const ManyShape& s, const W4Device& dev,
                       cudaStream_t stream) {
    ManyProblem p{};
    p.a = a;
    p.box = kRows;
    p.row_blocks = static_cast<int32_t>(ceil_div(a.N, kRows));
    p.cluster = s.cluster;
    p.depth = s.depth;
    p.tokens = s.tokens;
    p.stage_bytes = s.stage_bytes;
    p.off_sums = s.depth * kParts * p.stage_bytes;
    p.off_misc = p.off_sums + C::kSumBytes;
    const uint32_t bytes = p.off_misc + static_cast<uint32_t>(sizeof(ManyMisc)) + 1024;
    const uint64_t rows = static_cast<uint64_t>(a.groups) * a.N, k2 = a.K / 2, m = a.M;
    const cuuint64_t dims_b[2] = {k2, rows}, stride_b[1] = {k2};
    const cuuint64_t dims_a[2] = {2 * k2, m}, stride_a[1] = {4 * k2};
    const cuuint32_t box_b[2] = {64, kRows}, box_a[2] = {64, static_cast<cuuint32_t>(s.tokens)};
    const CUtensorMapDataType type =
        C::kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (encode(dev.encode, &p.tm_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.B, dims_b, stride_b,
               box_b, CU_TENSOR_MAP_SWIZZLE_64B) ||
        encode(dev.encode, &p.tm_tokens, type, 2, a.A, dims_a, stride_a, box_a,
               CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    static ContextMarks attr_done;
    auto kernel = gemm_w4_many_kernel<C>;
    if (cudaError_t e = smem_opt_in(kernel, static_cast<int>(kSmemLimit), attr_done)) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(s.clusters * s.cluster)),
                         dim3(kThreads), bytes, stream, static_cast<unsigned>(s.cluster), dev.pdl,
                         p, dev.limit_ns, dev.err_word);
}

// K split over a CTA's warpgroups and up to four CTAs, or a unit to a warpgroup.
template <bool BF16, int GB, bool GROUPED>
cudaError_t launch_split(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    using Split = ManyCfg<BF16, GB, GROUPED, false>;
    using Alone = ManyCfg<BF16, GB, GROUPED, true>;
    ManyShape s{}, t{};
    bool found = false;
    for (int cluster = 1; cluster <= 4; cluster *= 2)
        if (shape_of<Split>(a, cluster, dev.sms, &t) && (!found || t.time < s.time)) {
            s = t;
            found = true;
        }
    if (shape_of<Alone>(a, 1, dev.sms, &t) && (!found || t.time < s.time))
        return launch_cfg<Alone>(a, t, dev, stream);
    return found ? launch_cfg<Split>(a, s, dev, stream) : cudaErrorInvalidConfiguration;
}
template <bool BF16, int GB>
cudaError_t launch_groups(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    return a.offsets ? launch_split<BF16, GB, true>(a, dev, stream)
                     : launch_split<BF16, GB, false>(a, dev, stream);
}
template <bool BF16>
cudaError_t launch_scales(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    return a.group == 32   ? launch_groups<BF16, 1>(a, dev, stream)
           : a.group == 64 ? launch_groups<BF16, 2>(a, dev, stream)
                           : launch_groups<BF16, 4>(a, dev, stream);
}

}  // namespace

cudaError_t launch_gemm_w4_many(const W4Args& a, bool bf16, const W4Device& dev,
                                cudaStream_t stream) {
    return bf16 ? launch_scales<true>(a, dev, stream) : launch_scales<false>(a, dev, stream);
}

}  // namespace tmagemm
