// Products of a few tokens with 4-bit weights and group scales:
//   D[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] (q[n][k] - z[n][g]).
//
// q - z is a whole number of five bits, exact in 16 bits, so the inner sums run on
// mma.sync with FP32 accumulators and the scale is applied to a whole group's sum in
// FP32.  (tcgen05 would need the widened weights in shared memory, four times the bytes
// that are read; up to 32 tokens the time is that of reading the weights.)
//
// A unit is a block of weight rows and up to 8 NT tokens.  The warps of a CTA are WR along
// the rows, 16 MT each, and WK along K, 128 k of a stage each.  One thread keeps a ring of
// stages filled by TMA: codes as 128-byte rows (256 k), tokens as 64-byte rows (32 k), both
// swizzled so that the rows of one access are in different banks.  In a block of 32 k the
// lanes of a quad hold eight k each (one word of codes): the product's order of k is free,
// so the pairs that one mask takes out of a word (nibbles i and i + 4) become the pairs of
// an MMA operand, and the tokens' values are brought into the same order with byte
// permutes.
// The WK partial sums meet in shared memory in a fixed order; with a cluster its CTAs
// split K and add theirs through distributed shared memory.
// The loop over stages is one loop for prologue and body, not unrolled: a kernel of a few
// microseconds otherwise waits for its instructions.
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

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMaxGroups = 384;
constexpr int kMaxDepth = 8;
constexpr uint32_t kSmemLimit = 232448;

template <int MT_, int NT_, int WARPS_, bool BF16_, int GB_, bool GROUPED_>
struct W4Cfg {
    static constexpr int MT = MT_, NT = NT_, kWarps = WARPS_, kThreads = 32 * WARPS_;
    static constexpr int GB = GB_;                         // blocks of 32 k of a scale
    static constexpr bool kBF16 = BF16_, kGrouped = GROUPED_, kClusters = NT > 1;
    static constexpr int kWarpRows = 16 * MT, kTokens = 8 * NT;
    // Partial sums of eight tokens: a float per warp, row and token.
    static constexpr int kValues = kWarpRows * 8;          // of a warp
    static constexpr uint32_t kPartBytes = kWarps * kValues * 4;
};

struct W4Problem {
    CUtensorMap tm_blocks;   // codes {128 bytes, rows of all groups, K / 256}, box {128, box, KC / 256}
    CUtensorMap tm_rows;     // codes {K / 2, rows}, box {128, box}: where K ends inside a block
    CUtensorMap tm_tokens;   // A {32, M, K / 32}, box {32, tokens, KC / 32}
    W4Args a;
    int32_t box, tokens;     // rows and tokens of a stage
    int32_t row_blocks;      // of a group
    int32_t cluster, depth;  // CTAs that split K, stages of the ring
    int32_t wr, wk_shift;    // warps along the rows; warps along K = 1 << wk_shift
    uint32_t w_bytes, stage_bytes, off_part, off_exchange, off_misc;
};

// Barriers, flags and the groups' table, behind the rest of shared memory.
struct W4Misc {
    uint64_t full[kMaxDepth], empty[kMaxDepth], sum_full, sum_empty;
    int abort_flag;
    int32_t first[kMaxGroups + 1];    // first row of each group
    int32_t chunk[kMaxGroups + 1];    // blocks of tokens before each group
};

// A unit of work: `rows` weight rows from n of group g, `tokens` tokens from m.
struct Unit {
    int32_t n, m, g, rows, tokens;
};

// The units of a cluster, in order: token block by token block of each group, and row
// block by row block of each.
template <class C>
struct Units {
    int32_t left, block, m, g;          // the next unit is a later one if block >= row_blocks
    __device__ Units(const W4Problem& p, const W4Misc& misc) {
        const int32_t id = static_cast<int32_t>(blockIdx.x) / p.cluster;
        const int32_t step = static_cast<int32_t>(gridDim.x) / p.cluster;
        const int32_t chunks =
            C::kGrouped ? misc.chunk[p.a.groups] : (p.a.M + C::kTokens - 1) / C::kTokens;
        const int64_t all = static_cast<int64_t>(chunks) * p.row_blocks;
        left = all <= id ? 0
                         : all <= 0x7fffffff - step
                               ? (static_cast<int32_t>(all) - id + step - 1) / step
                               : static_cast<int32_t>((all - id + step - 1) / step);
        block = id;
        g = 0;
        m = C::kGrouped ? misc.first[0] : 0;
    }
    // The next unit (left > 0).
    __device__ __forceinline__ Unit next(const W4Problem& p, const W4Misc& misc) {
        int32_t end = C::kGrouped ? misc.first[g + 1] : p.a.M;
        while (block >= p.row_blocks || m >= end) {
            if (m < end) {
                block -= p.row_blocks;
                m += C::kTokens;
            }
            if (C::kGrouped && m >= end) {
                ++g;
                m = end;
                end = misc.first[g + 1];
            }
        }
        const Unit t{block * p.box, m, g, min(p.box, p.a.N - block * p.box),
                     min(C::kTokens, end - m)};
        block += static_cast<int32_t>(gridDim.x) / p.cluster;
        --left;
        return t;
    }
};

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

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (a & mask) | base in one instruction.
template <uint32_t MASK, uint32_t BASE>
__device__ __forceinline__ uint32_t and_or(uint32_t a) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "n"(MASK), "n"(BASE));
    return r;
}
// a * b + c of two packed 16-bit numbers each, rounded once.
template <bool BF16>
__device__ __forceinline__ uint32_t fma16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    if constexpr (BF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// What turns the eight codes of a word into pairs of (q - z), exactly.  A lower code is put
// into the low bits of 1024 (fp16) or 128 (bf16); an upper one stays four bits up, as
// 1024 + 16 q, or in bf16, whose significand has no room for that, as the subnormal
// 16 q 2^-133.  One multiply-add for each pair takes the power of two and the zero point out:
//   fp16  1 (1024 + q) - (1024 + z)            1/16 (1024 + 16 q) - (64 + z)
//   bf16  1/4 (128 + q) - (128 + z) / 4        2^127 (16 q 2^-133) - z / 4
// (in bf16 a quarter of q - z: 2^129, which would make it whole, is no bf16 number).
template <bool BF16>
struct Widen {
    uint32_t low, high;    // the pairs of addends
    static constexpr float kScale = BF16 ? 4.0f : 1.0f;   // what the products are multiplied with
    Widen() = default;
    __device__ __forceinline__ explicit Widen(uint32_t z) {
        // z / 4 is in the last places of -32 in bf16, z in those of -1024 in fp16.
        low = z * 0x10001u + (BF16 ? 0xc200c200u : 0xe400e400u);
        high = fma16x2<BF16>(low, BF16 ? 0x3f803f80u : 0x3c003c00u,      // low + 32, or + 960
                             BF16 ? 0x42004200u : 0x63806380u);
    }
    // Codes (0, 4), (1, 5), (2, 6), (3, 7) of a word.
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&out)[4]) const {
        const uint32_t v = w >> 8;
        if constexpr (BF16) {
            out[0] = fma16x2<BF16>(and_or<0x000f000fu, 0x43004300u>(w), 0x3e803e80u, low);
            out[1] = fma16x2<BF16>(w & 0x00f000f0u, 0x7f007f00u, high);
            out[2] = fma16x2<BF16>(and_or<0x000f000fu, 0x43004300u>(v), 0x3e803e80u, low);
            out[3] = fma16x2<BF16>(v & 0x00f000f0u, 0x7f007f00u, high);
        } else {
            out[0] = fma16x2<BF16>(and_or<0x000f000fu, 0x64006400u>(w), 0x3c003c00u, low);
            out[1] = fma16x2<BF16>(and_or<0x00f000f0u, 0x64006400u>(w), 0x2c002c00u, high);
            out[2] = fma16x2<BF16>(and_or<0x000f000fu, 0x64006400u>(v), 0x3c003c00u, low);
            out[3] = fma16x2<BF16>(and_or<0x00f000f0u, 0x64006400u>(v), 0x2c002c00u, high);
        }
    }
};
// Eight values of a token in the same pairs.
__device__ __forceinline__ void pair_up(const uint4& x, uint32_t (&out)[4]) {
    out[0] = __byte_perm(x.x, x.z, 0x5410);
    out[1] = __byte_perm(x.x, x.z, 0x7632);
    out[2] = __byte_perm(x.y, x.w, 0x5410);
    out[3] = __byte_perm(x.y, x.w, 0x7632);
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at));
    return v;
}

template <bool BF16>
__device__ __forceinline__ float scale_value(uint32_t bits) {
    if constexpr (BF16) return __uint_as_float(bits << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

// The groups' rows and blocks of tokens, by one warp.  (An offset counts as the largest
// so far, within [0, M].)
template <class C>
__device__ __forceinline__ void find_groups(const W4Args& a, W4Misc& misc, int lane) {
    int32_t last = 0, chunks = 0;
#pragma unroll 1
    for (int i0 = 0; i0 <= a.groups; i0 += 32) {
        const int i = i0 + lane;
        int32_t v = min(max(i <= a.groups ? a.offsets[i] : 0, last), a.M);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(kAll, v, d);
            if (lane >= d) v = max(v, o);
        }
        int32_t before = __shfl_up_sync(kAll, v, 1);
        if (lane == 0) before = i == 0 ? v : last;
        int32_t n = (v - before + C::kTokens - 1) / C::kTokens;   // of the group that ends here
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(kAll, n, d);
            if (lane >= d) n += o;
        }
        if (i <= a.groups) {
            misc.first[i] = v;
            misc.chunk[i] = chunks + n;
        }
        last = __shfl_sync(kAll, v, 31);
        chunks += __shfl_sync(kAll, n, 31);
    }
}

// The end of a unit: the warps' sums meet, eight tokens at a time, and then those of a
// cluster's CTAs.  Value j of a lane (of 4 MT: tile, row half, token) of warp (wk, wr) is
// at [wk][wr][j][lane].  False after a wait that failed, in this warp or another.
template <class C>
__device__ __forceinline__ bool finish(const W4Problem& p, W4Misc& misc, uint8_t* smem,
                                       float (&acc)[C::MT][C::NT][4], const Unit& t, int warp,
                                       int lane, int wr, int wk, int32_t rank, uint32_t sums,
                                       bool ok, uint64_t limit_ns, uint32_t* err) {
    const W4Args& a = p.a;
    const int tid = warp * 32 + lane, values = p.wr * C::kValues;
    const bool clusters = C::kClusters && p.cluster > 1;
    volatile int* abort_flag = &misc.abort_flag;
    float* exchange = reinterpret_cast<float*>(smem + p.off_exchange);
    float* part = reinterpret_cast<float*>(smem + p.off_part);
    if (clusters && sums > 0)
        ok = __all_sync(kAll, wait_cluster(smem_u32(&misc.sum_empty), (sums - 1) & 1u, abort_flag,
                                           err, limit_ns)) &&
             ok;
    auto store = [&](int v, int n, float sum) {
        const int l = v & 31, j = (v >> 5) & (4 * C::MT - 1), r = v / C::kValues;
        const int rr = r * C::kWarpRows + (j >> 2) * 16 + ((j >> 1) & 1) * 8 + (l >> 2);
        const int tok = n * 8 + (l & 3) * 2 + (j & 1);
        if (rr < t.rows && tok < t.tokens &&
            check_ok(t.n + rr < a.N && t.m + tok < a.M, err, kSiteCheckBounds))
            a.D[static_cast<int64_t>(t.m + tok) * a.N + t.n + rr] =
                cvt16_rn<C::kBF16>(__float_as_uint(sum));
    };
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        if (n > 0 && 8 * n >= t.tokens) break;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[((wk * p.wr + wr) * 4 * C::MT + 4 * i + e) * 32 + lane] =
                    acc[i][n][e] * Widen<C::kBF16>::kScale;
        __syncwarp();
        if (!named_bar_and(1, C::kThreads, ok)) return false;
#pragma unroll 1
        for (int v = tid; v < values; v += C::kThreads) {
            float sum = part[v];
#pragma unroll 4
            for (int q = 1; q < (1 << p.wk_shift); ++q) sum += part[q * values + v];
            if (clusters)
                exchange[n * values + v] = sum;
            else
                store(v, n, sum);
        }
        __syncthreads();
    }
    if (clusters) {
        // All sums of this CTA are in place: tell the cluster; add the CTAs' sums, a part of
        // the values each, when all have.
        if (tid < p.cluster) mbar_arrive_cluster(map_to_rank(smem_u32(&misc.sum_full), tid));
        ok = __all_sync(kAll, wait_cluster(smem_u32(&misc.sum_full), sums & 1u, abort_flag, err,
                                           limit_ns));
        if (ok) {
            const int all = (t.tokens + 7) / 8 * values;
            const int v1 = all * (rank + 1) / p.cluster;
#pragma unroll 1
            for (int v = all * rank / p.cluster + tid; v < v1; v += C::kThreads) {
                float sum = 0.0f;
                for (int q = 0; q < p.cluster; ++q) {
                    float other;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(other)
                                 : "r"(map_to_rank(smem_u32(exchange + v), q))
                                 : "memory");
                    sum += other;
                }
                store(v % values, v / values, sum);
            }
        }
        __syncwarp();
        if (!named_bar_and(1, C::kThreads, ok)) return false;
        if (tid < p.cluster) mbar_arrive_cluster(map_to_rank(smem_u32(&misc.sum_empty), tid));
    }
    return true;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
gemm_w4_kernel(const __grid_constant__ W4Problem p, const uint64_t limit_ns,
               uint32_t* __restrict__ err) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
    W4Misc& misc = *reinterpret_cast<W4Misc*>(smem + p.off_misc);
    volatile int* abort_flag = &misc.abort_flag;
    const W4Args& a = p.a;
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = __shfl_sync(kAll, tid / 32, 0), lane = tid % 32;
    const int row = lane >> 2, quad = lane & 3;
    const int wr = warp & (p.wr - 1), wk = warp / p.wr;
    const bool clusters = C::kClusters && p.cluster > 1;
    const int32_t rank = clusters ? static_cast<int32_t>(cluster_ctarank()) : 0;

    grid_launch_dependents();
    if (tid == 0) {
        for (int s = 0; s < p.depth; ++s) {
            mbar_init(smem_u32(&misc.full[s]), 1);
            mbar_init(smem_u32(&misc.empty[s]), C::kWarps);
        }
        mbar_init(smem_u32(&misc.sum_full), p.cluster);
        mbar_init(smem_u32(&misc.sum_empty), p.cluster);
        misc.abort_flag = 0;
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    if (C::kGrouped && warp == 0) find_groups<C>(a, misc, lane);
    __syncthreads();
    if (clusters) cluster_sync_after_init();

    // This CTA's blocks of 256 k, a stage of 1 << (wk_shift - 1) blocks at a time.
    const int32_t stage_shift = p.wk_shift - 1, k256 = (a.K + 255) / 256;
    const int32_t b0 = clusters ? k256 * rank / p.cluster : 0;
    const int32_t b1 = clusters ? k256 * (rank + 1) / p.cluster : k256;
    const int32_t per_unit = max((b1 - b0 + (1 << stage_shift) - 1) >> stage_shift, 1);

    Units<C> units(p, misc);
    const int64_t total = static_cast<int64_t>(units.left) * per_unit;   // stages

    // ---- copies, by one thread ----
    Units<C> ahead = units;
    Unit at{};
    int32_t copied = 0, copy_slot = 0;
    uint32_t copy_phase = 1;
    auto copy_next = [&]() {
        const uint32_t full = smem_u32(&misc.full[copy_slot]);
        if (!wait_or_abort(smem_u32(&misc.empty[copy_slot]), copy_phase, abort_flag, err,
                           kSiteProducerEmpty, limit_ns))
            return;
        if (copied == 0) at = ahead.next(p, misc);
        const int32_t b = b0 + (copied << stage_shift), n = min(b1 - b, 1 << stage_shift);
        if (++copied == per_unit) copied = 0;
        const uint32_t dst = sbase + copy_slot * p.stage_bytes;
        if (++copy_slot == p.depth) {
            copy_slot = 0;
            copy_phase ^= 1u;
        }
        const int32_t r = at.g * a.N + at.n;
        // Blocks that are whole and all of the stage in one copy, else one by one.
        const bool whole = n == 1 << stage_shift && (b + n) * 256 <= a.K;
        const uint32_t w = static_cast<uint32_t>(p.box) * 128u;
        mbar_arrive_expect_tx(full, max(n, 0) * w + (p.stage_bytes - p.w_bytes));
        if (whole) {
            tma_load_3d(dst, &p.tm_blocks, 0, r, b, full);
        } else {
            for (int i = 0; i < n; ++i)
                tma_load_2d(dst + i * w, &p.tm_rows, (b + i) * 128, r, full);
        }
        tma_load_3d(dst + p.w_bytes, &p.tm_tokens, 0, at.m, b * 8, full);
    };

    // ---- products ----
    constexpr int kScales = 4 / C::GB;              // of a row and 128 k
    // Where this lane's words of codes and parts of tokens are in a stage, by block of 32 k
    // (a stage starts at a multiple of 1024 bytes, so that the swizzle, which goes by the
    // address, is the same in each).
    // (Tokens past the stage's are not looked at: what is read there is other data.)
    uint32_t w_at[4], x_at[4];
    const uint32_t w_row =
        sbase + static_cast<uint32_t>((wk >> 1) * p.box + wr * C::kWarpRows + row) * 128;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        w_at[b] = (w_row | ((wk & 1) * 64 + b * 16 + quad * 4)) ^ ((w_row >> 3) & 0x70u);
        const uint32_t at = sbase + p.w_bytes + quad * 16 +
                            ((wk * 4 + b) * p.tokens + (C::NT == 1 ? min(row, p.tokens - 1) : row)) * 64;
        x_at[b] = at ^ ((at >> 3) & 0x30u);
    }
    // Scales and zero points of this warp's part of the next stage: of rows row + 8 i,
    // group `quad` of the 128 k.
    uint32_t s_next[2 * C::MT] = {}, z_next[2 * C::MT] = {}, s_off[2 * C::MT];
    int64_t s_base = 0;
    int32_t group = 0;
    auto scales_of = [&](const Unit& u) {
        s_base = (static_cast<int64_t>(u.g) * a.N + u.n) * a.scale_groups;
        group = (b0 * 8 + wk * 4) / C::GB + min(quad, kScales - 1);
#pragma unroll
        for (int i = 0; i < 2 * C::MT; ++i)
            s_off[i] = min(wr * C::kWarpRows + row + 8 * i, u.rows - 1) * a.scale_groups + group;
    };
    auto read_scales = [&]() {
        if (group < a.scale_groups) {     // (past K the tokens are zeros)
#pragma unroll
            for (int i = 0; i < 2 * C::MT; ++i) {
                s_next[i] = a.S[s_base + s_off[i]];
                z_next[i] = a.Z ? a.Z[s_base + s_off[i]] : 8;
            }
        }
    };
    Unit t{}, next{};
    float acc[C::MT][C::NT][4] = {};
    uint32_t sums = 0, phase = 0;
    int slot = 0;
    bool ok = true;
    bool more = units.left > 0;
    if (more) {
        next = units.next(p, misc);
        scales_of(next);
        read_scales();
    }
    if (tid == 0)
        for (int i = 0; i < p.depth && i < total; ++i) copy_next();
    int64_t issued = p.depth;
#pragma unroll 1
    while (ok && more) {
        t = next;
        more = units.left > 0;
        if (more) next = units.next(p, misc);
        const bool mine = wr * C::kWarpRows < t.rows;
        int32_t c = (b0 << 1) + wk;      // 128 k of this warp
#pragma unroll 1
        for (int32_t st = 0; st < per_unit; ++st) {
            ok = __all_sync(kAll, wait_many(smem_u32(&misc.full[slot]), phase, abort_flag, err,
                                            kSiteMmaFull, limit_ns));
            if (!ok) break;
            uint32_t both[kScales][2 * C::MT];
#pragma unroll
            for (int j = 0; j < kScales; ++j)
#pragma unroll
                for (int i = 0; i < 2 * C::MT; ++i)
                    both[j][i] = __shfl_sync(kAll, s_next[i] | (z_next[i] << 16), (lane & ~3) + j);
            if (st + 1 < per_unit) {
                group += 4 / C::GB << p.wk_shift;
#pragma unroll
                for (int i = 0; i < 2 * C::MT; ++i) s_off[i] += 4 / C::GB << p.wk_shift;
                read_scales();
            } else if (more) {
                scales_of(next);
                read_scales();
            }
            if (mine && c < 2 * b1 && c * 128 < a.K) {
                const uint32_t stage = slot * p.stage_bytes;
#pragma unroll
                for (int j = 0; j < kScales; ++j) {
                    float part[C::MT][C::NT][4] = {};
                    Widen<C::kBF16> widen[2 * C::MT];
#pragma unroll
                    for (int i = 0; i < 2 * C::MT; ++i) widen[i] = Widen<C::kBF16>(both[j][i] >> 16);
#pragma unroll
                    for (int b = j * C::GB; b < (j + 1) * C::GB; ++b) {
                        uint32_t v[2 * C::MT][4];
#pragma unroll
                        for (int i = 0; i < 2 * C::MT; ++i)
                            widen[i](ld_shared_u32(w_at[b] + stage + i * 1024), v[i]);
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            if (n > 0 && 8 * n >= t.tokens) break;
                            uint32_t x[4];
                            pair_up(ld_shared_v4(x_at[b] + stage + n * 512), x);
#pragma unroll
                            for (int i = 0; i < C::MT; ++i) {
                                mma_16816<C::kBF16>(part[i][n], v[2 * i][0], v[2 * i + 1][0],
                                                    v[2 * i][1], v[2 * i + 1][1], x[0], x[1]);
                                mma_16816<C::kBF16>(part[i][n], v[2 * i][2], v[2 * i + 1][2],
                                                    v[2 * i][3], v[2 * i + 1][3], x[2], x[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2 * C::MT; ++i) {
                        const float f = scale_value<C::kBF16>(both[j][i] & 0xffffu);
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float& out = acc[i / 2][n][2 * (i & 1) + e];
                                out = fmaf(part[i / 2][n][2 * (i & 1) + e], f, out);
                            }
                    }
                }
            }
            __syncwarp();     // every lane is done with the stage
            if (lane == 0) mbar_arrive(smem_u32(&misc.empty[slot]));
            if (++slot == p.depth) {
                slot = 0;
                phase ^= 1u;
            }
            c += 1 << p.wk_shift;
            // The stage before this one, which the other warps are done with by now, is filled
            // again.
            if (tid == 0) {
                if (issued > p.depth && issued <= total) copy_next();
                ++issued;
            }
            __syncwarp();
        }
        ok = finish<C>(p, misc, smem, acc, t, warp, lane, wr, wk, rank, sums, ok, limit_ns, err);
        if (ok && tid == 0 && rank == 0)
            check_count_unit(err, static_cast<int32_t>((blockIdx.x + sums * gridDim.x) / p.cluster));
        ++sums;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
    }
    // After a failed wait: the copies in flight must have landed before this CTA ends.
    if (*abort_flag && tid == 0) {
        const int64_t n = min(total, static_cast<int64_t>(p.depth));
        for (int s = 0; s < n; ++s)
            wait_bounded(smem_u32(&misc.full[s]), s < copy_slot ? copy_phase ^ 1u : copy_phase, err,
                         kSiteDrainFull, limit_ns);
    }
    // Peers' shared memory stays alive until every CTA is done with it.
    __syncwarp();
    if (clusters) cluster_sync();
}

// Clusters of `size` (1, 2 or 4) CTAs with all of an SM's shared memory that the current
// device holds at once, asked once per context.
int resident_clusters(int size, int sms) {
    if (size == 1) return sms;
    static ContextMarks known[5], attr_done;
    static std::atomic<int> held[64][5];
    auto kernel = gemm_w4_kernel<W4Cfg<2, 2, 16, false, 4, false>>;
    int dev = 0;
    const uint64_t ctx = current_context_id();
    const bool tracked = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && ctx != 0;
    if (tracked && known[size][dev].load(std::memory_order_acquire) == ctx)
        return held[dev][size].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(512);
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

// A map of up to three dimensions; 0, or -1 on failure.
int encode(EncodeTiled fn, CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
           const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
           CUtensorMapSwizzle swizzle) {
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? 0
               : -1;
}

// The shape of a launch, and the time it is expected to take, in stages.
struct W4Shape {
    int wr, wk_shift, cluster, depth;
    int64_t clusters, box;
    uint32_t w_bytes, x_bytes, pitch, exchange;   // of a stage: codes, tokens, both; of a unit
    int32_t tokens;
    double time;
};

template <class C>
bool shape_of(const W4Args& a, int wr, int cluster, int sms, W4Shape* s) {
    s->wr = wr;
    s->wk_shift = 0;
    while ((wr << s->wk_shift) < C::kWarps) ++s->wk_shift;
    s->cluster = cluster;
    s->clusters = resident_clusters(cluster, sms);
    if (s->clusters < 1) return false;
    const int64_t rows = C::kWarpRows * wr, least = ceil_div(a.N, rows);
    // Units: of the groups, those that can have rows; dense, all blocks of tokens.
    const int64_t chunks =
        a.offsets ? (a.groups < a.M ? a.groups : a.M) : ceil_div(a.M, C::kTokens);
    const int64_t rounds = ceil_div(chunks * least, s->clusters);
    // Dense: as many blocks of rows as those rounds have room for.
    int64_t blocks = a.offsets ? least : rounds * s->clusters / chunks;
    if (blocks > a.N) blocks = a.N;
    s->box = ceil_div(a.N, blocks);
    const int32_t kc = 128 << s->wk_shift;
    // (Of several tiles of eight tokens, whole ones: their rows are 512 bytes apart.)
    s->tokens = C::NT == 1 && a.M < 8 ? a.M : static_cast<int32_t>(ceil_div(a.M, 8) * 8);
    if (s->tokens > C::kTokens) s->tokens = C::kTokens;
    s->x_bytes = static_cast<uint32_t>(s->tokens * kc * 2);
    s->pitch = (static_cast<uint32_t>(s->box * (kc / 2)) + s->x_bytes + 1023u) / 1024u * 1024u;
    s->w_bytes = s->pitch - s->x_bytes;      // (tokens at a multiple of 512 bytes)
    s->exchange = cluster > 1 ? static_cast<uint32_t>(wr) * C::kValues * C::NT * 4u : 0u;
    const uint32_t rest =
        C::kPartBytes + s->exchange + static_cast<uint32_t>(sizeof(W4Misc)) + 1024;
    const uint32_t depth = (kSmemLimit - rest) / s->pitch;
    s->depth = static_cast<int>(depth < kMaxDepth ? depth : kMaxDepth);
    // A stage takes about the same time whatever its shape (1.1 us for up to 8 tokens, 1.8
    // for 16, 2.7 for 32); the end of a unit half of one, or twice one with a cluster.
    const int64_t stages = ceil_div(ceil_div(ceil_div(a.K, 256), cluster), kc / 256);
    s->time = rounds * (stages + (cluster > 1 ? 2.2 : 0.5));
    return s->depth >= 2;
}

template <class C>
cudaError_t launch_cfg(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    // The warps along the rows and the CTAs along K that are expected to take least time:
    // 1 x 4096 x 14336 13.2 us with one warp along the rows and 20 with two, 5 x 5003 x 2080
    // 10.6 and 7.7; 16 x 4096 x 14336 28 us without a cluster and 19 in pairs, 32 tokens 75
    // and 27 in fours, 27 x 14336 x 4096 30 without and 44 in pairs.
    W4Shape s{};
    bool found = false;
    for (int wr = 1; C::kWarpRows * wr <= 256 && 2 * wr <= C::kWarps; wr *= 2)
        for (int cluster = 1; cluster <= (C::kClusters && !a.offsets ? 4 : 1); cluster *= 2) {
            W4Shape t{};
            if (shape_of<C>(a, wr, cluster, dev.sms, &t) && (!found || t.time < s.time)) {
                s = t;
                found = true;
            }
        }
    if (!found) return cudaErrorInvalidConfiguration;
    W4Problem p{};
    p.a = a;
    p.cluster = s.cluster;
    p.wr = s.wr;
    p.wk_shift = s.wk_shift;
    p.depth = s.depth;
    p.box = static_cast<int32_t>(s.box);
    p.row_blocks = static_cast<int32_t>(ceil_div(a.N, s.box));
    p.tokens = s.tokens;
    p.w_bytes = s.w_bytes;
    p.stage_bytes = s.pitch;
    p.off_part = s.depth * s.pitch;
    p.off_exchange = p.off_part + C::kPartBytes;
    p.off_misc = p.off_exchange + s.exchange;
    const uint32_t bytes = p.off_misc + static_cast<uint32_t>(sizeof(W4Misc)) + 1024;
    const uint32_t kc = 128u << s.wk_shift, box = static_cast<uint32_t>(s.box);
    const uint64_t rows = static_cast<uint64_t>(a.groups) * a.N, k2 = a.K / 2, m = a.M;
    const cuuint64_t dims3[3] = {128, rows, k2 / 128}, dims2[2] = {k2, rows};
    const cuuint64_t dimsx[3] = {32, m, k2 / 16};
    const cuuint64_t stride3[2] = {k2, 128}, stride2[1] = {k2}, stridex[2] = {4 * k2, 64};
    const cuuint32_t box3[3] = {128, box, kc / 256}, box2[2] = {128, box};
    const cuuint32_t boxx[3] = {32, static_cast<cuuint32_t>(s.tokens), kc / 32};
    const CUtensorMapDataType type =
        C::kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // (With K below 256 no block is whole and the blocks' map is not used.)
    if ((a.K >= 256 && encode(dev.encode, &p.tm_blocks, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.B,
                              dims3, stride3, box3, CU_TENSOR_MAP_SWIZZLE_128B)) ||
        encode(dev.encode, &p.tm_rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.B, dims2, stride2, box2,
               CU_TENSOR_MAP_SWIZZLE_128B) ||
        encode(dev.encode, &p.tm_tokens, type, 3, a.A, dimsx, stridex, boxx,
               CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    static ContextMarks attr_done;
    auto kernel = gemm_w4_kernel<C>;
    if (cudaError_t e = smem_opt_in(kernel, static_cast<int>(kSmemLimit), attr_done)) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(s.clusters * s.cluster)),
                         dim3(C::kThreads), bytes, stream, static_cast<unsigned>(s.cluster),
                         dev.pdl, p, dev.limit_ns, dev.err_word);
}

template <int MT, int NT, int WARPS, bool BF16, int GB>
cudaError_t launch_groups(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    return a.offsets ? launch_cfg<W4Cfg<MT, NT, WARPS, BF16, GB, true>>(a, dev, stream)
                     : launch_cfg<W4Cfg<MT, NT, WARPS, BF16, GB, false>>(a, dev, stream);
}
template <int MT, int NT, int WARPS, bool BF16>
cudaError_t launch_scales(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    return a.group == 32   ? launch_groups<MT, NT, WARPS, BF16, 1>(a, dev, stream)
           : a.group == 64 ? launch_groups<MT, NT, WARPS, BF16, 2>(a, dev, stream)
                           : launch_groups<MT, NT, WARPS, BF16, 4>(a, dev, stream);
}
template <int MT, int NT, int WARPS>
cudaError_t launch_typed(const W4Args& a, bool bf16, const W4Device& dev, cudaStream_t stream) {
    return bf16 ? launch_scales<MT, NT, WARPS, true>(a, dev, stream)
                : launch_scales<MT, NT, WARPS, false>(a, dev, stream);
}

}  // namespace

cudaError_t launch_gemm_w4(const W4Args& a, bool bf16, const W4Device& dev, cudaStream_t stream) {
    // Tokens of a unit: what the groups have on average, in tiles of eight; more are taken
    // in several units, which read the weights again (from L2).
    const int64_t tokens = a.offsets ? ceil_div(a.M, a.groups) : a.M;
    if (tokens <= 8) return launch_typed<2, 1, 16>(a, bf16, dev, stream);
    if (tokens <= 16) return launch_typed<2, 2, 16>(a, bf16, dev, stream);
    return launch_typed<4, 4, 8>(a, bf16, dev, stream);
}

}  // namespace tmagemm
