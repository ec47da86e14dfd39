// Products of up to eight tokens with 4-bit weights and group scales:
//   D[m][n] = sum_g s[n][g] sum_{k in g} A[m][k] (q[n][k] - z[n][g]).
//
// q - z is a whole number of five bits, exact in 16 bits, so the inner sums run on
// mma.sync with FP32 accumulators and the scale is applied to a whole group's sum in
// FP32.  (gemm_w4_many.cu has more tokens, groups of rows, and many rows of weights with a long K.)
//
// A unit is a block of weight rows and up to eight tokens.  The warps of a CTA are WR along
// the rows, 16 MT each, and WK along K, 128 k of a stage each.  One thread keeps a ring of
// stages filled by TMA: codes as 128-byte rows (256 k), tokens as 64-byte rows (32 k), both
// swizzled so that the rows of one access are in different banks.  In a block of 32 k the
// lanes of a quad hold eight k each (one word of codes): the product's order of k is free,
// so the pairs that one mask takes out of a word (nibbles i and i + 4) become the pairs of
// an MMA operand, and the tokens' values are brought into the same order with byte
// permutes.  The WK partial sums meet in shared memory in a fixed order.
// Its 358 instructions for 32 rows by 128 k, 9 to widen eight codes, are about as long as the
// bytes (4.4 us at 4096 x 14336 if every slot issued); with 16 warps an SM half the slots do,
// and what bounds it is the latency from a stage's arrival over widening to the sums.
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
#include "w4.cuh"

namespace tmagemm {

namespace {

template <bool BF16_, int GB_, bool GROUPED_>
struct W4Cfg {
    static constexpr int MT = 2, kTokens = 8, kWarps = 16, kThreads = 32 * kWarps;
    static constexpr int GB = GB_;                         // blocks of 32 k of a scale
    static constexpr bool kBF16 = BF16_, kGrouped = GROUPED_;
    static constexpr int kWarpRows = 16 * MT;
    static constexpr int kValues = kWarpRows * kTokens;    // partial sums of a warp
    static constexpr uint32_t kPartBytes = kWarps * kValues * 4;
};

struct W4Problem {
    CUtensorMap tm_blocks;   // codes {128 bytes, rows of all groups, K / 256}, box {128, box, KC / 256}
    CUtensorMap tm_rows;     // codes {K / 2, rows}, box {128, box}: where K ends inside a block
    CUtensorMap tm_tokens;   // A {32, M, K / 32}, box {32, tokens, KC / 32}
    W4Args a;
    int32_t box, tokens;     // rows and tokens of a stage
    int32_t row_blocks;      // of a group
    int32_t depth;           // stages of the ring
    int32_t wr, wk_shift;    // warps along the rows; warps along K = 1 << wk_shift
    uint32_t w_bytes, stage_bytes, off_part, off_misc;
};

// Barriers, flags and the groups' table, behind the rest of shared memory.
struct W4Misc {
    uint64_t full[kMaxDepth], empty[kMaxDepth];
    int abort_flag;
    W4Groups groups;
};

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

// The end of a unit: the warps' sums meet.  Value j of a lane (of 4 MT: tile, row half,
// token) of warp (wk, wr) is at [wk][wr][j][lane].  False after a wait that failed, in this
// warp or another.
template <class C>
__device__ __forceinline__ bool finish(const W4Problem& p, float* part, float (&acc)[C::MT][4],
                                       const Unit& t, int warp, int lane, int wr, int wk, bool ok,
                                       uint32_t* err) {
    const W4Args& a = p.a;
    const int values = p.wr * C::kValues;
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            part[((wk * p.wr + wr) * 4 * C::MT + 4 * i + e) * 32 + lane] =
                acc[i][e] * Widen<C::kBF16>::kScale;
    __syncwarp();
    if (!named_bar_and(1, C::kThreads, ok)) return false;
#pragma unroll 1
    for (int v = warp * 32 + lane; v < values; v += C::kThreads) {
        float sum = part[v];
#pragma unroll 4
        for (int q = 1; q < (1 << p.wk_shift); ++q) sum += part[q * values + v];
        const int l = v & 31, j = (v >> 5) & (4 * C::MT - 1), r = v / C::kValues;
        const int rr = r * C::kWarpRows + (j >> 2) * 16 + ((j >> 1) & 1) * 8 + (l >> 2);
        const int tok = (l & 3) * 2 + (j & 1);
        if (rr < t.rows && tok < t.tokens &&
            check_ok(t.n + rr < a.N && t.m + tok < a.M, err, kSiteCheckBounds))
            a.D[static_cast<int64_t>(t.m + tok) * a.N + t.n + rr] =
                cvt16_rn<C::kBF16>(__float_as_uint(sum));
    }
    __syncthreads();
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

    grid_launch_dependents();
    if (tid == 0) {
        for (int s = 0; s < p.depth; ++s) {
            mbar_init(smem_u32(&misc.full[s]), 1);
            mbar_init(smem_u32(&misc.empty[s]), C::kWarps);
        }
        misc.abort_flag = 0;
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    if (C::kGrouped && warp == 0) find_groups<C>(a, misc.groups, lane);
    __syncthreads();

    // Blocks of 256 k, a stage of 1 << (wk_shift - 1) blocks at a time.
    const int32_t stage_shift = p.wk_shift - 1, k256 = (a.K + 255) / 256;
    const int32_t per_unit = (k256 + (1 << stage_shift) - 1) >> stage_shift;

    Units<C, W4Problem> units(p, misc.groups, static_cast<int32_t>(blockIdx.x),
                               static_cast<int32_t>(gridDim.x));
    const int64_t total = static_cast<int64_t>(units.left) * per_unit;   // stages

    // ---- copies, by one thread ----
    Units<C, W4Problem> ahead = units;
    Unit at{};
    int32_t copied = 0, copy_slot = 0;
    uint32_t copy_phase = 1;
    auto copy_next = [&]() {
        const uint32_t full = smem_u32(&misc.full[copy_slot]);
        if (!wait_or_abort(smem_u32(&misc.empty[copy_slot]), copy_phase, abort_flag, err,
                           kSiteProducerEmpty, limit_ns))
            return;
        if (copied == 0) at = ahead.next(p, misc.groups);
        const int32_t b = copied << stage_shift, n = min(k256 - b, 1 << stage_shift);
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
        mbar_arrive_expect_tx(full, n * w + (p.stage_bytes - p.w_bytes));
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
    uint32_t w_at[4], x_at[4];
    const uint32_t w_row =
        sbase + static_cast<uint32_t>((wk >> 1) * p.box + wr * C::kWarpRows + row) * 128;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        w_at[b] = (w_row | ((wk & 1) * 64 + b * 16 + quad * 4)) ^ ((w_row >> 3) & 0x70u);
        const uint32_t at = sbase + p.w_bytes + quad * 16 +
                            ((wk * 4 + b) * p.tokens + min(row, p.tokens - 1)) * 64;
        x_at[b] = at ^ ((at >> 3) & 0x30u);
    }
    // Scales and zero points of this warp's part of the next stage: of rows row + 8 i,
    // group `quad` of the 128 k.
    uint32_t s_next[2 * C::MT] = {}, z_next[2 * C::MT] = {}, s_off[2 * C::MT];
    int64_t s_base = 0;
    int32_t group = 0;
    auto scales_of = [&](const Unit& u) {
        s_base = (static_cast<int64_t>(u.g) * a.N + u.n) * a.scale_groups;
        group = wk * 4 / C::GB + min(quad, kScales - 1);
#pragma unroll
        for (int i = 0; i < 2 * C::MT; ++i)
            s_off[i] = min(wr * C::kWarpRows + row + 8 * i, u.rows - 1) * a.scale_groups + group;
    };
    auto read_scales = [&]() {
        const bool in = group < a.scale_groups;     // (past K the tokens are zeros)
#pragma unroll
        for (int i = 0; i < 2 * C::MT; ++i) {
            s_next[i] = in ? a.S[s_base + s_off[i]] : 0;
            z_next[i] = in && a.Z ? a.Z[s_base + s_off[i]] : 8;
        }
    };
    float* part = reinterpret_cast<float*>(smem + p.off_part);
    Unit t{}, next{};
    float acc[C::MT][4] = {};
    uint32_t done = 0, phase = 0;
    int slot = 0;
    bool ok = true;
    bool more = units.left > 0;
    if (more) {
        next = units.next(p, misc.groups);
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
        if (more) next = units.next(p, misc.groups);
        const bool mine = wr * C::kWarpRows < t.rows;
        int32_t c = wk;                  // 128 k of this warp
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
            if (mine && c * 128 < a.K) {
                const uint32_t stage = slot * p.stage_bytes;
#pragma unroll
                for (int j = 0; j < kScales; ++j) {
                    float part[C::MT][4] = {};
                    Widen<C::kBF16> widen[2 * C::MT];
#pragma unroll
                    for (int i = 0; i < 2 * C::MT; ++i) widen[i] = Widen<C::kBF16>(both[j][i] >> 16);
#pragma unroll
                    for (int b = j * C::GB; b < (j + 1) * C::GB; ++b) {
                        uint32_t v[2 * C::MT][4];
#pragma unroll
                        for (int i = 0; i < 2 * C::MT; ++i)
                            widen[i](ld_shared_u32(w_at[b] + stage + i * 1024), v[i]);
                        uint32_t x[4];
                        pair_up(ld_shared_v4(x_at[b] + stage), x);
#pragma unroll
                        for (int i = 0; i < C::MT; ++i) {
                            mma_16816<C::kBF16>(part[i], v[2 * i][0], v[2 * i + 1][0], v[2 * i][1],
                                                v[2 * i + 1][1], x[0], x[1]);
                            mma_16816<C::kBF16>(part[i], v[2 * i][2], v[2 * i + 1][2], v[2 * i][3],
                                                v[2 * i + 1][3], x[2], x[3]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2 * C::MT; ++i) {
                        const float f = scale_value<C::kBF16>(both[j][i] & 0xffffu);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& out = acc[i / 2][2 * (i & 1) + e];
                            out = fmaf(part[i / 2][2 * (i & 1) + e], f, out);
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
        ok = finish<C>(p, part, acc, t, warp, lane, wr, wk, ok, err);
        if (ok && tid == 0)
            check_count_unit(err, static_cast<int32_t>(blockIdx.x + done * gridDim.x));
        ++done;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
    }
    // After a failed wait: the copies in flight must have landed before this CTA ends.
    if (*abort_flag && tid == 0) {
        const int64_t n = min(total, static_cast<int64_t>(p.depth));
        for (int s = 0; s < n; ++s)
            wait_bounded(smem_u32(&misc.full[s]), s < copy_slot ? copy_phase ^ 1u : copy_phase, err,
                         kSiteDrainFull, limit_ns);
    }
    __syncwarp();
}

// The shape of a launch, and the time it is expected to take, in stages.
struct W4Shape {
    int wr, wk_shift, depth;
    int64_t box;
    uint32_t w_bytes, pitch;      // of a stage: codes, codes and tokens
    int32_t tokens;
    double time;
};

template <class C>
W4Shape shape_of(const W4Args& a, int wr, int sms) {
    W4Shape s{};
    s.wr = wr;
    while ((wr << s.wk_shift) < C::kWarps) ++s.wk_shift;
    const int64_t rows = C::kWarpRows * wr, least = ceil_div(a.N, rows);
    // Units: of the groups, those that can have rows; dense, all blocks of tokens.
    const int64_t chunks =
        a.offsets ? (a.groups < a.M ? a.groups : a.M) : ceil_div(a.M, C::kTokens);
    const int64_t rounds = ceil_div(chunks * least, sms);
    // Dense: as many blocks of rows as those rounds have room for.
    int64_t blocks = a.offsets ? least : rounds * sms / chunks;
    if (blocks > a.N) blocks = a.N;
    s.box = ceil_div(a.N, blocks);
    const int32_t kc = 128 << s.wk_shift;
    s.tokens = a.M < C::kTokens ? a.M : C::kTokens;
    const uint32_t x_bytes = static_cast<uint32_t>(s.tokens * kc * 2);
    s.pitch = (static_cast<uint32_t>(s.box * (kc / 2)) + x_bytes + 1023u) / 1024u * 1024u;
    s.w_bytes = s.pitch - x_bytes;       // (tokens at a multiple of 512 bytes)
    const uint32_t depth = (kSmemLimit - C::kPartBytes - sizeof(W4Misc) - 1024) / s.pitch;
    s.depth = static_cast<int>(depth < kMaxDepth ? depth : kMaxDepth);
    // A stage takes about the same time whatever its shape (1.1 us), the end of a unit half
    // of that.
    s.time = rounds * (ceil_div(ceil_div(a.K, 256), kc / 256) + 0.5);
    return s;
}

template <class C>
cudaError_t launch_cfg(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    // The warps along the rows that are expected to take least time: 1 x 4096 x 14336 13.2 us
    // with one and 20 with two, 5 x 5003 x 2080 10.6 and 7.7.
    W4Shape s{};
    for (int wr = 1; C::kWarpRows * wr <= 256 && 2 * wr <= C::kWarps; wr *= 2) {
        const W4Shape t = shape_of<C>(a, wr, dev.sms);
        if (t.depth >= 2 && (s.depth == 0 || t.time < s.time)) s = t;
    }
    if (s.depth == 0) return cudaErrorInvalidConfiguration;
    W4Problem p{};
    p.a = a;
    p.wr = s.wr;
    p.wk_shift = s.wk_shift;
    p.depth = s.depth;
    p.box = static_cast<int32_t>(s.box);
    p.row_blocks = static_cast<int32_t>(ceil_div(a.N, s.box));
    p.tokens = s.tokens;
    p.w_bytes = s.w_bytes;
    p.stage_bytes = s.pitch;
    p.off_part = s.depth * s.pitch;
    p.off_misc = p.off_part + C::kPartBytes;
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
    return launch_kernel(kernel, dim3(static_cast<unsigned>(dev.sms)), dim3(C::kThreads), bytes,
                         stream, 1, dev.pdl, p, dev.limit_ns, dev.err_word);
}

template <bool BF16>
cudaError_t launch_scales(const W4Args& a, const W4Device& dev, cudaStream_t stream) {
    return a.offsets         ? launch_cfg<W4Cfg<BF16, 1, true>>(a, dev, stream)
           : a.group == 32   ? launch_cfg<W4Cfg<BF16, 1, false>>(a, dev, stream)
           : a.group == 64   ? launch_cfg<W4Cfg<BF16, 2, false>>(a, dev, stream)
                             : launch_cfg<W4Cfg<BF16, 4, false>>(a, dev, stream);
}

}  // namespace

cudaError_t launch_gemm_w4(const W4Args& a, bool bf16, const W4Device& dev, cudaStream_t stream) {
    // Up to eight tokens here, more on tcgen05: N x K = 4096 x 4096, groups of 128, 6.9 us here
    // and 8.1 there with 8 tokens, 9.4 and 8.2 with 12; 14336 x 4096, groups of 32, 15.7 and
    // 22.5, 28.6 and 22.5.  With groups of 128, whose sums are read back least, there too where
    // its blocks of 128 rows take more than half the SMs and K is long: one token, 8192 x 4096
    // 8.9 and 9.9, 9856 x 1024 5.6 and 5.4, 11008 x 4096 12.8 and 10.8, 19456 x 8192 24.1 and
    // 19.9; 14336 x 512 4.4 and 4.5, 28672 x 512 6.2 and 7.1, x 768 7.8 and 8.6, x 896 8.8 and
    // 8.4, x 8192 35.2 and 33.7.  Past two blocks an SM whatever K is: 38912 x 512 6.7 and 7.4,
    // 39040 x 512 8.9 and 7.4, x 256 6.8 and 5.0.  (The same with four and eight tokens.)
    // By group of rows, with N x K = 4096 x 2048: scales of 32 k up to two rows on average (64
    // groups with two each 91 and 100 us, with 256 rows in 50 of them 115 and 100), of 64 and
    // 128 none (64 groups, 128 rows: 68 and 44, 65 and 43; 8 rows 19 and 18, 18 and 16).
    const int64_t blocks = ceil_div(a.N, 128);
    const bool wide =
        a.group == 128 && 2 * blocks > dev.sms && (a.K > 768 || blocks > 2ll * dev.sms);
    const int64_t few = a.offsets ? (a.group == 32 ? 2 : 0) : wide ? 0 : 8;
    if (ceil_div(a.M, a.offsets ? a.groups : 1) > few)
        return launch_gemm_w4_many(a, bf16, dev, stream);
    return bf16 ? launch_scales<true>(a, dev, stream) : launch_scales<false>(a, dev, stream);
}

}  // namespace tmagemm
