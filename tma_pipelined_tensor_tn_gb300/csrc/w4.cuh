// What the products with 4-bit weights share: the units of work, the groups' rows, and the
// exact widening of codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace tmagemm {

// Products of more tokens, on tcgen05.
cudaError_t launch_gemm_w4_many(const W4Args& a, bool bf16, const W4Device& dev,
                                cudaStream_t stream);

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMaxGroups = 384;
constexpr int kMaxDepth = 8;
constexpr uint32_t kSmemLimit = 232448;

// First row of each group, and blocks of tokens of all.
struct W4Groups {
    int32_t chunks;
    int32_t first[kMaxGroups + 1];
};

// A unit of work: `rows` weight rows from n of group g, `tokens` tokens from m.
struct Unit {
    int32_t n, m, g, rows, tokens;
};

// Every `step`-th unit from `id` on, in order: token block by token block of each group, and
// row block by row block of each.
template <class C, class P>
struct Units {
    int32_t left, step, block, m, g;    // the next unit is a later one if block >= row_blocks
    __device__ Units(const P& p, const W4Groups& groups, int32_t id, int32_t every) : step(every) {
        const int32_t chunks =
            C::kGrouped ? groups.chunks : (p.a.M + C::kTokens - 1) / C::kTokens;
        const int64_t all = static_cast<int64_t>(chunks) * p.row_blocks;
        left = all <= id ? 0
                         : all <= 0x7fffffff - step
                               ? (static_cast<int32_t>(all) - id + step - 1) / step
                               : static_cast<int32_t>((all - id + step - 1) / step);
        block = id;
        g = 0;
        m = C::kGrouped ? groups.first[0] : 0;
    }
    // The next unit (left > 0).
    __device__ __forceinline__ Unit next(const P& p, const W4Groups& groups) {
        int32_t end = C::kGrouped ? groups.first[g + 1] : p.a.M;
        while (block >= p.row_blocks || m >= end) {
            if (m < end) {
                block -= p.row_blocks;
                m += C::kTokens;
            }
            if (C::kGrouped && m >= end) {
                ++g;
                m = end;
                end = groups.first[g + 1];
            }
        }
        const Unit t{block * p.box, m, g, min(p.box, p.a.N - block * p.box),
                     min(C::kTokens, end - m)};
        block += step;
        --left;
        return t;
    }
};

// The groups' rows and blocks of tokens, by one warp.  (An offset counts as the largest
// so far, within [0, M].)
template <class C>
__device__ __forceinline__ void find_groups(const W4Args& a, W4Groups& groups, int lane) {
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
        if (i <= a.groups) groups.first[i] = v;
        last = __shfl_sync(kAll, v, 31);
        chunks += __shfl_sync(kAll, n, 31);
    }
    if (lane == 0) groups.chunks = chunks;
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
template <bool BF16>
__device__ __forceinline__ float scale_value(uint32_t bits) {
    if constexpr (BF16) return __uint_as_float(bits << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at));
    return v;
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

}  // namespace

}  // namespace tmagemm
