// Device helpers of the block-scaled 8-bit format: e4m3 codes with one FP32
// scale per block of 128 values along K (or per 128 x 128 values).
//
// Quantisation of a block whose largest magnitude is `a`:
//   a' = max(a, 2^-100),  S = fl32(a' / 448),  Q = e4m3_rn(fl32(x * fl32(448 / a'))).
// 448 is the largest finite e4m3 value.  The floor 2^-100 keeps both quotients
// normal FP32 numbers (an all-zero block gets codes 0 and a tiny scale).  One
// division per block and one multiplication per element, each rounded once to
// FP32, so the codes are the same on every machine with IEEE arithmetic.
// A NaN in the block makes a, and with it the scale, NaN; an infinity makes
// the scale infinite and its own code NaN (inf * 0): neither can pass unseen.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

namespace tmagemm {

constexpr int kFp8Block = 128;              // values per scale along K
constexpr float kFp8Max = 448.0f;           // largest finite e4m3 value
constexpr float kFp8AmaxFloor = 0x1p-100f;  // smallest magnitude a scale is made from

struct BlockScale {
    float scale;    // what a code is multiplied with
    float inverse;  // what a value is multiplied with before it is rounded to a code
};

__device__ __forceinline__ BlockScale block_scale(float amax) {
    // A comparison, not fmaxf: NaN has to stay.
    const float a = amax < kFp8AmaxFloor ? kFp8AmaxFloor : amax;
    return {__fdiv_rn(a, kFp8Max), __fdiv_rn(kFp8Max, a)};
}

// Four values -> four e4m3 codes (nearest even; |v| <= 448 (1 + 2^-22) rounds to 448).
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v2, v3), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// |v| as ordered bits: unsigned comparison orders magnitudes, NaN above infinity.
__device__ __forceinline__ uint32_t magnitude_bits(float v) {
    return __float_as_uint(v) & 0x7fffffffu;
}

// Eight packed 16-bit values -> FP32.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// Eight FP32 -> packed 16-bit values, each rounded once to nearest even.
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint4 p;
    p.x = pack2_rn<BF16>(__float_as_uint(v[0]), __float_as_uint(v[1]));
    p.y = pack2_rn<BF16>(__float_as_uint(v[2]), __float_as_uint(v[3]));
    p.z = pack2_rn<BF16>(__float_as_uint(v[4]), __float_as_uint(v[5]));
    p.w = pack2_rn<BF16>(__float_as_uint(v[6]), __float_as_uint(v[7]));
    return p;
}

// Largest magnitude bits over the 16 lanes of a half warp (all 32 lanes active).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m) {
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// acc += t * s, with t from TMEM.  Volatile, so that it stays behind the wait
// for the load that brought t.  (Multiply-adds of packed pairs are half as
// many instructions for the same cycles, but each loaded register is then
// copied to form its pair.)
__device__ __forceinline__ void scale_add(float& acc, uint32_t t, float s) {
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(t)), "f"(s));
}

}  // namespace tmagemm
