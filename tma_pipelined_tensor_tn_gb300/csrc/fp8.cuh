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

#include "ptx.cuh"

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

// Two packed floats: one arithmetic instruction for both, each half rounded
// once to nearest even.
using f32x2 = uint64_t;

__device__ __forceinline__ f32x2 pack_f32x2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
    float lo, hi;
    unpack_f32x2(v, lo, hi);
    return lo + hi;
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

// The same, in pairs.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& p, f32x2 (&v)[4]) {
    float f[8];
    unpack8<BF16>(p, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_f32x2(f[2 * i], f[2 * i + 1]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const f32x2 (&v)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_f32x2(v[i], f[2 * i], f[2 * i + 1]);
    return pack8<BF16>(f);
}

// Largest magnitude bits over the 16 lanes of a half warp (all 32 lanes active).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m) {
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// wait_or_abort for many warps that wait often: a few tries of three
// instructions each before the first look at the abort flag and the clock, so
// that the waiting warps leave the issue slots to the working ones.
__device__ __forceinline__ bool wait_many(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* err_word, uint32_t site, uint64_t limit_ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P, Q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 64;\n"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 P, [%1], %2;\n\t"
        "@P bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 Q, n, 0;\n\t"
        "@Q bra TRY;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    return wait_or_abort(bar, parity, abort_flag, err_word, site, limit_ns);
}

// Instruction descriptor of kind::f8f6f4 with e4m3 operands and FP32 sums
// (both K-major): the fields are those of kind::f16, with operand format 0 =
// e4m3.
constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// acc += {t0, t1} * s, each half rounded once, with t0 and t1 from TMEM.  Volatile, so that it stays
// behind the wait for the load that brought them.
__device__ __forceinline__ void scale_add(f32x2& acc, uint32_t t0, uint32_t t1, f32x2 s) {
    asm volatile(
        "{\n\t.reg .b64 t;\n\t"
        "mov.b64 t, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(t0), "r"(t1), "l"(s));
}

}  // namespace tmagemm
