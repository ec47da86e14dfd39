// Products of a few tokens with 4-bit weights and group scales:
//   D[m][n] = sum_k A[m][k] (q[n][k] - z[n][g]) s[n][g],  g = k / group.
//
// A warp has one row of weights and up to eight tokens of a group of rows; its lanes
// take blocks of 32 k in turn (16 bytes of codes each), multiply in FP32 and apply the
// scale to the block's sum.
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

constexpr int kWarps = 8;
constexpr int kTokens = 8;
constexpr uint32_t kAll = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float value16(uint16_t bits) {
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(bits) << 16);
    return __half2float(__ushort_as_half(bits));
}

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32) gemm_w4_kernel(const __grid_constant__ W4Args a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const int32_t blocks = a.K / 32, kg = a.scale_groups;
    for (int32_t g = blockIdx.y; g < a.groups; g += gridDim.y) {
        int32_t lo = 0, hi = a.M;
        if (a.offsets) {
            // An offset counts as the largest so far, within [0, M].
            for (int32_t i = 0; i <= g; ++i) lo = min(max(lo, a.offsets[i]), a.M);
            hi = min(max(lo, a.offsets[g + 1]), a.M);
        }
        const int64_t row = g * static_cast<int64_t>(a.N) + n;
        const uint4* w = a.B + row * blocks;
        for (int32_t m0 = lo; m0 < hi; m0 += kTokens) {
            const int count = min(kTokens, hi - m0);
            float acc[kTokens] = {};
            for (int32_t b = lane; b < blocks; b += 32) {
                const uint4 q = w[b];
                const uint32_t word[4] = {q.x, q.y, q.z, q.w};
                const int64_t at = row * kg + b * 32 / a.group;
                const float s = value16<BF16>(a.S[at]);
                const float z = a.Z ? static_cast<float>(a.Z[at]) : 8.0f;
                for (int m = 0; m < count; ++m) {
                    const uint4* x = a.A + (static_cast<int64_t>(m0 + m) * blocks + b) * 4;
                    float part = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[8];
                        unpack8<BF16>(x[i], v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            part = fmaf(v[e], static_cast<float>((word[i] >> (4 * e)) & 15u) - z,
                                        part);
                    }
                    acc[m] = fmaf(part, s, acc[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                float v = acc[m];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
                if (lane == 0 && m < count)
                    a.D[static_cast<int64_t>(m0 + m) * a.N + n] = cvt16_rn<BF16>(__float_as_uint(v));
            }
        }
    }
}

}  // namespace

cudaError_t launch_gemm_w4(const W4Args& a, bool bf16, const W4Device& dev, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.N, kWarps)),
                    static_cast<unsigned>(a.groups));
    return launch_kernel(bf16 ? gemm_w4_kernel<true> : gemm_w4_kernel<false>, grid,
                         dim3(kWarps * 32), 0, stream, 1u, dev.pdl, a);
}

}  // namespace tmagemm
