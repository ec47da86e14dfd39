// Block quantisation to e4m3: X (M x K, fp16 or bf16) -> codes Q (M x K) and
// FP32 scales, one per 1 x 128 values (activations) or per 128 x 128 values
// (weights).  The format is described in fp8.cuh.
//
// Bound by memory: each value is read once (2 bytes) and written once (1
// byte); a block's values stay in registers between the maximum and the
// rounding.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"

namespace tmagemm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Magnitude bits of the largest of eight values.
template <bool BF16>
__device__ __forceinline__ uint32_t max8(const uint4& p) {
    float v[8];
    unpack8<BF16>(p, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude_bits(v[i]));
    return m;
}

template <bool BF16>
__device__ __forceinline__ uint2 quantize8(const uint4& p, float inverse) {
    float v[8];
    unpack8<BF16>(p, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], inverse);
    return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// One scale per row and 128 columns.  A CTA takes 32 rows x 256 columns: each
// warp four rows, a lane eight values (16 bytes) of each, so a block is one
// half warp and four loads per lane are in flight.  The 64 scales are gathered
// in shared memory and written 32 rows at a time, whole lines in the layout
// with consecutive rows next to each other.
constexpr int kRowTile = 32, kRowsPerWarp = kRowTile / kWarps;

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const uint4* X, uint2* Q, float* S, int32_t M, int32_t K8, int32_t blocks,
                     int64_t s_row, int64_t s_blk) {
    __shared__ float scales[2][kRowTile];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const int32_t c = static_cast<int32_t>(blockIdx.x) * 32 + lane;   // 8-value chunk of the row
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRowTile; row0 < M;
         row0 += static_cast<int64_t>(gridDim.y) * kRowTile) {
        uint4 x[kRowsPerWarp];
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            const int64_t r = row0 + warp * kRowsPerWarp + i;
            x[i] = r < M && c < K8 ? ld_stream(X + r * K8 + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            const int64_t r = row0 + warp * kRowsPerWarp + i;
            const BlockScale b = block_scale(__uint_as_float(half_warp_max(max8<BF16>(x[i]))));
            if (r < M && c < K8) Q[r * K8 + c] = quantize8<BF16>(x[i], b.inverse);
            if ((lane & 15) == 0) scales[lane >> 4][warp * kRowsPerWarp + i] = b.scale;
        }
        __syncthreads();
        if (threadIdx.x < 2 * kRowTile) {
            const int32_t blk = static_cast<int32_t>(blockIdx.x) * 2 + (threadIdx.x >> 5);
            const int64_t r = row0 + lane;
            if (blk < blocks && r < M) S[r * s_row + blk * s_blk] = scales[threadIdx.x >> 5][lane];
        }
        __syncthreads();
    }
}

// One scale per 128 x 128 values: one CTA per block, 16 rows at a time, the
// whole block (8 x 16 bytes per thread) in registers.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
quantize_tiles_kernel(const uint4* X, uint2* Q, float* S, int32_t M, int32_t K8, int64_t s_row,
                      int64_t s_blk) {
    __shared__ uint32_t warp_max[kWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const int32_t c = static_cast<int32_t>(blockIdx.x) * 16 + (lane & 15);
    for (int64_t tile = blockIdx.y; tile * kFp8Block < M; tile += gridDim.y) {
        const int64_t row0 = tile * kFp8Block + (threadIdx.x >> 4);
        uint4 x[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = row0 + 16 * i;
            x[i] = r < M && c < K8 ? ld_stream(X + r * K8 + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, max8<BF16>(x[i]));
        m = half_warp_max(m);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = max(m, warp_max[w]);
        const BlockScale b = block_scale(__uint_as_float(m));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = row0 + 16 * i;
            if (r < M && c < K8) Q[r * K8 + c] = quantize8<BF16>(x[i], b.inverse);
        }
        if (threadIdx.x == 0) S[tile * s_row + blockIdx.x * s_blk] = b.scale;
        __syncthreads();
    }
}

constexpr int64_t kMaxGridY = 65535;

}  // namespace

cudaError_t launch_quantize(int64_t M, int64_t K, const void* X, bool bf16, int block_rows,
                            void* Q, float* S, int64_t s_row, int64_t s_blk, bool pdl,
                            cudaStream_t stream) {
    const auto* x = static_cast<const uint4*>(X);
    auto* q = static_cast<uint2*>(Q);
    const int32_t m = static_cast<int32_t>(M), k8 = static_cast<int32_t>(K / 8);
    const int64_t blocks = (K + kFp8Block - 1) / kFp8Block;
    if (block_rows == 1) {
        const int64_t rows = (M + kRowTile - 1) / kRowTile;
        const dim3 grid(static_cast<unsigned>((blocks + 1) / 2),
                        static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY));
        return launch_kernel(bf16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>, grid,
                             dim3(kThreads), 0, stream, 1, pdl, x, q, S, m, k8,
                             static_cast<int32_t>(blocks), s_row, s_blk);
    }
    const int64_t rows = (M + kFp8Block - 1) / kFp8Block;
    const dim3 grid(static_cast<unsigned>(blocks),
                    static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY));
    return launch_kernel(bf16 ? quantize_tiles_kernel<true> : quantize_tiles_kernel<false>, grid,
                         dim3(kThreads), 0, stream, 1, pdl, x, q, S, m, k8, s_row, s_blk);
}

}  // namespace tmagemm
