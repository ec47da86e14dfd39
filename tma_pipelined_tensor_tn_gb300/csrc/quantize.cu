// Block quantisation to e4m3: X (M x K, fp16 or bf16) -> codes Q (M x K) and
// FP32 scales, one per 1 x 128 values (activations) or per 128 x 128 values
// (weights).  The format is described in fp8.cuh.
//
// Bound by memory: each value is read once (2 bytes) and written once (1
// byte); a block's values stay in registers between the maximum and the
// rounding, but for what four CTAs an SM leave no room for (64 registers a thread:
// 68 bytes spilled of an fp16 128 x 128 block, 12 of a tile of rows).  Measured on
// GB300 (device time, cold): rows of 8192 x 14336 57.8 us (6.1 TB/s), 128 x 128
// blocks of 4100 x 4096 9.6 us in fp16 (5.2 TB/s) and 9.3 in bf16, one row of 4096
// values 1.2 us.
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

// One scale per row and 128 columns.  A CTA takes 8 ROWS rows x 256 VECS
// columns: each warp ROWS rows, a lane eight values (16 bytes) of each 256
// columns, so a block is one half warp and ROWS x VECS loads per lane are in
// flight.  The scales are gathered in shared memory and written all rows of a
// block together, whole sectors in the layout with consecutive rows next to
// each other.
//
// 16 x 1024 tiles (2 KB of a row read together, four CTAs per SM) for large
// problems: 8192 x 14336 58 us (6.1 TB/s) against 65 us for 32 x 256.  8 x 256
// tiles where those would leave SMs idle: 1 x 4096 1.8 against 2.4 us.
template <bool BF16, int ROWS, int VECS>
__global__ void __launch_bounds__(kThreads, 4)
quantize_rows_kernel(const uint4* X, uint2* Q, float* S, int32_t M, int32_t K8, int32_t blocks,
                     int64_t s_row, int64_t s_blk) {
    constexpr int kRowTile = ROWS * kWarps;
    constexpr int kTileBlocks = 2 * VECS;   // 128-column blocks of a tile
    __shared__ float scales[kTileBlocks][kRowTile];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const int32_t c0 = static_cast<int32_t>(blockIdx.x) * (32 * VECS) + lane;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRowTile; row0 < M;
         row0 += static_cast<int64_t>(gridDim.y) * kRowTile) {
        uint4 x[ROWS][VECS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                const int64_t r = row0 + warp * ROWS + i;
                const int32_t c = c0 + 32 * v;   // 8-value chunk of the row
                x[i][v] = r < M && c < K8 ? ld_stream(X + r * K8 + c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                const int64_t r = row0 + warp * ROWS + i;
                const int32_t c = c0 + 32 * v;
                const BlockScale b =
                    block_scale(__uint_as_float(half_warp_max(max8<BF16>(x[i][v]))));
                if (r < M && c < K8) Q[r * K8 + c] = quantize8<BF16>(x[i][v], b.inverse);
                if ((lane & 15) == 0)
                    scales[2 * v + (lane >> 4)][warp * ROWS + i] = b.scale;
            }
        __syncthreads();
        if (threadIdx.x < kTileBlocks * kRowTile) {
            const int32_t i = static_cast<int32_t>(threadIdx.x) / kRowTile;
            const int32_t blk = static_cast<int32_t>(blockIdx.x) * kTileBlocks + i;
            const int64_t r = row0 + threadIdx.x % kRowTile;
            if (blk < blocks && r < M)
                S[r * s_row + blk * s_blk] = scales[i][threadIdx.x % kRowTile];
        }
        __syncthreads();
    }
}

// One scale per 128 x 128 values: one CTA per block, 16 rows at a time, the
// whole block (8 x 16 bytes per thread) held between the two passes.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4)
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

template <bool BF16, int ROWS, int VECS>
cudaError_t launch_row_tiles(int64_t M, int64_t K, const uint4* x, uint2* q, float* S,
                             int64_t s_row, int64_t s_blk, bool pdl, cudaStream_t stream) {
    const int64_t rows = ceil_div(M, ROWS * kWarps);
    const dim3 grid(static_cast<unsigned>(ceil_div(K, 256 * VECS)),
                    static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY));
    return launch_kernel(quantize_rows_kernel<BF16, ROWS, VECS>, grid, dim3(kThreads), 0, stream,
                         1, pdl, x, q, S, static_cast<int32_t>(M), static_cast<int32_t>(K / 8),
                         static_cast<int32_t>(ceil_div(K, kFp8Block)), s_row, s_blk);
}

template <bool BF16>
cudaError_t launch_typed(int64_t M, int64_t K, const uint4* x, int block_rows, uint2* q, float* S,
                         int64_t s_row, int64_t s_blk, int sms, bool pdl, cudaStream_t stream) {
    if (block_rows == 1) {
        if (ceil_div(M, 16) * ceil_div(K, 1024) >= 2ll * sms)
            return launch_row_tiles<BF16, 2, 4>(M, K, x, q, S, s_row, s_blk, pdl, stream);
        return launch_row_tiles<BF16, 1, 1>(M, K, x, q, S, s_row, s_blk, pdl, stream);
    }
    const int64_t rows = ceil_div(M, kFp8Block);
    const dim3 grid(static_cast<unsigned>(ceil_div(K, kFp8Block)),
                    static_cast<unsigned>(rows < kMaxGridY ? rows : kMaxGridY));
    return launch_kernel(quantize_tiles_kernel<BF16>, grid, dim3(kThreads), 0, stream, 1, pdl, x,
                         q, S, static_cast<int32_t>(M), static_cast<int32_t>(K / 8), s_row, s_blk);
}

}  // namespace

cudaError_t launch_quantize(int64_t M, int64_t K, const void* X, bool bf16, int block_rows,
                            void* Q, float* S, int64_t s_row, int64_t s_blk, int sms, bool pdl,
                            cudaStream_t stream) {
    const auto* x = static_cast<const uint4*>(X);
    auto* q = static_cast<uint2*>(Q);
    return bf16 ? launch_typed<true>(M, K, x, block_rows, q, S, s_row, s_blk, sms, pdl, stream)
                : launch_typed<false>(M, K, x, block_rows, q, S, s_row, s_blk, sms, pdl, stream);
}

}  // namespace tmagemm
