// The element-wise work between two blocks of a network, fused into one pass:
//   u  = y * rsqrt(mean(y^2) + eps) * w_post      (u = y without w_post)
//   h' = h + alpha * g * u                        (g: none, per channel, token or element)
//   x  = h' * rsqrt(mean(h'^2) + eps) * w_pre
// and its gradients.  All arithmetic is FP32; h' is rounded once when it is
// written, and x is computed from the unrounded h'.  x leaves in 16 bits or as
// e4m3 codes with a scale per 128 channels (fp8.cuh), ready for gemm_fp8.
//
// Bound by memory: a row of C channels stays in the registers of one CTA
// between the loads, the two sums and the stores, so each operand is read
// once and each result written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "fp8.cuh"

namespace tmagemm {

namespace {

constexpr int kMaxWarps = 32;

// Sum over the CTA, the same in every thread: each warp by shuffles, then
// every warp adds the warps' sums in the same order.  `slot` alternates, so
// one barrier separates the uses of a slot.
__device__ __forceinline__ float cta_sum(float v, float (*slots)[kMaxWarps], uint32_t& slot) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if (warps == 1) return v;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    float* s = slots[slot];
    slot ^= 1u;
    if (lane == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = lane < warps ? s[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    return t;
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v) {
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else
        return __half2float(__ushort_as_half(v));
}

// The gate of one row: per element of an 8-channel vector, or one number.
template <bool BF16>
__device__ __forceinline__ void gate8(const NormArgs& p, int64_t row, int32_t c, float (&g)[8]) {
    if (p.gate_mode == kGateChannel) {
        unpack8<BF16>(static_cast<const uint4*>(p.gate)[c], g);
    } else if (p.gate_mode == kGateElement) {
        unpack8<BF16>(static_cast<const uint4*>(p.gate)[row * p.C8 + c], g);
    } else {
        const float v = p.gate_mode == kGateToken
                            ? to_float<BF16>(static_cast<const uint16_t*>(p.gate)[row])
                            : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = v;
    }
}

// One CTA per row at a time; thread t holds the 8-channel vectors t + i *
// blockDim.x, i < V, so the 16 lanes of a half warp hold one 128-channel block.
template <bool BF16, int V>
__global__ void __launch_bounds__(1024)
norm_forward_kernel(const NormArgs p) {
    __shared__ float slots[2][kMaxWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    uint32_t slot = 0;
    const int32_t C8 = p.C8;
    const float inv_c = 1.0f / (8.0f * static_cast<float>(C8));
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        float h[V][8], y[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            unpack8<BF16>(c < C8 ? p.h[row * C8 + c] : z, h[i]);
            if (p.y) unpack8<BF16>(c < C8 ? p.y[row * C8 + c] : z, y[i]);
        }
        if (p.y) {
            float r = 1.0f;
            if (p.w_post) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(y[i][e], y[i][e], ss);
                r = rsqrtf(cta_sum(ss, slots, slot) * inv_c + p.eps);
                if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = r;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
                if (c >= C8) continue;
                float g[8], w[8];
                gate8<BF16>(p, row, c, g);
                if (p.w_post) {
                    unpack8<BF16>(p.w_post[c], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r * w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = fmaf(p.alpha, g[e] * y[i][e], h[i][e]);
                p.h_out[row * C8 + c] = pack8<BF16>(h[i]);
            }
        }
        if (!p.w_pre) continue;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
        const float r = rsqrtf(cta_sum(ss, slots, slot) * inv_c + p.eps);
        if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[row] = r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            float x[8] = {};
            if (c < C8) {
                float w[8];
                unpack8<BF16>(p.w_pre[c], w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = h[i][e] * r * w[e];
            }
            if (p.x) {
                if (c < C8) p.x[row * C8 + c] = pack8<BF16>(x);
                continue;
            }
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, magnitude_bits(x[e]));
            const BlockScale b = block_scale(__uint_as_float(half_warp_max(m)));
            if (c < C8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], b.inverse);
                p.q[row * C8 + c] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]),
                                               e4m3x4(x[4], x[5], x[6], x[7]));
                if ((threadIdx.x & 15) == 0) p.scales[row * p.s_row + (c >> 4) * p.s_blk] = b.scale;
            }
        }
    }
}

// Gradients.  With t the gradient of h' (through both of its uses),
//   p = dx * w_pre,  n = h' rh,  t = dh' + rh (p - n mean(p n))
//   dh = t,  du = alpha g t,  dgate = alpha u t
//   q = du * w_post,  m = y ry,  dy = ry (q - m mean(q m))    (dy = du without w_post)
//   dw_pre = sum over rows of dx n,  dw_post = sum over rows of du m.
// q m = alpha g t u, so its row sum is also a per-token gate's gradient times
// g; and with a per-channel gate both dw_post = g S and dgate = w_post S come
// from the one column sum S = sum alpha t m.  So a row needs two sums and a
// column two accumulators.  h' is recomputed from h and y, unrounded.
// A CTA walks rows blockIdx.x, + gridDim.x, ... with the column accumulators
// in registers, and leaves them in `partial` [CTA][2][C]; the second kernel
// adds them in CTA order, so the sums are the same from run to run.
template <bool BF16, int V>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024)
norm_backward_kernel(const NormArgs p) {
    __shared__ float slots[2][kMaxWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    uint32_t slot = 0;
    const int32_t C8 = p.C8;
    const float inv_c = 1.0f / (8.0f * static_cast<float>(C8));
    float col_a[V][8] = {}, col_b[V][8] = {};
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        const float ry = p.w_post ? p.rstd_post[row] : 1.0f;
        const float rh = p.w_pre ? p.rstd_pre[row] : 1.0f;
        float u[V][8], t[V][8], n[V][8];
        float sum1 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            const bool in = c < C8;
            float hv[8], g[8], w[8];
            unpack8<BF16>(in ? p.h[row * C8 + c] : z, hv);
            unpack8<BF16>(in && p.y ? p.y[row * C8 + c] : z, u[i]);
            unpack8<BF16>(in && p.dh ? p.dh[row * C8 + c] : z, t[i]);
            if (p.w_post) {
                unpack8<BF16>(in ? p.w_post[c] : z, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * ry * w[e];
            }
            if (p.w_pre) {
                float dx[8];
                if (in) gate8<BF16>(p, row, c, g);
                unpack8<BF16>(in ? p.dx[row * C8 + c] : z, dx);
                unpack8<BF16>(in ? p.w_pre[c] : z, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float h2 = in ? fmaf(p.alpha, g[e] * u[i][e], hv[e]) : 0.0f;
                    n[i][e] = h2 * rh;
                    col_b[i][e] = fmaf(dx[e], n[i][e], col_b[i][e]);
                    sum1 = fmaf(dx[e] * w[e], n[i][e], sum1);
                    t[i][e] = fmaf(rh, dx[e] * w[e], t[i][e]);
                }
            }
        }
        if (p.w_pre) {
            const float c1 = cta_sum(sum1, slots, slot) * inv_c;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = fmaf(-rh * c1, n[i][e], t[i][e]);
        }
        // sum of alpha t u (times g, where g differs within the row)
        float sum2 = 0.0f;
        const bool g_row = p.gate_mode == kGateNone || p.gate_mode == kGateToken;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            if (c >= C8) continue;
            p.dh_in[row * C8 + c] = pack8<BF16>(t[i]);
            if (!p.y) continue;
            float g[8];
            gate8<BF16>(p, row, c, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum2 = fmaf(p.alpha * t[i][e], g_row ? u[i][e] : g[e] * u[i][e], sum2);
        }
        if (!p.y) continue;
        float c2 = 0.0f;
        if (p.w_post || p.gate_mode == kGateToken) {
            c2 = cta_sum(sum2, slots, slot);
            if (p.gate_mode == kGateToken) {
                if (threadIdx.x == 0) static_cast<float*>(p.dgate)[row] = c2;
                c2 *= to_float<BF16>(static_cast<const uint16_t*>(p.gate)[row]);
            }
            c2 *= inv_c;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            if (c >= C8) continue;
            float g[8], w[8], m[8], dy[8], dg[8];
            gate8<BF16>(p, row, c, g);
            unpack8<BF16>(p.y[row * C8 + c], m);
            if (p.w_post) unpack8<BF16>(p.w_post[c], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float at = p.alpha * t[i][e];
                dg[e] = at * u[i][e];
                const float du = at * g[e];
                if (p.w_post) {
                    m[e] *= ry;
                    dy[e] = ry * (du * w[e] - m[e] * c2);
                } else {
                    dy[e] = du;
                }
                col_a[i][e] = fmaf(p.gate_mode == kGateChannel ? at : du, m[e], col_a[i][e]);
            }
            p.dy[row * C8 + c] = pack8<BF16>(dy);
            if (p.gate_mode == kGateElement) static_cast<uint4*>(p.dgate)[row * C8 + c] = pack8<BF16>(dg);
        }
    }
    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 16 * C8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
        if (c >= C8) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            part[8 * c + e] = col_a[i][e];
            part[8 * (C8 + c) + e] = col_b[i][e];
        }
    }
}

// Column sums of the partials, in CTA order: 32 columns x 8 slices of the CTAs
// per block, the slices added in order.
template <bool BF16>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormArgs p, int32_t ctas) {
    __shared__ float s[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C = 8 * p.C8;
    const int lane = static_cast<int>(threadIdx.x) & 31, slice = static_cast<int>(threadIdx.x) >> 5;
    const int32_t col = static_cast<int32_t>(blockIdx.x) * 32 + lane;   // 0 .. 2 C
    const int32_t per = (ctas + 7) / 8;
    float v = 0.0f;
    if (col < 2 * C)
        for (int32_t i = slice * per; i < min(ctas, (slice + 1) * per); ++i)
            v += p.partial[static_cast<int64_t>(i) * 2 * C + col];
    s[slice][lane] = v;
    __syncthreads();
    if (slice != 0 || col >= 2 * C) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][lane];
    if (col >= C) {
        if (p.dw_pre) p.dw_pre[col - C] = v;
        return;
    }
    const bool channel = p.gate_mode == kGateChannel;
    if (p.dw_post)
        p.dw_post[col] =
            channel ? v * to_float<BF16>(static_cast<const uint16_t*>(p.gate)[col]) : v;
    if (channel)
        static_cast<float*>(p.dgate)[col] =
            p.w_post ? v * to_float<BF16>(reinterpret_cast<const uint16_t*>(p.w_post)[col]) : v;
}

unsigned row_threads(int64_t C8, int V) {
    return static_cast<unsigned>(((C8 + V - 1) / V + 31) / 32 * 32);
}

template <bool BF16>
cudaError_t forward_typed(const NormArgs& p, int sms, bool pdl, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(p.T < (1 << 30) ? p.T : (1 << 30));
    const bool one = p.C8 <= 1024 && (p.C8 <= 128 || p.T <= 2 * sms);
    if (one)
        return launch_kernel(norm_forward_kernel<BF16, 1>, dim3(grid), dim3(row_threads(p.C8, 1)),
                             0, stream, 1, pdl, p);
    return launch_kernel(norm_forward_kernel<BF16, 2>, dim3(grid), dim3(row_threads(p.C8, 2)), 0,
                         stream, 1, pdl, p);
}

template <bool BF16>
cudaError_t backward_typed(const NormArgs& p, int ctas, bool pdl, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (ctas == 0) {
        // no rows: the column sums below come out as zeros
    } else if (p.C8 <= 512)
        e = launch_kernel(norm_backward_kernel<BF16, 1>, dim3(ctas), dim3(row_threads(p.C8, 1)), 0,
                          stream, 1, pdl, p);
    else
        e = launch_kernel(norm_backward_kernel<BF16, 2>, dim3(ctas), dim3(row_threads(p.C8, 2)), 0,
                          stream, 1, pdl, p);
    const bool columns = p.dw_pre || p.dw_post || p.gate_mode == kGateChannel;
    if (e != cudaSuccess || !columns) return e;
    return launch_kernel(norm_columns_kernel<BF16>, dim3((16 * p.C8 + 31) / 32), dim3(256), 0,
                         stream, 1, pdl, p, static_cast<int32_t>(ctas));
}

}  // namespace

int norm_backward_ctas(int64_t T, int sms) {
    const int64_t most = 2 * static_cast<int64_t>(sms);
    return static_cast<int>(T < most ? T : most);
}

cudaError_t launch_norm_forward(const NormArgs& p, bool bf16, int sms, bool pdl,
                                cudaStream_t stream) {
    return bf16 ? forward_typed<true>(p, sms, pdl, stream)
                : forward_typed<false>(p, sms, pdl, stream);
}

cudaError_t launch_norm_backward(const NormArgs& p, bool bf16, int sms, bool pdl,
                                 cudaStream_t stream) {
    const int ctas = norm_backward_ctas(p.T, sms);
    return bf16 ? backward_typed<true>(p, ctas, pdl, stream)
                : backward_typed<false>(p, ctas, pdl, stream);
}

}  // namespace tmagemm
