// The element-wise work between two blocks of a network, fused into one pass:
//   u  = y * rsqrt(mean(y^2) + eps) * w_post      (u = y without w_post)
//   h' = h + alpha * g * u                        (g: none, per channel, token or element)
//   x  = h' * rsqrt(mean(h'^2) + eps) * w_pre
// and its gradients.  All arithmetic is FP32; h' is rounded once when it is
// written, and x is computed from the unrounded h'.  x leaves in 16 bits or as
// e4m3 codes with a scale per 128 channels (fp8.cuh), ready for gemm_fp8.
//
// Bound by memory, each operand read once and each result written once.  A CTA
// walks rows blockIdx.x, + gridDim.x, ...; thread t owns the 8-channel vectors
// t + i * blockDim.x of every row, so weights and column sums stay in its
// registers, and it copies its own vectors of the next row into shared memory
// (cp.async) while the CTA works on this one: no thread reads another's copy,
// so only the two row sums need a barrier.
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

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All copies of this thread but those of its latest N groups have arrived.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kMaxRowInputs = 5;

// The T x C operands of a row: their order in a stage, -1 where absent.
struct RowInputs {
    const uint4* base[kMaxRowInputs];
    int n;
    int h, y, gate, dh, dx;
    int stages;   // rows in shared memory: 2, or 1 where two do not fit
};

// This thread's vectors of the rows of its CTA, in shared memory one row ahead
// (with one stage, the next row's are fetched when this one is done):
// vector i of operand a at ring[(stage * n + a) * V + i][thread].
template <int V>
struct RowPipe {
    const RowInputs& in;
    uint32_t base;    // shared-memory address of this thread's column
    uint32_t step;    // bytes between consecutive vectors of a thread
    int32_t C8;
    uint32_t stage = 0;

    __device__ __forceinline__ RowPipe(const RowInputs& inputs, uint4* ring, int32_t c8)
        : in(inputs), base(smem_u32(ring) + threadIdx.x * 16u), step(blockDim.x * 16u), C8(c8) {}
    __device__ __forceinline__ uint32_t at(uint32_t st, int a, int i) const {
        return base + ((st * in.n + a) * V + i) * step;
    }
    __device__ __forceinline__ void issue(int64_t row, int64_t T, uint32_t st) {
        if (row < T) {
            for (int a = 0; a < in.n; ++a)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
                    if (c < C8) cp_async_16(at(st, a, i), in.base[a] + row * C8 + c);
                }
        }
        cp_async_commit();
    }
    // Before a row: starts on the copies of row `next`, waits for this row's.
    __device__ __forceinline__ void begin(int64_t next, int64_t T) {
        if (in.stages == 2) {
            issue(next, T, stage ^ 1u);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
    }
    // After a row (its vectors have been read).
    __device__ __forceinline__ void end(int64_t next, int64_t T) {
        if (in.stages == 2)
            stage ^= 1u;
        else
            issue(next, T, 0);
    }
    template <bool BF16>
    __device__ __forceinline__ void read(int a, int i, float (&v)[8]) const {
        uint4 p;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(p.x), "=r"(p.y), "=r"(p.z), "=r"(p.w)
                     : "r"(at(stage, a, i))
                     : "memory");
        unpack8<BF16>(p, v);
    }
};

// This thread's vectors of the per-channel operands, kept packed.
template <int V>
struct Channels {
    uint4 w_post[V], w_pre[V], gate[V];
    __device__ __forceinline__ explicit Channels(const NormArgs& p) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            w_post[i] = p.w_post && c < p.C8 ? p.w_post[c] : z;
            w_pre[i] = p.w_pre && c < p.C8 ? p.w_pre[c] : z;
            gate[i] = p.gate_mode == kGateChannel && c < p.C8
                          ? static_cast<const uint4*>(p.gate)[c]
                          : z;
        }
    }
};

// The gate of vector i of the current row; `token` is a per-token gate (or 1).
template <bool BF16, int V>
__device__ __forceinline__ void gate8(const NormArgs& p, const Channels<V>& ch,
                                      const RowPipe<V>& pipe, float token, int i,
                                      float (&g)[8]) {
    if (p.gate_mode == kGateChannel) {
        unpack8<BF16>(ch.gate[i], g);
    } else if (p.gate_mode == kGateElement) {
        pipe.template read<BF16>(pipe.in.gate, i, g);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = token;
    }
}

template <bool BF16>
__device__ __forceinline__ float token_gate(const NormArgs& p, int64_t row) {
    return p.gate_mode == kGateToken && row < p.T
               ? to_float<BF16>(static_cast<const uint16_t*>(p.gate)[row])
               : 1.0f;
}

// The 16 lanes of a half warp hold one 128-channel block, so its largest
// magnitude takes four shuffles.
template <bool BF16, int V, int MAX_THREADS, int MIN_CTAS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_CTAS)
norm_forward_kernel(const __grid_constant__ NormArgs p, const __grid_constant__ RowInputs in) {
    extern __shared__ uint4 ring[];
    __shared__ float slots[2][kMaxWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C8 = p.C8;
    const float channels = 8.0f * static_cast<float>(C8);
    uint32_t slot = 0;
    RowPipe<V> pipe(in, ring, C8);
    pipe.issue(blockIdx.x, p.T, 0);
    float token_next = token_gate<BF16>(p, blockIdx.x);
    const Channels<V> ch(p);
    for (int64_t row = blockIdx.x; row < p.T; pipe.end(row + gridDim.x, p.T), row += gridDim.x) {
        pipe.begin(row + gridDim.x, p.T);
        const float token = token_next;
        token_next = token_gate<BF16>(p, row + gridDim.x);
        float h[V][8];
        float r = 1.0f;
        if (p.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (static_cast<int32_t>(threadIdx.x + i * blockDim.x) >= C8) continue;
                float y[8];
                pipe.template read<BF16>(in.y, i, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
            }
            r = __frsqrt_rn(cta_sum(ss, slots, slot) / channels + p.eps);
            if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = r;
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
            if (c >= C8) continue;
            pipe.template read<BF16>(in.h, i, h[i]);
            if (p.y) {
                float y[8], g[8];
                pipe.template read<BF16>(in.y, i, y);
                gate8<BF16>(p, ch, pipe, token, i, g);
                if (p.w_post) {
                    float w[8];
                    unpack8<BF16>(ch.w_post[i], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = fmaf(p.alpha, g[e] * y[e], h[i][e]);
                p.h_out[row * C8 + c] = pack8<BF16>(h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
        }
        if (!p.w_pre) continue;
        r = __frsqrt_rn(cta_sum(ss, slots, slot) / channels + p.eps);
        if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[row] = r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            float x[8], w[8];
            unpack8<BF16>(ch.w_pre[i], w);   // zeros past the last channel
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = h[i][e] * r * w[e];
            if (p.x) {
                if (c < C8) p.x[row * C8 + c] = pack8<BF16>(x);
                continue;
            }
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, c < C8 ? magnitude_bits(x[e]) : 0u);
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
// The column accumulators are left in `partial` [CTA][2][C]; the second kernel
// adds them in CTA order, so the sums are the same from run to run.
// POST (w_post given) and GATE are fixed at compile time: read at run time they
// cost half as many instructions again.
template <bool BF16, bool POST, int GATE, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, 1)
norm_backward_kernel(const __grid_constant__ NormArgs p, const __grid_constant__ RowInputs in) {
    constexpr int V = 2;
    constexpr bool kTokenLike = GATE == kGateNone || GATE == kGateToken;   // one gate per row
    extern __shared__ uint4 ring[];
    __shared__ float slots[2][kMaxWarps];
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C8 = p.C8;
    const float inv_c = 1.0f / (8.0f * static_cast<float>(C8));
    uint32_t slot = 0;
    RowPipe<V> pipe(in, ring, C8);
    pipe.issue(blockIdx.x, p.T, 0);
    // The row's two factors and its gate, one row ahead like its operands.
    float token_next = 1.0f, ry_next = 1.0f, rh_next = 1.0f;
    auto fetch = [&](int64_t row) {
        if (row >= p.T) return;
        if constexpr (GATE == kGateToken) token_next = token_gate<BF16>(p, row);
        if constexpr (POST) ry_next = p.rstd_post[row];
        if (p.w_pre) rh_next = p.rstd_pre[row];
    };
    fetch(blockIdx.x);
    const Channels<V> ch(p);
    float col_a[V][8] = {}, col_b[V][8] = {};
    for (int64_t row = blockIdx.x; row < p.T; pipe.end(row + gridDim.x, p.T), row += gridDim.x) {
        pipe.begin(row + gridDim.x, p.T);
        // alpha times the row's gate where that is one number
        const float ry = ry_next, rh = rh_next, ag = p.alpha * token_next;
        fetch(row + gridDim.x);
        // alpha g of vector i
        auto scaled_gate = [&](int i, float (&g)[8]) {
            if constexpr (GATE == kGateChannel) unpack8<BF16>(ch.gate[i], g);
            if constexpr (GATE == kGateElement) pipe.template read<BF16>(in.gate, i, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = kTokenLike ? ag : p.alpha * g[e];
        };
        float u[V][8] = {}, t[V][8] = {}, n[V][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (static_cast<int32_t>(threadIdx.x + i * blockDim.x) >= C8) continue;
            float w[8];
            if (POST || in.y >= 0) pipe.template read<BF16>(in.y, i, u[i]);
            if constexpr (POST) {
                unpack8<BF16>(ch.w_post[i], w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[i][e] *= ry * w[e];
            }
            if (in.dh >= 0) pipe.template read<BF16>(in.dh, i, t[i]);
            if (p.w_pre) {
                float dx[8], g[8];
                pipe.template read<BF16>(in.h, i, n[i]);
                scaled_gate(i, g);
                pipe.template read<BF16>(in.dx, i, dx);
                unpack8<BF16>(ch.w_pre[i], w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[i][e] = fmaf(g[e], u[i][e], n[i][e]) * rh;
                    col_b[i][e] = fmaf(dx[e], n[i][e], col_b[i][e]);
                    dx[e] *= w[e];
                    sum = fmaf(dx[e], n[i][e], sum);
                    t[i][e] = fmaf(rh, dx[e], t[i][e]);
                }
            }
        }
        float c1 = 0.0f;
        if (p.w_pre) c1 = -rh * (cta_sum(sum, slots, slot) * inv_c);
        // t, and the sum of t u (times alpha g where g differs within the row)
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            if (c >= C8) continue;
            if (p.w_pre) {
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = fmaf(c1, n[i][e], t[i][e]);
            }
            p.dh_in[row * C8 + c] = pack8<BF16>(t[i]);
            if constexpr (kTokenLike) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(t[i][e], u[i][e], sum);
            } else if constexpr (POST) {
                float g[8];
                scaled_gate(i, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(t[i][e] * g[e], u[i][e], sum);
            }
        }
        if (!POST && in.y < 0) continue;
        float c2 = 0.0f;
        if constexpr (POST || GATE == kGateToken) {
            c2 = cta_sum(sum, slots, slot);
            if (GATE == kGateToken && threadIdx.x == 0)
                static_cast<float*>(p.dgate)[row] = p.alpha * c2;
            c2 *= -inv_c * ry * ry * (kTokenLike ? ag : 1.0f);
        }
        // dy = ry (du w_post - (y ry) mean(q m)), the last product through c2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            if (c >= C8) continue;
            float g[8], w[8], y[8], out[8];
            scaled_gate(i, g);
            if constexpr (GATE == kGateElement) {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = p.alpha * t[i][e] * u[i][e];
                static_cast<uint4*>(p.dgate)[row * C8 + c] = pack8<BF16>(out);
            }
            if constexpr (POST) unpack8<BF16>(ch.w_post[i], w);
            pipe.template read<BF16>(in.y, i, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                out[e] = t[i][e] * g[e];   // du
                // (a column of a per-channel gate's du m, without the gate)
                const float s = GATE == kGateChannel ? p.alpha * t[i][e] : out[e];
                if constexpr (POST) {
                    col_a[i][e] = fmaf(s * ry, y[e], col_a[i][e]);
                    out[e] = fmaf(out[e] * ry, w[e], c2 * y[e]);
                } else if constexpr (GATE == kGateChannel) {
                    col_a[i][e] = fmaf(s, y[e], col_a[i][e]);
                }
            }
            p.dy[row * C8 + c] = pack8<BF16>(out);
        }
    }
    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 16 * C8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
        if (c >= C8) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            *reinterpret_cast<float4*>(part + 8 * c + e) =
                make_float4(col_a[i][e], col_a[i][e + 1], col_a[i][e + 2], col_a[i][e + 3]);
            *reinterpret_cast<float4*>(part + 8 * (C8 + c) + e) =
                make_float4(col_b[i][e], col_b[i][e + 1], col_b[i][e + 2], col_b[i][e + 3]);
        }
    }
}

// Column sums of the partials in a fixed order: 32 columns x 32 slices of the
// CTAs per block, each slice a run of CTAs read eight at a time, the slices
// added in order.
constexpr int kSlices = 32;

template <bool BF16>
__global__ void __launch_bounds__(32 * kSlices) norm_columns_kernel(const NormArgs p,
                                                                    int32_t ctas) {
    __shared__ float s[kSlices][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C = 8 * p.C8;
    const int lane = static_cast<int>(threadIdx.x) & 31, slice = static_cast<int>(threadIdx.x) >> 5;
    const int32_t col = static_cast<int32_t>(blockIdx.x) * 32 + lane;   // 0 .. 2 C
    const int32_t per = (ctas + kSlices - 1) / kSlices;
    const int32_t end = min(ctas, (slice + 1) * per);
    float v = 0.0f;
    if (col < 2 * C)
        for (int32_t i = slice * per; i < end; i += 8) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = i + k < end ? p.partial[static_cast<int64_t>(i + k) * 2 * C + col] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) v += x[k];
        }
    s[slice][lane] = v;
    __syncthreads();
    if (slice != 0 || col >= 2 * C) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) v += s[i][lane];
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

// Threads of a CTA whose threads own V vectors of each row.
int row_threads(int64_t C8, int V) {
    return static_cast<int>(((C8 + V - 1) / V + 31) / 32 * 32);
}

RowInputs row_inputs(const NormArgs& p, bool backward) {
    RowInputs in{};
    auto add = [&](const void* q) {
        if (!q) return -1;
        in.base[in.n] = static_cast<const uint4*>(q);
        return in.n++;
    };
    in.h = add(!backward || p.w_pre ? p.h : nullptr);   // dh' alone needs no h
    in.y = add(p.y);
    in.gate = add(p.gate_mode == kGateElement ? p.gate : nullptr);
    in.dh = add(backward ? p.dh : nullptr);
    in.dx = add(backward ? p.dx : nullptr);
    return in;
}

template <class K>
cudaError_t launch_rows(K kernel, ContextMarks& done, const NormArgs& p, RowInputs in,
                        int64_t ctas, int threads, int V, bool pdl, cudaStream_t stream) {
    constexpr int kMost = 227 * 1024 - 1024;   // dynamic shared memory, beside the static
    const int row = in.n * V * threads * 16;   // at most 160 KB (five operands, 16384 channels)
    in.stages = 2 * row <= kMost ? 2 : 1;
    const size_t smem = static_cast<size_t>(in.stages) * row;
    if (cudaError_t e = smem_opt_in(kernel, kMost, done, false)) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)),
                         dim3(static_cast<unsigned>(threads)), smem, stream, 1, pdl, p, in);
}

template <bool BF16>
cudaError_t forward_typed(const NormArgs& p, int sms, bool pdl, cudaStream_t stream) {
    const RowInputs in = row_inputs(p, false);
    // Few rows: a vector per thread, the shortest time for one row.
    static ContextMarks done1, done256, done512, done1024;
    if (p.C8 <= 1024 && (p.C8 <= 32 || p.T <= sms))
        return launch_rows(norm_forward_kernel<BF16, 1, 1024, 1>, done1, p, in,
                           p.T < 8 * sms ? p.T : 8 * sms, row_threads(p.C8, 1), 1, pdl, stream);
    // Two CTAs of 256 threads with 128 registers, or two of 512 with 64: at 8192
    // x 4096 55 us against 66 us for four of 256 with 64 registers, at 4096 x
    // 8192 43 us against 50 us for one of 512 with 128.
    const int threads = row_threads(p.C8, 2);
    const int64_t most = static_cast<int64_t>(sms) * (threads < 256 ? 512 / threads
                                                      : threads <= 512 ? 2 : 1);
    const int64_t ctas = p.T < most ? p.T : most;
    if (threads <= 256)
        return launch_rows(norm_forward_kernel<BF16, 2, 256, 2>, done256, p, in, ctas, threads, 2,
                           pdl, stream);
    if (threads <= 512)
        return launch_rows(norm_forward_kernel<BF16, 2, 512, 2>, done512, p, in, ctas, threads, 2,
                           pdl, stream);
    return launch_rows(norm_forward_kernel<BF16, 2, 1024, 1>, done1024, p, in, ctas, threads, 2,
                       pdl, stream);
}

template <bool BF16, bool POST, int GATE>
cudaError_t backward_rows(const NormArgs& p, int64_t ctas, int threads, bool pdl,
                          cudaStream_t stream) {
    const RowInputs in = row_inputs(p, true);
    static ContextMarks done512, done1024;
    if (threads <= 512)
        return launch_rows(norm_backward_kernel<BF16, POST, GATE, 512>, done512, p, in, ctas,
                           threads, 2, pdl, stream);
    return launch_rows(norm_backward_kernel<BF16, POST, GATE, 1024>, done1024, p, in, ctas,
                       threads, 2, pdl, stream);
}

template <bool BF16, bool POST>
cudaError_t backward_gated(const NormArgs& p, int64_t ctas, int threads, bool pdl,
                           cudaStream_t stream) {
    switch (p.gate_mode) {
        case kGateChannel: return backward_rows<BF16, POST, kGateChannel>(p, ctas, threads, pdl, stream);
        case kGateToken: return backward_rows<BF16, POST, kGateToken>(p, ctas, threads, pdl, stream);
        case kGateElement: return backward_rows<BF16, POST, kGateElement>(p, ctas, threads, pdl, stream);
        default: return backward_rows<BF16, POST, kGateNone>(p, ctas, threads, pdl, stream);
    }
}

template <bool BF16>
cudaError_t backward_typed(const NormArgs& p, int sms, bool pdl, cudaStream_t stream) {
    const int ctas = norm_backward_ctas(p.T, 8ll * p.C8, sms);
    const int threads = row_threads(p.C8, 2);
    cudaError_t e = cudaSuccess;
    if (ctas > 0)   // (no rows: the column sums come out as zeros)
        e = p.w_post ? backward_gated<BF16, true>(p, ctas, threads, pdl, stream)
                     : backward_gated<BF16, false>(p, ctas, threads, pdl, stream);
    const bool columns = p.dw_pre || p.dw_post || p.gate_mode == kGateChannel;
    if (e != cudaSuccess || !columns) return e;
    return launch_kernel(norm_columns_kernel<BF16>, dim3((16 * p.C8 + 31) / 32),
                         dim3(32 * kSlices), 0, stream, 1, pdl, p, static_cast<int32_t>(ctas));
}

}  // namespace

int norm_backward_ctas(int64_t T, int64_t C, int sms) {
    const int threads = row_threads(C / 8, 2);
    const int64_t most = static_cast<int64_t>(sms) * (threads < 512 ? 512 / threads : 1);
    return static_cast<int>(T < most ? T : most);
}

cudaError_t launch_norm_forward(const NormArgs& p, bool bf16, int sms, bool pdl,
                                cudaStream_t stream) {
    return bf16 ? forward_typed<true>(p, sms, pdl, stream)
                : forward_typed<false>(p, sms, pdl, stream);
}

cudaError_t launch_norm_backward(const NormArgs& p, bool bf16, int sms, bool pdl,
                                 cudaStream_t stream) {
    return bf16 ? backward_typed<true>(p, sms, pdl, stream)
                : backward_typed<false>(p, sms, pdl, stream);
}

}  // namespace tmagemm
