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
// t + i * blockDim.x of every row, so column sums stay in its registers, and it
// copies its own vectors of the next rows into shared memory (cp.async) while
// the CTA works on this one: no thread reads another's copy, so only the row
// sums need a barrier.  The per-channel weights and gate lie in shared memory
// too (in registers they made the compiler spill, and a spilled value's load
// waits behind the row copies in flight: the backward at 4096 x 8192 took 95
// us, and takes 67).  Beyond 8192 channels the backward spills all the same (64 to
// 304 bytes a thread: 1024 threads have 64 registers each, 32 of them column sums),
// and shared memory holds one row, so that copies do not run ahead: 4096 x 12288
// 172 us and 4096 x 16384 228 us (3.5 TB/s).  Vectors past the last channel are zeros, so that a
// thread's vectors are worked on together, without branches between them.
// Arithmetic is on packed pairs, half the instructions of scalar FP32.
//
// Measured on GB300 (device time, operands colder than L2), h and y 16-bit:
// forward 8192 x 4096 with a (T, C) gate 53 us (6.3 TB/s), 4096 x 8192 into
// codes 41 us (5.7 TB/s); backward 8192 x 4096 with both weights 68 us without a
// gate (5.9 TB/s) and 100 us with a (T, C) gate (5.3 TB/s, where a kernel that
// only copies the same five operands to three takes 91); 4096 x 16384 forward with
// both weights 85 us (6.3 TB/s), into codes 99; one row of 4096 channels 2.7 us.
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

// N sums over the CTA, the same in every thread: each warp by shuffles, then
// every warp adds the warps' sums in the same order.  `slot` alternates, so
// one barrier separates the uses of a slot.
template <int N>
using SumSlots = float[2][N][kMaxWarps];

template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], SumSlots<N>& slots, uint32_t& slot) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if (warps == 1) return;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    auto& s = slots[slot];
    slot ^= 1u;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < warps ? s[k][lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
}
__device__ __forceinline__ float cta_sum(float v, SumSlots<1>& slots, uint32_t& slot) {
    float s[1] = {v};
    cta_sums<1>(s, slots, slot);
    return s[0];
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
// The same through L1, for what the CTAs of an SM share.
__device__ __forceinline__ void cp_async_16_shared(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All copies of this thread but those of its latest N groups have arrived.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kMaxRowInputs = 5, kMaxChannelInputs = 3;

// Where the operands lie in shared memory.  An operand takes V * threads
// 16-byte slots, vector i of thread t in slot i * threads + t; a stage holds
// the T x C operands of one row, and the per-channel ones come after the
// stages.  Offsets are in bytes from a stage (h to dx) or from the start
// (w_post to gate_c), -1 where absent.
struct RowInputs {
    const uint4* row[kMaxRowInputs];
    const uint4* channel[kMaxChannelInputs];
    int rows, channels;
    int h, y, gate, dh, dx;
    int w_post, w_pre, gate_c;
    int step, stage_bytes;   // from a thread's vector to its next, from a stage to the next
    int stages;              // 1 to 3
};

// This thread's vectors of the rows of its CTA, copied to shared memory up to
// two rows ahead (with one stage, the next row's are fetched when this one is
// done).  Vectors past the last channel are zeros.
template <int V>
struct RowPipe {
    const RowInputs& in;
    const uint8_t* mine;   // this thread's first slot
    uint32_t base;         // its shared-memory address
    int32_t C8;
    uint32_t at, to;  // offsets of the stages read now and filled next

    __device__ __forceinline__ RowPipe(const RowInputs& inputs, uint4* ring, int32_t c8)
        : in(inputs), mine(reinterpret_cast<const uint8_t*>(ring + threadIdx.x)),
          base(smem_u32(ring + threadIdx.x)), C8(c8), at(0), to(0) {}
    __device__ __forceinline__ bool exists(int i) const {
        return static_cast<int32_t>(threadIdx.x + i * blockDim.x) < C8;
    }
    __device__ __forceinline__ void next(uint32_t& stage) const {
        stage += in.stage_bytes;
        if (stage == static_cast<uint32_t>(in.stages * in.stage_bytes)) stage = 0;
    }
    __device__ __forceinline__ void issue(int64_t row, int64_t T) {
        if (row < T) {
            const int64_t first = row * C8 + threadIdx.x;
            uint32_t dst = base + to;
            for (int a = 0; a < in.rows; ++a)
#pragma unroll
                for (int i = 0; i < V; ++i, dst += in.step)
                    if (exists(i)) cp_async_16(dst, in.row[a] + first + i * blockDim.x);
        }
        cp_async_commit();
        next(to);
    }
    __device__ __forceinline__ void start(int64_t row, int64_t T) {
        const int32_t all = in.stages * in.rows + in.channels;
        for (int i = 0; i < V; ++i)
            if (!exists(i))
                for (int a = 0; a < all; ++a)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                                 ::"r"(base + (a * V + i) * in.step), "r"(0u)
                                 : "memory");
        uint32_t dst = base + in.stages * in.stage_bytes;
        for (int a = 0; a < in.channels; ++a)
#pragma unroll
            for (int i = 0; i < V; ++i, dst += in.step)
                if (exists(i))
                    cp_async_16_shared(dst, in.channel[a] + threadIdx.x + i * blockDim.x);
        issue(row, T);
        if (in.stages == 3) issue(row + gridDim.x, T);
    }
    // Before a row: starts on a later one's copies, waits for this one's.
    __device__ __forceinline__ void begin(int64_t row, int64_t T) {
        if (in.stages == 3) {
            issue(row + 2 * gridDim.x, T);
            cp_async_wait<2>();
        } else if (in.stages == 2) {
            issue(row + gridDim.x, T);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
    }
    // After a row (its vectors have been read).
    __device__ __forceinline__ void end(int64_t row, int64_t T) {
        next(at);
        if (in.stages == 1) issue(row + gridDim.x, T);
    }
    template <bool BF16>
    __device__ __forceinline__ void load(uint32_t from, f32x2 (&v)[4]) const {
        unpack8<BF16>(*reinterpret_cast<const uint4*>(mine + from), v);
    }
    // Vector i of a row's operand, and of a per-channel one.
    template <bool BF16>
    __device__ __forceinline__ void read(int operand, int i, f32x2 (&v)[4]) const {
        load<BF16>(at + operand + i * in.step, v);
    }
    template <bool BF16>
    __device__ __forceinline__ void channels(int operand, int i, f32x2 (&v)[4]) const {
        load<BF16>(operand + i * in.step, v);
    }
};

// The gate of vector i of the current row; `token` is a per-token gate (or 1).
template <bool BF16, int V>
__device__ __forceinline__ void gate8(const NormArgs& p, const RowPipe<V>& pipe, float token,
                                      int i, f32x2 (&g)[4]) {
    if (p.gate_mode == kGateChannel) {
        pipe.template channels<BF16>(pipe.in.gate_c, i, g);
    } else if (p.gate_mode == kGateElement) {
        pipe.template read<BF16>(pipe.in.gate, i, g);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = pack_f32x2(token, token);
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
    __shared__ SumSlots<1> slots;
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C8 = p.C8;
    const float channels = 8.0f * static_cast<float>(C8);
    const f32x2 alpha = pack_f32x2(p.alpha, p.alpha);
    uint32_t slot = 0;
    RowPipe<V> pipe(in, ring, C8);
    pipe.start(blockIdx.x, p.T);
    float token_next = token_gate<BF16>(p, blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.T; pipe.end(row, p.T), row += gridDim.x) {
        pipe.begin(row, p.T);
        const float token = token_next;
        token_next = token_gate<BF16>(p, row + gridDim.x);
        f32x2 h[V][4];
        float r = 1.0f;
        if (p.w_post) {
            f32x2 ss = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f32x2 y[4];
                pipe.template read<BF16>(in.y, i, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = fma2(y[e], y[e], ss);
            }
            r = __frsqrt_rn(cta_sum(sum2(ss), slots, slot) / channels + p.eps);
            if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = r;
        }
        f32x2 ss = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            pipe.template read<BF16>(in.h, i, h[i]);
            if (p.y) {
                f32x2 y[4], g[4];
                pipe.template read<BF16>(in.y, i, y);
                gate8<BF16>(p, pipe, token, i, g);
                if (p.w_post) {
                    f32x2 w[4];
                    pipe.template channels<BF16>(in.w_post, i, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(y[e], pack_f32x2(r, r)), w[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) h[i][e] = fma2(alpha, mul2(g[e], y[e]), h[i][e]);
                if (c < C8) p.h_out[row * C8 + c] = pack8<BF16>(h[i]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fma2(h[i][e], h[i][e], ss);
        }
        if (!p.w_pre) continue;
        r = __frsqrt_rn(cta_sum(sum2(ss), slots, slot) / channels + p.eps);
        if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[row] = r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            f32x2 x[4], w[4];
            pipe.template channels<BF16>(in.w_pre, i, w);   // zeros past the last channel
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(h[i][e], pack_f32x2(r, r)), w[e]);
            if (p.x) {
                if (c < C8) p.x[row * C8 + c] = pack8<BF16>(x);
                continue;
            }
            float v[8];
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                unpack_f32x2(x[e], v[2 * e], v[2 * e + 1]);
                m = max(m, max(magnitude_bits(v[2 * e]), magnitude_bits(v[2 * e + 1])));
            }
            // (A lane past the last channel takes no part.)
            const BlockScale b = block_scale(__uint_as_float(half_warp_max(c < C8 ? m : 0u)));
            if (c < C8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], b.inverse);
                p.q[row * C8 + c] = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]),
                                               e4m3x4(v[4], v[5], v[6], v[7]));
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
// The second sum waits for t, and t for the first; but with t0 = dh' + rh p,
//   sum(t g u) = sum(t0 g u) - rh mean(p n) sum(n g u),
// so three sums of what is known at once replace them, with one barrier per row
// (8192 x 4096, both weights: 85 against 90 us with two).
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
    // Whether sum(t g u) is wanted.
    constexpr bool kSecond = POST || GATE == kGateToken;
    constexpr int kSums = kSecond ? 3 : 1;
    __shared__ SumSlots<kSums> slots;
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C8 = p.C8;
    const float inv_c = 1.0f / (8.0f * static_cast<float>(C8));
    uint32_t slot = 0;
    RowPipe<V> pipe(in, ring, C8);
    pipe.start(blockIdx.x, p.T);
    // The factors and gates of the CTA's next 32 rows, one row per lane.
    const int lane = static_cast<int>(threadIdx.x) & 31;
    float ry_lane = 1.0f, rh_lane = 1.0f, token_lane = 1.0f;
    int at = 0;
    f32x2 col_a[V][4] = {}, col_b[V][4] = {};
    for (int64_t row = blockIdx.x; row < p.T; pipe.end(row, p.T), row += gridDim.x) {
        pipe.begin(row, p.T);
        if (at == 0) {
            const int64_t r = row + static_cast<int64_t>(lane) * gridDim.x;
            if (r < p.T) {
                if constexpr (GATE == kGateToken) token_lane = token_gate<BF16>(p, r);
                if constexpr (POST) ry_lane = p.rstd_post[r];
                if (p.w_pre) rh_lane = p.rstd_pre[r];
            }
        }
        // alpha, times the row's gate where that is one number
        const float ry = POST ? __shfl_sync(0xffffffffu, ry_lane, at) : 1.0f;
        const float rh = __shfl_sync(0xffffffffu, rh_lane, at);
        const float ag = GATE == kGateToken
                             ? p.alpha * __shfl_sync(0xffffffffu, token_lane, at) : p.alpha;
        at = (at + 1) & 31;
        const f32x2 ry2 = pack_f32x2(ry, ry), rh2 = pack_f32x2(rh, rh), ag2 = pack_f32x2(ag, ag);
        auto vector_gate = [&](int i, f32x2 (&g)[4]) {   // of vector i
            if constexpr (GATE == kGateChannel)
                pipe.template channels<BF16>(in.gate_c, i, g);
            if constexpr (GATE == kGateElement) pipe.template read<BF16>(in.gate, i, g);
        };
        // gu: u, times the gate where that differs within the row
        f32x2 gu[V][4] = {}, t[V][4] = {}, n[V][4];
        f32x2 pn = 0, tu = 0, nu = 0;   // sums of p n, t gu (without n's part) and n gu
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f32x2 w[4];
            if (POST || in.y >= 0) pipe.template read<BF16>(in.y, i, gu[i]);
            if constexpr (POST) {
                pipe.template channels<BF16>(in.w_post, i, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) gu[i][e] = mul2(mul2(gu[i][e], ry2), w[e]);
            }
            if constexpr (!kTokenLike) {
                f32x2 g[4];
                vector_gate(i, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) gu[i][e] = mul2(gu[i][e], g[e]);
            }
            if (in.dh >= 0) pipe.template read<BF16>(in.dh, i, t[i]);
            if (p.w_pre) {
                f32x2 dx[4];
                pipe.template read<BF16>(in.h, i, n[i]);
                pipe.template read<BF16>(in.dx, i, dx);
                pipe.template channels<BF16>(in.w_pre, i, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    n[i][e] = mul2(fma2(ag2, gu[i][e], n[i][e]), rh2);
                    col_b[i][e] = fma2(dx[e], n[i][e], col_b[i][e]);
                    dx[e] = mul2(dx[e], w[e]);
                    pn = fma2(dx[e], n[i][e], pn);
                    t[i][e] = fma2(rh2, dx[e], t[i][e]);
                    if constexpr (kSecond) nu = fma2(n[i][e], gu[i][e], nu);
                }
            }
            if constexpr (kSecond) {
#pragma unroll
                for (int e = 0; e < 4; ++e) tu = fma2(t[i][e], gu[i][e], tu);
            }
        }
        float sums[kSums];
        sums[0] = sum2(pn);
        if constexpr (kSecond) {
            sums[1] = sum2(tu);
            sums[2] = sum2(nu);
        }
        if (kSecond || p.w_pre) cta_sums<kSums>(sums, slots, slot);
        const float c1 = -rh * (sums[0] * inv_c);   // (0 without w_pre)
        const f32x2 c1_2 = pack_f32x2(c1, c1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            if (p.w_pre) {
#pragma unroll
                for (int e = 0; e < 4; ++e) t[i][e] = fma2(c1_2, n[i][e], t[i][e]);
            }
            if (c < C8) p.dh_in[row * C8 + c] = pack8<BF16>(t[i]);
        }
        if (!POST && in.y < 0) continue;
        float c2 = 0.0f;
        if constexpr (kSecond) {
            c2 = fmaf(c1, sums[2], sums[1]);
            if (GATE == kGateToken && threadIdx.x == 0)
                static_cast<float*>(p.dgate)[row] = p.alpha * c2;
            c2 *= -inv_c * ag;   // - mean(q m)
        }
        const f32x2 c2_2 = pack_f32x2(c2, c2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
            f32x2 m[4], w[4], g[4], out[4];
            pipe.template read<BF16>(in.y, i, m);
            vector_gate(i, g);
            if constexpr (POST) pipe.template channels<BF16>(in.w_post, i, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (POST) m[e] = mul2(m[e], ry2);
                t[i][e] = mul2(t[i][e], ag2);
            }
            if constexpr (GATE == kGateElement) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    out[e] = mul2(t[i][e], POST ? mul2(m[e], w[e]) : m[e]);
                if (c < C8) static_cast<uint4*>(p.dgate)[row * C8 + c] = pack8<BF16>(out);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                out[e] = kTokenLike ? t[i][e] : mul2(t[i][e], g[e]);   // du
                if constexpr (GATE == kGateChannel)
                    col_a[i][e] = fma2(t[i][e], m[e], col_a[i][e]);
                else if constexpr (POST)
                    col_a[i][e] = fma2(out[e], m[e], col_a[i][e]);
                if constexpr (POST)
                    out[e] = mul2(fma2(out[e], w[e], mul2(c2_2, m[e])), ry2);
            }
            if (c < C8) p.dy[row * C8 + c] = pack8<BF16>(out);
        }
    }
    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 16 * C8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = static_cast<int32_t>(threadIdx.x + i * blockDim.x);
        if (c >= C8) continue;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {   // (16-byte aligned)
            *reinterpret_cast<ulonglong2*>(part + 8 * c + 2 * e) =
                make_ulonglong2(col_a[i][e], col_a[i][e + 1]);
            *reinterpret_cast<ulonglong2*>(part + 8 * (C8 + c) + 2 * e) =
                make_ulonglong2(col_b[i][e], col_b[i][e + 1]);
        }
    }
}

// Column sums of the partials in a fixed order: LANES columns x 1024 / LANES
// slices of the CTAs per block, each slice a run of CTAs read eight at a time, the
// slices added in order.
constexpr int kColumnThreads = 1024;

template <bool BF16, int LANES>
__global__ void __launch_bounds__(kColumnThreads) norm_columns_kernel(const NormArgs p,
                                                                      int32_t ctas) {
    constexpr int kSlices = kColumnThreads / LANES;
    __shared__ float s[kSlices][LANES];
    grid_launch_dependents();
    grid_dependency_wait();
    const int32_t C = 8 * p.C8;
    const int lane = static_cast<int>(threadIdx.x) % LANES;
    const int slice = static_cast<int>(threadIdx.x) / LANES;
    const int32_t col = static_cast<int32_t>(blockIdx.x) * LANES + lane;   // 0 .. 2 C
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
    // Groups of 32 slices in order, then the groups in order.
    __syncthreads();
    if constexpr (kSlices > 32) {
        v = 0.0f;
        if (slice % 32 == 0)
#pragma unroll
            for (int i = 0; i < 32; ++i) v += s[slice + i][lane];
        __syncthreads();
        if (slice % 32 == 0) s[slice / 32][lane] = v;
        __syncthreads();
    }
    if (slice != 0 || col >= 2 * C) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < (kSlices > 32 ? kSlices / 32 : 32); ++i) v += s[i][lane];
    if (col >= C) {
        if (p.dw_pre) p.dw_pre[col - C] = v;
        return;
    }
    const bool channel = p.gate_mode == kGateChannel && ctas > 0;   // (no rows: all sums are 0)
    if (p.dw_post)
        p.dw_post[col] =
            channel ? v * to_float<BF16>(static_cast<const uint16_t*>(p.gate)[col]) : v;
    if (p.gate_mode == kGateChannel)
        static_cast<float*>(p.dgate)[col] =
            channel && p.w_post
                ? v * to_float<BF16>(reinterpret_cast<const uint16_t*>(p.w_post)[col])
                : v;
}

// Threads of a CTA whose threads own V vectors of each row.
int row_threads(int64_t C8, int V) {
    return static_cast<int>(((C8 + V - 1) / V + 31) / 32 * 32);
}

// The operands' places for CTAs of `threads` with V vectors each, `per_sm` of
// them sharing an SM's shared memory.
RowInputs row_inputs(const NormArgs& p, bool backward, int threads, int V, int per_sm) {
    constexpr int kMost = 227 * 1024, kEach = 2048;   // (static and reserved, per CTA)
    RowInputs in{};
    in.step = threads * 16;
    const int operand = V * in.step;
    auto add = [&](const void* q) {
        if (!q) return -1;
        in.row[in.rows] = static_cast<const uint4*>(q);
        return operand * in.rows++;
    };
    in.h = add(!backward || p.w_pre ? p.h : nullptr);   // dh' alone needs no h
    in.y = add(p.y);
    in.gate = add(p.gate_mode == kGateElement ? p.gate : nullptr);
    in.dh = add(backward ? p.dh : nullptr);
    in.dx = add(backward ? p.dx : nullptr);
    in.stage_bytes = operand * in.rows;
    const void* channel[kMaxChannelInputs] = {
        p.w_post, p.w_pre, p.gate_mode == kGateChannel ? p.gate : nullptr};
    for (const void* c : channel) in.channels += c != nullptr;
    // (One stage always fits: at 16384 channels at most seven operands of 32 KB.)
    // A third stage pays in the forward (8192 x 2048 into codes 26.6 against 28.5
    // us, 8192 x 4096 without a gate 10 us of 50), not in the backward (8192 x 4096
    // without w_post 75.2 against 70.4 us).
    const int room = kMost / per_sm - kEach - operand * in.channels;
    in.stages = !backward && 3 * in.stage_bytes <= room ? 3 : 2 * in.stage_bytes <= room ? 2 : 1;
    int at = in.stages * in.stage_bytes, k = 0;
    auto place = [&](const void* q) {
        if (!q) return -1;
        in.channel[k++] = static_cast<const uint4*>(q);
        at += operand;
        return at - operand;
    };
    in.w_post = place(channel[0]);
    in.w_pre = place(channel[1]);
    in.gate_c = place(channel[2]);
    return in;
}

template <class K>
cudaError_t launch_rows(K kernel, ContextMarks& done, const NormArgs& p, bool backward,
                        int64_t ctas, int threads, int V, int per_sm, bool pdl,
                        cudaStream_t stream) {
    const RowInputs in = row_inputs(p, backward, threads, V, per_sm);
    const int smem = in.stages * in.stage_bytes + in.channels * V * in.step;
    if (cudaError_t e = smem_opt_in(kernel, 225 * 1024, done, false)) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)),
                         dim3(static_cast<unsigned>(threads)), smem, stream, 1, pdl, p, in);
}

template <bool BF16>
cudaError_t forward_typed(const NormArgs& p, int sms, bool pdl, cudaStream_t stream) {
    // Few rows: a vector per thread, the shortest time for one row.
    static ContextMarks done1, done256, done512, done1024;
    if (p.C8 <= 1024 && (p.C8 <= 32 || p.T <= sms))
        return launch_rows(norm_forward_kernel<BF16, 1, 1024, 1>, done1, p, false,
                           p.T < 8 * sms ? p.T : 8 * sms, row_threads(p.C8, 1), 1,
                           p.T <= sms ? 1 : 8, pdl, stream);
    // How many CTAs share an SM: 1024 threads of narrow CTAs, 768 of 160 to 256
    // threads, two wider ones.  8192 x 2048 into codes 25.2 us with 1024 threads, 26.1
    // with 768 and 35.0 with 512; 8192 x 4096 with a (T, C) gate 52.9 us with 768, 56.4
    // with 512, and 56.8 with 1024, whose rings hold a row less.
    const int threads = row_threads(p.C8, 2);
    const int per_sm = threads <= 128 ? 1024 / threads : threads <= 256 ? 768 / threads
                       : threads <= 512 ? 2 : 1;
    const int64_t most = static_cast<int64_t>(sms) * per_sm;
    const int64_t ctas = p.T < most ? p.T : most;
    if (threads <= 256)
        return launch_rows(norm_forward_kernel<BF16, 2, 256, 4>, done256, p, false, ctas, threads,
                           2, per_sm, pdl, stream);
    if (threads <= 512)
        return launch_rows(norm_forward_kernel<BF16, 2, 512, 2>, done512, p, false, ctas, threads,
                           2, per_sm, pdl, stream);
    return launch_rows(norm_forward_kernel<BF16, 2, 1024, 1>, done1024, p, false, ctas, threads,
                       2, per_sm, pdl, stream);
}

template <bool BF16, bool POST, int GATE>
cudaError_t backward_rows(const NormArgs& p, int64_t ctas, int threads, bool pdl,
                          cudaStream_t stream) {
    static ContextMarks done512, done1024;
    if (threads <= 512)
        return launch_rows(norm_backward_kernel<BF16, POST, GATE, 512>, done512, p, true, ctas,
                           threads, 2, 512 / threads, pdl, stream);
    return launch_rows(norm_backward_kernel<BF16, POST, GATE, 1024>, done1024, p, true, ctas,
                       threads, 2, 1, pdl, stream);
}

template <bool BF16, bool POST>
cudaError_t backward_gated(const NormArgs& p, int64_t ctas, int threads, bool pdl,
                           cudaStream_t stream) {
    switch (p.gate_mode) {
        case kGateChannel:
            return backward_rows<BF16, POST, kGateChannel>(p, ctas, threads, pdl, stream);
        case kGateToken:
            return backward_rows<BF16, POST, kGateToken>(p, ctas, threads, pdl, stream);
        case kGateElement:
            return backward_rows<BF16, POST, kGateElement>(p, ctas, threads, pdl, stream);
        default:
            return backward_rows<BF16, POST, kGateNone>(p, ctas, threads, pdl, stream);
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
    const unsigned cols = 16u * static_cast<unsigned>(p.C8);
    const int32_t n = static_cast<int32_t>(ctas);
    // Narrow blocks where wide ones would leave SMs idle: 8192 x 1024 24.7 against 29.0
    // us for the whole backward, 8192 x 4096 103.7 against 100.0.
    if (cols < 32u * static_cast<unsigned>(sms))
        return launch_kernel(norm_columns_kernel<BF16, 8>, dim3(cols / 8), dim3(kColumnThreads),
                             0, stream, 1, pdl, p, n);
    return launch_kernel(norm_columns_kernel<BF16, 32>, dim3((cols + 31) / 32),
                         dim3(kColumnThreads), 0, stream, 1, pdl, p, n);
}

}  // namespace

int norm_backward_ctas(int64_t T, int64_t C, int sms) {
    const int threads = row_threads(C / 8, 2);
    int64_t most = static_cast<int64_t>(sms) * (threads < 512 ? 512 / threads : 1);
    // Two rows each at least once all SMs have a CTA, for fewer partial sums to add:
    // 3424 x 264 9.9 against 10.7 us (four: 11.6).
    const int64_t few = (T + 1) / 2 > sms ? (T + 1) / 2 : sms;
    if (few < most) most = few;
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
