// Binding of the 8-bit and 4-bit operators, the norms and the router's operators for
// torch tensors: checks the
// operands, allocates the results on the current stream of their device and
// calls the C ABI (include/tmagemm.h) there.  Native because these calls are
// often smaller than their own marshalling: at one token a kernel takes 1 to 3
// us and the same steps in Python 13 to 18 us.
//
// The library's functions come in as addresses (bind), so that the module works
// with either build of the library and links to neither.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <cstdint>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/tmagemm.h"

namespace {

using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

struct Library {
    decltype(&::quantize_fp8) quantize;
    decltype(&::gemm_fp8) gemm;
    decltype(&::gemm_fp8_grouped) gemm_grouped;
    decltype(&::norm_residual) norm;
    decltype(&::norm_residual_backward) norm_backward;
    decltype(&::norm_residual_backward_workspace_size) norm_workspace;
    decltype(&::route_topk) route;
    decltype(&::route_topk_backward) route_backward;
    decltype(&::dispatch_rows) dispatch;
    decltype(&::dispatch_rows_workspace_size) dispatch_workspace;
    decltype(&::combine_rows) combine;
    decltype(&::combine_rows_backward) combine_backward;
    decltype(&::gemm_w4) w4;
    decltype(&::gemm_w4_grouped) w4_grouped;
} lib;

struct StatusError {
    int status;
    const char* what;
};

void require(int status, const char* what) {
    if (status != TMAGEMM_OK) throw StatusError{status, what};
}

constexpr int64_t kBlock = 128;
int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

// A call's first operand: a CUDA tensor of `dims` dimensions.
void check_first(const char* name, const Tensor& t, int64_t dims) {
    if (!t.is_cuda()) throw py::type_error(std::string(name) + " must be a CUDA tensor");
    if (t.dim() != dims)
        throw py::value_error(std::string(name) + " must have " + std::to_string(dims) +
                              " dimensions, got " + std::to_string(t.dim()));
}

void check(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape,
           const at::Device& device, bool contiguous = true) {
    if (!t.is_cuda()) throw py::type_error(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != type)
        throw py::type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
                             c10::toString(t.scalar_type()));
    if (t.device() != device)
        throw py::value_error(std::string(name) + " is on " + t.device().str() + ", expected " +
                              device.str());
    if (t.sizes() != shape)
        throw py::value_error(std::string(name) + " must be " + text(shape) + ", got " +
                              text(t.sizes()));
    if (contiguous && !t.is_contiguous())
        throw py::value_error(std::string(name) + " must be contiguous (row-major)");
}

// 1 for bf16, 0 for fp16; other types are refused.
int bf16_flag(at::ScalarType type) {
    if (type == at::kBFloat16) return 1;
    if (type == at::kHalf) return 0;
    throw py::type_error(std::string("the type must be float16 or bfloat16, got ") +
                         c10::toString(type));
}

void* stream_of(const at::Device& device) {
    return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}

void* ptr(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }

// New tensors on the device of `like`, past the dispatcher (a call makes up to
// seven).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
Tensor same(const Tensor& like) { return empty(like.sizes(), like.scalar_type(), like); }

// Row scales, consecutive rows next to each other.
Tensor row_scales(int64_t rows, int64_t cols, const Tensor& like) {
    return Tensor(at::detail::empty_strided_cuda({rows, blocks(cols)},
                                                 {1, std::max<int64_t>(rows, 1)}, at::kFloat,
                                                 like.device()));
}

std::tuple<Tensor, Tensor> quantize(const Tensor& X, int block_rows) {
    check_first("X", X, 2);
    const int bf16 = bf16_flag(X.scalar_type());
    if (!X.is_contiguous()) throw py::value_error("X must be contiguous (row-major)");
    if (block_rows != 1 && block_rows != kBlock)
        throw py::value_error("block_rows must be 1 or 128");
    const c10::cuda::CUDAGuard guard(X.device());
    const int64_t M = X.size(0), K = X.size(1);
    Tensor Q = empty({M, K}, at::kFloat8_e4m3fn, X);
    Tensor S = block_rows == 1 ? row_scales(M, K, X)
                               : empty({blocks(M), blocks(K)}, at::kFloat, X);
    require(lib.quantize(M, K, X.data_ptr(), bf16, block_rows, Q.data_ptr(),
                         static_cast<float*>(S.data_ptr()),
                         block_rows == 1 ? 1 : std::max<int64_t>(blocks(K), 1),
                         block_rows == 1 ? std::max<int64_t>(M, 1) : 1, stream_of(X.device())),
            "quantize_fp8");
    return {Q, S};
}

// gemm_fp8 (no offsets) and gemm_fp8_grouped; bf16 < 0: the type of `out`.
Tensor product(const Tensor& A, const Tensor& SA, const Tensor& B, const Tensor& SB,
               const MaybeTensor& offsets, int bf16, const MaybeTensor& out) {
    check_first("A", A, 2);
    check_first("B", B, offsets ? 3 : 2);
    const at::Device device = A.device();
    const int64_t M = A.size(0), K = A.size(1), N = B.size(-2), kb = blocks(K), nb = blocks(N);
    check("A", A, at::kFloat8_e4m3fn, A.sizes(), device);
    check("SA", SA, at::kFloat, {M, kb}, device, false);
    if (offsets) {
        const int64_t G = B.size(0);
        check("B", B, at::kFloat8_e4m3fn, {G, N, K}, device);
        check("SB", SB, at::kFloat, {G, nb, kb}, device);
        check("m_offsets", *offsets, at::kInt, {G + 1}, device);
    } else {
        check("B", B, at::kFloat8_e4m3fn, {N, K}, device);
        check("SB", SB, at::kFloat, {nb, kb}, device);
    }
    if (bf16 < 0) bf16 = bf16_flag(out->scalar_type());
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kHalf;
    if (out) check("out", *out, type, {M, N}, device);
    const c10::cuda::CUDAGuard guard(device);
    Tensor D = out ? *out : empty({M, N}, type, A);
    // A stride that is never stepped (a dimension of one) counts as 1.
    // Broadcast (zero) strides are refused by the library.
    const int64_t row = M > 1 ? SA.stride(0) : 1, block = kb > 1 ? SA.stride(1) : 1;
    const auto* sa = static_cast<const float*>(SA.data_ptr());
    const auto* sb = static_cast<const float*>(SB.data_ptr());
    if (offsets)
        require(lib.gemm_grouped(B.size(0), static_cast<const int32_t*>(offsets->data_ptr()), M, N,
                                 K, A.data_ptr(), sa, row, block, B.data_ptr(), sb, D.data_ptr(),
                                 bf16, stream_of(device)),
                "gemm_fp8_grouped");
    else
        require(lib.gemm(M, N, K, A.data_ptr(), sa, row, block, B.data_ptr(), sb, D.data_ptr(),
                         bf16, stream_of(device)),
                "gemm_fp8");
    return D;
}

enum Gate : int32_t { kNone = 0, kChannel = 1, kToken = 2, kElement = 3 };

// The checked operands that norm_residual and its backward share.
tmagemm_norm norm_operands(const Tensor& h, const MaybeTensor& y, const MaybeTensor& gate,
                           const MaybeTensor& w_post, const MaybeTensor& w_pre, double alpha,
                           double eps) {
    check_first("h", h, 2);
    const at::ScalarType type = h.scalar_type();
    const at::Device device = h.device();
    const int64_t T = h.size(0), C = h.size(1);
    tmagemm_norm p{};
    p.T = T;
    p.C = C;
    p.bf16 = bf16_flag(type);
    p.alpha = static_cast<float>(alpha);
    p.eps = static_cast<float>(eps);
    check("h", h, type, h.sizes(), device);
    if (!y && (!w_pre || w_post || gate))
        throw py::value_error("without y there is neither w_post nor gate, and w_pre is needed");
    if (y) check("y", *y, type, {T, C}, device);
    if (w_post) check("w_post", *w_post, type, {C}, device);
    if (w_pre) check("w_pre", *w_pre, type, {C}, device);
    if (gate) {
        // (A per-channel gate has one dimension: as (1, C) it would be per element, with
        // a gradient of another type, for one token.)
        const at::IntArrayRef shape = gate->sizes();
        if (shape == at::IntArrayRef({T, C}))
            p.gate_mode = kElement;
        else if (shape == at::IntArrayRef({C}))
            p.gate_mode = kChannel;
        else if (shape == at::IntArrayRef({T, 1}))
            p.gate_mode = kToken;
        else
            throw py::value_error("gate must be (C,), (T, 1) or (T, C), got " + text(shape));
        check("gate", *gate, type, shape, device);
    }
    p.h = h.data_ptr();
    p.y = ptr(y);
    p.gate = ptr(gate);
    p.w_post = ptr(w_post);
    p.w_pre = ptr(w_pre);
    return p;
}

float* floats(MaybeTensor& t, at::IntArrayRef shape, const Tensor& like) {
    t = empty(shape, at::kFloat, like);
    return static_cast<float*>(t->data_ptr());
}

std::tuple<Tensor, MaybeTensor, MaybeTensor, MaybeTensor, MaybeTensor> norm(
    const Tensor& h, const MaybeTensor& y, const MaybeTensor& gate, const MaybeTensor& w_post,
    const MaybeTensor& w_pre, double alpha, double eps, bool quantize, bool save_rstd) {
    tmagemm_norm p = norm_operands(h, y, gate, w_post, w_pre, alpha, eps);
    if (quantize && !w_pre) throw py::value_error("quantize needs w_pre");
    const c10::cuda::CUDAGuard guard(h.device());
    Tensor h_out = h;
    MaybeTensor x, scales, rstd_post, rstd_pre;
    if (y) {
        h_out = same(h);
        p.h_out = h_out.data_ptr();
    }
    if (w_pre && quantize) {
        x = empty(h.sizes(), at::kFloat8_e4m3fn, h);
        scales = row_scales(p.T, p.C, h);
        p.q = x->data_ptr();
        p.scales = static_cast<float*>(scales->data_ptr());
        p.s_row_stride = 1;
        p.s_block_stride = std::max<int64_t>(p.T, 1);
    } else if (w_pre) {
        x = same(h);
        p.x = x->data_ptr();
    }
    if (save_rstd && w_post) p.rstd_post = floats(rstd_post, {p.T}, h);
    if (save_rstd && w_pre) p.rstd_pre = floats(rstd_pre, {p.T}, h);
    require(lib.norm(&p, stream_of(h.device())), "norm_residual");
    return {h_out, x, scales, rstd_post, rstd_pre};
}

std::tuple<Tensor, MaybeTensor, MaybeTensor, MaybeTensor, MaybeTensor> norm_backward(
    const Tensor& h, const MaybeTensor& y, const MaybeTensor& dh, const MaybeTensor& dx,
    const MaybeTensor& gate, const MaybeTensor& w_post, const MaybeTensor& w_pre, double alpha,
    const MaybeTensor& rstd_post, const MaybeTensor& rstd_pre) {
    tmagemm_norm p = norm_operands(h, y, gate, w_post, w_pre, alpha, 0.0);
    const at::Device device = h.device();
    if (dx.has_value() != w_pre.has_value())
        throw py::value_error("dx is given if and only if w_pre is");
    if ((w_post && !rstd_post) || (w_pre && !rstd_pre))
        throw py::value_error("the rsqrt factors of the norms (save_rstd) are needed");
    if (dh) check("dh", *dh, h.scalar_type(), {p.T, p.C}, device);
    if (dx) check("dx", *dx, h.scalar_type(), {p.T, p.C}, device);
    if (w_post) check("rstd_post", *rstd_post, at::kFloat, {p.T}, device);
    if (w_pre) check("rstd_pre", *rstd_pre, at::kFloat, {p.T}, device);
    p.dh_out = ptr(dh);
    p.dx = ptr(dx);
    p.rstd_post = w_post ? static_cast<float*>(rstd_post->data_ptr()) : nullptr;
    p.rstd_pre = w_pre ? static_cast<float*>(rstd_pre->data_ptr()) : nullptr;
    const c10::cuda::CUDAGuard guard(device);
    const int64_t need = lib.norm_workspace(p.T, p.C);
    if (need < 0) require(static_cast<int>(need), "norm_residual_backward_workspace_size");
    Tensor workspace = empty({need}, at::kByte, h);
    Tensor dh_in = same(h);
    MaybeTensor dy, dgate, dw_post, dw_pre;
    p.dh = dh_in.data_ptr();
    if (y) {
        dy = same(h);
        p.dy = dy->data_ptr();
    }
    if (gate && p.gate_mode == kElement) {
        dgate = same(h);
        p.dgate = dgate->data_ptr();
    } else if (gate) {
        p.dgate = floats(dgate, gate->sizes(), h);
    }
    if (w_post) p.dw_post = floats(dw_post, {p.C}, h);
    if (w_pre) p.dw_pre = floats(dw_pre, {p.C}, h);
    require(lib.norm_backward(&p, workspace.data_ptr(), need, stream_of(device)),
            "norm_residual_backward");
    return {dh_in, dy, dgate, dw_post, dw_pre};
}

// ---- routed experts ----

// The operands that route_topk and its backward share.
tmagemm_route route_operands(const Tensor& logits, int64_t k, bool sigmoid, bool renormalize,
                             double scale) {
    check_first("logits", logits, 2);
    const at::ScalarType type = logits.scalar_type();
    tmagemm_route p{};
    p.type = type == at::kFloat ? 2 : -1;
    if (p.type < 0) {
        if (type != at::kBFloat16 && type != at::kHalf)
            throw py::type_error(std::string("logits must be float32, float16 or bfloat16, got ") +
                                 c10::toString(type));
        p.type = type == at::kBFloat16;
    }
    if (!logits.is_contiguous()) throw py::value_error("logits must be contiguous (row-major)");
    p.T = logits.size(0);
    p.E = logits.size(1);
    if (k < 1 || k > p.E)
        throw py::value_error("k must be from 1 to the number of experts, got " +
                              std::to_string(k));
    p.k = static_cast<int32_t>(std::min<int64_t>(k, INT32_MAX));
    p.score = sigmoid;
    p.renormalize = renormalize;
    p.scale = static_cast<float>(scale);
    p.logits = logits.data_ptr();
    return p;
}

std::tuple<Tensor, Tensor> route(const Tensor& logits, int64_t k, bool sigmoid,
                                 const MaybeTensor& bias, int64_t groups, int64_t top_groups,
                                 int64_t group_sum, bool renormalize, double scale) {
    tmagemm_route p = route_operands(logits, k, sigmoid, renormalize, scale);
    if (groups < 1 || groups > p.E || p.E % groups != 0)
        throw py::value_error("groups must divide the number of experts");
    if (top_groups < 1 || top_groups > groups || k > p.E / groups * top_groups)
        throw py::value_error("top_groups must be from 1 to groups and hold k experts");
    if (group_sum != 1 && group_sum != 2) throw py::value_error("group_sum must be 1 or 2");
    if (bias) check("bias", *bias, at::kFloat, {p.E}, logits.device());
    const c10::cuda::CUDAGuard guard(logits.device());
    Tensor ids = empty({p.T, k}, at::kInt, logits), weights = empty({p.T, k}, at::kFloat, logits);
    p.groups = static_cast<int32_t>(groups);
    p.top_groups = static_cast<int32_t>(top_groups);
    p.group_sum = static_cast<int32_t>(group_sum);
    p.bias = static_cast<const float*>(ptr(bias));
    p.ids = static_cast<int32_t*>(ids.data_ptr());
    p.weights = static_cast<float*>(weights.data_ptr());
    require(lib.route(&p, stream_of(logits.device())), "route_topk");
    return {ids, weights};
}

Tensor route_backward(const Tensor& logits, const Tensor& ids, const Tensor& dweights,
                      bool sigmoid, bool renormalize, double scale) {
    check_first("ids", ids, 2);
    tmagemm_route p = route_operands(logits, ids.size(1), sigmoid, renormalize, scale);
    check("ids", ids, at::kInt, {p.T, p.k}, logits.device());
    check("dweights", dweights, at::kFloat, {p.T, p.k}, logits.device());
    const c10::cuda::CUDAGuard guard(logits.device());
    Tensor dlogits = same(logits);
    p.ids = static_cast<int32_t*>(ids.data_ptr());
    p.dweights = static_cast<const float*>(dweights.data_ptr());
    p.dlogits = dlogits.data_ptr();
    require(lib.route_backward(&p, stream_of(logits.device())), "route_topk_backward");
    return dlogits;
}

std::tuple<Tensor, MaybeTensor, Tensor, Tensor> dispatch(const Tensor& x, const Tensor& ids,
                                                         int64_t experts, bool quantize) {
    check_first("x", x, 2);
    check_first("ids", ids, 2);
    const at::ScalarType type = x.scalar_type();
    const at::Device device = x.device();
    const int bf16 = bf16_flag(type);
    const int64_t T = x.size(0), C = x.size(1), k = ids.size(1);
    check("x", x, type, x.sizes(), device);
    check("ids", ids, at::kInt, {T, k}, device);
    const c10::cuda::CUDAGuard guard(device);
    const int64_t need = lib.dispatch_workspace(T, k, experts);
    if (need < 0) require(static_cast<int>(need), "dispatch_rows_workspace_size");
    Tensor workspace, rows = empty({T * k, C}, quantize ? at::kFloat8_e4m3fn : type, x);
    if (need > 0) workspace = empty({need}, at::kByte, x);
    MaybeTensor scales;
    if (quantize) scales = row_scales(T * k, C, x);
    Tensor offsets = empty({experts + 1}, at::kInt, x), row_of = empty({T, k}, at::kInt, x);
    require(lib.dispatch(T, k, experts, C, static_cast<const int32_t*>(ids.data_ptr()),
                         x.data_ptr(), bf16, rows.data_ptr(), static_cast<float*>(ptr(scales)), 1,
                         std::max<int64_t>(T * k, 1), static_cast<int32_t*>(offsets.data_ptr()),
                         static_cast<int32_t*>(row_of.data_ptr()),
                         need > 0 ? workspace.data_ptr() : nullptr, need, stream_of(device)),
            "dispatch_rows");
    return {rows, scales, offsets, row_of};
}

// The checked operands of combine_rows and its backward.
struct Rows {
    int64_t T, k, C, R;
    int bf16;
};
Rows combine_operands(const Tensor& rows, const Tensor& row_of, const MaybeTensor& weights) {
    check_first("rows", rows, 2);
    check_first("row_of", row_of, 2);
    const Rows n{row_of.size(0), row_of.size(1), rows.size(1), rows.size(0),
                 bf16_flag(rows.scalar_type())};
    check("rows", rows, rows.scalar_type(), rows.sizes(), rows.device());
    check("row_of", row_of, at::kInt, row_of.sizes(), rows.device());
    if (weights) check("weights", *weights, at::kFloat, {n.T, n.k}, rows.device());
    return n;
}

Tensor combine(const Tensor& rows, const Tensor& row_of, const MaybeTensor& weights) {
    const Rows n = combine_operands(rows, row_of, weights);
    const c10::cuda::CUDAGuard guard(rows.device());
    Tensor y = empty({n.T, n.C}, rows.scalar_type(), rows);
    require(lib.combine(n.T, n.k, n.C, n.R, rows.data_ptr(),
                        static_cast<const int32_t*>(row_of.data_ptr()),
                        static_cast<const float*>(ptr(weights)), y.data_ptr(), n.bf16,
                        stream_of(rows.device())),
            "combine_rows");
    return y;
}

std::tuple<Tensor, Tensor> combine_backward(const Tensor& dy, const Tensor& rows,
                                            const Tensor& row_of, const Tensor& weights) {
    const Rows n = combine_operands(rows, row_of, weights);
    check("dy", dy, rows.scalar_type(), {n.T, n.C}, rows.device());
    const c10::cuda::CUDAGuard guard(rows.device());
    Tensor drows = same(rows), dweights = empty({n.T, n.k}, at::kFloat, rows);
    require(lib.combine_backward(n.T, n.k, n.C, n.R, dy.data_ptr(), rows.data_ptr(),
                                 static_cast<const int32_t*>(row_of.data_ptr()),
                                 static_cast<const float*>(weights.data_ptr()), drows.data_ptr(),
                                 static_cast<float*>(dweights.data_ptr()), n.bf16,
                                 stream_of(rows.device())),
            "combine_rows_backward");
    return {drows, dweights};
}

// ---- 4-bit weights ----

// gemm_w4 (no offsets) and gemm_w4_grouped.
Tensor product_w4(const Tensor& A, const Tensor& B, const Tensor& SB, const MaybeTensor& ZB,
                  const MaybeTensor& offsets, int64_t group, const MaybeTensor& out) {
    check_first("A", A, 2);
    check_first("B", B, offsets ? 3 : 2);
    const at::ScalarType type = A.scalar_type();
    const at::Device device = A.device();
    const int bf16 = bf16_flag(type);
    const int64_t M = A.size(0), K = A.size(1), N = B.size(-2), G = offsets ? B.size(0) : 1;
    if (group != 32 && group != 64 && group != 128)
        throw py::value_error("group must be 32, 64 or 128");
    if (K % 32 != 0) throw py::value_error("A must have a multiple of 32 columns");
    const int64_t kg = (K + group - 1) / group;
    check("A", A, type, A.sizes(), device);
    const int64_t codes[3] = {G, N, K / 2}, scales[3] = {G, N, kg};
    const int skip = offsets ? 0 : 1;
    check("B", B, at::kByte, at::IntArrayRef(codes + skip, 3 - skip), device);
    check("SB", SB, type, at::IntArrayRef(scales + skip, 3 - skip), device);
    if (ZB) check("ZB", *ZB, at::kByte, at::IntArrayRef(scales + skip, 3 - skip), device);
    if (offsets) check("m_offsets", *offsets, at::kInt, {G + 1}, device);
    if (out) check("out", *out, type, {M, N}, device);
    const c10::cuda::CUDAGuard guard(device);
    Tensor D = out ? *out : empty({M, N}, type, A);
    if (offsets)
        require(lib.w4_grouped(G, static_cast<const int32_t*>(offsets->data_ptr()), M, N, K, group,
                               A.data_ptr(), B.data_ptr(), SB.data_ptr(), ptr(ZB), D.data_ptr(),
                               bf16, stream_of(device)),
                "gemm_w4_grouped");
    else
        require(lib.w4(M, N, K, group, A.data_ptr(), B.data_ptr(), SB.data_ptr(), ptr(ZB),
                       D.data_ptr(), bf16, stream_of(device)),
                "gemm_w4");
    return D;
}

py::object& error_class() {
    static py::object* cls = new py::object();   // lives as long as the process
    return *cls;
}

template <class F>
void take(F& f, const py::dict& functions, const char* name) {
    f = reinterpret_cast<F>(functions[name].cast<uintptr_t>());
}

// The addresses of the library's functions, and what to raise for a status.
void bind(const py::dict& functions, py::object error) {
    take(lib.quantize, functions, "quantize_fp8");
    take(lib.gemm, functions, "gemm_fp8");
    take(lib.gemm_grouped, functions, "gemm_fp8_grouped");
    take(lib.norm, functions, "norm_residual");
    take(lib.norm_backward, functions, "norm_residual_backward");
    take(lib.norm_workspace, functions, "norm_residual_backward_workspace_size");
    take(lib.route, functions, "route_topk");
    take(lib.route_backward, functions, "route_topk_backward");
    take(lib.dispatch, functions, "dispatch_rows");
    take(lib.dispatch_workspace, functions, "dispatch_rows_workspace_size");
    take(lib.combine, functions, "combine_rows");
    take(lib.combine_backward, functions, "combine_rows_backward");
    take(lib.w4, functions, "gemm_w4");
    take(lib.w4_grouped, functions, "gemm_w4_grouped");
    error_class() = std::move(error);
}

}  // namespace

PYBIND11_MODULE(_torch_ops, m) {
    py::register_exception_translator([](std::exception_ptr e) {
        try {
            if (e) std::rethrow_exception(e);
        } catch (const StatusError& s) {
            const py::object error = error_class()(s.status, s.what);
            PyErr_SetObject(error_class().ptr(), error.ptr());
        }
    });
    m.def("bind", &bind);
    m.def("quantize_fp8", &quantize);
    m.def("product", &product);
    m.def("norm_residual", &norm);
    m.def("norm_residual_backward", &norm_backward);
    m.def("route_topk", &route);
    m.def("route_topk_backward", &route_backward);
    m.def("dispatch_rows", &dispatch);
    m.def("combine_rows", &combine);
    m.def("combine_rows_backward", &combine_backward);
    m.def("product_w4", &product_w4);
}
