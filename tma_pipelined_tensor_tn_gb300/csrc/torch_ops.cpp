// Binding of the 8-bit operators and the norms for torch tensors: checks the
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
}
