// operators_torch.cpp - the layer-free operators on torch tensors: the compiled part
// of sparse_mixture_experts_gate_b200/operators.py.
//
// Argument checks, output tensors and the calls of the C ABI (include/moe.h), on
// the current stream of the tensors' device. For a call on a few tokens the host's
// work is what counts: the same through Python and ctypes took 12 us for the routing
// of one token, and takes 5 us here, 3 of them the launch.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>
#include <string>

#include "moe.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

constexpr int kBlock[2] = {32, 16};  // elements per scale of MXFP4, NVFP4

template <class... A>
[[noreturn]] void refuse(const A &...parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw py::value_error(s.str());
}

// A status of the C ABI as the binding's MoEError.
void check(int rc, const char *where) {
    if (rc == MOE_OK) return;
    const py::object type = py::module_::import("sparse_mixture_experts_gate_b200.binding").attr("MoEError");
    const py::object error = type(rc, where, std::string(moe_last_error()));
    PyErr_SetObject(type.ptr(), error.ptr());
    throw py::error_already_set();
}

int dtype_of(const char *name, at::ScalarType t) {
    if (t == at::kBFloat16) return MOE_DTYPE_BF16;
    if (t == at::kFloat) return MOE_DTYPE_FP32;
    refuse(name, ": bf16 or fp32, got ", t);
}

// The row stride of a matrix of contiguous rows.
int64_t rows_of(const char *name, const Tensor &t, int64_t cols = -1) {
    if (t.dim() != 2 || (cols >= 0 && t.size(1) != cols)) {
        if (cols >= 0) refuse(name, ": a matrix of ", cols, " columns is needed, got ", t.sizes());
        refuse(name, ": a matrix is needed, got ", t.sizes());
    }
    dtype_of(name, t.scalar_type());
    if (t.size(1) > 1 && t.stride(1) != 1) refuse(name, ": rows have to be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// The address of a contiguous array; shape {-1}: any.
template <class T>
T *array(const char *name, const Tensor &t, const Tensor &like, at::ScalarType type, at::IntArrayRef shape) {
    if (t.scalar_type() != type || !t.is_contiguous() || t.device() != like.device() ||
        (!(shape.size() == 1 && shape[0] < 0) && t.sizes() != shape))
        refuse(name, ": a contiguous ", type, " tensor", shape[0] < 0 ? "" : " of this call's sizes", " on ", like.device(),
               " is needed, got ", t.scalar_type(), " ", t.sizes(), " on ", t.device());
    return static_cast<T *>(t.data_ptr());
}

template <class T>
T *array(const char *name, const Maybe &t, const Tensor &like, at::ScalarType type, at::IntArrayRef shape) {
    return t ? array<T>(name, *t, like, type, shape) : nullptr;
}

int32_t count(const char *name, int64_t n) {
    if (n > INT32_MAX) refuse(name, ": more than 2^31 - 1");
    return static_cast<int32_t>(n);
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Tensor &like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// The tensors' device current, and its current stream.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;
    explicit On(const Tensor &t) {
        if (!t.is_cuda()) refuse("the operators take CUDA tensors");
        if (t.get_device() != c10::cuda::current_device()) guard.set_device(t.device());
        stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
    }
};

int64_t scale_bytes(int format, int64_t rows, int64_t cols) {
    const int64_t tile = 4 * kBlock[format];
    return (rows + 127) / 128 * ((cols + tile - 1) / tile) * 512;
}

py::tuple route(const Tensor &logits, uintptr_t config, const Maybe &bias, bool counts, const Maybe &out_w,
                const Maybe &out_idx, const Maybe &out_n) {
    moe_route_config_t c = *reinterpret_cast<const moe_route_config_t *>(config);
    const int64_t ld = rows_of("logits", logits, c.num_experts);
    c.dtype = dtype_of("logits", logits.scalar_type());
    const int64_t T = logits.size(0), E = c.num_experts, k = c.num_active;
    if (out_w.has_value() != out_idx.has_value() || (out_n && !out_w))
        refuse("out: weights and topk_idx go together, counts with them");
    const float *b = array<float>("bias", bias, logits, at::kFloat, {E});
    float *pw = array<float>("weights", out_w, logits, at::kFloat, {T, k});
    int32_t *pi = array<int32_t>("topk_idx", out_idx, logits, at::kInt, {T, k});
    int32_t *pn = array<int32_t>("counts", out_n, logits, at::kInt, {E});
    On on(logits);
    Tensor w, idx, n;
    if (out_w) {
        w = *out_w;
        idx = *out_idx;
        if (out_n) n = *out_n;
    } else {
        if (k < 1) refuse("num_active must be at least 1");
        w = empty({T, k}, at::kFloat, logits);
        idx = empty({T, k}, at::kInt, logits);
        if (counts) n = empty({E}, at::kInt, logits);
        pw = static_cast<float *>(w.data_ptr());
        pi = static_cast<int32_t *>(idx.data_ptr());
        pn = counts ? static_cast<int32_t *>(n.data_ptr()) : nullptr;
    }
    check(moe_route(&c, logits.data_ptr(), ld, count("logits", T), b, pw, pi, pn, on.stream), "moe_route");
    return py::make_tuple(w, idx, n.defined() ? py::cast(n) : py::none());
}

Tensor route_backward(const Tensor &grad, const Tensor &logits, const Tensor &idx, uintptr_t config, const Maybe &out) {
    moe_route_config_t c = *reinterpret_cast<const moe_route_config_t *>(config);
    const int64_t ld = rows_of("logits", logits, c.num_experts), T = logits.size(0), E = c.num_experts;
    c.dtype = dtype_of("logits", logits.scalar_type());
    const float *g = array<float>("grad_weights", grad, logits, at::kFloat, {T, c.num_active});
    const int32_t *i = array<int32_t>("topk_idx", idx, logits, at::kInt, {T, c.num_active});
    if (out && (out->scalar_type() != logits.scalar_type() || out->sizes() != logits.sizes() ||
                out->device() != logits.device()))
        refuse("out has to be like logits");
    On on(logits);
    const Tensor d = out ? *out : empty({T, E}, logits.scalar_type(), logits);
    check(moe_route_backward(&c, g, logits.data_ptr(), ld, i, count("logits", T), d.data_ptr(), rows_of("out", d),
                             on.stream),
          "moe_route_backward");
    return d;
}

// Codes and scales, given or made.
py::tuple quantize(const Tensor &x, int format, const Maybe &row_index, int scale_exp, const Maybe &values,
                   const Maybe &out_codes, const Maybe &out_scales) {
    const int64_t ld = rows_of("x", x), x_rows = x.size(0), cols = x.size(1);
    if (cols < 32 || cols % 32) refuse("a row needs a positive multiple of 32 elements, got ", cols);
    const int64_t rows = row_index ? row_index->numel() : x_rows;
    const int32_t *index = array<int32_t>("row_index", row_index, x, at::kInt, {-1});
    if (values && (values->scalar_type() != x.scalar_type() || values->dim() != 2 || values->size(0) != rows ||
                   values->size(1) != cols || values->device() != x.device()))
        refuse("values: a matrix like x's rows in the outputs' order is needed");
    On on(x);
    const Tensor codes = out_codes ? *out_codes : empty({rows, cols / 2}, at::kByte, x);
    const Tensor scales = out_scales ? *out_scales : empty({scale_bytes(format, rows, cols)}, at::kByte, x);
    const int type = dtype_of("x", x.scalar_type());
    const int32_t n = count("rows", rows), nx = count("rows", x_rows), nc = count("columns", cols);
    if (index && !values && rows >= 3 * x_rows && x_rows * cols >= 1 << 21) {
        // Rows that are wanted several times are quantised once and copied: 8192 x 2048 NVFP4 to six times as many
        // rows 27 us, 49 without, 32768 x 7168 MXFP4 to three times 210 and 254; to twice as many it is little or no
        // gain (170 and 172). Below this size it is not worth the launch (1024 x 2048 to 6144 rows 8 and 10 us, 256 x
        // 7168 to 2048 12 and 10). The index's length counts: it may have many rows that are none (padded segments),
        // and how many only the device knows.
        const int64_t bytes = static_cast<int64_t>(moe_mx_once_bytes(format, x_rows, cols));
        const Tensor workspace = empty({bytes}, at::kByte, x);
        check(moe_mx_quantize_once(format, x.data_ptr(), type, ld, nx, nc, index, n, scale_exp, codes.data_ptr(),
                                   scales.data_ptr(), workspace.data_ptr(), bytes, on.stream),
              "moe_mx_quantize_once");
    } else {
        check(moe_mx_quantize(format, x.data_ptr(), type, ld, nx, nc, index, n, scale_exp, codes.data_ptr(),
                              scales.data_ptr(), values ? values->data_ptr() : nullptr,
                              values ? rows_of("values", *values) : 0, on.stream),
              "moe_mx_quantize");
    }
    return py::make_tuple(codes, scales, rows, cols);
}

py::tuple gather(const Tensor &codes, const Tensor &scales, int format, int64_t src_rows, int64_t cols,
                 const Tensor &row_index, const Maybe &out_codes, const Maybe &out_scales) {
    const int64_t rows = row_index.numel();
    const int32_t *index = array<int32_t>("row_index", row_index, codes, at::kInt, {-1});
    On on(codes);
    const Tensor c = out_codes ? *out_codes : empty({rows, cols / 2}, at::kByte, codes);
    const Tensor s = out_scales ? *out_scales : empty({scale_bytes(format, rows, cols)}, at::kByte, codes);
    check(moe_mx_gather(format, codes.data_ptr(), scales.data_ptr(), count("rows", src_rows), count("columns", cols), index,
                        count("rows", rows), c.data_ptr(), s.data_ptr(), on.stream),
          "moe_mx_gather");
    return py::make_tuple(c, s);
}

void dequantize(const Tensor &codes, const Tensor &scales, int format, int64_t rows, int64_t cols, int scale_exp,
                const Tensor &out) {
    On on(codes);
    check(moe_mx_dequantize(format, codes.data_ptr(), scales.data_ptr(), count("rows", rows), count("columns", cols),
                            scale_exp, out.data_ptr(), dtype_of("out", out.scalar_type()), cols, on.stream),
          "moe_mx_dequantize");
}

Tensor gemm(const Tensor &a_codes, const Tensor &a_scales, const Tensor &w_codes, const Tensor &w_scales, int format,
            int64_t rows, int64_t n, int64_t k, int64_t groups, int scale_exp, const Maybe &group_start,
            const Maybe &group_rows, const Maybe &bias, const Maybe &alpha, int activation, const Maybe &out, bool fp32,
            const Maybe &status) {
    if (w_codes.device() != a_codes.device()) refuse("operands on different devices");
    moe_mx_gemm_t p;
    p.group_start = array<int32_t>("group_start", group_start, a_codes, at::kInt, {-1});
    p.group_rows = array<int32_t>("group_rows", group_rows, a_codes, at::kInt, {-1});
    if ((group_start && group_start->numel() < groups) || (group_rows && group_rows->numel() < groups))
        refuse("group_start and group_rows: one entry for each of ", groups, " groups is needed");
    p.bias = array<float>("bias", bias, a_codes, at::kFloat, {groups, n});
    p.alpha = array<float>("alpha", alpha, a_codes, at::kFloat, {groups});
    p.status = reinterpret_cast<uint32_t *>(array<int32_t>("status", status, a_codes, at::kInt, {1}));
    if (out && (out->device() != a_codes.device() || out->dim() != 2 || out->size(0) != rows))
        refuse("out: ", rows, " rows on ", a_codes.device(), " are needed");
    On on(a_codes);
    const Tensor y = out ? *out : empty({rows, n}, fp32 ? at::kFloat : at::kBFloat16, a_codes);
    p.out_ld = rows_of("out", y, n);
    p.format = format;
    p.rows = count("rows", rows);
    p.n = count("n", n);
    p.k = count("k", k);
    p.groups = count("groups", groups);
    p.scale_exp = scale_exp;
    p.activation = activation;
    p.out_dtype = dtype_of("out", y.scalar_type());
    p.a_codes = a_codes.data_ptr();
    p.a_scales = a_scales.data_ptr();
    p.w_codes = w_codes.data_ptr();
    p.w_scales = w_scales.data_ptr();
    p.out = y.data_ptr();
    check(moe_mx_gemm(&p, on.stream), "moe_mx_gemm");
    return y;
}

}  // namespace

PYBIND11_MODULE(_operators, m) {
    m.def("route", &route);
    m.def("route_backward", &route_backward);
    m.def("quantize", &quantize);
    m.def("gather", &gather);
    m.def("dequantize", &dequantize);
    m.def("gemm", &gemm);
}
