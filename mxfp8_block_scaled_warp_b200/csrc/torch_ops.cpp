// torch_ops.cpp -- the Python module _fpq_torch: the calls of one to ten
// microseconds (norm, gate, combination, matrix-vector products) with their
// argument checks, output allocation and current stream in C++.  Through
// ctypes and Python these cost 10 to 17 us per call, several times the
// kernel's time for a decoded token; here 4 to 6 us, most of it the launch.
// Each function checks its tensors, allocates the outputs and calls the C
// ABI of include/fpq.h on the current stream of the tensors' device.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>

#include "../../include/fpq.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
namespace py = pybind11;

void need(bool ok, const char* what) {
    if (!ok) throw py::value_error(what);
}

// FpqError(status, where, detail) of the package.
void check(fpq_status st, const char* where) {
    if (st == FPQ_OK) return;
    py::object type = py::module_::import("mxfp8_block_scaled_warp_b200").attr("FpqError");
    PyErr_SetObject(type.ptr(), type(st, where, fpq_last_error_detail()).ptr());
    throw py::error_already_set();
}

// The tensors must be contiguous and share one CUDA device, which becomes
// current (the library launches on the current device).
struct Call {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;
    Call(const Tensor& first, std::initializer_list<const Tensor*> rest) {
        need(first.is_cuda(), "tensors passed to the library must live on a CUDA device");
        for (const Tensor* t : rest) {
            if (!t) continue;
            need(t->is_cuda(), "tensors passed to the library must live on a CUDA device");
            need(t->get_device() == first.get_device(), "tensors must live on the same device");
            need(t->is_contiguous(), "tensors passed to the library must be contiguous");
        }
        if (first.get_device() != c10::cuda::current_device()) guard.set_index(first.get_device());
        stream = c10::cuda::getCurrentCUDAStream(first.get_device()).stream();
    }
};

const Tensor* ptr(const OptTensor& t) { return t ? &*t : nullptr; }
void* addr(const OptTensor& t) { return t ? t->data_ptr() : nullptr; }
template <typename T> T* as(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T> T* as(const OptTensor& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// For what the kernels write in full: without the dispatcher, half the time
// of at::empty.
Tensor empty(const Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

int32_t out_type(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kFloat, "expected bfloat16 or float32");
    return t == at::kFloat ? FPQ_OUT_F32 : FPQ_OUT_BF16;
}

bool is(const Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
    return t.scalar_type() == type && t.sizes() == shape;
}

// Row stride of a bf16 matrix whose rows are contiguous.
int64_t row_stride(const Tensor& x) {
    need(x.scalar_type() == at::kBFloat16 && x.dim() == 2, "need x bf16 [rows, cols]");
    need(x.stride(1) == 1 || x.size(1) == 1, "the rows of x must be contiguous");
    return x.size(0) > 1 ? x.stride(0) : x.size(1);
}

py::tuple rmsnorm_quantize(const Tensor& x, const Tensor& weight, std::optional<int> fmt, double eps,
                           const OptTensor& residual, bool want_y, bool want_rstd) {
    const int64_t ld = row_stride(x), rows = x.size(0), cols = x.size(1);
    need(is(weight, at::kBFloat16, {cols}), "need weight bf16 [cols]");
    need(!residual || is(*residual, at::kBFloat16, x.sizes()), "need residual bf16 of x's shape");
    need(!fmt || *fmt == FPQ_FP8_1x128 || *fmt == FPQ_MXFP8, "need fmt None, FP8_1x128 or MXFP8");
    const int64_t block = fmt && *fmt == FPQ_MXFP8 ? 32 : 128;
    need(!fmt || cols % block == 0, "cols is not a multiple of the format's block width");
    Call call(x, {&weight, ptr(residual)});
    OptTensor y, q, scales, h, rstd;
    if (fmt) {
        q = empty(x, {rows, cols}, at::kByte);
        scales = empty(x, {rows, cols / block}, block == 32 ? at::kByte : at::kFloat);
    }
    if (want_y || !fmt) y = empty(x, {rows, cols}, at::kBFloat16);
    if (residual) h = empty(x, {rows, cols}, at::kBFloat16);
    if (want_rstd) rstd = empty(x, {rows}, at::kFloat);
    check(fpq_rmsnorm_quantize(fmt.value_or(0), x.data_ptr(), ld, addr(residual), weight.data_ptr(), rows, cols,
                               (float)eps, addr(h), addr(y), addr(q), addr(scales), as<float>(rstd), call.stream),
          "fpq_rmsnorm_quantize");
    return py::make_tuple(y, q, scales, h, rstd);
}

py::tuple rmsnorm_backward(const Tensor& dy, const Tensor& x, const Tensor& weight, const Tensor& rstd,
                           const OptTensor& dres) {
    const int64_t ld = row_stride(x), rows = x.size(0), cols = x.size(1);
    need(is(dy, at::kBFloat16, x.sizes()), "need dy bf16 of x's shape");
    need(is(weight, at::kBFloat16, {cols}), "need weight bf16 [cols]");
    need(is(rstd, at::kFloat, {rows}), "need rstd fp32 [rows]");
    need(!dres || is(*dres, at::kBFloat16, x.sizes()), "need dres bf16 of x's shape");
    Call call(x, {&dy, &weight, &rstd, ptr(dres)});
    Tensor dx = empty(x, {rows, cols}, at::kBFloat16), dw = empty(x, {cols}, at::kFloat);
    const int64_t bytes = (int64_t)fpq_rmsnorm_backward_workspace_bytes(rows, cols);
    Tensor ws = empty(x, {bytes}, at::kByte);
    check(fpq_rmsnorm_backward(dy.data_ptr(), x.data_ptr(), ld, weight.data_ptr(), as<float>(rstd), addr(dres), rows,
                               cols, dx.data_ptr(), as<float>(dw), ws.data_ptr(), (size_t)bytes, call.stream),
          "fpq_rmsnorm_backward");
    return py::make_tuple(dx, dw);
}

Tensor gemv_nvfp4(const Tensor& x, const Tensor& wq, const Tensor& ws, const Tensor& wg, const OptTensor& ids,
                  at::ScalarType out_dtype) {
    const int32_t type = out_type(out_dtype);
    need(x.scalar_type() == at::kBFloat16 && wq.scalar_type() == at::kByte && ws.scalar_type() == at::kByte &&
             wg.scalar_type() == at::kFloat, "need x bf16, wq and ws uint8, wg fp32");
    const int64_t d = ids ? 3 : 2;
    need(wq.dim() == d && ws.dim() == d && x.dim() >= 2,
         "need wq [n, k/2] and ws [n, k/16], or [E, n, k/2] and [E, n, k/16] with ids");
    const int64_t n = wq.size(-2), k = wq.size(-1) * 2;
    need(k % 32 == 0 && x.size(-1) == k && ws.size(-1) == k / 16 && ws.size(-2) == n &&
             (d == 2 || ws.size(0) == wq.size(0)),
         "the shapes of x, wq and ws do not belong together (k a multiple of 32)");
    need(x.is_contiguous(), "tensors passed to the library must be contiguous");
    Call call(x, {&wq, &ws, &wg, ptr(ids)});
    if (!ids) {
        need(x.dim() == 2 && wg.numel() == 1, "need x [m, k] and wg of one element");
        Tensor y = empty(x, {x.size(0), n}, out_dtype);
        check(fpq_gemv_nvfp4(x.data_ptr(), x.size(0), wq.data_ptr(), ws.data_ptr(), as<float>(wg), n, k,
                             y.data_ptr(), type, call.stream), "fpq_gemv_nvfp4");
        return y;
    }
    need(ids->scalar_type() == at::kInt && ids->dim() == 2, "need ids int32 [tokens, topk]");
    const int64_t experts = wq.size(0), tokens = ids->size(0), topk = ids->size(1);
    need(wg.dim() == 1 && wg.size(0) == experts, "need wg [E]");
    need(x.size(0) == tokens && (x.dim() == 2 || (x.dim() == 3 && x.size(1) == topk)),
         "need x [tokens, k] or [tokens, topk, k]");
    Tensor y = empty(x, {tokens, topk, n}, out_dtype);
    check(fpq_moe_gemv_nvfp4(x.data_ptr(), x.dim() == 3, as<int32_t>(*ids), tokens, (int32_t)topk, (int32_t)experts,
                             wq.data_ptr(), ws.data_ptr(), as<float>(wg), n, k, y.data_ptr(), type, call.stream),
          "fpq_moe_gemv_nvfp4");
    return y;
}

py::tuple moe_gate(const Tensor& logits, int topk, const OptTensor& bias, int score, int n_group, int topk_group,
                   int group_top, bool renormalize, double scale) {
    need(logits.dim() == 2, "need logits [tokens, E]");
    const int32_t type = out_type(logits.scalar_type());
    const int64_t tokens = logits.size(0), experts = logits.size(1);
    need(!bias || is(*bias, at::kFloat, {experts}), "need bias fp32 [E]");
    need(topk >= 1 && topk <= experts && experts <= INT32_MAX, "need topk in [1, E]");
    need(logits.is_contiguous(), "tensors passed to the library must be contiguous");
    Call call(logits, {ptr(bias)});
    Tensor ids = empty(logits, {tokens, topk}, at::kInt), weights = empty(logits, {tokens, topk}, at::kFloat);
    check(fpq_moe_gate(logits.data_ptr(), type, as<float>(bias), tokens, (int32_t)experts, score, n_group, topk_group,
                       group_top, topk, renormalize, (float)scale, as<int32_t>(ids), as<float>(weights), call.stream),
          "fpq_moe_gate");
    return py::make_tuple(ids, weights);
}

Tensor moe_gate_backward(const Tensor& dweights, const Tensor& logits, const Tensor& ids, int score,
                         bool renormalize, double scale) {
    need(logits.dim() == 2, "need logits [tokens, E]");
    const int32_t type = out_type(logits.scalar_type());
    const int64_t tokens = logits.size(0), experts = logits.size(1);
    need(ids.scalar_type() == at::kInt && ids.dim() == 2 && ids.size(0) == tokens, "need ids int32 [tokens, topk]");
    need(is(dweights, at::kFloat, ids.sizes()), "need dweights fp32 of ids' shape");
    need(experts <= INT32_MAX && ids.size(1) <= INT32_MAX, "too many experts");
    need(logits.is_contiguous(), "tensors passed to the library must be contiguous");
    Call call(logits, {&ids, &dweights});
    Tensor d = empty(logits, {tokens, experts}, logits.scalar_type());
    check(fpq_moe_gate_backward(logits.data_ptr(), type, as<int32_t>(ids), as<float>(dweights), tokens,
                                (int32_t)experts, score, (int32_t)ids.size(1), renormalize, (float)scale,
                                d.data_ptr(), call.stream), "fpq_moe_gate_backward");
    return d;
}

// Checks that the combination and its backward pass share; rows of y.
int64_t pair_rows(const Tensor& y, const Tensor& weights, const OptTensor& rows) {
    need(weights.scalar_type() == at::kFloat && weights.dim() == 2, "need weights fp32 [tokens, topk]");
    need(y.dim() == 2 || (y.dim() == 3 && !rows && y.size(0) == weights.size(0) && y.size(1) == weights.size(1)),
         "need y [rows, hidden], or [tokens, topk, hidden] without a row map");
    need(!rows || is(*rows, at::kInt, weights.sizes()), "need rows int32 of weights' shape");
    need(y.is_contiguous(), "tensors passed to the library must be contiguous");
    need(weights.size(1) <= INT32_MAX, "too many choices");
    return y.dim() == 2 ? y.size(0) : y.size(0) * y.size(1);
}

Tensor moe_combine(const Tensor& y, const Tensor& weights, const OptTensor& rows, const OptTensor& add,
                   at::ScalarType out_dtype) {
    const int64_t y_rows = pair_rows(y, weights, rows), tokens = weights.size(0), hidden = y.size(-1);
    need(!add || is(*add, at::kBFloat16, {tokens, hidden}), "need add bf16 [tokens, hidden]");
    const int32_t type = out_type(y.scalar_type()), o_type = out_type(out_dtype);
    Call call(y, {&weights, ptr(rows), ptr(add)});
    Tensor out = empty(y, {tokens, hidden}, out_dtype);
    check(fpq_moe_combine(y.data_ptr(), type, y_rows, as<int32_t>(rows), as<float>(weights), tokens,
                          (int32_t)weights.size(1), hidden, addr(add), out.data_ptr(), o_type, call.stream),
          "fpq_moe_combine");
    return out;
}

py::tuple moe_combine_backward(const Tensor& dout, const Tensor& y, const Tensor& weights, const OptTensor& rows,
                               const OptTensor& dy_buffer) {
    const int64_t y_rows = pair_rows(y, weights, rows), tokens = weights.size(0), hidden = y.size(-1);
    need(dout.dim() == 2 && dout.size(0) == tokens && dout.size(1) == hidden, "need dout [tokens, hidden]");
    need(!dy_buffer || is(*dy_buffer, y.scalar_type(), y.sizes()), "need dy of y's type and shape");
    const int32_t type = out_type(y.scalar_type()), d_type = out_type(dout.scalar_type());
    Call call(y, {&dout, &weights, ptr(rows), ptr(dy_buffer)});
    Tensor dweights = empty(y, weights.sizes(), at::kFloat);
    if (dy_buffer) {
        check(fpq_moe_combine_backward(dout.data_ptr(), d_type, y.data_ptr(), type, y_rows, as<int32_t>(rows),
                                       as<float>(weights), tokens, (int32_t)weights.size(1), hidden,
                                       dy_buffer->data_ptr(), as<float>(dweights), call.stream),
              "fpq_moe_combine_backward");
        return py::make_tuple(*dy_buffer, dweights);
    }
    Tensor dy = empty(y, y.sizes(), y.scalar_type());
    const int64_t bytes = rows ? 4 * y_rows : 0;
    Tensor ws = empty(y, {bytes}, at::kByte);
    check(fpq_moe_combine_backward_full(dout.data_ptr(), d_type, y.data_ptr(), type, y_rows, as<int32_t>(rows),
                                        as<float>(weights), tokens, (int32_t)weights.size(1), hidden, dy.data_ptr(),
                                        as<float>(dweights), ws.data_ptr(), (size_t)bytes, call.stream),
          "fpq_moe_combine_backward_full");
    return py::make_tuple(dy, dweights);
}

}  // namespace

PYBIND11_MODULE(_fpq_torch, m) {
    m.def("rmsnorm_quantize", &rmsnorm_quantize);
    m.def("rmsnorm_backward", &rmsnorm_backward);
    m.def("gemv_nvfp4", &gemv_nvfp4);
    m.def("moe_gate", &moe_gate);
    m.def("moe_gate_backward", &moe_gate_backward);
    m.def("moe_combine", &moe_combine);
    m.def("moe_combine_backward", &moe_combine_backward);
}
