// Python binding of the feed-forward operators: checks of the tensors, outputs
// and workspaces from torch's allocator, and one C-ABI call on the current
// stream each.  Native because the decode step is short: the same steps in
// Python take longer than its kernels (11 us a call against 4, and 190 us
// against 20 for the 240 tensors of a gradient list).
//
// Wrong types raise TypeError, wrong shapes or devices ValueError, and a status
// of the library its Fp8Error.
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <vector>

#include "fp8bsq_ffn.h"
#include "spans.h"

namespace py = pybind11;
using at::Tensor;

namespace {

void check_status(int status) {
  if (status != FP8BSQ_OK) py::module_::import("fp8_block_scaled_quant_amd._lib").attr("check")(status);
}

[[noreturn]] void value(const char *text) { throw py::value_error(text); }
[[noreturn]] void type(const char *text) { throw py::type_error(text); }

// FP8BSQ_F32 or FP8BSQ_BF16, or -1
int dtype_of(const Tensor &t) {
  return t.scalar_type() == at::kFloat ? FP8BSQ_F32 : t.scalar_type() == at::kBFloat16 ? FP8BSQ_BF16 : -1;
}
at::ScalarType scalar_type(int dtype) { return dtype == FP8BSQ_F32 ? at::kFloat : at::kBFloat16; }

void require_gpu(const Tensor &t, c10::Device device) {
  if (!t.is_cuda()) value("fp8_block_scaled_quant_amd runs on the GPU only: tensor is on the CPU");
  if (!t.is_contiguous()) value("tensors must be contiguous");
  if (t.device() != device) value("all tensors must be on the same device");
}

void require_codes(const Tensor &t) {
  if (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte)
    type("E4M3 operands must be torch.float8_e4m3fn (or uint8 codes)");
}

Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, c10::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
}

// In use until the work queued on the current stream has passed it, as torch's
// allocator tracks.
Tensor workspace(size_t bytes, c10::Device device) { return empty({(int64_t)bytes}, at::kByte, device); }

void *stream_of(c10::Device device) { return c10::hip::getCurrentHIPStream(device.index()).stream(); }

std::vector<int64_t> with_last(const Tensor &t, int64_t last) {
  std::vector<int64_t> shape = t.sizes().vec();
  shape.back() = last;
  return shape;
}

struct Weight {
  const uint8_t *codes;
  const float *scales;
};

Weight weight(const Tensor &w, const Tensor &s, int64_t f, int64_t k) {
  if (w.dim() != 2 || w.size(0) != f || w.size(1) != k) value("weights must be [F, K] with x's K, both of one shape");
  if (s.scalar_type() != at::kFloat) type("scales must be float32");
  if (s.dim() != 2 || s.size(0) != (f + 127) / 128 || s.size(1) != k / 128)
    value("a weight's scales must be [ceil(F/128), K/128]");
  return {(const uint8_t *)w.data_ptr(), (const float *)s.data_ptr()};
}

py::object gated_ffn(const Tensor &x, const Tensor &w_gate, const Tensor &w_gate_s, const Tensor &w_up,
                     const Tensor &w_up_s, int scale_fmt, int out_dtype, bool save) {
  require_codes(w_gate);
  require_codes(w_up);
  const c10::Device device = x.device();
  for (const Tensor *t : {&x, &w_gate, &w_gate_s, &w_up, &w_up_s}) require_gpu(*t, device);
  const int x_dtype = dtype_of(x);
  if (x_dtype < 0) type("gated_ffn takes bf16 or fp32 activations");
  const int64_t k = x.dim() ? x.size(-1) : 0;
  if (k <= 0 || k % 128 != 0) value("K must be a positive multiple of 128");
  if (w_gate.dim() != 2) value("weights must be [F, K] with x's K, both of one shape");
  const int64_t f = w_gate.size(0), m = x.numel() / k;
  const Weight wg = weight(w_gate, w_gate_s, f, k), wu = weight(w_up, w_up_s, f, k);
  const c10::DeviceGuard guard(device);
  const std::vector<int64_t> shape = with_last(x, f);
  const Tensor h = empty(shape, scalar_type(out_dtype), device);
  Tensor g, u;
  if (save) {
    g = empty(shape, scalar_type(out_dtype), device);
    u = empty(shape, scalar_type(out_dtype), device);
  }
  if (m && f) {
    const size_t bytes = fp8_gated_ffn_workspace(m, f, k);
    const Tensor ws = workspace(bytes, device);
    check_status(fp8_gated_ffn(x.data_ptr(), x_dtype, scale_fmt, wg.codes, wg.scales, wu.codes, wu.scales,
                               h.data_ptr(), save ? g.data_ptr() : nullptr, save ? u.data_ptr() : nullptr, out_dtype,
                               m, f, k, ws.data_ptr(), bytes, stream_of(device)));
  }
  if (save) return py::make_tuple(h, g, u);
  return py::cast(h);
}

py::tuple gated_ffn_backward(const Tensor &dh, const Tensor &x, const Tensor &g, const Tensor &u,
                             const Tensor &w_gate, const Tensor &w_gate_s, const Tensor &w_up, const Tensor &w_up_s,
                             int out_dtype, bool input_grad, bool weight_grad) {
  require_codes(w_gate);
  require_codes(w_up);
  const c10::Device device = dh.device();
  for (const Tensor *t : {&dh, &x, &g, &u, &w_gate, &w_gate_s, &w_up, &w_up_s}) require_gpu(*t, device);
  const int dtype = dtype_of(dh);
  if (dtype < 0 || dtype_of(x) != dtype || dtype_of(g) != dtype || dtype_of(u) != dtype)
    type("dh, x, g and u must all be bf16 or all fp32");
  const int64_t f = dh.dim() ? dh.size(-1) : 0, k = x.dim() ? x.size(-1) : 0;
  if (f <= 0 || f % 128 != 0 || k <= 0 || k % 128 != 0) value("F and K must be positive multiples of 128");
  if (g.sizes() != dh.sizes() || u.sizes() != dh.sizes() ||
      x.sizes().slice(0, x.dim() - 1) != dh.sizes().slice(0, dh.dim() - 1))
    value("g and u must have dh's shape, and x its leading dimensions");
  const Weight wg = weight(w_gate, w_gate_s, f, k), wu = weight(w_up, w_up_s, f, k);
  const int64_t m = x.numel() / k;
  const c10::DeviceGuard guard(device);
  Tensor dx, dwg, dwu;
  if (input_grad) dx = empty(x.sizes(), scalar_type(out_dtype), device);
  if (weight_grad) {
    dwg = empty({f, k}, scalar_type(out_dtype), device);
    dwu = empty({f, k}, scalar_type(out_dtype), device);
  }
  if (weight_grad || (input_grad && m)) {
    const size_t bytes = fp8_gated_ffn_backward_workspace(m, f, k);
    const Tensor ws = workspace(bytes, device);
    check_status(fp8_gated_ffn_backward(
        dh.data_ptr(), x.data_ptr(), g.data_ptr(), u.data_ptr(), dtype, wg.codes, wg.scales, wu.codes, wu.scales,
        input_grad ? dx.data_ptr() : nullptr, weight_grad ? dwg.data_ptr() : nullptr,
        weight_grad ? dwu.data_ptr() : nullptr, out_dtype, m, f, k, ws.data_ptr(), bytes, stream_of(device)));
  }
  auto or_none = [](const Tensor &t) { return t.defined() ? py::cast(t) : py::object(py::none()); };
  return py::make_tuple(or_none(dx), or_none(dwg), or_none(dwu));
}

py::tuple fp4_quantize(const Tensor &w) {
  require_gpu(w, w.device());
  const int dtype = dtype_of(w);
  if (dtype < 0) type("fp4_weight_quant takes bf16 or fp32 input");
  if (w.dim() != 2) value("weight must be 2-D");
  const int64_t n = w.size(0), k = w.size(1);
  if (k % 32 != 0) value("K must be a multiple of 32");
  const c10::DeviceGuard guard(w.device());
  const Tensor q = empty({n, k / 2}, at::kByte, w.device()), s = empty({n, k / 32}, at::kByte, w.device());
  if (n && k)
    check_status(fp4_weight_quant(w.data_ptr(), dtype, n, k, (uint8_t *)q.data_ptr(), (uint8_t *)s.data_ptr(),
                                  stream_of(w.device())));
  return py::make_tuple(q, s);
}

Tensor fp4_product(const Tensor &x, const Tensor &q, const Tensor &s, int out_dtype, const std::optional<Tensor> &bias) {
  const c10::Device device = x.device();
  for (const Tensor *t : {&x, &q, &s}) require_gpu(*t, device);
  if (bias) require_gpu(*bias, device);
  const int x_dtype = dtype_of(x);
  if (x_dtype < 0) type("fp4_gemv takes bf16 or fp32 activations");
  if (q.scalar_type() != at::kByte || s.scalar_type() != at::kByte) type("4-bit codes and their scales are uint8");
  const int64_t k = x.dim() ? x.size(-1) : 0;
  if (k <= 0 || k % 32 != 0) value("K must be a positive multiple of 32");
  if (q.dim() != 2 || q.size(1) != k / 2) value("q must be [N, K/2] with x's K");
  const int64_t n = q.size(0), m = x.numel() / k;
  if (s.dim() != 2 || s.size(0) != n || s.size(1) != k / 32) value("s must be [N, K/32]");
  if (bias && (dtype_of(*bias) != out_dtype || bias->dim() != 1 || bias->size(0) != n))
    value("bias must be [N] of the output dtype");
  const c10::DeviceGuard guard(device);
  const Tensor y = empty(with_last(x, n), scalar_type(out_dtype), device);
  if (m && n)
    check_status(fp4_gemv(x.data_ptr(), x_dtype, (const uint8_t *)q.data_ptr(), (const uint8_t *)s.data_ptr(),
                          bias ? bias->data_ptr() : nullptr, y.data_ptr(), out_dtype, m, n, k, stream_of(device)));
  return y;
}

const Tensor &tensor_of(py::handle h) {
  if (!THPVariable_Check(h.ptr())) type("gradients must be tensors");
  return THPVariable_Unpack(h.ptr());
}

// outs: none (the norm only), or a list, which may be `grads` itself.
Tensor clip(const py::list &grads, const std::optional<py::list> &outs, double max_norm, double eps) {
  const size_t count = grads.size();
  if (count == 0) value("no gradients given");
  if (outs && outs->size() != count) value("out must match the gradients' number, shapes and dtypes");
  const bool in_place = outs && outs->ptr() == grads.ptr();
  const c10::Device device = tensor_of(grads[0]).device();
  std::vector<const void *> in(count);
  std::vector<void *> out(outs ? count : 0);
  std::vector<int64_t> numels(count);
  std::vector<int32_t> dtypes(count);
  std::vector<c10::TensorImpl *> changed(out.size());
  std::vector<fp8bsq::Span> spans;
  if (in_place) spans.reserve(count);
  for (size_t i = 0; i < count; ++i) {
    const Tensor &t = tensor_of(PyList_GET_ITEM(grads.ptr(), i));
    require_gpu(t, device);
    dtypes[i] = dtype_of(t);
    if (dtypes[i] < 0) type("gradients must be bf16 or fp32");
    in[i] = t.data_ptr();
    numels[i] = t.numel();
    if (!outs) continue;
    const Tensor &o = in_place ? t : tensor_of(PyList_GET_ITEM(outs->ptr(), i));
    if (!in_place) {
      require_gpu(o, device);
      if (o.sizes() != t.sizes() || o.scalar_type() != t.scalar_type())
        value("out must match the gradients' number, shapes and dtypes");
    }
    out[i] = o.data_ptr();
    if (out[i] == in[i] && numels[i])
      spans.push_back({(uintptr_t)in[i], (uintptr_t)in[i] + (uintptr_t)numels[i] * (dtypes[i] == FP8BSQ_F32 ? 4 : 2)});
    changed[i] = o.is_inference() ? nullptr : o.unsafeGetTensorImpl();
  }
  // a shared weight's gradient listed twice: two workgroups would scale it, at once
  if (fp8bsq::overlapping(std::move(spans))) value("gradients that are clipped in place must not overlap");
  const c10::DeviceGuard guard(device);
  const Tensor norm = empty({}, at::kFloat, device);
  const size_t bytes = fp8bsq_clip_grad_norm_workspace((int64_t)count);
  const Tensor ws = workspace(bytes, device);
  check_status(fp8bsq_clip_grad_norm(in.data(), outs ? out.data() : nullptr, numels.data(), dtypes.data(),
                                     (int64_t)count, (float)max_norm, (float)eps, (float *)norm.data_ptr(),
                                     ws.data_ptr(), bytes, stream_of(device)));
  // a tensor that autograd saved is seen to have changed, as after torch's own in-place operations
  for (c10::TensorImpl *t : changed)
    if (t) t->bump_version();
  return norm;
}

}  // namespace

PYBIND11_MODULE(_ffn_ext, m) {
  m.def("gated_ffn", &gated_ffn);
  m.def("gated_ffn_backward", &gated_ffn_backward);
  m.def("fp4_weight_quant", &fp4_quantize);
  m.def("fp4_gemv", &fp4_product);
  m.def("clip_grad_norm", &clip);
}
