// Python binding of the feed-forward operators: checks of the tensors, outputs
// and workspaces from torch's allocator, and one C-ABI call on the current
// stream each.  Native because the decode step is short: the same steps in
// Python take longer than its kernels (11 us a call against 4, and 190 us
// against 20 for the 240 tensors of a gradient list).
//
// Wrong types raise TypeError, wrong shapes or devices ValueError, and a status
// of the library its Fp8Error.
#include <ATen/EmptyTensor.h>
#include <ATen/core/grad_mode.h>
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

py::object or_none(const Tensor &t) { return t.defined() ? py::cast(t) : py::object(py::none()); }

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

// ---------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------

// A contiguous int32 tensor of its own over part of another's storage, from its
// `offset`-th element on.  Of one type with it: torch does not save tensors that share
// a storage and differ in type.
Tensor piece(const Tensor &all, int64_t offset, at::IntArrayRef shape) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                      c10::scalarTypeToTypeMeta(at::kInt));
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// A tensor from the allocator of a call's first output, but not through torch's
// dispatcher, which a decode step's call, bound by the host, would feel a second time
// (16 tokens' 8 choices of 7168, quantized: 4.2 us a call for 4.5).
Tensor beside(const Tensor &first, at::IntArrayRef shape, at::ScalarType dtype) {
  return at::detail::empty_generic(shape, first.storage().allocator(), c10::DispatchKeySet(c10::DispatchKey::CUDA), dtype,
                                   std::nullopt);
}

// The library's ranges (fp8bsq_ffn.h), so that a size beyond them is refused before
// memory for its outputs is asked for.
constexpr int64_t kMaxExperts = 1024, kMaxChoices = (int64_t)1 << 31, kMaxFeatures = (int64_t)1 << 21;
constexpr int64_t kMaxProductRows = (int64_t)65535 * 16;

void require_range(bool ok) {
  if (!ok) check_status(FP8BSQ_ERANGE);
}

// n sorted rows of h; none of them, or none of a length, are within every range.
void require_rows(int64_t n, int64_t h) { require_range(n == 0 || h == 0 || (n < kMaxChoices && h <= kMaxFeatures)); }

py::tuple expert_sort(const Tensor &experts, int64_t num_experts) {
  const c10::Device device = experts.device();
  require_gpu(experts, device);
  const bool wide = experts.scalar_type() == at::kLong;
  if (!wide && experts.scalar_type() != at::kInt) type("expert numbers must be int32 or int64");
  if (experts.dim() == 0) value("expert numbers must be [..., top_k]");
  if (num_experts <= 0) value("num_experts must be positive");
  const int64_t n = experts.numel();
  require_range(num_experts <= kMaxExperts && n < kMaxChoices);
  const c10::DeviceGuard guard(device);
  // one allocation for the three, which any of them keeps in use: one token's call is
  // bound by the host (4.0 us; with three allocations 4.5, through the dispatcher 5.0)
  const Tensor all = empty({num_experts + 1 + 2 * n}, at::kInt, device);
  const Tensor offsets = piece(all, 0, {num_experts + 1}),
               rows = piece(all, num_experts + 1, experts.sizes()),
               choices = piece(all, num_experts + 1 + n, {n});
  const size_t bytes = fp8bsq_expert_sort_workspace(n, num_experts);
  Tensor ws;
  if (bytes) ws = workspace(bytes, device);
  check_status(fp8bsq_expert_sort(experts.data_ptr(), wide ? 8 : 4, n, num_experts, (int32_t *)offsets.data_ptr(),
                                  (int32_t *)rows.data_ptr(), (int32_t *)choices.data_ptr(),
                                  bytes ? ws.data_ptr() : nullptr, bytes, stream_of(device)));
  return py::make_tuple(offsets, rows, choices);
}

struct Choices {
  const int32_t *rows;
  int64_t tokens, top_k;
};

// rows [..., top_k]; a token's tensors have its leading dimensions.
Choices choices_of(const Tensor &rows) {
  if (rows.scalar_type() != at::kInt) type("rows must be int32, as expert_sort returns them");
  if (rows.dim() == 0 || rows.size(-1) == 0) value("rows must be [..., top_k]");
  return {(const int32_t *)rows.data_ptr(), rows.numel() / rows.size(-1), rows.size(-1)};
}

void require_tokens(const Tensor &x, const Tensor &rows) {
  if (x.dim() == 0 || x.sizes().slice(0, x.dim() - 1) != rows.sizes().slice(0, rows.dim() - 1))
    value("a token's tensors must have the leading dimensions of rows");
}

void require_sorted(const Tensor &y, const Choices &c) {
  if (y.dim() != 2 || y.size(0) != c.tokens * c.top_k) value("sorted rows must be [T * top_k, H]");
}

// The weights' type; fp32 where there are none.
int require_weights(const std::optional<Tensor> &weights, const Tensor &rows, c10::Device device) {
  if (!weights) return FP8BSQ_F32;
  require_gpu(*weights, device);
  if (dtype_of(*weights) < 0) type("weights must be bf16 or fp32");
  if (weights->sizes() != rows.sizes()) value("weights must have the shape of rows");
  return dtype_of(*weights);
}

const void *data_or_null(const std::optional<Tensor> &t) { return t ? t->data_ptr() : nullptr; }

// Whether autograd has to see an operation on t: a gradient is asked for, or a
// forward-mode tangent comes along (which the function refuses and a plain call
// would drop).
bool tracked(const Tensor &t) { return (at::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(0).defined(); }

// None where `ask` and autograd has to see the call.
py::object expert_dispatch(const Tensor &x, const Tensor &rows, bool ask) {
  if (ask && tracked(x)) return py::none();
  const c10::Device device = x.device();
  for (const Tensor *t : {&x, &rows}) require_gpu(*t, device);
  const int dtype = dtype_of(x);
  if (dtype < 0) type("expert_dispatch takes bf16 or fp32 rows");
  const Choices c = choices_of(rows);
  require_tokens(x, rows);
  const int64_t h = x.size(-1), n = c.tokens * c.top_k;
  require_rows(n, h);
  const c10::DeviceGuard guard(device);
  const Tensor y = empty({n, h}, x.scalar_type(), device);
  check_status(fp8bsq_expert_dispatch(x.data_ptr(), dtype, c.rows, c.tokens, c.top_k, h, y.data_ptr(), stream_of(device)));
  return py::cast(y);
}

py::tuple expert_dispatch_quant(const Tensor &x, const Tensor &rows, int scale_fmt) {
  const c10::Device device = x.device();
  for (const Tensor *t : {&x, &rows}) require_gpu(*t, device);
  const int dtype = dtype_of(x);
  if (dtype < 0) type("expert_dispatch_quant takes bf16 or fp32 rows");
  const Choices c = choices_of(rows);
  require_tokens(x, rows);
  const int64_t h = x.size(-1), n = c.tokens * c.top_k;
  if (h % 128 != 0) value("H must be a multiple of 128");
  require_rows(n, h);
  const c10::DeviceGuard guard(device);
  const Tensor y = empty({n, h}, at::kFloat8_e4m3fn, device), s = beside(y, {n, h / 128}, at::kFloat);
  check_status(fp8_expert_dispatch_quant(x.data_ptr(), dtype, scale_fmt, c.rows, c.tokens, c.top_k, h,
                                         (uint8_t *)y.data_ptr(), (float *)s.data_ptr(), stream_of(device)));
  return py::make_tuple(y, s);
}

py::object expert_combine(const Tensor &y, const Tensor &rows, const std::optional<Tensor> &weights, bool ask) {
  if (ask && (tracked(y) || (weights && tracked(*weights)))) return py::none();
  const c10::Device device = y.device();
  for (const Tensor *t : {&y, &rows}) require_gpu(*t, device);
  const int dtype = dtype_of(y);
  if (dtype < 0) type("expert_combine takes bf16 or fp32 rows");
  const Choices c = choices_of(rows);
  require_sorted(y, c);
  const int w_dtype = require_weights(weights, rows, device);
  const int64_t h = y.size(1);
  require_rows(y.size(0), h);
  const c10::DeviceGuard guard(device);
  const Tensor out = empty(with_last(rows, h), y.scalar_type(), device);
  check_status(fp8bsq_expert_combine(y.data_ptr(), dtype, c.rows, data_or_null(weights), w_dtype, c.tokens, c.top_k, h,
                                     out.data_ptr(), stream_of(device)));
  return py::cast(out);
}

py::tuple expert_combine_backward(const Tensor &dout, const Tensor &y, const Tensor &rows,
                                  const std::optional<Tensor> &weights, bool row_grad, bool weight_grad) {
  const c10::Device device = dout.device();
  for (const Tensor *t : {&dout, &y, &rows}) require_gpu(*t, device);
  const int dtype = dtype_of(dout);
  if (dtype < 0 || dtype_of(y) != dtype) type("dout and y must both be bf16 or both fp32");
  const Choices c = choices_of(rows);
  require_tokens(dout, rows);
  require_sorted(y, c);
  if (y.size(1) != dout.size(-1)) value("dout and y must have rows of one length");
  const int w_dtype = require_weights(weights, rows, device);
  const int64_t h = y.size(1);
  require_rows(y.size(0), h);
  const c10::DeviceGuard guard(device);
  Tensor dy, dw;
  if (row_grad) dy = empty(y.sizes(), y.scalar_type(), device);
  if (weight_grad) dw = empty(rows.sizes(), scalar_type(w_dtype), device);
  check_status(fp8bsq_expert_combine_backward(dout.data_ptr(), y.data_ptr(), dtype, c.rows, data_or_null(weights),
                                              w_dtype, c.tokens, c.top_k, h, row_grad ? dy.data_ptr() : nullptr,
                                              weight_grad ? dw.data_ptr() : nullptr, stream_of(device)));
  return py::make_tuple(or_none(dy), or_none(dw));
}

// [E, F, K] codes and their scales; f, k and experts from the first.
Weight expert_weight(const Tensor &w, const Tensor &s, at::IntArrayRef shape) {
  if (w.dim() != 3 || w.sizes() != shape) value("weights must be [E, F, K] with a's K, all of one shape");
  if (s.scalar_type() != at::kFloat) type("scales must be float32");
  if (s.dim() != 3 || s.size(0) != shape[0] || s.size(1) != (shape[1] + 127) / 128 || s.size(2) != shape[2] / 128)
    value("the weights' scales must be [E, ceil(F/128), K/128]");
  return {(const uint8_t *)w.data_ptr(), (const float *)s.data_ptr()};
}

// The product with one weight (w1 null), or the gated one.
Tensor expert_product(const Tensor &a, const Tensor &a_s, const Tensor &offsets, const Tensor &w0, const Tensor &w0_s,
                      const Tensor *w1, const Tensor *w1_s, int out_dtype) {
  for (const Tensor *t : {&a, &w0}) require_codes(*t);
  if (w1) require_codes(*w1);
  const c10::Device device = a.device();
  for (const Tensor *t : {&a, &a_s, &offsets, &w0, &w0_s}) require_gpu(*t, device);
  if (w1)
    for (const Tensor *t : {w1, w1_s}) require_gpu(*t, device);
  if (a.dim() != 2 || a.size(1) <= 0 || a.size(1) % 128 != 0) value("a must be [R, K], K a positive multiple of 128");
  const int64_t rows = a.size(0), k = a.size(1);
  if (a_s.scalar_type() != at::kFloat) type("scales must be float32");
  if (a_s.dim() != 2 || a_s.size(0) != rows || a_s.size(1) != k / 128) value("a_s must be [R, K/128]");
  if (w0.dim() != 3 || w0.size(0) <= 0 || w0.size(2) != k) value("weights must be [E, F, K] with a's K, all of one shape");
  const int64_t experts = w0.size(0), f = w0.size(1);
  const Weight first = expert_weight(w0, w0_s, w0.sizes());
  const Weight second = w1 ? expert_weight(*w1, *w1_s, w0.sizes()) : Weight{nullptr, nullptr};
  if (offsets.scalar_type() != at::kInt) type("offsets must be int32, as expert_sort returns them");
  if (offsets.dim() != 1 || offsets.size(0) != experts + 1) value("offsets must be [E + 1]");
  // nothing to do is within every range
  require_range(rows == 0 || f == 0 || (rows <= kMaxProductRows && experts <= kMaxExperts && f <= kMaxFeatures && k <= kMaxFeatures));
  const c10::DeviceGuard guard(device);
  const Tensor out = empty({rows, f}, scalar_type(out_dtype), device);
  const uint8_t *codes = (const uint8_t *)a.data_ptr();
  const float *scales = (const float *)a_s.data_ptr();
  const int32_t *begin = (const int32_t *)offsets.data_ptr();
  check_status(w1 ? fp8_expert_gated_ffn(codes, scales, begin, first.codes, first.scales, second.codes, second.scales,
                                         out.data_ptr(), out_dtype, rows, experts, f, k, stream_of(device))
                  : fp8_expert_gemm(codes, scales, begin, first.codes, first.scales, out.data_ptr(), out_dtype, rows,
                                    experts, f, k, stream_of(device)));
  return out;
}

Tensor expert_gemm(const Tensor &a, const Tensor &a_s, const Tensor &offsets, const Tensor &b, const Tensor &b_s,
                   int out_dtype) {
  return expert_product(a, a_s, offsets, b, b_s, nullptr, nullptr, out_dtype);
}

Tensor expert_gated_ffn(const Tensor &a, const Tensor &a_s, const Tensor &offsets, const Tensor &w_gate,
                        const Tensor &w_gate_s, const Tensor &w_up, const Tensor &w_up_s, int out_dtype) {
  return expert_product(a, a_s, offsets, w_gate, w_gate_s, &w_up, &w_up_s, out_dtype);
}

}  // namespace

PYBIND11_MODULE(_ffn_ext, m) {
  m.def("gated_ffn", &gated_ffn);
  m.def("gated_ffn_backward", &gated_ffn_backward);
  m.def("fp4_weight_quant", &fp4_quantize);
  m.def("fp4_gemv", &fp4_product);
  m.def("clip_grad_norm", &clip);
  m.def("expert_sort", &expert_sort);
  m.def("expert_dispatch", &expert_dispatch);
  m.def("expert_dispatch_quant", &expert_dispatch_quant);
  m.def("expert_combine", &expert_combine);
  m.def("expert_combine_backward", &expert_combine_backward);
  m.def("expert_gemm", &expert_gemm);
  m.def("expert_gated_ffn", &expert_gated_ffn);
}
