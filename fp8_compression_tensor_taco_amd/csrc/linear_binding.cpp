// Python's way into the 8-bit linear layer's C ABI (taco_linear.h): checks of
// the tensors, outputs and workspaces from torch's allocator, and the call.
// Marshalling only.  In C++ because small calls are bound by it: a call's checks
// and four outputs took 9 us in Python, besides 4 us for the launch.
//
// Every function takes the handle of the current stream last.  Tensors that are
// not contiguous, or not 16-byte aligned, are copied.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "taco_linear.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Given = std::optional<Tensor>;
constexpr int64_t kBlock = 128;

int64_t fp8_cols(int64_t cols) { return (cols + kBlock - 1) / kBlock * kBlock; }
int64_t fp8_scale_cols(int64_t cols) { return (fp8_cols(cols) / kBlock + 3) / 4 * 4; }

taco_stream_t stream_of(uint64_t handle) { return reinterpret_cast<taco_stream_t>(handle); }

void check(taco_status_t status) {      // raises TacoError
  if (status != TACO_OK)
    py::module_::import("fp8_compression_tensor_taco_amd._binding").attr("_check")(static_cast<int>(status));
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

[[noreturn]] void refuse(const char* name, const std::string& what) {
  throw py::value_error(std::string(name) + " must " + what);
}

const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : "torch.uint8";
}

// An input as the kernels take it.
Tensor input(const Tensor& t, const char* name, at::ScalarType type, int64_t dims = 2) {
  if (t.scalar_type() != type) refuse(name, std::string("be ") + type_name(type));
  if (!t.is_cuda()) throw py::value_error("libtaco works on GPU tensors only (no CPU fallback)");
  if (t.dim() != dims) refuse(name, "have " + std::to_string(dims) + " dimensions, got " + std::to_string(t.dim()));
  if (!t.is_contiguous()) return t.contiguous();
  return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 ? t : t.clone();
}

// The same, of a given shape and on the call's device.
Tensor input(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  Tensor c = input(t, name, type, static_cast<int64_t>(shape.size()));
  if (c.sizes() != shape) refuse(name, "have shape " + text(shape) + ", got " + text(c.sizes()));
  if (c.device() != device) throw py::value_error("all tensors must be on the same device");
  return c;
}

Tensor output(const Given& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  if (!t) return at::empty(shape, at::TensorOptions(type).device(device));
  if (t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous() || t->device() != device)
    refuse(name, std::string("be a contiguous ") + type_name(type) + " tensor of shape " + text(shape) + " on " +
                     device.str());
  return *t;
}

// The given workspace, or a new one per call: torch's allocator hands it out
// again in the stream's order, and a captured graph keeps its own.
struct Workspace {
  Tensor held;
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(const Given& given, size_t need, at::Device device) {
    if (given) {
      if (!given->is_contiguous() || given->device() != device)
        refuse("workspace", "be contiguous and on " + device.str());
      held = *given;
    } else if (need > 0) {
      held = at::empty({static_cast<int64_t>(need)}, at::TensorOptions(at::kByte).device(device));
    } else {
      return;
    }
    at = held.data_ptr();
    bytes = held.nbytes();
  }
};

uint8_t* bytes_of(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }
float* floats_of(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }
py::object maybe(const Tensor& t) { return t.defined() ? py::cast(t) : py::none(); }
uint8_t* maybe_bytes(const Tensor& t) { return t.defined() ? bytes_of(t) : nullptr; }

std::tuple<Tensor, Tensor> quantize_rows(const Tensor& x_, const Given& q_, const Given& scale_, uint64_t stream) {
  const Tensor x = input(x_, "x", at::kBFloat16);
  const int64_t rows = x.size(0), cols = x.size(1);
  const Tensor q = output(q_, "q", at::kByte, {rows, fp8_cols(cols)}, x.device());
  const Tensor scale = output(scale_, "scale", at::kByte, {rows, fp8_scale_cols(cols)}, x.device());
  check(taco_quantize_rows(x.data_ptr(), rows, cols, bytes_of(q), bytes_of(scale), stream_of(stream)));
  return {q, scale};
}

py::tuple quantize_weight(const Tensor& w_, bool transposed, const Given& q_, const Given& scale_, const Given& qt_,
                          const Given& scale_t_, uint64_t stream) {
  const Tensor w = input(w_, "w", at::kBFloat16);
  const int64_t rows = w.size(0), cols = w.size(1);
  const Tensor q = output(q_, "q", at::kByte, {rows, fp8_cols(cols)}, w.device());
  const Tensor scale = output(scale_, "scale", at::kByte, {fp8_cols(rows) / kBlock, fp8_scale_cols(cols)}, w.device());
  Tensor qt, scale_t;
  if (transposed) {
    qt = output(qt_, "qt", at::kByte, {cols, fp8_cols(rows)}, w.device());
    scale_t = output(scale_t_, "scale_t", at::kByte, {fp8_cols(cols) / kBlock, fp8_scale_cols(rows)}, w.device());
  } else if (qt_ || scale_t_) {
    throw py::value_error("qt and scale_t are outputs of transposed=True");
  }
  check(taco_quantize_weight(w.data_ptr(), rows, cols, bytes_of(q), bytes_of(scale), maybe_bytes(qt),
                             maybe_bytes(scale_t), stream_of(stream)));
  return py::make_tuple(q, scale, maybe(qt), maybe(scale_t));
}

std::tuple<Tensor, Tensor, Tensor, Tensor> rmsnorm_quantize(const Tensor& x_, const Tensor& weight_, double eps,
                                                            const Given& residual_, const Given& z_, const Given& rstd_,
                                                            const Given& q_, const Given& scale_, uint64_t stream) {
  const Tensor x = input(x_, "x", at::kBFloat16);
  const int64_t tokens = x.size(0), hidden = x.size(1);
  const at::Device device = x.device();
  const Tensor weight = input(weight_, "weight", at::kBFloat16, {hidden}, device);
  Tensor residual, z;
  if (residual_) {
    residual = input(*residual_, "residual", at::kBFloat16, {tokens, hidden}, device);
    z = output(z_, "z", at::kBFloat16, {tokens, hidden}, device);
  } else if (z_) {
    throw py::value_error("z is an output of the call with a residual");
  }
  const Tensor rstd = output(rstd_, "rstd", at::kFloat, {tokens}, device);
  const Tensor q = output(q_, "q", at::kByte, {tokens, fp8_cols(hidden)}, device);
  const Tensor scale = output(scale_, "scale", at::kByte, {tokens, fp8_scale_cols(hidden)}, device);
  check(taco_rmsnorm_quantize(x.data_ptr(), residual.defined() ? residual.data_ptr() : nullptr, weight.data_ptr(),
                              tokens, hidden, static_cast<float>(eps), z.defined() ? z.data_ptr() : nullptr,
                              floats_of(rstd), bytes_of(q), bytes_of(scale), stream_of(stream)));
  return {z.defined() ? z : x_, rstd, q, scale};      // x itself, also where the kernel took a copy
}

std::tuple<Tensor, Tensor> rmsnorm_backward(const Tensor& dy_, const Tensor& z_, const Tensor& rstd_,
                                            const Tensor& weight_, const Given& dz_, const Given& dx_,
                                            const Given& dweight_, const Given& workspace_, uint64_t stream) {
  const Tensor dy = input(dy_, "dy", at::kBFloat16);
  const int64_t tokens = dy.size(0), hidden = dy.size(1);
  const at::Device device = dy.device();
  const Tensor z = input(z_, "z", at::kBFloat16, {tokens, hidden}, device);
  const Tensor rstd = input(rstd_, "rstd", at::kFloat, {tokens}, device);
  const Tensor weight = input(weight_, "weight", at::kBFloat16, {hidden}, device);
  Tensor dz;
  if (dz_) dz = input(*dz_, "dz", at::kBFloat16, {tokens, hidden}, device);
  const Tensor dx = output(dx_, "dx", at::kBFloat16, {tokens, hidden}, device);
  const Tensor dweight = output(dweight_, "dweight", at::kFloat, {hidden}, device);
  const Workspace ws(workspace_, taco_rmsnorm_backward_workspace_bytes(tokens, hidden), device);
  check(taco_rmsnorm_backward(dy.data_ptr(), z.data_ptr(), floats_of(rstd), weight.data_ptr(),
                              dz.defined() ? dz.data_ptr() : nullptr, tokens, hidden, dx.data_ptr(),
                              floats_of(dweight), ws.at, ws.bytes, stream_of(stream)));
  return {dx, dweight};
}

Tensor matmul_fp8(const Tensor& qa_, const Tensor& sa_, const Tensor& qb_, const Tensor& sb_, const Given& out_,
                  const Given& workspace_, uint64_t stream) {
  const Tensor qa = input(qa_, "qa", at::kByte), qb = input(qb_, "qb", at::kByte);
  const int64_t m = qa.size(0), n = qb.size(0), k = qa.size(1);
  const at::Device device = qa.device();
  if (k == 0 || k % kBlock != 0 || qb.size(1) != k)
    throw py::value_error("qa and qb must have the same number of columns, a multiple of 128: got " +
                          std::to_string(k) + " and " + std::to_string(qb.size(1)));
  const Tensor sa = input(sa_, "sa", at::kByte, {m, fp8_scale_cols(k)}, device);
  const Tensor sb = input(sb_, "sb", at::kByte, {fp8_cols(n) / kBlock, fp8_scale_cols(k)}, device);
  if (qb.device() != device) throw py::value_error("all tensors must be on the same device");
  const Tensor out = output(out_, "out", at::kBFloat16, {m, n}, device);
  const Workspace ws(workspace_, taco_matmul_fp8_workspace_bytes(m, n, k), device);
  check(taco_matmul_fp8(bytes_of(qa), bytes_of(sa), bytes_of(qb), bytes_of(sb), m, n, k, out.data_ptr(), ws.at,
                        ws.bytes, stream_of(stream)));
  return out;
}

Tensor wgrad_fp8(const Tensor& dy_, const Tensor& q_, const Tensor& scale_, int64_t cols, const Given& dw_,
                 bool accumulate, const Given& workspace_, uint64_t stream) {
  const Tensor dy = input(dy_, "dy", at::kBFloat16);
  const int64_t tokens = dy.size(0), n = dy.size(1);
  const at::Device device = dy.device();
  if (cols < 1) throw py::value_error("cols must be at least 1");
  const Tensor q = input(q_, "q", at::kByte, {tokens, fp8_cols(cols)}, device);
  const Tensor scale = input(scale_, "scale", at::kByte, {tokens, fp8_scale_cols(cols)}, device);
  if (accumulate && !dw_) throw py::value_error("accumulate=True adds to dw: pass it");
  const Tensor dw = output(dw_, "dw", at::kFloat, {n, cols}, device);
  const Workspace ws(workspace_, taco_wgrad_fp8_workspace_bytes(tokens, n, cols), device);
  check(taco_wgrad_fp8(dy.data_ptr(), bytes_of(q), bytes_of(scale), tokens, n, cols, floats_of(dw), accumulate ? 1 : 0,
                       ws.at, ws.bytes, stream_of(stream)));
  return dw;
}

py::tuple swiglu_quantize(const Tensor& gu_, bool checkpoint, const Given& hq_, const Given& hs_, const Given& cq_,
                          const Given& cs_, uint64_t stream) {
  const Tensor gu = input(gu_, "gu", at::kBFloat16);
  const int64_t tokens = gu.size(0), both = gu.size(1);
  const at::Device device = gu.device();
  if (both == 0 || both % 2 != 0) throw py::value_error("gu must have an even number of columns: gate, then up");
  const int64_t inner = both / 2, wide = fp8_cols(inner);
  const Tensor hq = output(hq_, "hq", at::kByte, {tokens, wide}, device);
  const Tensor hs = output(hs_, "hs", at::kByte, {tokens, fp8_scale_cols(inner)}, device);
  Tensor cq, cs;
  if (checkpoint) {
    cq = output(cq_, "cq", at::kByte, {tokens, 2 * wide}, device);
    cs = output(cs_, "cs", at::kByte, {tokens, fp8_scale_cols(2 * wide)}, device);
  } else if (cq_ || cs_) {
    throw py::value_error("cq and cs are outputs of checkpoint=True");
  }
  check(taco_swiglu_quantize(gu.data_ptr(), tokens, inner, bytes_of(hq), bytes_of(hs), maybe_bytes(cq),
                             maybe_bytes(cs), stream_of(stream)));
  return py::make_tuple(hq, hs, maybe(cq), maybe(cs));
}

py::tuple swiglu_backward(const Tensor& dh_, const Tensor& cq_, const Tensor& cs_, bool quantize, const Given& dgu_,
                          const Given& dq_, const Given& ds_, uint64_t stream) {
  const Tensor dh = input(dh_, "dh", at::kBFloat16);
  const int64_t tokens = dh.size(0), inner = dh.size(1), wide = fp8_cols(inner);
  const at::Device device = dh.device();
  const Tensor cq = input(cq_, "cq", at::kByte, {tokens, 2 * wide}, device);
  const Tensor cs = input(cs_, "cs", at::kByte, {tokens, fp8_scale_cols(2 * wide)}, device);
  const Tensor dgu = output(dgu_, "dgu", at::kBFloat16, {tokens, 2 * inner}, device);
  Tensor dq, ds;
  if (quantize) {
    dq = output(dq_, "dq", at::kByte, {tokens, fp8_cols(2 * inner)}, device);
    ds = output(ds_, "ds", at::kByte, {tokens, fp8_scale_cols(2 * inner)}, device);
  } else if (dq_ || ds_) {
    throw py::value_error("dq and ds are outputs of quantize=True");
  }
  check(taco_swiglu_backward(dh.data_ptr(), bytes_of(cq), bytes_of(cs), tokens, inner, dgu.data_ptr(),
                             maybe_bytes(dq), maybe_bytes(ds), stream_of(stream)));
  return py::make_tuple(dgu, maybe(dq), maybe(ds));
}

}  // namespace

PYBIND11_MODULE(_linear_binding, m) {
  m.def("quantize_rows", &quantize_rows);
  m.def("quantize_weight", &quantize_weight);
  m.def("rmsnorm_quantize", &rmsnorm_quantize);
  m.def("rmsnorm_backward", &rmsnorm_backward);
  m.def("matmul_fp8", &matmul_fp8);
  m.def("wgrad_fp8", &wgrad_fp8);
  m.def("swiglu_quantize", &swiglu_quantize);
  m.def("swiglu_backward", &swiglu_backward);
}
