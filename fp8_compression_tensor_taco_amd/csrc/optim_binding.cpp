// Python's way into the update of a training step (taco_optim.h), in the same
// module as the linear layer's.  Marshalling only; lists of tensors are walked
// without a reference taken to each, which is most of a short call's time.
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "binding.h"
#include "taco_optim.h"

namespace {

// A Python list or tuple, held while its items are looked at.
class Items {
 public:
  Items(const py::handle& of, const char* name)
      : held_(py::reinterpret_steal<py::object>(PySequence_Fast(of.ptr(), "not a sequence"))), name_(name) {
    if (!held_) {
      PyErr_Clear();
      refuse(name, "be a list or tuple");
    }
  }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(held_.ptr()); }
  PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(held_.ptr(), i); }
  const char* name() const { return name_; }
  const Tensor& tensor(Py_ssize_t i) const {
    if (!THPVariable_Check(at(i))) refuse((name_ + ("[" + std::to_string(i) + "]")).c_str(), "be a tensor");
    return THPVariable_Unpack(at(i));
  }

 private:
  py::object held_;
  const char* name_;
};

[[noreturn]] void refuse_item(const char* name, Py_ssize_t i, const std::string& what) {
  refuse((std::string(name) + "[" + std::to_string(i) + "]").c_str(), what);
}

bool real(const Tensor& t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }
int32_t type_of(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? TACO_TYPE_BF16 : TACO_TYPE_FP32; }

void check_device(const Tensor& t, at::Device device) {
  if (!t.is_cuda()) throw py::value_error("libtaco works on GPU tensors only (no CPU fallback)");
  if (t.device() != device) throw py::value_error("all tensors must be on the same device");
}

// A tensor that is written in place, or read as it lies.
void* lying(const Tensor& t, const char* name, Py_ssize_t i, at::ScalarType type, int64_t count, at::Device device) {
  check_device(t, device);
  if (t.scalar_type() != type || t.numel() != count || !t.is_contiguous())
    refuse_item(name, i, std::string("be a contiguous ") + type_name(type) + " tensor of " + std::to_string(count) + " elements");
  return t.data_ptr();
}

// A gradient: contiguous, or a contiguous copy, kept until the call was made.
const void* gradient(const Tensor& t, const char* name, Py_ssize_t i, at::Device device, std::vector<Tensor>& copies) {
  check_device(t, device);
  if (!real(t)) refuse_item(name, i, "be torch.float32 or torch.bfloat16");
  if (t.is_contiguous()) return t.data_ptr();
  copies.push_back(t.contiguous());
  return copies.back().data_ptr();
}

// A state: fp32, or a pair of codes and scale bytes.
void state(const Items& of, Py_ssize_t i, int64_t count, at::Device device, void*& data, uint8_t*& scale) {
  PyObject* item = of.at(i);
  if (THPVariable_Check(item)) {
    data = lying(THPVariable_Unpack(item), of.name(), i, at::kFloat, count, device);
    scale = nullptr;
    return;
  }
  if (!PyTuple_Check(item) || PyTuple_GET_SIZE(item) != 2 || !THPVariable_Check(PyTuple_GET_ITEM(item, 0)) ||
      !THPVariable_Check(PyTuple_GET_ITEM(item, 1)))
    refuse_item(of.name(), i, "be a tensor, or a tuple of codes and scale bytes");
  data = lying(THPVariable_Unpack(PyTuple_GET_ITEM(item, 0)), of.name(), i, at::kByte, fp8_cols(count), device);
  scale = static_cast<uint8_t*>(
      lying(THPVariable_Unpack(PyTuple_GET_ITEM(item, 1)), of.name(), i, at::kByte, fp8_scale_cols(count), device));
}

// One element on the device, or a number.
template <typename T>
const T* on_device(const py::object& value, const char* name, at::ScalarType type, at::Device device) {
  if (!THPVariable_Check(value.ptr())) return nullptr;
  const Tensor& t = THPVariable_Unpack(value.ptr());
  check_device(t, device);
  if (t.scalar_type() != type || t.numel() != 1)
    refuse(name, std::string("have one element of ") + (type == at::kLong ? "torch.int64" : "torch.float32"));
  return static_cast<const T*>(t.data_ptr());
}

template <typename T>
T number(const py::object& value, const char* name) {
  try {
    return value.cast<T>();
  } catch (const py::cast_error&) {
    refuse(name, "be a number or a tensor");
  }
}

void adamw_step(const py::object& params_, const py::object& grads_, const py::object& m_, const py::object& v_,
                const py::object& lr, const py::object& step, double beta1, double beta2, double eps,
                double weight_decay, const py::object& grad_scale, const py::object& copies_, uint64_t seed,
                uint64_t stream) {
  const Items params(params_, "params"), grads(grads_, "grads"), m(m_, "m"), v(v_, "v");
  const Py_ssize_t count = params.size();
  std::optional<Items> copies;
  if (!copies_.is_none()) copies.emplace(copies_, "copies");
  if (grads.size() != count || m.size() != count || v.size() != count || (copies && copies->size() != count))
    throw py::value_error("params, grads, m, v and copies must have the same length");
  if (count == 0) return;
  const at::Device device = params.tensor(0).device();
  std::vector<taco_adamw_tensor_t> tensors(static_cast<size_t>(count));
  std::vector<Tensor> held;
  for (Py_ssize_t i = 0; i < count; ++i) {
    taco_adamw_tensor_t& t = tensors[static_cast<size_t>(i)];
    const Tensor &p = params.tensor(i), &g = grads.tensor(i);
    if (!real(p)) refuse_item("params", i, "be torch.float32 or torch.bfloat16");
    t.count = p.numel();
    t.param = lying(p, "params", i, p.scalar_type(), t.count, device);
    if (g.sizes() != p.sizes()) refuse_item("grads", i, "have the parameter's shape, " + text(p.sizes()));
    t.grad = gradient(g, "grads", i, device, held);
    t.param_type = type_of(p);
    t.grad_type = type_of(g);
    state(m, i, t.count, device, t.m, t.m_scale);
    state(v, i, t.count, device, t.v, t.v_scale);
    if ((t.m_scale == nullptr) != (t.v_scale == nullptr)) refuse_item("v", i, "be of as many bits as m");
    if (copies && copies->at(i) != Py_None) {
      if (t.param_type == TACO_TYPE_BF16) refuse_item("copies", i, "be None for a torch.bfloat16 parameter");
      t.copy = lying(copies->tensor(i), "copies", i, at::kBFloat16, t.count, device);
    }
  }
  taco_adamw_options_t o{};
  o.lr_device = on_device<float>(lr, "lr", at::kFloat, device);
  if (!o.lr_device) o.lr = number<double>(lr, "lr");
  o.step_device = on_device<int64_t>(step, "step", at::kLong, device);
  if (!o.step_device) o.step = number<int64_t>(step, "step");
  o.beta1 = beta1;
  o.beta2 = beta2;
  o.eps = eps;
  o.weight_decay = weight_decay;
  o.seed = seed;
  if (!grad_scale.is_none()) {
    o.grad_scale = on_device<float>(grad_scale, "grad_scale", at::kFloat, device);
    if (!o.grad_scale) refuse("grad_scale", "be a tensor");
  }
  check(taco_adamw_step(tensors.data(), count, &o, stream_of(stream)));
}

Tensor gradient_norm(const py::object& grads_, double max_norm, const Given& out_, const Given& workspace_,
                     uint64_t stream) {
  const Items grads(grads_, "grads");
  const Py_ssize_t count = grads.size();
  if (count == 0) throw py::value_error("grads must have at least one tensor");
  const at::Device device = grads.tensor(0).device();
  std::vector<taco_norm_tensor_t> tensors(static_cast<size_t>(count));
  std::vector<Tensor> held;
  for (Py_ssize_t i = 0; i < count; ++i) {
    const Tensor& g = grads.tensor(i);
    tensors[static_cast<size_t>(i)] = {gradient(g, "grads", i, device, held), g.numel(), type_of(g)};
  }
  const Tensor out = output(out_, "out", at::kFloat, {2}, device);
  const Workspace ws(workspace_, taco_gradient_norm_workspace_bytes(count), device);
  check(taco_gradient_norm(tensors.data(), count, max_norm, static_cast<float*>(out.data_ptr()), ws.at, ws.bytes,
                           stream_of(stream)));
  return out;
}

}  // namespace

void define_optimizer(py::module_& m) {
  m.def("adamw_step", &adamw_step);
  m.def("gradient_norm", &gradient_norm);
}
