// torch_binding.cpp -- the tensor side of the serving and affine-MSR calls: checks of shapes, types,
// layouts and devices, and the call into libretnet.so on the tensors' device and stream.
//
// These calls are made once a decode step and layer, where the host's time is the call's time: the
// same checks and ctypes marshalling in Python took 9 us beside a 4 us kernel, here they take about 1.
// Argument errors are ValueErrors; the library's status is returned.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/numpy.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "retnet.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;
using Floats = py::array_t<float, py::array::c_style | py::array::forcecast>;
using Stream = std::optional<uintptr_t>;  // a raw stream; none: the device's current one

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

retnet_dtype_t dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return RETNET_F32;
  if (t.scalar_type() == at::kBFloat16) return RETNET_BF16;
  throw py::type_error("unsupported dtype: the library takes float32 or bfloat16");
}

template <typename T>
T* pointer(const Maybe& t) {
  return t.has_value() ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// Every tensor on one CUDA device, made current while this lives; and the call's stream there.
class Place {
 public:
  Place(const Tensor& first, std::initializer_list<const Tensor*> others, const Stream& stream) : stream_(stream) {
    bool ok = first.is_cuda();
    for (const Tensor* t : others) ok = ok && (!t || !t->defined() || (t->is_cuda() && t->device() == first.device()));
    if (!ok) refuse("tensors must be CUDA tensors of one device");
    guard_.emplace(first.device());
    device_ = first.device();
  }
  void* raw() const {
    return stream_ ? reinterpret_cast<void*>(*stream_) : static_cast<void*>(c10::cuda::getCurrentCUDAStream(device_.index()).stream());
  }
  // fn() with the call's stream current, so that memory it allocates belongs to that stream.
  template <typename F>
  auto allocate(F fn) const {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    if (stream_) guard.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*stream_), device_.index()));
    return fn();
  }
  // A new contiguous tensor, past the dispatcher (0.4 us less a tensor).
  Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) const {
    return Tensor(at::detail::empty_cuda(sizes, type, device_, std::nullopt));
  }
  Tensor bytes(size_t n) const {
    return allocate([&] { return fresh({static_cast<int64_t>(n)}, at::kByte); });
  }

 private:
  Stream stream_;
  c10::Device device_{c10::kCPU};
  std::optional<c10::cuda::CUDAGuard> guard_;
};

const Tensor* address(const Maybe& t) { return t.has_value() ? &*t : nullptr; }

// Elements between the rows of (rows, heads, width), whose heads are contiguous.
int64_t token_stride(const Tensor& t, const char* name) {
  const int64_t rows = t.size(0), heads = t.size(1), width = t.size(2);
  const int64_t row = t.stride(0), head = t.stride(1), one = t.stride(2);
  if ((width > 1 && one != 1) || (heads > 1 && head != width) || (rows > 1 && row < heads * width))
    refuse(std::string(name) + ": the heads of a row must be contiguous, and rows must not overlap");
  return rows > 1 ? row : heads * width;
}

void check_index(const Tensor& t, at::ScalarType type, int64_t n, const char* name) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + (type == at::kInt ? "int32" : "int64") + " tensor of " +
           std::to_string(n) + " entries");
}

const float* host_values(const std::optional<Floats>& a, int64_t n, const char* name) {
  if (!a.has_value()) return nullptr;
  if (a->size() < n) refuse(std::string(name) + " has " + std::to_string(a->size()) + " entries, needs " + std::to_string(n));
  return a->data();
}

retnet_packed_t packed_dims(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& pool,
                            int64_t seqs) {
  if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3 || o.dim() != 3) refuse("q, k, v and o must have three dimensions");
  const int64_t rows = q.size(0), heads = q.size(1), dk = q.size(2), kv = v.size(1), dv = v.size(2);
  if (k.size(0) != rows || k.size(1) != kv || k.size(2) != dk || v.size(0) != rows || o.size(0) != rows || o.size(1) != heads ||
      o.size(2) != dv)
    refuse("shape mismatch between q, k, v, o");
  if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || o.scalar_type() != q.scalar_type())
    refuse("q, k, v and o must have one dtype");
  if (pool.scalar_type() != at::kFloat || pool.dim() != 4 || pool.size(1) != kv || pool.size(2) != dk || pool.size(3) != dv ||
      !pool.is_contiguous())
    refuse("pool must be a contiguous float32 (slots, heads_kv, d_k, d_v)");
  return retnet_packed_t{rows, seqs, heads, kv, dk, dv, pool.size(0), token_stride(q, "q"), token_stride(k, "k"),
                         token_stride(v, "v"), token_stride(o, "o")};
}

int retention_packed(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& pool, const Tensor& cu,
                     const Tensor& slots, const Maybe& pos, const std::optional<Floats>& gamma,
                     const std::optional<Floats>& theta, uint32_t flags, const Maybe& workspace, const Stream& stream) {
  if (slots.dim() != 1) refuse("slots must have one dimension");
  const int64_t seqs = slots.size(0);
  const retnet_packed_t d = packed_dims(q, k, v, o, pool, seqs);
  check_index(cu, at::kInt, seqs + 1, "cu_seqlens");
  check_index(slots, at::kInt, seqs, "slots");
  if (pos.has_value()) check_index(*pos, at::kLong, seqs, "pos");
  if (workspace.has_value() && !workspace->is_contiguous()) refuse("workspace must be contiguous");
  const float* g = host_values(gamma, d.heads_kv, "gamma");
  const float* th = host_values(theta, d.d_k / 2, "theta");
  const Place place(q, {&k, &v, &o, &pool, &cu, &slots, address(pos), address(workspace)}, stream);
  Tensor ws;
  if (workspace.has_value()) {
    ws = *workspace;
  } else {
    uintptr_t at = 0;
    for (const Tensor* t : {&q, &k, &v, &o}) at |= reinterpret_cast<uintptr_t>(t->data_ptr());
    size_t need = 0;
    const retnet_status_t st =
        retnet_packed_call_workspace_size(d, dtype_of(q), at % 16 ? flags | RETNET_F_PRECISE : flags, g, &need);
    if (st != RETNET_OK) return st;
    ws = place.bytes(need);
  }
  return retnet_retention_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), d, dtype_of(q), g, th, flags,
                                 static_cast<const int32_t*>(cu.data_ptr()), static_cast<const int32_t*>(slots.data_ptr()),
                                 pointer<const int64_t>(pos), static_cast<float*>(pool.data_ptr()), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), place.raw());
}

int retention_step_slots(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& o, const Tensor& pool,
                         const Tensor& slots, const Maybe& pos, const std::optional<Floats>& gamma,
                         const std::optional<Floats>& theta, uint32_t flags, const Stream& stream) {
  const retnet_packed_t d = packed_dims(q, k, v, o, pool, q.dim() == 3 ? q.size(0) : 0);
  check_index(slots, at::kInt, d.seqs, "slots");
  if (pos.has_value()) check_index(*pos, at::kLong, d.seqs, "pos");
  const float* g = host_values(gamma, d.heads_kv, "gamma");
  const float* th = host_values(theta, d.d_k / 2, "theta");
  const Place place(q, {&k, &v, &o, &pool, &slots, address(pos)}, stream);
  return retnet_retention_step_slots(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), d, dtype_of(q), g, th, flags,
                                     static_cast<const int32_t*>(slots.data_ptr()), pointer<const int64_t>(pos),
                                     static_cast<float*>(pool.data_ptr()), place.raw());
}

int state_slots_copy(const Tensor& pool, const Tensor& src, const Tensor& dst, const Stream& stream) {
  if (pool.scalar_type() != at::kFloat || pool.dim() < 1 || !pool.is_contiguous()) refuse("pool must be a contiguous float32 tensor");
  if (src.dim() != 1) refuse("src must have one dimension");
  const int64_t n = src.size(0), slots = pool.size(0);
  check_index(src, at::kInt, n, "src");
  check_index(dst, at::kInt, n, "dst");
  const Place place(pool, {&src, &dst}, stream);
  return retnet_state_slots_copy(static_cast<float*>(pool.data_ptr()), slots, slots ? pool.numel() / slots : 0,
                                 static_cast<const int32_t*>(src.data_ptr()), static_cast<const int32_t*>(dst.data_ptr()), n,
                                 place.raw());
}

void check_msr(const Tensor& y, std::initializer_list<const Tensor*> same, std::initializer_list<const Maybe*> params) {
  if (y.dim() != 3 || !y.is_contiguous()) refuse("y must be a contiguous (tokens, heads, d_v)");
  for (const Tensor* t : same)
    if (t->sizes() != y.sizes() || t->scalar_type() != y.scalar_type() || !t->is_contiguous())
      refuse("y, g, out, dout, dy and dg must be contiguous and have one shape and dtype");
  for (const Maybe* t : params)
    if (t->has_value() && ((*t)->dim() != 2 || (*t)->size(0) != y.size(1) || (*t)->size(1) != y.size(2) ||
                           (*t)->scalar_type() != at::kFloat || !(*t)->is_contiguous()))
      refuse("weight, bias, dweight and dbias must be contiguous float32 (heads, d_v)");
}

int run_msr_affine(const Place& place, const Tensor& y, const Tensor& g, const Maybe& weight, const Maybe& bias, const Tensor& out,
                   float eps) {
  return retnet_msr_affine(y.data_ptr(), g.data_ptr(), pointer<const float>(weight), pointer<const float>(bias), out.data_ptr(),
                           y.size(0), y.size(1), y.size(2), eps, dtype_of(y), place.raw());
}
int msr_affine(const Tensor& y, const Tensor& g, const Maybe& weight, const Maybe& bias, const Tensor& out, float eps,
               const Stream& stream) {
  check_msr(y, {&g, &out}, {&weight, &bias});
  const Place place(y, {&g, &out, address(weight), address(bias)}, stream);
  return run_msr_affine(place, y, g, weight, bias, out, eps);
}
std::tuple<int, Tensor> msr_affine_new(const Tensor& y, const Tensor& g, const Maybe& weight, const Maybe& bias, float eps,
                                       const Stream& stream) {
  check_msr(y, {&g}, {&weight, &bias});
  const Place place(y, {&g, address(weight), address(bias)}, stream);
  const Tensor out = place.allocate([&] { return place.fresh(y.sizes(), y.scalar_type()); });
  return {run_msr_affine(place, y, g, weight, bias, out, eps), out};
}

int run_msr_affine_backward(const Place& place, const Tensor& y, const Tensor& g, const Maybe& weight, const Maybe& bias,
                            const Tensor& dout, const Tensor& dy, const Tensor& dg, float* dweight, float* dbias, float eps,
                            const Maybe& workspace) {
  Tensor ws;
  if (workspace.has_value()) {
    if (!workspace->is_contiguous()) refuse("workspace must be contiguous");
    ws = *workspace;
  } else if (dweight || dbias) {
    size_t need = 0;
    const retnet_status_t st = retnet_msr_affine_workspace_size(y.size(0), y.size(1), y.size(2), &need);
    if (st != RETNET_OK) return st;
    ws = place.bytes(need);
  }
  return retnet_msr_affine_backward(y.data_ptr(), g.data_ptr(), pointer<const float>(weight), pointer<const float>(bias),
                                    dout.data_ptr(), dy.data_ptr(), dg.data_ptr(), dweight, dbias, y.size(0), y.size(1), y.size(2),
                                    eps, dtype_of(y), ws.defined() ? ws.data_ptr() : nullptr,
                                    ws.defined() ? ws.numel() * ws.element_size() : 0, place.raw());
}
int msr_affine_backward(const Tensor& y, const Tensor& g, const Maybe& weight, const Maybe& bias, const Tensor& dout,
                        const Tensor& dy, const Tensor& dg, const Maybe& dweight, const Maybe& dbias, float eps,
                        const Maybe& workspace, const Stream& stream) {
  check_msr(y, {&g, &dout, &dy, &dg}, {&weight, &bias, &dweight, &dbias});
  const Place place(y, {&g, &dout, &dy, &dg, address(weight), address(bias), address(dweight), address(dbias), address(workspace)},
                    stream);
  return run_msr_affine_backward(place, y, g, weight, bias, dout, dy, dg, pointer<float>(dweight), pointer<float>(dbias), eps,
                                 workspace);
}
std::tuple<int, Tensor, Tensor, Tensor, Tensor> msr_affine_backward_new(const Tensor& y, const Tensor& g, const Maybe& weight,
                                                                        const Maybe& bias, const Tensor& dout, float eps,
                                                                        const Maybe& workspace, const Stream& stream) {
  check_msr(y, {&g, &dout}, {&weight, &bias});
  const Place place(y, {&g, &dout, address(weight), address(bias), address(workspace)}, stream);
  auto [dy, dg, dw, db] = place.allocate([&] {
    return std::make_tuple(place.fresh(y.sizes(), y.scalar_type()), place.fresh(y.sizes(), y.scalar_type()),
                           place.fresh({y.size(1), y.size(2)}, at::kFloat), place.fresh({y.size(1), y.size(2)}, at::kFloat));
  });
  const int st = run_msr_affine_backward(place, y, g, weight, bias, dout, dy, dg, static_cast<float*>(dw.data_ptr()),
                                         static_cast<float*>(db.data_ptr()), eps, workspace);
  return {st, dy, dg, dw, db};
}

}  // namespace

PYBIND11_MODULE(_torch_binding, m) {
  m.attr("built_for") = RETNET_BINDING_KEY;
  m.def("retention_packed", &retention_packed);
  m.def("retention_step_slots", &retention_step_slots);
  m.def("state_slots_copy", &state_slots_copy);
  m.def("msr_affine", &msr_affine);
  m.def("msr_affine_new", &msr_affine_new);
  m.def("msr_affine_backward", &msr_affine_backward);
  m.def("msr_affine_backward_new", &msr_affine_backward_new);
}
