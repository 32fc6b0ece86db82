// The feed-forward operators' calls on torch tensors: checks of the arguments,
// the outputs, and one call of the C ABI on torch's current stream of the
// tensors' device.  Marshalling only, in C++ because a small call's kernel takes
// 2 to 4 us and the same steps in Python 8 to 13.  The entry points come as
// addresses from the library that the Python side has loaded.
#include <ATen/Functions.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include "../../include/effort.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

decltype(&effort_block_norm) f_block_norm = nullptr;
decltype(&effort_fp8_matmul) f_fp8_matmul = nullptr;
decltype(&effort_moe_forward) f_moe_forward = nullptr;
decltype(&effort_moe_scratch_bytes) f_moe_scratch = nullptr;

void init(uintptr_t norm, uintptr_t matmul, uintptr_t moe, uintptr_t scratch) {
  f_block_norm = reinterpret_cast<decltype(f_block_norm)>(norm);
  f_fp8_matmul = reinterpret_cast<decltype(f_fp8_matmul)>(matmul);
  f_moe_forward = reinterpret_cast<decltype(f_moe_forward)>(moe);
  f_moe_scratch = reinterpret_cast<decltype(f_moe_scratch)>(scratch);
}

int dtype_of(at::ScalarType t) {
  return t == at::kFloat ? EFFORT_F32 : t == at::kHalf ? EFFORT_F16 : t == at::kBFloat16 ? EFFORT_BF16 : -1;
}
effort_dtype_t need_dtype(at::ScalarType t, const char* name) {
  const int d = dtype_of(t);
  TORCH_CHECK_TYPE(d >= 0, name, " must be float32, float16 or bfloat16, got ", t);
  return (effort_dtype_t)d;
}

// Tensors whose values do not lie in memory as they are: subclasses with a dispatch
// of their own (fake tensors among them), vmap's and other transforms' wrappers,
// lazily negated views.
const c10::DispatchKeySet kWrapped({c10::DispatchKey::Python, c10::DispatchKey::FuncTorchBatched, c10::DispatchKey::FuncTorchGradWrapper,
                                    c10::DispatchKey::Functionalize, c10::DispatchKey::Negative, c10::DispatchKey::Conjugate});
void need_plain(const Tensor& t, const char* name) {
  TORCH_CHECK_TYPE(!t.key_set().has_any(kWrapped), name, " must be a plain tensor, whose values lie in memory as they are");
  TORCH_CHECK(!(t.requires_grad() && c10::GradMode::is_enabled()), name,
              " asks for a gradient, but this operator has no backward pass: detach it, or call under torch.no_grad()");
}

// t is [rows, dim] on this device (any if negative), its rows' elements adjacent
void need_rows(const Tensor& t, const char* name, int64_t rows, int64_t dim, int device) {
  need_plain(t, name);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
  TORCH_CHECK_VALUE(device < 0 || t.get_device() == device, name, " is on cuda:", (int)t.get_device(), ", expected cuda:", device);
  TORCH_CHECK_VALUE(t.dim() == 2 && (dim < 0 || t.size(1) == dim) && (rows < 0 || t.size(0) == rows), name, " must be [",
                    rows < 0 ? "rows" : std::to_string(rows), ", ", dim < 0 ? "dim" : std::to_string(dim), "], got ", t.sizes());
  TORCH_CHECK_VALUE(t.size(1) <= 1 || t.stride(1) == 1, "the elements of a row of ", name, " must be adjacent");
}
void need_type(const Tensor& t, const char* name, at::ScalarType type) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ", expected ", type);
}
// the row stride; one row's is never used and may be anything
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

const void* need_vector(const Opt& w, const char* name, int64_t dim, int device, std::optional<at::ScalarType>& type) {
  if (!w) return nullptr;
  need_plain(*w, name);
  if (!type) {
    type = w->scalar_type();
    need_dtype(*type, name);
  }
  TORCH_CHECK_VALUE(w->is_cuda() && w->get_device() == device && w->is_contiguous() && w->scalar_type() == *type &&
                        w->dim() == 1 && w->size(0) == dim,
                    name, " must be a contiguous vector of ", dim, " ", *type, " on cuda:", device);
  return w->data_ptr();
}

Tensor make(int64_t rows, int64_t dim, at::ScalarType type, const Tensor& like) {
  return at::empty({rows, dim}, like.options().dtype(type));
}

// kinds: 0 none, 1 rms, 2 layer.  Returns (status, x', h, q, scales).
py::tuple block_norm(Tensor x, Opt y, int post, const Opt& post_weight, const Opt& post_bias, Opt gate, double residual_scale,
                     double branch_scale, int pre, const Opt& pre_weight, const Opt& pre_bias, double eps, double offset,
                     std::optional<at::ScalarType> out_dtype, bool quantize, Opt x_out, Opt h_out) {
  const bool flat = x.dim() == 1;
  if (flat) {
    x = x.unsqueeze(0);
    if (y) y = y->unsqueeze(0);
    if (gate) gate = gate->reshape({1, -1});
    if (x_out) x_out = x_out->unsqueeze(0);
    if (h_out) h_out = h_out->unsqueeze(0);
  }
  need_rows(x, "x", -1, -1, -1);
  const int64_t rows = x.size(0), dim = x.size(1);
  const int dev = x.get_device();
  const auto type = x.scalar_type();
  effort_block_norm_t a = {};
  a.rows = rows;
  a.dim = dim;
  a.dtype = need_dtype(type, "x");
  a.post_kind = (effort_norm_kind_t)post;
  a.pre_kind = (effort_norm_kind_t)pre;
  a.eps = (float)eps;
  a.weight_offset = (float)offset;
  a.residual_scale = (float)residual_scale;
  a.branch_scale = (float)branch_scale;
  a.x = x.data_ptr();
  a.x_stride = row_stride(x);
  if (y) {
    need_rows(*y, "y", rows, dim, dev);
    need_type(*y, "y", type);
    a.y = y->data_ptr();
    a.y_stride = row_stride(*y);
  } else {
    TORCH_CHECK_VALUE(post == 0 && !gate && !post_weight && !post_bias, "post and gate work on y");
  }
  if (gate) {
    need_rows(*gate, "gate", gate->dim() == 2 && gate->size(0) == 1 ? 1 : rows, dim, dev);
    need_type(*gate, "gate", type);
    a.gate = gate->data_ptr();
    a.gate_stride = gate->size(0) == 1 ? 0 : gate->stride(0);
  }
  TORCH_CHECK_VALUE((post != 0 || (!post_weight && !post_bias)) && (pre != 0 || (!pre_weight && !pre_bias)),
                    "a weight or bias without its norm");
  std::optional<at::ScalarType> wt;
  a.post_weight = need_vector(post_weight, "post_weight", dim, dev, wt);
  a.post_bias = need_vector(post_bias, "post_bias", dim, dev, wt);
  a.pre_weight = need_vector(pre_weight, "pre_weight", dim, dev, wt);
  a.pre_bias = need_vector(pre_bias, "pre_bias", dim, dev, wt);
  a.weight_dtype = wt ? (effort_dtype_t)dtype_of(*wt) : a.dtype;
  Tensor xo = x;  // where nothing is added or scaled, x itself
  if (x_out) {
    need_rows(*x_out, "x_out", rows, dim, dev);
    need_type(*x_out, "x_out", type);
    xo = *x_out;
  } else if (y || residual_scale != 1.0) {
    xo = make(rows, dim, type, x);
  }
  if (x_out || xo.data_ptr() != x.data_ptr()) {
    a.x_out = xo.data_ptr();
    a.x_out_stride = row_stride(xo);
  }
  Tensor h, q, s;
  if (quantize) {
    TORCH_CHECK_VALUE(!h_out && !out_dtype, "quantize gives q and scales, no h");
    const int64_t pitch = (dim + 15) / 16 * 16, blocks = (dim + EFFORT_BLOCK - 1) / EFFORT_BLOCK;
    q = make(rows, pitch, at::kFloat8_e4m3fn, x);
    if (pitch != dim) q = q.narrow(1, 0, dim);
    s = make(rows, blocks, at::kFloat, x);
    a.q_out = q.data_ptr();
    a.q_stride = pitch;
    a.q_scales = s.data_ptr<float>();
    a.q_scales_stride = blocks;
  } else {
    const auto ht = out_dtype ? *out_dtype : h_out ? h_out->scalar_type() : type;
    a.h_dtype = need_dtype(ht, "out_dtype");
    if (h_out) {
      need_rows(*h_out, "h_out", rows, dim, dev);
      need_type(*h_out, "h_out", ht);
      h = *h_out;
    } else {
      h = make(rows, dim, ht, x);
    }
    a.h_out = h.data_ptr();
    a.h_stride = row_stride(h);
  }
  int st = 0;
  if (rows) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    st = f_block_norm(&a, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
  }
  if (flat) {
    xo = xo.squeeze(0);
    if (quantize) q = q.squeeze(0), s = s.squeeze(0);
    else h = h.squeeze(0);
  }
  auto obj = [](const Tensor& t) -> py::object { return t.defined() ? py::cast(t) : py::none(); };
  return py::make_tuple(st, obj(xo), obj(h), obj(q), obj(s));
}

// Returns (status, out).
py::tuple fp8_matmul(uintptr_t handle, int64_t in_dim, int64_t out_dim, int dev, const Tensor& x, const Tensor& x_scales,
                     const Opt& out, at::ScalarType out_dtype) {
  need_rows(x, "x", -1, in_dim, dev);
  need_type(x, "x", at::kFloat8_e4m3fn);
  const int64_t rows = x.size(0);
  need_rows(x_scales, "x_scales", rows, (in_dim + EFFORT_BLOCK - 1) / EFFORT_BLOCK, dev);
  need_type(x_scales, "x_scales", at::kFloat);
  if (out) need_rows(*out, "out", rows, out_dim, dev);
  const auto type = out ? out->scalar_type() : out_dtype;
  const effort_dtype_t dt = need_dtype(type, "out_dtype");
  Tensor o = out ? *out : make(rows, out_dim, type, x);
  int st = 0;
  if (rows)
    st = f_fp8_matmul(reinterpret_cast<effort_fp8_t>(handle), x.data_ptr(), rows > 1 ? x.stride(0) : (in_dim + 15) / 16 * 16,
                      x_scales.data_ptr<float>(), row_stride(x_scales), rows, dt, o.data_ptr(), row_stride(o),
                      c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
  return py::make_tuple(st, o);
}

// mode: effort_gate_mode_t; ids and gates are given with EFFORT_GATE_GIVEN, else
// made.  Returns (status, out, ids, gates).
py::tuple moe_forward(uintptr_t handle, int64_t in_dim, int dev, const Tensor& x, int64_t top_k, int mode, const Opt& ids_in,
                      const Opt& gates_in, const Opt& out, std::optional<at::ScalarType> out_dtype) {
  need_rows(x, "x", -1, in_dim, dev);
  const auto type = x.scalar_type();
  const effort_dtype_t xdt = need_dtype(type, "x");
  const int64_t n = x.size(0);
  const auto h = reinterpret_cast<effort_moe_t>(handle);
  Tensor ids, gates;
  if (mode == EFFORT_GATE_GIVEN) {
    ids = *ids_in;
    gates = *gates_in;
    need_plain(ids, "ids");
    need_plain(gates, "gates");
    top_k = ids.dim() == 2 ? ids.size(1) : -1;
    auto good = [&](const Tensor& t, at::ScalarType want) {
      return t.is_cuda() && t.get_device() == dev && t.is_contiguous() && t.scalar_type() == want && t.dim() == 2 &&
             t.size(0) == n && t.size(1) == top_k;
    };
    TORCH_CHECK_VALUE(good(ids, at::kInt) && good(gates, at::kFloat),
                      "ids and gates must be contiguous int32 and float32 [tokens, top_k] on cuda:", dev);
  }
  if (out) need_rows(*out, "out", n, in_dim, dev);
  const auto ot = out ? out->scalar_type() : out_dtype ? *out_dtype : type;
  const effort_dtype_t odt = need_dtype(ot, "out_dtype");
  // tokens and top_k are checked before anything of their size is made
  const int32_t k = top_k < 0 ? 0 : top_k > INT32_MAX ? INT32_MAX : (int32_t)top_k;
  size_t bytes = 0;
  int st = n ? f_moe_scratch(h, n, k, &bytes) : 0;
  if (st != 0) return py::make_tuple(st, py::none(), py::none(), py::none());
  if (mode != EFFORT_GATE_GIVEN) {
    ids = make(n, k, at::kInt, x);
    gates = make(n, k, at::kFloat, x);
  }
  Tensor o = out ? *out : make(n, in_dim, ot, x);
  if (n) {
    // scratch of this call's own: the caching allocator keeps it apart from
    // other streams' and other graphs' calls
    const Tensor scratch = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte));
    st = f_moe_forward(h, x.data_ptr(), xdt, row_stride(x), n, k, (effort_gate_mode_t)mode, ids.data_ptr<int32_t>(),
                       gates.data_ptr<float>(), o.data_ptr(), odt, row_stride(o), scratch.data_ptr(), bytes,
                       c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
  }
  return py::make_tuple(st, o, ids, gates);
}

}  // namespace

PYBIND11_MODULE(_effort_torch, m) {
  m.def("init", &init);
  m.def("block_norm", &block_norm);
  m.def("fp8_matmul", &fp8_matmul);
  m.def("moe_forward", &moe_forward);
}
