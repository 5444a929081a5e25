// The short way from Python to the layer norm, token log probability and AdamW
// entry points: checks, output allocation and the call in one compiled step, for
// calls whose kernels run a few microseconds (a layer norm of one token: 7 us of
// host time against 12 through ctypes).  Every function returns None where an
// argument is not what it expects; the caller then takes the checked way, which
// says what is wrong.  Nothing is computed here.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <algorithm>
#include <cstring>
#include <utility>
#include <vector>

#include "../../include/dora_finetune.h"

namespace {

struct Api {
  decltype(&dora_layernorm_forward) layernorm_forward;
  decltype(&dora_layernorm_backward) layernorm_backward;
  decltype(&dora_layernorm_workspace_bytes) layernorm_workspace_bytes;
  decltype(&dora_token_logprob_forward) logprob_forward;
  decltype(&dora_token_logprob_backward) logprob_backward;
  decltype(&dora_token_logprob_workspace_bytes) logprob_workspace_bytes;
  decltype(&dora_grad_norm) grad_norm;
  decltype(&dora_adamw_step) adamw_step;
  decltype(&dora_adamw_dequantize) dequantize;
};
Api g_api = {};

int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? DORA_BF16 : t == at::kFloat ? DORA_F32 : -1;
}

// A tensor argument, or null for None; `ok` is cleared if it is neither.
const at::Tensor* tensor(PyObject* o, bool& ok) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    ok = false;
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// [rows, width] on the GPU with contiguous rows that do not overlap; its row
// stride in ld.
bool rows_ok(const at::Tensor& t, int64_t& ld) {
  if (!t.is_cuda() || t.dim() != 2 || dtype_code(t.scalar_type()) < 0) return false;
  const int64_t R = t.size(0), D = t.size(1);
  if (D > 1 && t.stride(1) != 1) return false;
  ld = R <= 1 ? D : t.stride(0);
  return ld >= D;
}

// A contiguous vector of n elements of that type, on x's device.
bool vector_ok(const at::Tensor* t, int64_t n, at::ScalarType dt, const at::Tensor& x) {
  return t && t->scalar_type() == dt && t->dim() == 1 && t->size(0) == n && t->is_contiguous() &&
         t->device() == x.device();
}

const void* ptr(const at::Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
float* floats(const at::Tensor& t) { return static_cast<float*>(t.mutable_data_ptr()); }
const float* floats(const at::Tensor* t) { return static_cast<const float*>(ptr(t)); }
void* stream_of(PyObject* o) { return reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(o)); }

// Float32 tensors that share one allocation: `whole` has all their elements, and each takes
// the next ones: 0.5 us of host time less for every allocation saved.
at::Tensor take(const at::Tensor& whole, int64_t& from, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()),
                                                          whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(from);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  from += t.numel();
  return t;
}

PyObject* give(std::initializer_list<const at::Tensor*> out) {
  PyObject* t = PyTuple_New((Py_ssize_t)out.size());
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* x : out) {
    PyObject* o = x && x->defined() ? THPVariable_Wrap(*x) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// layernorm(x, weight, bias, eps, stream) -> (y, mean, rstd)
PyObject* layernorm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 5 && PyFloat_Check(args[3]);
  const at::Tensor* x = ok ? tensor(args[0], ok) : nullptr;
  const at::Tensor* w = ok ? tensor(args[1], ok) : nullptr;
  const at::Tensor* b = ok ? tensor(args[2], ok) : nullptr;
  dora_layernorm_shape s = {};
  if (!ok || !x || !rows_ok(*x, s.ld_x)) Py_RETURN_NONE;
  s.rows = x->size(0);
  s.width = x->size(1);
  s.ld_gy = s.ld_x;
  s.dtype = dtype_code(x->scalar_type());
  s.eps = (float)PyFloat_AS_DOUBLE(args[3]);
  if ((w && !vector_ok(w, s.width, x->scalar_type(), *x)) ||
      (b && !vector_ok(b, s.width, x->scalar_type(), *x)))
    Py_RETURN_NONE;
  const auto f32 = x->options().dtype(at::kFloat);
  const at::Tensor y = at::empty({s.rows, s.width}, x->options());
  const at::Tensor stats = at::empty({2 * s.rows}, f32);
  int64_t from = 0;
  const at::Tensor mean = take(stats, from, {s.rows}), rstd = take(stats, from, {s.rows});
  if (g_api.layernorm_forward(&s, x->const_data_ptr(), ptr(w), ptr(b), y.mutable_data_ptr(),
                              floats(mean), floats(rstd), stream_of(args[4])) != DORA_OK)
    Py_RETURN_NONE;
  return give({&y, &mean, &rstd});
  END_HANDLE_TH_ERRORS
}

// layernorm_backward(grad_y, x, weight, mean, rstd, want_x, want_weight, want_bias, stream)
// -> (grad_x, grad_weight, grad_bias)
PyObject* layernorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 9;
  const at::Tensor* t[5] = {};
  for (int i = 0; ok && i < 5; ++i) t[i] = tensor(args[i], ok);
  const at::Tensor *gy = t[0], *x = t[1], *w = t[2], *mean = t[3], *rstd = t[4];
  dora_layernorm_shape s = {};
  if (!ok || !gy || !x || !rows_ok(*x, s.ld_x) || !rows_ok(*gy, s.ld_gy)) Py_RETURN_NONE;
  s.rows = x->size(0);
  s.width = x->size(1);
  s.dtype = dtype_code(x->scalar_type());
  const auto dt = x->scalar_type();
  if (gy->size(0) != s.rows || gy->size(1) != s.width || gy->scalar_type() != dt ||
      gy->device() != x->device() || (w && !vector_ok(w, s.width, dt, *x)) ||
      !vector_ok(mean, s.rows, at::kFloat, *x) || !vector_ok(rstd, s.rows, at::kFloat, *x))
    Py_RETURN_NONE;
  at::Tensor gx, gw, gb, ws;
  if (args[5] == Py_True) gx = at::empty({s.rows, s.width}, x->options());
  if (args[6] == Py_True) gw = at::empty({s.width}, x->options());
  if (args[7] == Py_True) gb = at::empty({s.width}, x->options());
  const bool alone = !gw.defined() && !gb.defined() && s.width <= DORA_LAYERNORM_NO_WS_WIDTH(s.dtype);
  const size_t need = alone ? 0 : g_api.layernorm_workspace_bytes(&s);
  if (need) ws = at::empty({(int64_t)need}, x->options().dtype(at::kByte));
  auto out = [](const at::Tensor& o) { return o.defined() ? o.mutable_data_ptr() : nullptr; };
  if (g_api.layernorm_backward(&s, gy->const_data_ptr(), x->const_data_ptr(), ptr(w), floats(mean),
                               floats(rstd), out(gx), out(gw), out(gb), out(ws), need,
                               stream_of(args[8])) != DORA_OK)
    Py_RETURN_NONE;
  return give({&gx, &gw, &gb});
  END_HANDLE_TH_ERRORS
}

// token_logprob(logits, targets, scale, top, stream)
// -> (logp, entropy, lse, top_logp or None, top_index or None)
PyObject* token_logprob(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 5 && PyFloat_Check(args[2]) && PyLong_Check(args[3]);
  const at::Tensor* z = ok ? tensor(args[0], ok) : nullptr;
  const at::Tensor* y = ok ? tensor(args[1], ok) : nullptr;
  dora_logprob_shape s = {};
  if (!ok || !z || !rows_ok(*z, s.ld)) Py_RETURN_NONE;
  s.rows = z->size(0);
  s.vocab = z->size(1);
  s.dtype = dtype_code(z->scalar_type());
  s.scale = (float)PyFloat_AS_DOUBLE(args[2]);
  const long top = PyLong_AsLong(args[3]);
  if (top == -1 && PyErr_Occurred()) PyErr_Clear();
  if (top < 0 || top > DORA_LOGPROB_MAX_TOP || !vector_ok(y, s.rows, at::kLong, *z)) Py_RETURN_NONE;
  s.top = (int32_t)top;
  const auto f32 = z->options().dtype(at::kFloat);
  const at::Tensor whole = at::empty({s.rows * (3 + top)}, f32);
  int64_t from = 0;
  const at::Tensor logp = take(whole, from, {s.rows}), entropy = take(whole, from, {s.rows}),
                   lse = take(whole, from, {s.rows});
  at::Tensor top_logp, top_index, ws;
  if (top) {
    top_logp = take(whole, from, {s.rows, top});
    top_index = at::empty({s.rows, top}, z->options().dtype(at::kLong));
  }
  const size_t need = g_api.logprob_workspace_bytes(&s);
  if (need) ws = at::empty({(int64_t)need}, z->options().dtype(at::kByte));
  if (g_api.logprob_forward(&s, z->const_data_ptr(), y->const_data_ptr<int64_t>(), floats(logp),
                            floats(entropy), floats(lse), top ? floats(top_logp) : nullptr,
                            top ? top_index.mutable_data_ptr<int64_t>() : nullptr,
                            need ? ws.mutable_data_ptr() : nullptr, need,
                            stream_of(args[4])) != DORA_OK)
    Py_RETURN_NONE;
  return give({&logp, &entropy, &lse, &top_logp, &top_index});
  END_HANDLE_TH_ERRORS
}

// token_logprob_backward(grad_logp, grad_entropy, logits, targets, lse, entropy, scale, stream)
// -> grad_logits
PyObject* token_logprob_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 8 && PyFloat_Check(args[6]);
  const at::Tensor* t[6] = {};
  for (int i = 0; ok && i < 6; ++i) t[i] = tensor(args[i], ok);
  const at::Tensor *ga = t[0], *gh = t[1], *z = t[2], *y = t[3], *lse = t[4], *entropy = t[5];
  dora_logprob_shape s = {};
  if (!ok || !z || !rows_ok(*z, s.ld)) Py_RETURN_NONE;
  s.rows = z->size(0);
  s.vocab = z->size(1);
  s.dtype = dtype_code(z->scalar_type());
  s.scale = (float)PyFloat_AS_DOUBLE(args[6]);
  auto floats_ok = [&](const at::Tensor* v) { return vector_ok(v, s.rows, at::kFloat, *z); };
  if (!vector_ok(y, s.rows, at::kLong, *z) || !floats_ok(lse) || (ga && !floats_ok(ga)) ||
      (gh && !floats_ok(gh)) || (entropy && !floats_ok(entropy)))
    Py_RETURN_NONE;
  const at::Tensor g = at::empty({s.rows, s.vocab}, z->options());
  if (g_api.logprob_backward(&s, floats(ga), floats(gh), z->const_data_ptr(),
                             y->const_data_ptr<int64_t>(), floats(lse), floats(entropy),
                             g.mutable_data_ptr(), stream_of(args[7])) != DORA_OK)
    Py_RETURN_NONE;
  return THPVariable_Wrap(g);
  END_HANDLE_TH_ERRORS
}

// The lists of an AdamW step: params, exp_avg, exp_avg_sq, exp_avg_scales, exp_avg_sq_scales,
// masters (the last three may be None; without scales the moments are float32, with them int8 and
// uint8).
struct Lists {
  PyObject* const* list;   // kCount of them
  static constexpr int kCount = 6;
  Py_ssize_t count = 0;
  bool small = false;
  const at::Tensor* first = nullptr;   // the first param

  explicit Lists(PyObject* const* args) : list(args) {}
  bool open() {
    if (!PyList_Check(list[0])) return false;
    count = PyList_GET_SIZE(list[0]);
    for (int i = 1; i < kCount; ++i)
      if (!(i > 2 && list[i] == Py_None) &&
          !(PyList_Check(list[i]) && PyList_GET_SIZE(list[i]) == count))
        return false;
    small = list[3] != Py_None;
    return small == (list[4] != Py_None);
  }
  // Tensor i as the table's entry (its gradient left out); false unless all are contiguous, on
  // one device, of their types and sizes.
  bool entry(Py_ssize_t i, dora_adamw_tensor& e) {
    bool ok = true;
    const at::Tensor* t[kCount] = {};
    for (int k = 0; k < kCount; ++k)
      if (list[k] != Py_None) t[k] = tensor(PyList_GET_ITEM(list[k], i), ok);
    if (!ok || !t[0]) return false;
    if (!first) first = t[0];
    const int64_t size = t[0]->numel(), blocks = (size + DORA_STATE_BLOCK - 1) / DORA_STATE_BLOCK;
    if (!t[0]->is_cuda() || t[0]->scalar_type() != first->scalar_type()) return false;
    const at::ScalarType types[kCount] = {first->scalar_type(), small ? at::kChar : at::kFloat,
                                          small ? at::kByte : at::kFloat, at::kFloat, at::kFloat,
                                          at::kFloat};
    for (int k = 0; k < kCount; ++k) {
      if (list[k] == Py_None) continue;
      const int64_t need = k == 3 || k == 4 ? blocks : size;
      if (!t[k] || t[k]->scalar_type() != types[k] || t[k]->numel() != need ||
          !t[k]->is_contiguous() || t[k]->device() != first->device())
        return false;
    }
    auto at = [&](int k) { return t[k] ? t[k]->data_ptr() : nullptr; };
    e.param = at(0);
    e.exp_avg = at(1);
    e.exp_avg_sq = at(2);
    e.exp_avg_scale = static_cast<float*>(at(3));
    e.exp_avg_sq_scale = static_cast<float*>(at(4));
    e.master = static_cast<float*>(at(5));
    e.n = size;
    return true;
  }
  // Whether tensor i still is what the table's entry says (the same address is the same device).
  bool same(Py_ssize_t i, const dora_adamw_tensor& e) {
    const void* at[kCount] = {e.param,         e.exp_avg,          e.exp_avg_sq,
                              e.exp_avg_scale, e.exp_avg_sq_scale, e.master};
    const int64_t blocks = (e.n + DORA_STATE_BLOCK - 1) / DORA_STATE_BLOCK;
    for (int k = 0; k < kCount; ++k) {
      if (list[k] == Py_None) continue;
      PyObject* o = PyList_GET_ITEM(list[k], i);
      if (!THPVariable_Check(o)) return false;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!first) first = &t;
      const at::ScalarType type = k == 0              ? first->scalar_type()
                                  : small && k == 1 ? at::kChar
                                  : small && k == 2 ? at::kByte
                                                    : at::kFloat;
      if (t.const_data_ptr() != at[k] || t.numel() != (k == 3 || k == 4 ? blocks : e.n) ||
          t.scalar_type() != type || !t.is_contiguous())
        return false;
    }
    return true;
  }
};

// Whether any two of the arrays that a step on these tensors writes share memory.
bool overlapping(const dora_adamw_tensor* table, Py_ssize_t count, int param_bytes, bool small) {
  std::vector<std::pair<const char*, const char*>> written;
  written.reserve((size_t)count * 6);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const dora_adamw_tensor& e = table[i];
    const int64_t blocks = (e.n + DORA_STATE_BLOCK - 1) / DORA_STATE_BLOCK;
    auto add = [&](const void* p, int64_t bytes) {
      const char* at = static_cast<const char*>(p);
      if (at && bytes > 0) written.emplace_back(at, at + bytes);
    };
    add(e.param, e.n * param_bytes);
    add(e.exp_avg, e.n * (small ? 1 : 4));
    add(e.exp_avg_sq, e.n * (small ? 1 : 4));
    add(e.exp_avg_scale, blocks * 4);
    add(e.exp_avg_sq_scale, blocks * 4);
    add(e.master, e.n * 4);
  }
  std::sort(written.begin(), written.end());
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].first < written[i - 1].second) return true;
  return false;
}

// make_table(the six lists, table address): fills the table.  Returns the parameters' dtype code,
// or None where the lists are not what they should be.
PyObject* make_table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Lists lists(args);
  if (n != Lists::kCount + 1 || !lists.open()) Py_RETURN_NONE;
  auto* table = static_cast<dora_adamw_tensor*>(PyLong_AsVoidPtr(args[6]));
  for (Py_ssize_t i = 0; i < lists.count; ++i)
    if (!lists.entry(i, table[i])) Py_RETURN_NONE;
  const int code = lists.first ? dtype_code(lists.first->scalar_type()) : -1;
  if (code < 0 || (args[5] != Py_None && code != DORA_BF16)) Py_RETURN_NONE;
  if (overlapping(table, lists.count, code == DORA_BF16 ? 2 : 4, lists.small)) Py_RETURN_NONE;
  return PyLong_FromLong(code);
  END_HANDLE_TH_ERRORS
}

// same_table(the six lists, table address) -> whether every tensor is where the table has it.
PyObject* same_table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Lists lists(args);
  if (n != Lists::kCount + 1 || !lists.open()) Py_RETURN_FALSE;
  const auto* table = static_cast<dora_adamw_tensor*>(PyLong_AsVoidPtr(args[6]));
  for (Py_ssize_t i = 0; i < lists.count; ++i)
    if (!lists.same(i, table[i])) Py_RETURN_FALSE;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// take_grads(the six lists, table address, grads, device index): notes the gradients' addresses in
// the table.  Returns their dtype code, or None unless every tensor is where the table has it and
// every gradient is contiguous, of its size, of one type and on the device.
PyObject* take_grads(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Lists lists(args);
  if (n != Lists::kCount + 3 || !lists.open() || !PyList_Check(args[7])) Py_RETURN_NONE;
  if (lists.count < 1 || PyList_GET_SIZE(args[7]) != lists.count) Py_RETURN_NONE;
  auto* table = static_cast<dora_adamw_tensor*>(PyLong_AsVoidPtr(args[6]));
  const long device = PyLong_AsLong(args[8]);
  int code = -1;
  for (Py_ssize_t i = 0; i < lists.count; ++i) {
    bool ok = true;
    const at::Tensor* g = tensor(PyList_GET_ITEM(args[7], i), ok);
    if (!g || !g->is_cuda()) Py_RETURN_NONE;
    const int c = dtype_code(g->scalar_type());
    if (i == 0) code = c;
    if (c < 0 || c != code || !lists.same(i, table[i]) || g->numel() != table[i].n ||
        !g->is_contiguous() || g->get_device() != device)
      Py_RETURN_NONE;
    table[i].grad = g->const_data_ptr();
  }
  return PyLong_FromLong(code);
  END_HANDLE_TH_ERRORS
}

// grad_norm(table address, count, dtype code, max_norm, workspace bytes, a param, stream)
// -> (norm, factor)
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 7;
  const at::Tensor* like = ok ? tensor(args[5], ok) : nullptr;
  if (!ok || !like) Py_RETURN_NONE;
  const int64_t bytes = PyLong_AsLongLong(args[4]);
  const auto f32 = like->options().dtype(at::kFloat);
  const at::Tensor both = at::empty({2}, f32);
  int64_t from = 0;
  const at::Tensor norm = take(both, from, {}), factor = take(both, from, {});
  const at::Tensor ws = at::empty({bytes > 0 ? bytes : 1}, f32.dtype(at::kByte));
  if (g_api.grad_norm(static_cast<dora_adamw_tensor*>(PyLong_AsVoidPtr(args[0])),
                      PyLong_AsLongLong(args[1]), (int32_t)PyLong_AsLong(args[2]),
                      PyFloat_AsDouble(args[3]), floats(norm), floats(factor),
                      ws.mutable_data_ptr(), (size_t)bytes, stream_of(args[6])) != DORA_OK)
    Py_RETURN_NONE;
  return give({&norm, &factor});
  END_HANDLE_TH_ERRORS
}

// adamw_step(table address, params, param code, grad code, state bits, step, lr, beta1, beta2, eps,
// weight_decay, grad_scale or None, stream) -> the return code.  The parameters' versions go up, so
// that a backward pass which saved one of them from before the step is refused.
PyObject* adamw_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 13 && PyList_Check(args[1]);
  const at::Tensor* scale = ok ? tensor(args[11], ok) : nullptr;
  if (!ok) Py_RETURN_NONE;
  const Py_ssize_t count = PyList_GET_SIZE(args[1]);
  dora_adamw_options o = {};
  o.param_dtype = (int32_t)PyLong_AsLong(args[2]);
  o.grad_dtype = (int32_t)PyLong_AsLong(args[3]);
  o.state_bits = (int32_t)PyLong_AsLong(args[4]);
  o.step = PyLong_AsLongLong(args[5]);
  o.lr = PyFloat_AsDouble(args[6]);
  o.beta1 = PyFloat_AsDouble(args[7]);
  o.beta2 = PyFloat_AsDouble(args[8]);
  o.eps = PyFloat_AsDouble(args[9]);
  o.weight_decay = PyFloat_AsDouble(args[10]);
  o.grad_scale = floats(scale);
  if (PyErr_Occurred()) return nullptr;
  const int rc = g_api.adamw_step(static_cast<dora_adamw_tensor*>(PyLong_AsVoidPtr(args[0])), count,
                                  &o, stream_of(args[12]));
  for (Py_ssize_t i = 0; rc == DORA_OK && i < count; ++i) {
    const at::Tensor* p = tensor(PyList_GET_ITEM(args[1], i), ok);
    if (p && !p->is_inference()) p->unsafeGetTensorImpl()->bump_version();
  }
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

// dequantize(codes, scales, bf16, stream) -> values
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 4;
  const at::Tensor* codes = ok ? tensor(args[0], ok) : nullptr;
  const at::Tensor* scales = ok ? tensor(args[1], ok) : nullptr;
  if (!ok || !codes || !codes->is_cuda() || !codes->is_contiguous()) Py_RETURN_NONE;
  const bool second = codes->scalar_type() == at::kByte;
  const int64_t blocks = (codes->numel() + DORA_STATE_BLOCK - 1) / DORA_STATE_BLOCK;
  if ((!second && codes->scalar_type() != at::kChar) ||
      !vector_ok(scales, blocks, at::kFloat, *codes))
    Py_RETURN_NONE;
  const bool bf16 = args[2] == Py_True;
  const at::Tensor out =
      at::empty(codes->sizes(), codes->options().dtype(bf16 ? at::kBFloat16 : at::kFloat));
  if (g_api.dequantize(codes->const_data_ptr(), floats(scales), codes->numel(), second,
                       out.mutable_data_ptr(), bf16 ? DORA_BF16 : DORA_F32,
                       stream_of(args[3])) != DORA_OK)
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// init(addresses of the entry points of Api, in its order)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kCount = sizeof(Api) / sizeof(void*);
  void* p[kCount];
  for (Py_ssize_t i = 0; i < kCount; ++i) {
    p[i] = n == kCount ? PyLong_AsVoidPtr(args[i]) : nullptr;
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "init takes an address per entry point");
      return nullptr;
    }
  }
  static_assert(sizeof p == sizeof g_api, "function pointers only");
  memcpy(&g_api, p, sizeof g_api);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(layernorm),     FAST(layernorm_backward),
                         FAST(token_logprob), FAST(token_logprob_backward),
                         FAST(make_table),    FAST(same_table),
                         FAST(take_grads),    FAST(grad_norm),
                         FAST(adamw_step),    FAST(dequantize),
                         FAST(init),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
