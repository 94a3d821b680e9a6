// Python binding of the layer operators: checks torch tensors and passes
// their addresses, sizes and strides to the C ABI (include/repro.h).
//
// Marshalling in Python took more time than the smallest of these calls run
// for: a one-token call took 8.4 us that way and takes 4.0-5.0 so, by the
// host's pace, of which the launch is 3.7; a 4096-row table 7.9 and 5.5-6.0, a
// short backward pass with gains 19.7 and 11.1-11.8.  The comparison
// of a call's views for shared memory is some 0.1 us of that.  The library's entry points come from layer.py
// as addresses (bind), so this module links to no library of ours.
//
// Every function returns its tensors, or the library's status as an int where
// that is not REPRO_OK; layer.py raises for it.  Argument errors are raised
// here, as TypeError and ValueError.
#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdarg.h>
#include <string.h>

#include <algorithm>
#include <string>
#include <vector>

#include "repro.h"

namespace {

decltype(&repro_rope_table) g_rope_table;
decltype(&repro_qk_norm_rope) g_qk;
decltype(&repro_qk_workspace_bytes) g_qk_workspace;
decltype(&repro_qk_norm_rope_backward) g_qk_backward;
decltype(&repro_grad_list_bytes) g_list_bytes;
decltype(&repro_grad_list_plan) g_list_plan;
decltype(&repro_grad_list_norm) g_list_norm;
decltype(&repro_clip_grad_list) g_list_clip;
PyObject* g_raw_stream;  // device index -> its current stream's address

// Raises a Python exception from C++.
[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}

int current_device() {
  const c10::impl::VirtualGuardImpl impl(c10::DeviceType::CUDA);
  return impl.getDevice().index();
}

void* current_stream(int device) {
  PyObject* index = PyLong_FromLong(device);
  if (index == nullptr) throw python_error();
  PyObject* out = PyObject_CallOneArg(g_raw_stream, index);
  Py_DECREF(index);
  if (out == nullptr) throw python_error();
  void* stream = PyLong_AsVoidPtr(out);
  Py_DECREF(out);
  if (stream == nullptr && PyErr_Occurred()) throw python_error();
  return stream;
}

// The tensor in o, which has to be on `device`, the current one (-1: not
// looked up yet).
const at::Tensor& tensor(PyObject* o, const char* name, int* device) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor on a ROCm device", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(PyExc_TypeError, "%s must be a tensor on a ROCm device", name);
  if (t.layout() != at::kStrided) fail(PyExc_TypeError, "%s must be a strided tensor", name);
  if (*device < 0) *device = current_device();
  if (t.get_device() != *device)
    fail(PyExc_ValueError, "%s is on cuda:%d, but the current device is cuda:%d", name, (int)t.get_device(), *device);
  return t;
}

int32_t kind_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return REPRO_F32;
  if (t.scalar_type() == at::kBFloat16) return REPRO_BF16;
  fail(PyExc_TypeError, "%s must be float32 or bfloat16", name);
}

void* address(const at::Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::DeviceType::CUDA, (c10::DeviceIndex)device));
}

// o, a contiguous tensor of this type and shape, or a new one for None.
at::Tensor contiguous_out(PyObject* o, const char* name, at::IntArrayRef sizes, at::ScalarType type, int* device) {
  if (o == Py_None) return make(sizes, type, *device);
  const at::Tensor& t = tensor(o, name, device);
  if (t.scalar_type() != type || t.sizes() != sizes || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be a contiguous tensor of the type and shape of this output", name);
  return t;
}

// A side's tensor as the library takes it.
repro_head_view view(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef sizes) {
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must have the queries' type", name);
  if (t.sizes() != sizes) fail(PyExc_ValueError, "%s must have the shape of its side", name);
  if (t.stride(3) != 1) fail(PyExc_ValueError, "%s needs unit stride along its last dimension", name);
  return {address(t), t.stride(0), t.stride(1), t.stride(2)};
}

const void* gain(PyObject* o, const char* name, int64_t dim, int32_t* kind, int* device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name, device);
  const int32_t mine = kind_of(t, name);
  if (*kind >= 0 && *kind != mine) fail(PyExc_TypeError, "the gains must be of one type");
  if (t.dim() != 1 || t.size(0) != dim || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be a contiguous tensor of %lld elements", name, (long long)dim);
  *kind = mine;
  return t.data_ptr();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// Borrows the items; they are released here.
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* out = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (out == nullptr || o == nullptr) {
      Py_XDECREF(o);
      continue;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  if (out != nullptr && i != (Py_ssize_t)items.size()) {
    Py_DECREF(out);
    return nullptr;
  }
  return out;
}

// A new reference to o, or to t as a Python tensor where o is None.
PyObject* result(PyObject* o, const at::Tensor& t) {
  if (o != Py_None) {
    Py_INCREF(o);
    return o;
  }
  return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "%lld arguments, not %lld", (long long)want, (long long)n);
}

// rope_table(inv_freq, length, start, cos, sin)
PyObject* rope_table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 5);
  int device = -1;
  const at::Tensor& f = tensor(args[0], "inv_freq", &device);
  if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
    fail(PyExc_TypeError, "inv_freq must be a contiguous 1-D float64 tensor");
  const int64_t length = whole(args[1]), start = whole(args[2]);
  if (length < 0) fail(PyExc_ValueError, "length must not be negative");
  const int64_t half = f.size(0) < 1 << 20 ? f.size(0) : 1 << 20;  // the library refuses it
  if (half < 1 || half > 4096) return PyLong_FromLong(REPRO_EINVAL);
  const int64_t sizes[2] = {length, half};
  const at::Tensor cos = contiguous_out(args[3], "cos", sizes, at::kFloat, &device);
  const at::Tensor sin = contiguous_out(args[4], "sin", sizes, at::kFloat, &device);
  const int status =
      g_rope_table(static_cast<const double*>(f.data_ptr()), (int32_t)half, start, length,
                   static_cast<float*>(address(cos)), static_cast<float*>(address(sin)), current_stream(device));
  if (status != REPRO_OK) return PyLong_FromLong(status);
  return tuple_of({result(args[3], cos), result(args[4], sin)});
  END_HANDLE_TH_ERRORS
}

// What both passes check alike: everything of `a` but out, dy, dgain and eps.
struct Sides {
  int device = -1;
  at::ScalarType type;
  at::Tensor q, k;
};

void fill(repro_qk_args* a, Sides* s, PyObject* q, PyObject* k, PyObject* cos_o, PyObject* sin_o, PyObject* positions,
          PyObject* q_gain, PyObject* k_gain, PyObject* interleaved) {
  memset(a, 0, sizeof(*a));
  s->q = tensor(q, "q", &s->device);
  if (s->q.dim() != 4) fail(PyExc_ValueError, "q must be (batch, seq, heads, dim)");
  a->dtype = kind_of(s->q, "q");
  s->type = s->q.scalar_type();
  s->k = tensor(k, "k", &s->device);
  const auto qs = s->q.sizes(), ks = s->k.sizes();
  if (s->k.dim() != 4 || ks[0] != qs[0] || ks[1] != qs[1] || ks[3] != qs[3])
    fail(PyExc_ValueError, "k must be (batch, seq, heads, dim) with q's batch, seq and dim");
  constexpr int64_t kMost = INT32_MAX;
  if (qs[2] > kMost || ks[2] > kMost || qs[3] > kMost) fail(PyExc_ValueError, "q and k have too many heads");
  a->batch = qs[0];
  a->seq = qs[1];
  a->heads[0] = (int32_t)qs[2];
  a->heads[1] = (int32_t)ks[2];
  a->dim = (int32_t)qs[3];
  a->x[0] = view(s->q, "q", s->type, qs);
  a->x[1] = view(s->k, "k", s->type, ks);
  a->interleaved = truth(interleaved);

  const at::Tensor& cos = tensor(cos_o, "cos", &s->device);
  const at::Tensor& sin = tensor(sin_o, "sin", &s->device);
  if (cos.scalar_type() != at::kFloat || sin.scalar_type() != at::kFloat)
    fail(PyExc_TypeError, "cos and sin must be torch.float32");
  if (cos.dim() != 2 || sin.sizes() != cos.sizes())
    fail(PyExc_ValueError, "cos and sin must be (positions, rotary / 2) and of one shape");
  const int64_t rows = cos.size(0), half = cos.size(1);
  // A dimension of one element has any stride.
  if ((half > 1 && (cos.stride(1) != 1 || sin.stride(1) != 1)) || (rows > 1 && sin.stride(0) != cos.stride(0)))
    fail(PyExc_ValueError, "cos and sin need unit stride along their last dimension and one row stride");
  if (half > REPRO_MAX_HEAD_DIM) fail(PyExc_ValueError, "cos and sin are wider than any head");
  a->rotary = (int32_t)(2 * half);
  a->cos = static_cast<const float*>(address(cos));
  a->sin = static_cast<const float*>(address(sin));
  a->table_rows = rows;
  a->table_stride = rows > 1 ? cos.stride(0) : half;

  if (positions != Py_None) {
    const at::Tensor& p = tensor(positions, "positions", &s->device);
    if (p.scalar_type() != at::kInt && p.scalar_type() != at::kLong)
      fail(PyExc_TypeError, "positions must be int32 or int64");
    a->position_bytes = p.scalar_type() == at::kInt ? 4 : 8;
    if (p.dim() == 2 && p.size(0) == a->batch && p.size(1) == a->seq) {
      a->position_batch_stride = p.stride(0);
      a->position_seq_stride = p.stride(1);
    } else if (p.dim() == 1 && p.size(0) == a->seq) {
      a->position_seq_stride = p.stride(0);
    } else {
      fail(PyExc_ValueError, "positions must be (batch, seq) or (seq,)");
    }
    a->positions = address(p);
  }
  int32_t kind = -1;
  a->gain[0] = gain(q_gain, "q_gain", a->dim, &kind, &s->device);
  a->gain[1] = gain(k_gain, "k_gain", a->dim, &kind, &s->device);
  a->gain_dtype = kind < 0 ? 0 : kind;
}

// o, of the shape of like, or a new tensor for None.
at::Tensor side_out(PyObject* o, const char* name, const at::Tensor& like, Sides* s) {
  if (o == Py_None) return make(like.sizes(), s->type, s->device);
  return tensor(o, name, &s->device);
}

// qk(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved, q_out, k_out)
PyObject* qk(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 11);
  repro_qk_args a;
  Sides s;
  fill(&a, &s, args[0], args[1], args[2], args[3], args[4], args[5], args[6], args[8]);
  a.eps = (float)number(args[7]);
  const at::Tensor q_out = side_out(args[9], "q_out", s.q, &s);
  const at::Tensor k_out = side_out(args[10], "k_out", s.k, &s);
  a.out[0] = view(q_out, "q_out", s.type, s.q.sizes());
  a.out[1] = view(k_out, "k_out", s.type, s.k.sizes());
  const int status = g_qk(&a, current_stream(s.device));
  if (status != REPRO_OK) return PyLong_FromLong(status);
  return tuple_of({result(args[9], q_out), result(args[10], k_out)});
  END_HANDLE_TH_ERRORS
}

at::Tensor gain_out(PyObject* gain_o, PyObject* o, const char* name, int64_t dim, Sides* s) {
  if (gain_o == Py_None) {
    if (o != Py_None) fail(PyExc_ValueError, "%s without its gain", name);
    return {};
  }
  return contiguous_out(o, name, dim, at::kFloat, &s->device);
}

// qk_backward(q, k, dq_out, dk_out, cos, sin, positions, q_gain, k_gain, eps, interleaved, dq, dk, dq_gain, dk_gain,
//             workspace)
PyObject* qk_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 16);
  repro_qk_args a;
  Sides s;
  fill(&a, &s, args[0], args[1], args[4], args[5], args[6], args[7], args[8], args[10]);
  a.eps = (float)number(args[9]);
  a.dy[0] = view(tensor(args[2], "dq_out", &s.device), "dq_out", s.type, s.q.sizes());
  a.dy[1] = view(tensor(args[3], "dk_out", &s.device), "dk_out", s.type, s.k.sizes());
  const at::Tensor dq = side_out(args[11], "dq", s.q, &s);
  const at::Tensor dk = side_out(args[12], "dk", s.k, &s);
  a.out[0] = view(dq, "dq", s.type, s.q.sizes());
  a.out[1] = view(dk, "dk", s.type, s.k.sizes());
  const at::Tensor grads[2] = {gain_out(args[7], args[13], "dq_gain", a.dim, &s),
                               gain_out(args[8], args[14], "dk_gain", a.dim, &s)};
  for (int i = 0; i < 2; ++i) a.dgain[i] = grads[i].defined() ? static_cast<float*>(grads[i].data_ptr()) : nullptr;
  at::Tensor workspace;
  if (args[15] != Py_None) {
    workspace = tensor(args[15], "workspace", &s.device);
    if (workspace.scalar_type() != at::kByte) fail(PyExc_TypeError, "workspace must be torch.uint8");
    if (!workspace.is_contiguous()) fail(PyExc_ValueError, "workspace must be contiguous");
  } else if (a.dgain[0] != nullptr || a.dgain[1] != nullptr) {
    const int64_t need = g_qk_workspace(&a);
    if (need > 0) workspace = make(need, at::kByte, s.device);
  }
  const int status = g_qk_backward(&a, workspace.defined() ? address(workspace) : nullptr,
                                   workspace.defined() ? workspace.numel() : 0, current_stream(s.device));
  if (status != REPRO_OK) return PyLong_FromLong(status);
  return tuple_of({result(args[11], dq), result(args[12], dk), result(args[13], grads[0]), result(args[14], grads[1])});
  END_HANDLE_TH_ERRORS
}

// An out may be its own gradient, but share no memory with another tensor of
// the list.
void refuse_overlap(const std::vector<const void*>& grads, const std::vector<void*>& outs,
                    const std::vector<int64_t>& bytes) {
  struct Span {
    uintptr_t first, end;
    bool out;
  };
  std::vector<Span> spans;
  for (size_t i = 0; i < grads.size(); ++i) {
    if (bytes[i] == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
    spans.push_back({o, o + bytes[i], true});
    if (g != o) spans.push_back({g, g + bytes[i], false});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.first < b.first; });
  uintptr_t reach = 0, reach_out = 0;  // of all spans so far, and of the outs
  for (const Span& s : spans) {
    if (s.first < (s.out ? reach : reach_out))
      fail(PyExc_ValueError, "an out overlaps another tensor of the list");
    reach = std::max(reach, s.end);
    if (s.out) reach_out = std::max(reach_out, s.end);
  }
}

// What a list was laid out for: each tensor's memory, size and type.
struct Held {
  const void* at;
  int64_t size, type;
};

Held held(const at::Tensor& t) { return {address(t), t.numel(), (int64_t)t.scalar_type()}; }

// Whether the tensors of `list` still have the memory that it was laid out
// for (resize_, set_, as_strided_ and .data take it from a tensor that the
// list keeps).
void refuse_moved(PyObject* list, const char* name, const Held* was, Py_ssize_t count) {
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor& t = THPVariable_Unpack(PyTuple_GET_ITEM(list, i));
    const Held now = held(t);
    if (now.at != was[i].at || now.size != was[i].size || now.type != was[i].type || !t.is_contiguous())
      fail(PyExc_ValueError, "%s[%lld] has moved since the list was made: make a new one", name, (long long)i);
  }
}

// The statistics are written while a list's tensors are read and written, so
// they lie in none of them.
void refuse_shared(PyObject* list, const char* name, const void* out3, Py_ssize_t count) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(out3), end = first + 3 * sizeof(float);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor& t = THPVariable_Unpack(PyTuple_GET_ITEM(list, i));
    const uintptr_t at = reinterpret_cast<uintptr_t>(address(t));
    if (first < at + t.nbytes() && at < end)
      fail(PyExc_ValueError, "out shares memory with %s[%lld]", name, (long long)i);
  }
}

// list_plan(grads, outs), both tuples of one length: (device, host plan,
// held), the plan as a uint8 tensor, held for grad_list.
PyObject* list_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 2);
  if (!PyTuple_Check(args[0]) || !PyTuple_Check(args[1])) fail(PyExc_TypeError, "grads and outs must be tuples");
  const Py_ssize_t count = PyTuple_GET_SIZE(args[0]);
  if (PyTuple_GET_SIZE(args[1]) != count) fail(PyExc_ValueError, "outs must have one tensor for each gradient");
  std::vector<const void*> grads(count);
  std::vector<void*> outs(count);
  std::vector<int64_t> sizes(count), bytes(count);
  std::vector<int32_t> kinds(count);
  std::vector<Held> was(2 * count);
  int device = -1;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject* go = PyTuple_GET_ITEM(args[0], i);
    PyObject* oo = PyTuple_GET_ITEM(args[1], i);
    const std::string name = "grads[" + std::to_string(i) + "]";
    const at::Tensor& g = tensor(go, name.c_str(), &device);
    kinds[i] = kind_of(g, name.c_str());
    if (!g.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name.c_str());
    sizes[i] = g.numel();
    bytes[i] = sizes[i] * (int64_t)g.element_size();
    grads[i] = outs[i] = address(g);
    was[i] = was[count + i] = held(g);
    if (go == oo) continue;
    const std::string out_name = "outs[" + std::to_string(i) + "]";
    const at::Tensor& o = tensor(oo, out_name.c_str(), &device);
    if (o.scalar_type() != g.scalar_type()) fail(PyExc_TypeError, "%s must have its gradient's type", out_name.c_str());
    if (!o.is_contiguous() || o.numel() != sizes[i])
      fail(PyExc_ValueError, "%s must be contiguous and of its gradient's size", out_name.c_str());
    outs[i] = address(o);
    was[count + i] = held(o);
  }
  refuse_overlap(grads, outs, bytes);
  if (device < 0) device = current_device();
  const int64_t need = g_list_bytes(sizes.data(), kinds.data(), count);
  if (need < 0) return PyLong_FromLong((long)need);
  const at::Tensor host = at::empty(need, at::TensorOptions().dtype(at::kByte));
  const int status =
      g_list_plan(grads.data(), outs.data(), sizes.data(), kinds.data(), count, host.data_ptr(), need);
  if (status != REPRO_OK) return PyLong_FromLong(status);
  return tuple_of({PyLong_FromLong(device), THPVariable_Wrap(host),
                   PyBytes_FromStringAndSize(reinterpret_cast<const char*>(was.data()),
                                             (Py_ssize_t)(was.size() * sizeof(Held)))});
  END_HANDLE_TH_ERRORS
}

// grad_list(head, plan, max_norm, out, grads, outs, held): the clip, or the
// norm alone where max_norm is None; head: the first bytes of the plan on the
// host.
PyObject* grad_list(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 7);
  if (!PyTuple_Check(args[4]) || !PyTuple_Check(args[5]) || !PyBytes_Check(args[6]))
    fail(PyExc_TypeError, "grads and outs must be tuples and held bytes");
  const Py_ssize_t count = PyTuple_GET_SIZE(args[4]);
  if (PyTuple_GET_SIZE(args[5]) != count || PyBytes_GET_SIZE(args[6]) != (Py_ssize_t)(2 * count * sizeof(Held)))
    fail(PyExc_TypeError, "held is not of these tensors");
  const Held* was = reinterpret_cast<const Held*>(PyBytes_AS_STRING(args[6]));
  refuse_moved(args[4], "grads", was, count);
  if (args[4] != args[5]) refuse_moved(args[5], "outs", was + count, count);
  if (!PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) < 64) fail(PyExc_TypeError, "head must be 64 bytes");
  int device = -1;
  const at::Tensor& plan = tensor(args[1], "the list", &device);
  at::Tensor out;
  if (args[3] == Py_None) {
    out = make(3, at::kFloat, device);
  } else {
    out = tensor(args[3], "out", &device);
    if (out.scalar_type() != at::kFloat) fail(PyExc_TypeError, "out must be torch.float32");
    if (!out.is_contiguous() || out.numel() < 3) fail(PyExc_ValueError, "out must hold 3 contiguous elements");
    refuse_shared(args[4], "grads", address(out), count);
    if (args[4] != args[5]) refuse_shared(args[5], "outs", address(out), count);
  }
  const void* head = PyBytes_AS_STRING(args[0]);
  float* out3 = static_cast<float*>(out.data_ptr());
  const int status =
      args[2] == Py_None
          ? g_list_norm(head, plan.data_ptr(), out3, current_stream(device))
          : g_list_clip(head, plan.data_ptr(), (float)number(args[2]), out3, current_stream(device));
  if (status != REPRO_OK) return PyLong_FromLong(status);
  return result(args[3], out);
  END_HANDLE_TH_ERRORS
}

// bind(rope_table, qk, qk_workspace, qk_backward, list_bytes, list_plan, list_norm, list_clip, raw_stream)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int kEntries = 8;
  expect(n, kEntries + 1);
  void* at[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (at[i] == nullptr) fail(PyExc_ValueError, "no entry point");
  }
  g_rope_table = reinterpret_cast<decltype(g_rope_table)>(at[0]);
  g_qk = reinterpret_cast<decltype(g_qk)>(at[1]);
  g_qk_workspace = reinterpret_cast<decltype(g_qk_workspace)>(at[2]);
  g_qk_backward = reinterpret_cast<decltype(g_qk_backward)>(at[3]);
  g_list_bytes = reinterpret_cast<decltype(g_list_bytes)>(at[4]);
  g_list_plan = reinterpret_cast<decltype(g_list_plan)>(at[5]);
  g_list_norm = reinterpret_cast<decltype(g_list_norm)>(at[6]);
  g_list_clip = reinterpret_cast<decltype(g_list_clip)>(at[7]);
  Py_INCREF(args[kEntries]);
  Py_XDECREF(g_raw_stream);
  g_raw_stream = args[kEntries];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(bind),      FAST(rope_table), FAST(qk), FAST(qk_backward),
                           FAST(list_plan), FAST(grad_list),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer(void) {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddIntConstant(m, "QK_ARGS_BYTES", sizeof(repro_qk_args)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
