// The hot calls of the attention half's binding: reads the tensors of a call,
// checks that they are what the call takes, and enters the C ABI.  A decode
// step makes five such calls a layer; in Python the same checks and the
// marshalling took longer than the kernels run.  A function returns the
// library's code, or kNotTaken where some argument is not what it must be; the
// Python side then finds the reasons and raises.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "mono_attn.h"

namespace {

constexpr long kNotTaken = LONG_MIN;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int64_t number(PyObject* o) { return o == Py_None ? 0 : PyLong_AsLongLong(o); }
void* address(PyObject* o) { return reinterpret_cast<void*>(number(o)); }

at::ScalarType type_of(int64_t code) { return code == MONO_F32 ? at::kFloat : at::kBFloat16; }

void* stream_of(PyObject* o, int64_t device) {
  return o == Py_None ? c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream() : address(o);
}

bool on(const at::Tensor* t, int64_t device) { return t && t->is_cuda() && t->get_device() == device; }

// int32, contiguous, [n] or [n][m]
bool entries(const at::Tensor* t, int64_t device, int64_t n, int64_t m) {
  return on(t, device) && t->scalar_type() == at::kInt && t->is_contiguous() && t->dim() == (m < 0 ? 1 : 2) &&
         t->size(0) == n && (m < 0 || t->size(1) == m);
}

// Memory that is written.  Taking its address gives a lazily cloned tensor
// storage of its own, so it comes before that of tensors which may share it.
void* written(const at::Tensor* t) { return t->mutable_data_ptr(); }

// [seqs][width][heads][head_dim] with a contiguous last dimension
bool rows(const at::Tensor* t, int64_t device, int64_t type, int64_t heads, int64_t head_dim, bool out, mono_rows* r) {
  if (!on(t, device) || t->scalar_type() != type_of(type) || t->dim() != 4 || t->size(2) != heads ||
      t->size(3) != head_dim || t->stride(3) != 1)
    return false;
  *r = mono_rows{out ? written(t) : const_cast<void*>(t->const_data_ptr()), t->stride(0), t->stride(1), t->stride(2)};
  return true;
}

template <typename F>
PyObject* guarded(F&& f) {
  long rc = kNotTaken;
  try {
    rc = f();
  } catch (...) {   // of torch's accessors
  }
  if (PyErr_Occurred()) return nullptr;
  return PyLong_FromLong(rc);
}

template <typename F>
long enter(F&& f) {
  if (PyErr_Occurred()) return kNotTaken;   // an argument that is no number
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  return rc;
}

// (rope, x, positions, out, transpose, stream)
PyObject* call_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    const at::Tensor *x = n == 6 ? tensor(a[1]) : nullptr, *pos = x ? tensor(a[2]) : nullptr, *out = pos ? tensor(a[3]) : nullptr;
    if (!out || !x->is_cuda() || x->dim() != 3 || out->dim() != 3) return kNotTaken;
    const int64_t dev = x->get_device(), tokens = x->size(0), heads = x->size(1);
    const auto type = x->scalar_type();
    if ((type != at::kFloat && type != at::kBFloat16) || out->scalar_type() != type || !on(out, dev) ||
        out->sizes() != x->sizes() || !entries(pos, dev, tokens, -1) || tokens > INT_MAX || heads > INT_MAX ||
        x->size(2) > INT_MAX || (tokens && heads && (x->stride(2) != 1 || out->stride(2) != 1)))
      return kNotTaken;
    const auto* rope = static_cast<const mono_rope*>(address(a[0]));
    const int transpose = PyObject_IsTrue(a[4]) == 1;
    void* stream = stream_of(a[5], dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    void* to = written(out);
    return enter([&] {
      return mono_rope_apply(rope, (int)tokens, (int)heads, (int)x->size(2), type == at::kFloat ? MONO_F32 : MONO_BF16,
                             x->const_data_ptr(), x->stride(0), x->stride(1), static_cast<const int*>(pos->const_data_ptr()),
                             to, out->stride(0), out->stride(1), transpose, stream);
    });
  });
}

// what append and attend share: (plan, cache, heads, head_dim, dtype, device,
// max_pages, x, y, lens, table, n_new, ...)
struct Call {
  mono_rows x, y;
  mono_seqs seqs;
  bool take(PyObject* const* a, bool y_out) {
    const int64_t heads = number(a[2]), head_dim = number(a[3]), type = number(a[4]), dev = number(a[5]);
    const at::Tensor *tx = tensor(a[7]), *ty = tensor(a[8]), *lens = tensor(a[9]), *table = tensor(a[10]);
    const at::Tensor* n_new = a[11] == Py_None ? nullptr : tensor(a[11]);
    if (!rows(ty, dev, type, heads, head_dim, y_out, &y) || !rows(tx, dev, type, heads, head_dim, false, &x)) return false;
    const int64_t n = tx->size(0), width = tx->size(1);
    if (ty->size(0) != n || ty->size(1) != width || n > INT_MAX || width > INT_MAX || !entries(lens, dev, n, -1) ||
        !entries(table, dev, n, number(a[6])) || (a[11] != Py_None && !entries(n_new, dev, n, -1)))
      return false;
    seqs = mono_seqs{(int)n, (int)width, static_cast<const int*>(lens->const_data_ptr()),
                     n_new ? static_cast<const int*>(n_new->const_data_ptr()) : nullptr,
                     static_cast<const int*>(table->const_data_ptr())};
    return true;
  }
};

// (..., rope, stream)
PyObject* call_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    Call c;
    if (n != 14 || !c.take(a, false)) return kNotTaken;
    auto* plan = static_cast<mono_attn_plan_t*>(address(a[0]));
    const auto* cache = static_cast<const mono_kv_cache*>(address(a[1]));
    const auto* rope = static_cast<const mono_rope*>(address(a[12]));
    void* stream = stream_of(a[13], number(a[5]));
    return enter([&] { return mono_attn_append(plan, cache, &c.seqs, &c.x, &c.y, rope, stream); });
  });
}

// (..., lse, stream)
PyObject* call_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    Call c;
    if (n != 14 || !c.take(a, true)) return kNotTaken;
    float* lse = nullptr;
    if (a[12] != Py_None) {
      const at::Tensor* t = tensor(a[12]);
      if (!on(t, number(a[5])) || t->scalar_type() != at::kFloat || t->dim() != 3 || t->size(0) != c.seqs.seqs ||
          t->size(1) != c.seqs.width || t->size(2) != number(a[2]) || !t->is_contiguous())
        return kNotTaken;
      lse = static_cast<float*>(written(t));
    }
    auto* plan = static_cast<mono_attn_plan_t*>(address(a[0]));
    const auto* cache = static_cast<const mono_kv_cache*>(address(a[1]));
    void* stream = stream_of(a[13], number(a[5]));
    return enter([&] { return mono_attn_attend(plan, cache, &c.seqs, &c.x, &c.y, lse, stream); });
  });
}

// (plan, n_out, n_in, dtype, device, x, y, stream)
PyObject* call_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> long {
    const at::Tensor *x = n == 8 ? tensor(a[5]) : nullptr, *y = x ? tensor(a[6]) : nullptr;
    if (!y) return kNotTaken;
    const int64_t n_out = number(a[1]), n_in = number(a[2]), dev = number(a[4]);
    const auto type = type_of(number(a[3]));
    if (!on(x, dev) || !on(y, dev) || x->scalar_type() != type || y->scalar_type() != type || x->dim() != 2 ||
        y->dim() != 2 || x->size(1) != n_in || y->size(1) != n_out || y->size(0) != x->size(0) || x->size(0) > INT_MAX ||
        x->stride(1) != 1 || (y->stride(1) != 1 && n_out != 1))
      return kNotTaken;
    auto* plan = static_cast<mono_proj_plan_t*>(address(a[0]));
    void* stream = stream_of(a[7], dev);
    void* to = written(y);
    return enter([&] {
      return mono_proj_step(plan, (int)x->size(0), x->const_data_ptr(), x->stride(0), to, y->stride(0), stream);
    });
  });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_attend)), METH_FASTCALL, nullptr},
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_step)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddObject(m, "NOT_TAKEN", PyLong_FromLong(kNotTaken)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
