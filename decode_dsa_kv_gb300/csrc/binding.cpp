// Python entry points of the paged cache's calls: the C ABI's functions with
// their arguments taken from tensors, ints and None, as the ctypes binding takes
// them. A call of a few microseconds on the GPU is bound by its caller: through
// ctypes a wrapper of twenty arguments takes 3.8 us before its launch, here 1.3.
//
// Arguments by the C type: a pointer is None, an address or anything with
// data_ptr(); a stream None (the current one), a handle or anything with
// cuda_stream; whole numbers as they are, flags what int() takes, a scale what
// float() takes. Those after the required ones default to None.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "dsakv.h"

namespace {

PyObject *s_data_ptr, *s_cuda_stream;          // names
PyObject *f_current_device, *f_raw_stream;     // torch's, looked up once

bool get_address(PyObject* o, uintptr_t* out) {
  *out = 0;
  if (o == Py_None) return true;
  if (PyLong_Check(o)) {
    *out = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o));
    return !PyErr_Occurred();
  }
  PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!p) return false;
  *out = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(p));
  Py_DECREF(p);
  return !PyErr_Occurred();
}

bool find_torch() {
  if (f_raw_stream) return true;
  PyObject* m = PyImport_ImportModule("torch._C");
  if (!m) return false;
  f_current_device = PyObject_GetAttrString(m, "_cuda_getDevice");
  PyObject* raw = f_current_device ? PyObject_GetAttrString(m, "_cuda_getCurrentRawStream") : nullptr;
  Py_DECREF(m);
  if (!raw) return false;
  PyObject* cuda = PyImport_ImportModule("torch.cuda");
  PyObject* done = cuda ? PyObject_CallMethod(cuda, "init", nullptr) : nullptr;
  Py_XDECREF(cuda);
  if (!done) {
    Py_DECREF(raw);
    return false;
  }
  Py_DECREF(done);
  f_raw_stream = raw;
  return true;
}

bool get_stream(PyObject* o, uintptr_t* out) {
  if (PyLong_Check(o)) return get_address(o, out);
  PyObject* h;
  if (o == Py_None) {
    if (!find_torch()) return false;
    PyObject* dev = PyObject_CallNoArgs(f_current_device);
    if (!dev) return false;
    h = PyObject_CallOneArg(f_raw_stream, dev);
    Py_DECREF(dev);
  } else {
    h = PyObject_GetAttr(o, s_cuda_stream);
  }
  if (!h) return false;
  *out = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(h));
  Py_DECREF(h);
  return !PyErr_Occurred();
}

template <class T>
bool get(PyObject* o, T* out) {
  if constexpr (std::is_same_v<T, cudaStream_t>) {
    uintptr_t v;
    if (!get_stream(o, &v)) return false;
    *out = reinterpret_cast<cudaStream_t>(v);
    return true;
  } else if constexpr (std::is_pointer_v<T>) {
    uintptr_t v;
    if (!get_address(o, &v)) return false;
    *out = reinterpret_cast<T>(v);
    return true;
  } else if constexpr (std::is_floating_point_v<T>) {
    PyObject* x = PyNumber_Float(o);
    if (!x) return false;
    *out = static_cast<T>(PyFloat_AS_DOUBLE(x));
    Py_DECREF(x);
    return true;
  } else {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    *out = static_cast<T>(v);
    if (static_cast<long long>(*out) != v) {
      PyErr_SetString(PyExc_OverflowError, "an argument does not fit its C type");
      return false;
    }
    return true;
  }
}

template <class F>
struct Signature;
template <class R, class... A>
struct Signature<R (*)(A...)> {
  static constexpr Py_ssize_t kCount = sizeof...(A);
  template <class F, size_t... I>
  static PyObject* call(F f, PyObject* const* o, std::index_sequence<I...>) {
    std::tuple<A...> v;
    if (!(get(o[I], &std::get<I>(v)) && ...)) return nullptr;
    R r;
    Py_BEGIN_ALLOW_THREADS;
    r = f(std::get<I>(v)...);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLongLong(static_cast<long long>(r));
  }
};

// A function, its parameters' names, which of them are flags and how many have no
// default.
struct Names {
  PyObject* name[32];
  uint32_t flags;
  Py_ssize_t required;
};

template <auto* kFunction>
struct Entry {
  using S = Signature<decltype(kFunction)>;
  static_assert(S::kCount < 32, "names");
  static Names names;
  static PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t given, PyObject* keywords) {
    PyObject* o[32];
    if (given > S::kCount) {
      PyErr_Format(PyExc_TypeError, "%zd arguments at most: %zd given", S::kCount, given);
      return nullptr;
    }
    for (Py_ssize_t i = 0; i < S::kCount; ++i)
      o[i] = i < given ? args[i] : i < names.required ? nullptr : Py_None;
    const Py_ssize_t more = keywords ? PyTuple_GET_SIZE(keywords) : 0;
    for (Py_ssize_t k = 0; k < more; ++k) {
      PyObject* key = PyTuple_GET_ITEM(keywords, k);
      Py_ssize_t i = 0;
      while (i < S::kCount && key != names.name[i] && PyUnicode_Compare(key, names.name[i]) != 0) ++i;
      if (i == S::kCount || i < given) {
        PyErr_Format(PyExc_TypeError, i == S::kCount ? "no argument %R" : "two values for argument %R",
                     key);
        return nullptr;
      }
      o[i] = args[given + k];
    }
    for (Py_ssize_t i = given; i < names.required; ++i)
      if (!o[i]) {
        PyErr_Format(PyExc_TypeError, "argument %R is missing", names.name[i]);
        return nullptr;
      }
    for (Py_ssize_t i = 0; names.flags >> i; ++i) {
      if (!(names.flags >> i & 1) || PyLong_Check(o[i])) continue;
      PyObject* x = PyNumber_Long(o[i]);
      if (!x) return nullptr;
      o[i] = PyObject_IsTrue(x) ? Py_True : Py_False;
      Py_DECREF(x);
    }
    return S::call(kFunction, o, std::make_index_sequence<S::kCount>());
  }
};
template <auto* kFunction>
Names Entry<kFunction>::names;

// Fills in the names ("a b ?c | err stream": c is a flag, those after the bar have
// defaults).
template <auto* kFunction>
bool name(const char* list) {
  Names& n = Entry<kFunction>::names;
  Py_ssize_t count = 0;
  n.required = -1;
  n.flags = 0;
  for (const char* p = list; *p;) {
    const char* end = p;
    while (*end && *end != ' ') ++end;
    if (*p == '|') {
      n.required = count;
    } else {
      if (count == 31) return false;
      if (*p == '?') {
        n.flags |= 1u << count;
        ++p;
      }
      n.name[count] = PyUnicode_FromStringAndSize(p, end - p);
      if (!n.name[count]) return false;
      PyUnicode_InternInPlace(&n.name[count++]);
    }
    p = *end ? end + 1 : end;
  }
  if (n.required < 0) n.required = count;
  if (count != Signature<decltype(kFunction)>::kCount) {
    PyErr_Format(PyExc_SystemError, "names of %s", list);
    return false;
  }
  return true;
}

#define ENTRY(f)                                                                            \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(Entry<&f>::run)),         \
   METH_FASTCALL | METH_KEYWORDS, nullptr}

PyMethodDef methods[] = {
    ENTRY(dsa_cache_write),   ENTRY(dsa_cache_read),         ENTRY(sfa_chunk_workspace_size),
    ENTRY(sfa_mla_chunk),     ENTRY(ts_verify_drafts),       ENTRY(dsa_tree_plan),
    ENTRY(dsa_cache_append),  ENTRY(sfa_mla_tree),           ENTRY(ts_verify_tree),
    ENTRY(dsa_cache_keep),    ENTRY(ts_beam_workspace_size), ENTRY(ts_beam_select),
    ENTRY(dsa_cache_fork),    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  const bool named =
      s_data_ptr && s_cuda_stream &&
      name<&dsa_cache_write>("latent latent_stride rope rope_stride slots n cache num_slots fmt | "
                             "err stream") &&
      name<&dsa_cache_read>("cache num_slots fmt block_table table_stride page_size pos ctx_len B k "
                            "sel | err stream") &&
      name<&sfa_chunk_workspace_size>("T B H") &&
      name<&sfa_mla_chunk>("q q_stride cu_q T B H cache num_slots fmt block_table table_stride "
                           "page_size ctx_len ?causal scale out lse ws ws_bytes | err stream") &&
      name<&ts_verify_drafts>("drafts n_draft target target_stride draft draft_stride u B n V "
                              "tokens accepted | err stream") &&
      name<&dsa_tree_plan>("parent cu_q T B ctx_len block_table table_stride page_size num_slots "
                           "pos slots mask words | err stream") &&
      name<&dsa_cache_append>("latent latent_stride rope rope_stride pos slots n freq ?pairs cache "
                              "num_slots fmt q_rope q_rope_stride q_rope_head H q q_stride | err "
                              "stream") &&
      name<&sfa_mla_tree>("q q_stride cu_q T B H cache num_slots fmt block_table table_stride "
                          "page_size ctx_len mask words scale out lse ws ws_bytes | err stream") &&
      name<&ts_verify_tree>("tokens parent cu_q T B target target_stride u V depth path next "
                            "accepted | err stream") &&
      name<&dsa_cache_keep>("cache num_slots fmt block_table table_stride page_size cu_q T ctx_len B "
                            "path depth accepted | new_len err stream") &&
      name<&ts_beam_workspace_size>("B K V n") &&
      name<&ts_beam_select>("logits dtype row_stride cum B K V n tokens parents scores ws ws_bytes | "
                            "err stream") &&
      name<&dsa_cache_fork>("cache num_slots fmt block_table table_stride page_size ctx_len parents "
                            "spare B K n | new_table new_len err stream");
  return named ? PyModule_Create(&module) : nullptr;
}
