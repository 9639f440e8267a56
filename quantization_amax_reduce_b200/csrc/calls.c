/* CPython calls of the paged KV cache's entry points.
 *
 * These calls take microseconds on the device, and ctypes converts an argument
 * in 0.15 us: 4.6 us for the 31 of fp8attn_kv_tree_fwd, 0.7 us here.  The checks
 * of a small int32 tensor cost 0.9 us in Python and 0.35 us here.  The addresses
 * of the library's functions come from the binding (bind), so this module links
 * against nothing. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>

#include "fp8attn.h"

static __typeof__(&fp8attn_kv_assign_pages) p_assign;
static __typeof__(&fp8attn_kv_write) p_write;
static __typeof__(&fp8attn_kv_write_bf16) p_write_bf16;
static __typeof__(&fp8attn_kv_tree_fwd) p_tree;
static __typeof__(&fp8attn_kv_tree_fwd_bf16) p_tree_bf16;
static __typeof__(&fp8attn_kv_keep_path) p_keep;
static PyObject *tensor_type, *int32_dtype;
static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_numel, *s_data_ptr;

/* Arguments after `spec`, a character each: p pointer, i int, l 64 bits,
 * f float (into *f). */
static int take(PyObject* const* a, Py_ssize_t n, const char* spec, int64_t* v, float* f) {
  Py_ssize_t k = 0;
  for (; spec[k]; ++k) {
    if (k >= n) break;
    if (spec[k] == 'f') {
      const double d = PyFloat_AsDouble(a[k]);
      if (d == -1.0 && PyErr_Occurred()) return 0;
      *f = (float)d;
      continue;
    }
    v[k] = PyLong_AsLongLong(a[k]);
    if (v[k] == -1 && PyErr_Occurred()) return 0;
    if (spec[k] == 'i' && (v[k] < INT_MIN || v[k] > INT_MAX)) {
      PyErr_Format(PyExc_ValueError, "argument %zd does not fit an int", k);
      return 0;
    }
  }
  if (spec[k] || k != n) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return 0;
  }
  return 1;
}

#define PTR(k) ((void*)(intptr_t)v[k])
#define I32(k) ((int)v[k])

static PyObject* assign_pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[17];
  int st;
  (void)self;
  if (!take(a, n, "ppii" "pli" "ppip" "lpppp" "p", v, NULL)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_assign(PTR(0), PTR(1), I32(2), I32(3), PTR(4), v[5], I32(6), PTR(7), PTR(8), I32(9),
                PTR(10), v[11], PTR(12), PTR(13), PTR(14), PTR(15), PTR(16));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* write_kv(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[18];
  int st;
  (void)self;
  if (!take(a, n, "ppllpliipplll" "iippp", v, NULL)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_write(PTR(0), PTR(1), v[2], v[3], PTR(4), v[5], I32(6), I32(7), PTR(8), PTR(9), v[10],
               v[11], v[12], I32(13), I32(14), PTR(15), PTR(16), PTR(17));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* A scale's place in the arguments of the bf16 calls, which take the same
 * ones: it must be 0. */
static int no_scale(int64_t scale) {
  if (scale) PyErr_SetString(PyExc_ValueError, "a bf16 cache takes no scale");
  return !scale;
}

static PyObject* write_bf16(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[18];
  int st;
  (void)self;
  if (!take(a, n, "ppllpliipplll" "iippp", v, NULL) || !no_scale(v[15])) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_write_bf16(PTR(0), PTR(1), v[2], v[3], PTR(4), v[5], I32(6), I32(7), PTR(8), PTR(9),
                    v[10], v[11], v[12], I32(13), I32(14), PTR(16), PTR(17));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* tree_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[31];
  float scale = 0.0f;
  int st;
  (void)self;
  if (!take(a, n, "pllpplll" "ii" "pli" "pp" "iii" "liii" "ppi" "f" "pplpp", v, &scale)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_tree(PTR(0), v[1], v[2], PTR(3), PTR(4), v[5], v[6], v[7], I32(8), I32(9), PTR(10),
              v[11], I32(12), PTR(13), PTR(14), I32(15), I32(16), I32(17), v[18], I32(19),
              I32(20), I32(21), PTR(22), PTR(23), I32(24), scale, PTR(26), PTR(27),
              (size_t)v[28], PTR(29), PTR(30));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* tree_fwd_bf16(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[31];
  float scale = 0.0f;
  int st;
  (void)self;
  if (!take(a, n, "pllpplll" "ii" "pli" "pp" "iii" "liii" "ppi" "f" "pplpp", v, &scale) ||
      !no_scale(v[22]))
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_tree_bf16(PTR(0), v[1], v[2], PTR(3), PTR(4), v[5], v[6], v[7], I32(8), I32(9), PTR(10),
                   v[11], I32(12), PTR(13), PTR(14), I32(15), I32(16), I32(17), v[18], I32(19),
                   I32(20), I32(21), PTR(23), I32(24), scale, PTR(26), PTR(27), (size_t)v[28],
                   PTR(29), PTR(30));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* keep_path(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[22];
  int st;
  (void)self;
  if (!take(a, n, "pplll" "iiiii" "pli" "ppi" "pli" "ppp", v, NULL)) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = p_keep(PTR(0), PTR(1), v[2], v[3], v[4], I32(5), I32(6), I32(7), I32(8), I32(9), PTR(10),
              v[11], I32(12), PTR(13), PTR(14), I32(15), PTR(16), v[17], I32(18), PTR(19), PTR(20),
              PTR(21));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* t.method() as a number; -2 with an error set if that fails. */
static long long number(PyObject* t, PyObject* method) {
  PyObject* r = PyObject_CallMethodNoArgs(t, method);
  if (!r) return -2;
  const long long x = PyLong_AsLongLong(r);   /* (True counts as 1) */
  Py_DECREF(r);
  return x == -1 && PyErr_Occurred() ? -2 : x;
}

/* int32_ptr(t, name, device, numel): pointer of a contiguous int32 tensor on
 * CUDA device `device`, of `numel` elements unless that is negative. */
static PyObject* int32_ptr(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[4];
  (void)self;
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "int32_ptr(t, name, device, numel)");
    return NULL;
  }
  if (!take(a + 2, 2, "ll", v, NULL)) return NULL;
  PyObject* t = a[0];
  int ok = PyObject_TypeCheck(t, (PyTypeObject*)tensor_type);
  if (ok) {
    PyObject* dtype = PyObject_GetAttr(t, s_dtype);
    if (!dtype) return NULL;
    ok = dtype == int32_dtype;
    Py_DECREF(dtype);
  }
  if (ok) {
    const long long on = number(t, s_get_device);
    if (on == -2) return NULL;
    ok = on == v[0];
  }
  if (!ok)
    return PyErr_Format(PyExc_ValueError, "%U must be an int32 tensor on cuda:%lld", a[1],
                        (long long)v[0]);
  const long long whole = number(t, s_is_contiguous);
  if (whole == -2) return NULL;
  ok = whole == 1;
  if (ok && v[1] >= 0) {
    const long long have = number(t, s_numel);
    if (have == -2) return NULL;
    ok = have == v[1];
  }
  if (!ok)
    return v[1] >= 0 ? PyErr_Format(PyExc_ValueError, "%U must be contiguous and hold %lld elements",
                                    a[1], (long long)v[1])
                     : PyErr_Format(PyExc_ValueError, "%U must be contiguous", a[1]);
  return PyObject_CallMethodNoArgs(t, s_data_ptr);
}

/* bind(assign_pages, write, write_bf16, tree_fwd, tree_fwd_bf16, keep_path,
 *      torch.Tensor, torch.int32) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t v[6];
  (void)self;
  if (n != 8 || !PyType_Check(a[6])) {
    PyErr_SetString(PyExc_TypeError, "bind(six addresses, tensor type, int32)");
    return NULL;
  }
  if (!take(a, 6, "pppppp", v, NULL)) return NULL;
  p_assign = (__typeof__(p_assign))(intptr_t)v[0];
  p_write = (__typeof__(p_write))(intptr_t)v[1];
  p_write_bf16 = (__typeof__(p_write_bf16))(intptr_t)v[2];
  p_tree = (__typeof__(p_tree))(intptr_t)v[3];
  p_tree_bf16 = (__typeof__(p_tree_bf16))(intptr_t)v[4];
  p_keep = (__typeof__(p_keep))(intptr_t)v[5];
  Py_INCREF(a[6]);
  Py_XSETREF(tensor_type, a[6]);
  Py_INCREF(a[7]);
  Py_XSETREF(int32_dtype, a[7]);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"assign_pages", (PyCFunction)(void (*)(void))assign_pages, METH_FASTCALL, NULL},
    {"write", (PyCFunction)(void (*)(void))write_kv, METH_FASTCALL, NULL},
    {"write_bf16", (PyCFunction)(void (*)(void))write_bf16, METH_FASTCALL, NULL},
    {"tree_fwd", (PyCFunction)(void (*)(void))tree_fwd, METH_FASTCALL, NULL},
    {"tree_fwd_bf16", (PyCFunction)(void (*)(void))tree_fwd_bf16, METH_FASTCALL, NULL},
    {"keep_path", (PyCFunction)(void (*)(void))keep_path, METH_FASTCALL, NULL},
    {"int32_ptr", (PyCFunction)(void (*)(void))int32_ptr, METH_FASTCALL, NULL},
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_numel = PyUnicode_InternFromString("numel");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_get_device || !s_is_contiguous || !s_numel || !s_data_ptr) return NULL;
  return PyModule_Create(&module);
}
