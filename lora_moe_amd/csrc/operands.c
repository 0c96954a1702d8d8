/* A library call from Python with its tensors looked at on the way.
 *
 * call(function, shape, args, device, kind) takes the address of a library
 * function, the shape structure (a buffer), which function it is (kinds[name];
 * left out: one that takes 17 pointers) and its further arguments: None
 * (a null pointer), an int, or a tuple (name, tensor, sizes, type) for a
 * tensor's address.  Every tensor has to have those sizes and that type (torch's
 * name of it), to be contiguous and to lie in memory of the given HIP device.  Sizes None:
 * a workspace, one-dimensional, whose bytes are the next argument.  It returns
 * the function's status, or None, without having called it, when something is
 * not so: the caller then finds out what, at leisure, and says it.
 *
 * Tensors are seen through DLPack's C exchange functions, which torch.Tensor
 * offers, so that one costs 0.1 us where the same questions asked one by one in
 * Python cost 1.2 us, several times what a small call's kernel takes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include <ATen/dlpack.h>

#include "moe_lora.h"

enum { MOST = 16 };

/* The functions by kind, and their arguments behind the shape: each is called
 * through its own type. */
enum { SORT, SORT_BACKWARD, UNSORT, UNSORT_BACKWARD, ROUTE_BACKWARD, PROJ_FORWARD, PROJ_BACKWARD, KINDS };
static const struct {
  const char* name;
  int args;
} functions[KINDS] = {{"moe_lora_sort", 9},           {"moe_lora_sort_backward", 4},  {"moe_lora_unsort", 5},
                      {"moe_lora_unsort_backward", 7}, {"moe_lora_route_backward", 5}, {"moe_lora_proj_forward", 11},
                      {"moe_lora_proj_backward", 14}};

typedef int (*pointers17)(const void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*,
                          void*, void*, void*, void*, void*);

static int run(int kind, uintptr_t f, const void* s, const uintptr_t* a) {
#define P(i) ((void*)a[i])
#define F(name) ((__typeof__(&name))f)
  switch (kind) {
    case SORT: return F(moe_lora_sort)(s, P(0), P(1), P(2), a[3], P(4), P(5), P(6), P(7), P(8));
    case SORT_BACKWARD: return F(moe_lora_sort_backward)(s, P(0), P(1), P(2), P(3));
    case UNSORT: return F(moe_lora_unsort)(s, P(0), P(1), P(2), P(3), P(4));
    case UNSORT_BACKWARD: return F(moe_lora_unsort_backward)(s, P(0), P(1), P(2), P(3), P(4), P(5), P(6));
    case ROUTE_BACKWARD: return F(moe_lora_route_backward)(s, P(0), P(1), P(2), P(3), P(4));
    case PROJ_FORWARD:
      return F(moe_lora_proj_forward)(s, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), a[8], P(9), P(10));
    case PROJ_BACKWARD:
      return F(moe_lora_proj_backward)(s, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), P(8), a[9], P(10), P(11),
                                       P(12), P(13));
  }
  return ((pointers17)f)(s, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), P(8), P(9), P(10), P(11), P(12), P(13),
                         P(14), P(15));
#undef F
#undef P
}

static const DLPackExchangeAPI* api;

static int is_type(DLDataType t, const char* name) {
  if (t.lanes != 1) return 0;
  if (!strcmp(name, "bfloat16")) return t.code == kDLBfloat && t.bits == 16;
  if (!strcmp(name, "float16")) return t.code == kDLFloat && t.bits == 16;
  if (!strcmp(name, "float32")) return t.code == kDLFloat && t.bits == 32;
  if (!strcmp(name, "int32")) return t.code == kDLInt && t.bits == 32;
  if (!strcmp(name, "uint8")) return t.code == kDLUInt && t.bits == 8;
  return 0;
}

/* The tensor's address if it is what the spec says: 1; else 0. */
static int address_of(PyObject* spec, int device, uintptr_t* out) {
  PyObject *tensor = PyTuple_GET_ITEM(spec, 1), *sizes = PyTuple_GET_ITEM(spec, 2);
  const char* type = PyUnicode_AsUTF8(PyTuple_GET_ITEM(spec, 3));
  DLTensor t;
  if (!type || tensor == Py_None) return 0;
  if (api->dltensor_from_py_object_no_sync(tensor, &t)) return 0;
  if (t.device.device_type != kDLROCM || t.device.device_id != device || !is_type(t.dtype, type)) return 0;
  if (sizes == Py_None) {
    if (t.ndim != 1) return 0;
    out[1] = (uintptr_t)t.shape[0];
  } else {
    if (!PyTuple_Check(sizes) || PyTuple_GET_SIZE(sizes) != t.ndim) return 0;
    for (int i = 0; i < t.ndim; ++i)
      if (PyLong_AsLongLong(PyTuple_GET_ITEM(sizes, i)) != t.shape[i]) return 0;
  }
  int64_t n = 1;
  int empty = 0, dense = 1;
  for (int i = t.ndim - 1; i >= 0; --i) {
    if (t.shape[i] == 0) empty = 1;
    if (t.strides && t.shape[i] != 1 && t.strides[i] != n) dense = 0;
    n *= t.shape[i];
  }
  /* a tensor without memory (torch's zeros that are none, fake tensors) would
   * pass for an argument that is not given */
  if (!empty && (!dense || !t.data)) return 0;
  *out = (uintptr_t)t.data + t.byte_offset;
  return 1;
}

static PyObject* call(PyObject* self, PyObject* const* argv, Py_ssize_t argc) {
  (void)self;
  if ((argc != 4 && argc != 5) || !PyTuple_Check(argv[2])) {
    PyErr_SetString(PyExc_TypeError, "call(function, shape, args, device, kind)");
    return NULL;
  }
  const uintptr_t f = (uintptr_t)PyLong_AsUnsignedLongLong(argv[0]);
  const long device = PyLong_AsLong(argv[3]);
  const Py_ssize_t n = PyTuple_GET_SIZE(argv[2]);
  const long kind = argc == 5 ? PyLong_AsLong(argv[4]) : KINDS;
  if (PyErr_Occurred()) return NULL;
  if (kind < 0 || kind > KINDS || (kind < KINDS ? n != functions[kind].args : n >= MOST)) {
    PyErr_SetString(PyExc_TypeError, "call: no such function, or not as many arguments as it takes");
    return NULL;
  }
  uintptr_t a[MOST] = {0};
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* v = PyTuple_GET_ITEM(argv[2], i);
    if (v == Py_None) continue;
    if (PyTuple_Check(v)) {
      if (PyTuple_GET_SIZE(v) != 4 || !address_of(v, (int)device, a + i)) {
        PyErr_Clear();
        Py_RETURN_NONE;
      }
      if (PyTuple_GET_ITEM(v, 2) == Py_None) ++i;  /* its bytes */
    } else {
      a[i] = (uintptr_t)PyLong_AsUnsignedLongLong(v);
      if (PyErr_Occurred()) return NULL;
    }
  }
  Py_buffer shape;
  if (PyObject_GetBuffer(argv[1], &shape, PyBUF_SIMPLE)) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = run((int)kind, f, shape.buf, a);
  Py_END_ALLOW_THREADS
  PyBuffer_Release(&shape);
  return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {{"call", (PyCFunction)(void*)call, METH_FASTCALL, "see operands.c"}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operands", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__operands(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* tensor = torch ? PyObject_GetAttrString(torch, "Tensor") : NULL;
  PyObject* capsule = tensor ? PyObject_GetAttrString(tensor, "__dlpack_c_exchange_api__") : NULL;
  if (capsule) api = (const DLPackExchangeAPI*)PyCapsule_GetPointer(capsule, "dlpack_exchange_api");
  Py_XDECREF(capsule);
  Py_XDECREF(tensor);
  Py_XDECREF(torch);
  if (!api) return NULL;
  if (api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync) {
    PyErr_SetString(PyExc_ImportError, "torch's DLPack exchange functions are of another version");
    return NULL;
  }
  PyObject *m = PyModule_Create(&module), *kinds = PyDict_New();
  for (int i = 0; kinds && i < KINDS; ++i) {
    PyObject* v = PyLong_FromLong(i);
    if (!v || PyDict_SetItemString(kinds, functions[i].name, v)) Py_CLEAR(kinds);
    Py_XDECREF(v);
  }
  if (!m || !kinds || PyModule_AddObject(m, "kinds", kinds)) {  /* (takes kinds over where it succeeds) */
    Py_XDECREF(kinds);
    Py_XDECREF(m);
    return NULL;
  }
  return m;
}
