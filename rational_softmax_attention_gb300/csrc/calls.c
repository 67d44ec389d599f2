/* The serving calls of include/raattn.h as a Python module.  A single token's kernels run for a few
 * microseconds, and ctypes takes four to six to convert a call's 20 to 30 arguments; this takes less than one.
 * Arguments are positional: addresses as int (None: NULL), numbers as int or float; the result is the
 * ra_status_t.  The interpreter is free while a call runs. */
#define PY_SSIZE_T_CLEAN
#define Py_LIMITED_API 0x030a0000
#include <Python.h>
#include <limits.h>
#include <string.h>

#include "raattn.h"

#define MOST 40

typedef union {
  void* p;
  int i;
  int64_t q;
  float f;
} slot;

/* p: address, i: int, q: int64_t, f: float */
static int take(PyObject* const* args, Py_ssize_t n, const char* kinds, slot* s) {
  if (n != (Py_ssize_t)strlen(kinds)) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, (Py_ssize_t)strlen(kinds));
    return -1;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    PyObject* a = args[k];
    if (kinds[k] == 'p') {
      s[k].p = a == Py_None ? NULL : PyLong_AsVoidPtr(a);
    } else if (kinds[k] == 'f') {
      s[k].f = (float)PyFloat_AsDouble(a);
    } else {
      const long long v = PyLong_AsLongLong(a);
      if (kinds[k] == 'i' && (v < INT_MIN || v > INT_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "a size is beyond int32");
        return -1;
      }
      if (kinds[k] == 'i') s[k].i = (int)v;
      else s[k].q = v;
    }
  }
  return PyErr_Occurred() ? -1 : 0;
}

#define ENTRY(NAME, KINDS, CALL)                                                  \
  static PyObject* py_##NAME(PyObject* self, PyObject* const* args, Py_ssize_t n) { \
    slot s[MOST];                                                                 \
    ra_status_t code;                                                             \
    (void)self;                                                                   \
    if (take(args, n, KINDS, s) < 0) return NULL;                                 \
    Py_BEGIN_ALLOW_THREADS code = CALL;                                           \
    Py_END_ALLOW_THREADS return PyLong_FromLong((long)code);                      \
  }

ENTRY(ra_qk_norm_rope_fwd, "pqqppppifppqqpiipppppiiiiiiip",
      ra_qk_norm_rope_fwd(s[0].p, s[1].q, s[2].q, s[3].p, s[4].p, s[5].p, s[6].p, (ra_norm_t)s[7].i, s[8].f, s[9].p,
                          s[10].p, s[11].q, s[12].q, s[13].p, s[14].i, s[15].i, s[16].p, s[17].p, s[18].p, s[19].p,
                          s[20].p, s[21].i, s[22].i, s[23].i, s[24].i, s[25].i, s[26].i, (ra_dtype_t)s[27].i, s[28].p))
ENTRY(ra_qk_norm_rope_bwd, "pqqppppifppqqpiippppppiiiiiip",
      ra_qk_norm_rope_bwd(s[0].p, s[1].q, s[2].q, s[3].p, s[4].p, s[5].p, s[6].p, (ra_norm_t)s[7].i, s[8].f, s[9].p,
                          s[10].p, s[11].q, s[12].q, s[13].p, s[14].i, s[15].i, s[16].p, s[17].p, s[18].p, s[19].p,
                          s[20].p, s[21].p, s[22].i, s[23].i, s[24].i, s[25].i, s[26].i, (ra_dtype_t)s[27].i, s[28].p))
ENTRY(ra_attention_decode, "pppppppppiiiiiifip",
      ra_attention_decode(s[0].p, s[1].p, s[2].p, s[3].p, s[4].p, s[5].p, s[6].p, s[7].p, s[8].p, s[9].i, s[10].i,
                          s[11].i, s[12].i, s[13].i, s[14].i, s[15].f, (ra_dtype_t)s[16].i, s[17].p))
ENTRY(ra_cache_evict, "pppppppppiiiiiiiip",
      ra_cache_evict(s[0].p, s[1].p, s[2].p, s[3].p, s[4].p, s[5].p, s[6].p, s[7].p, s[8].p, s[9].i, s[10].i, s[11].i,
                     s[12].i, s[13].i, s[14].i, s[15].i, (ra_dtype_t)s[16].i, s[17].p))

#define METHOD(NAME) {#NAME, (PyCFunction)(void (*)(void))py_##NAME, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(ra_qk_norm_rope_fwd), METHOD(ra_qk_norm_rope_bwd), METHOD(ra_attention_decode),
                                METHOD(ra_cache_evict), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
