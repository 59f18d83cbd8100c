"""Build the lat_attn shared library in-tree with nvcc (sm_103a only).

    python -m gqa_attention_lat_gb300.build          # build if stale
    python -m gqa_attention_lat_gb300.build --force  # rebuild

Each CUDA translation unit compiles in parallel to ``_build/*.o``; the objects link into
``liblat_attn.so`` next to this file (CUDA runtime linked statically, so the library needs
only the NVIDIA driver at run time).  ``_lat_call.so`` beside it is the same calls as functions
of a C extension, written out from the binding's signatures: it takes 0.8 us to hand 23
arguments over where ctypes and Python take 4.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblat_attn.so")
CALLER = os.path.join(HERE, "_lat_call.so")

SOURCES = ["api.cu", "kv_append.cu", "row_attention_f32.cu", "decode_bf16.cu", "prefill_tc.cu",
           "decode_static.cu", "qkv_producer.cu", "kv_q4.cu", "decode_q4.cu",
           "block_select.cu", "decode_blocks_f32.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                 "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files += [os.path.abspath(__file__), os.path.join(HERE, "binding.py")]
    return files


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLER):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLER))
    return any(os.path.getmtime(f) > t for f in _inputs())


_CALLER_HEAD = """\
/* Written by build.py from the signatures of binding.py; not to be edited. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include "lat_attn.h"
#include "lat_attn_testing.h"

static PyObject *s_data_ptr;

/* NULL for None, an address for an int, x.data_ptr() for a tensor */
static int as_ptr(PyObject *x, void **p) {
    if (x == Py_None) return *p = NULL, 1;
    if (PyLong_Check(x)) return *p = PyLong_AsVoidPtr(x), *p != NULL || !PyErr_Occurred();
    PyObject *a = PyObject_CallMethodNoArgs(x, s_data_ptr);
    if (a == NULL) return 0;
    *p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return *p != NULL || !PyErr_Occurred();
}
static int as_i64(PyObject *x, int64_t *v) { return *v = PyLong_AsLongLong(x), *v != -1 || !PyErr_Occurred(); }
static int as_i32(PyObject *x, int *v) {
    int64_t w;
    if (!as_i64(x, &w)) return 0;
    if (w < INT32_MIN || w > INT32_MAX) return PyErr_SetString(PyExc_OverflowError, "argument exceeds 32 bits"), 0;
    return *v = (int)w, 1;
}
static int as_u64(PyObject *x, uint64_t *v) {
    return *v = PyLong_AsUnsignedLongLong(x), *v != UINT64_MAX || !PyErr_Occurred();
}
static int as_f64(PyObject *x, double *v) { return *v = PyFloat_AsDouble(x), *v != -1.0 || !PyErr_Occurred(); }
"""


def _caller_source() -> str:
    """One function per call that returns a status: arguments by position, the status as an int."""
    import ctypes

    from .binding import _SIGNATURES

    kinds = {ctypes.c_void_p: ("void *", "as_ptr", ""), ctypes.c_int64: ("int64_t ", "as_i64", ""),
             ctypes.c_int: ("int ", "as_i32", ""), ctypes.c_float: ("double ", "as_f64", "(float)"),
             ctypes.c_double: ("double ", "as_f64", ""), ctypes.c_size_t: ("uint64_t ", "as_u64", "(size_t)"),
             ctypes.c_uint64: ("uint64_t ", "as_u64", "")}
    out, table = [_CALLER_HEAD], []
    for name, (res, args) in _SIGNATURES.items():
        if res is not ctypes.c_int or len(args) < 2:  # sizes and names: not on a hot path
            continue
        decl = " ".join("%sa%d;" % (kinds[t][0], i) for i, t in enumerate(args))
        take = " || ".join("!%s(v[%d], &a%d)" % (kinds[t][1], i, i) for i, t in enumerate(args))
        give = ", ".join("%sa%d" % (kinds[t][2], i) for i, t in enumerate(args))
        out.append("""
static PyObject *w_%s(PyObject *self, PyObject *const *v, Py_ssize_t n) {
    (void)self;
    if (n != %d) return PyErr_Format(PyExc_TypeError, "%s takes %d arguments, got %%zd", n);
    %s
    if (%s) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = (int)%s(%s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}
""" % (name, len(args), name, len(args), decl, take, name, give))
        table.append('    {"%s", (PyCFunction)(void (*)(void))w_%s, METH_FASTCALL, NULL},\n' % (name, name))
    out.append("""
static PyMethodDef methods[] = {
%s    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lat_call", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__lat_call(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    return s_data_ptr == NULL ? NULL : PyModule_Create(&module);
}
""" % "".join(table))
    return "".join(out)


def _build_caller(verbose: bool) -> None:
    src = os.path.join(BUILD, "lat_call.c")
    with open(src, "w") as f:
        f.write(_caller_source())
    tmp = CALLER + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CC") or "gcc", "-O2", "-shared", "-fPIC", "-Wall", "-I", INCLUDE, "-I",
           sysconfig.get_paths()["include"], src, "-o", tmp, "-L", HERE, "-l:liblat_attn.so",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, CALLER)


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc] + CFLAGS + list(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT)))
    failed = []
    objs = []
    for src, obj, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stdout.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
        objs.append(obj)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    _build_caller(verbose)
    return LIB


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
