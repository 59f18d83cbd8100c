"""Build the lat_attn shared library in-tree with nvcc (sm_103a only).

    python -m gqa_attention_lat_gb300.build          # build if stale
    python -m gqa_attention_lat_gb300.build --force  # rebuild

Each CUDA translation unit compiles in parallel to ``_build/*.o``; the objects link into
``liblat_attn.so`` next to this file (CUDA runtime linked statically, so the library needs
only the NVIDIA driver at run time).  ``_lat_call.*.so`` beside it is the same calls as functions
of a C extension, written out from the binding's signatures: it takes 0.8 us to hand 23
arguments over where ctypes and Python take 4.  Where there is no C compiler or no Python.h it
is left out, with a warning, and the binding calls by ctypes.
"""
from __future__ import annotations

import os
import shlex
import shutil
import subprocess
import sys
import sysconfig
import warnings

from .binding import CALLER_PATH, _SIGNATURES, _status_calls

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblat_attn.so")

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
    files.append(os.path.abspath(__file__))
    return files


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _caller_is_stale() -> bool:
    if not os.path.exists(CALLER_PATH):
        return True
    t = os.path.getmtime(CALLER_PATH)
    return any(os.path.getmtime(f) > t for f in _inputs() + [os.path.join(HERE, "binding.py")])


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
    PyObject *n = PyNumber_Index(x);  /* (the conversion below takes an int alone) */
    if (n == NULL) return 0;
    *v = PyLong_AsUnsignedLongLong(n);
    Py_DECREF(n);
    return *v != UINT64_MAX || !PyErr_Occurred();
}
static int as_f64(PyObject *x, double *v) { return *v = PyFloat_AsDouble(x), *v != -1.0 || !PyErr_Occurred(); }
"""


def _caller_source() -> str:
    """One function per call that returns a status: arguments by position, the status as an int."""
    import ctypes

    kinds = {ctypes.c_void_p: ("void *", "as_ptr", ""), ctypes.c_int64: ("int64_t ", "as_i64", ""),
             ctypes.c_int: ("int ", "as_i32", ""), ctypes.c_float: ("double ", "as_f64", "(float)"),
             ctypes.c_double: ("double ", "as_f64", ""), ctypes.c_size_t: ("uint64_t ", "as_u64", "(size_t)"),
             ctypes.c_uint64: ("uint64_t ", "as_u64", "")}
    out, table = [_CALLER_HEAD], []
    for name in _status_calls():
        args = _SIGNATURES[name][1]
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
    os.makedirs(BUILD, exist_ok=True)
    src = os.path.join(BUILD, "lat_call.c")
    with open(src, "w") as f:
        f.write(_caller_source())
    tmp = CALLER_PATH + ".tmp%d" % os.getpid()
    cmd = shlex.split(os.environ.get("CC") or "gcc") + [
        "-O2", "-shared", "-fPIC", "-Wall", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
        src, "-o", tmp, "-L", HERE, "-l:liblat_attn.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        subprocess.check_call(cmd)
    except (OSError, subprocess.CalledProcessError) as e:  # no compiler, or no Python.h
        if os.path.exists(CALLER_PATH):
            os.remove(CALLER_PATH)  # not to be taken for the one that could not be built
        warnings.warn("%s could not be built (%s): calls go by ctypes, 3 us longer each"
                      % (os.path.basename(CALLER_PATH), e))
        return
    os.replace(tmp, CALLER_PATH)


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if force or is_stale():
        _build_cuda(verbose, extra_flags)
    if force or _caller_is_stale():
        _build_caller(verbose)
    return LIB


def _build_cuda(verbose: bool, extra_flags) -> None:
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


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
