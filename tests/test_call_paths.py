"""The two ways from the binding into the library, the generated C extension and ctypes: the same
statuses and the same errors, and the one where the other is missing.  No GPU."""
import ctypes
import os
import shutil
import subprocess
import sys
import sysconfig

import numpy as np
import pytest
import torch

from gqa_attention_lat_gb300 import binding, build

# These addresses are never device memory: run only where no launch could reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer host checks run only without a GPU")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
WAYS = ["extension", "ctypes"]


@pytest.fixture(scope="module", params=WAYS)
def calls(request):
    build.build_library()
    lib = binding.library()
    if request.param == "ctypes":
        return binding._ctypes_calls(lib)
    assert binding._calls().__file__ == binding.CALLER_PATH  # it was built, and is what calls take
    return binding._calls()


def plain(name):
    """Arguments of the right types that the library refuses for its type argument or for a size."""
    return [{ctypes.c_void_p: None, ctypes.c_float: 1.0, ctypes.c_double: 1.0}.get(t, 7)
            for t in binding._SIGNATURES[name][1]]


@pytest.mark.parametrize("name", binding._status_calls())
def test_every_call_takes_its_arguments_and_no_others(calls, name):
    fn, args, types = getattr(calls, name), plain(name), binding._SIGNATURES[name][1]
    assert fn(*args) in (binding.LAT_ERR_INVALID_ARG, binding.LAT_ERR_UNSUPPORTED)
    with pytest.raises(TypeError):
        fn(*args[:-1])
    with pytest.raises(TypeError):
        fn(*args, None)
    for i, t in enumerate(types):
        def given(x):
            return fn(*(args[:i] + [x] + args[i + 1:]))
        if t is ctypes.c_void_p:
            with pytest.raises(AttributeError):
                given("x")
            with pytest.raises(AttributeError):
                given(1.5)
            continue
        with pytest.raises(TypeError):
            given(None)
        if t in (ctypes.c_float, ctypes.c_double):
            given(np.float32(0.5)), given(3)
            continue
        with pytest.raises(TypeError):
            given(1.5)
        given(np.int64(7))
        for x in {ctypes.c_int: (1 << 31, -(1 << 31) - 1, 1 << 70), ctypes.c_int64: (1 << 63, -(1 << 63) - 1),
                  ctypes.c_size_t: (1 << 64, -1), ctypes.c_uint64: (1 << 64, -1)}[t]:
            with pytest.raises(OverflowError):
                given(x)


def test_pointers(calls):
    """None, an address and a tensor: the choice of blocks refuses a missing and an unaligned query,
    and with a good one goes on to refuse its workspace."""
    t = torch.zeros(64, dtype=torch.float32)

    def select(q):
        return calls.lat_attn_select_blocks(binding.LAT_F32, q, 64, FAKE, 128, 128, 128, 16, FAKE, 64, FAKE, 1, 0, 0,
                                            1, 1, 1, 64, None, 0, None, None)
    assert t.data_ptr() % 16 == 0
    assert select(None) == select(t[1:]) == select(FAKE + 4) == binding.LAT_ERR_INVALID_ARG
    assert select(t) == select(t.data_ptr()) == select(FAKE) == binding.LAT_ERR_WORKSPACE


def child(code, **env):
    r = subprocess.run([sys.executable, "-W", "error::ImportWarning", "-c", code], cwd=ROOT, text=True,
                       env=dict(os.environ, **env), capture_output=True)
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


REFUSED = """
try:
    binding.lat_kv_append_q4(9, None, 0, 0, 0, 0, None, None, 0, None, 0, 0, 1, 64)
except binding.LatError as e:
    print(e.status)
print(sorted({l.split()[-1] for l in open('/proc/self/maps') if 'lat_' in l and '.so' in l}))
"""


def test_another_library_than_the_one_beside_it(tmp_path):
    """Sizes and launches come from the library that was asked for, and from no other."""
    build.build_library()
    other = str(tmp_path / "liblat_other.so")
    shutil.copy(binding.LIB_PATH, other)
    out = child("from gqa_attention_lat_gb300 import binding\nbinding.library(%r)\n" % other + REFUSED)
    assert out == [str(binding.LAT_ERR_INVALID_ARG), "['%s']" % other]


def test_a_tree_without_the_extension(tmp_path):
    build.build_library()
    out = child("from gqa_attention_lat_gb300 import binding\nbinding.CALLER_PATH = %r\n" % str(tmp_path / "no.so")
                + REFUSED)
    assert out == [str(binding.LAT_ERR_INVALID_ARG), "['%s']" % binding.LIB_PATH]


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_a_build_that_cannot_make_the_extension(tmp_path, monkeypatch, missing):
    """It warns, leaves none that could be out of date, and the library stands."""
    build.build_library()
    old = tmp_path / "_lat_call.so"
    old.write_bytes(b"older")
    monkeypatch.setattr(build, "CALLER_PATH", str(old))
    if missing == "compiler":
        monkeypatch.setenv("CC", "no-such-compiler")
    else:
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    os.utime(old, (1, 1))  # older than the sources
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build_library() == binding.LIB_PATH
    assert not old.exists() and not build.is_stale()


def test_the_extension_names_its_interpreter():
    assert sysconfig.get_config_var("EXT_SUFFIX") in binding.CALLER_PATH
    assert binding.CALLER_PATH.endswith(".so")
