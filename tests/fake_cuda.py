"""The dense operators' host code over a CUDA runtime that launches nothing (fake_cuda.cpp), so
that what a call asks of the runtime, and in which order, can be tested without a GPU."""

import ctypes as C
import os
import subprocess

from collective_datapath_copy_gb300 import _lib
from collective_datapath_copy_gb300 import build as b

OBJECTS = [s + ".o" for s in b.CU_SOURCES if s.startswith("dense")]


_built = None


def load(folder):
    """libdense over the fake runtime, in `folder`: a fresh one for every folder."""
    global _built
    out = os.path.join(folder, "libdense_fake.so")
    if _built is None:
        _link(out)
        with open(out, "rb") as f:
            _built = f.read()
    else:
        with open(out, "wb") as f:
            f.write(_built)
    h = C.CDLL(out)
    for name, (res, args) in _lib._SIGS.items():
        if hasattr(h, name):
            getattr(h, name).restype, getattr(h, name).argtypes = res, args
    h.fake_launch_kernel.restype = C.c_char_p
    return h


def _link(out):
    b.build()
    objs = [os.path.join(b.BUILD, o) for o in OBJECTS]
    if not all(os.path.exists(o) for o in objs):
        b.build(force=True)
    here = os.path.dirname(os.path.abspath(__file__))
    toolkit = os.path.dirname(os.path.dirname(b._nvcc()))
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC",
                    "-Wl,-z,defs", "-Wl,-Bsymbolic", f"-I{toolkit}/include",
                    os.path.join(here, "fake_cuda.cpp"), *objs, "-o", out], check=True)


def launches(h):
    """(kernel, device) of every launch since the last reset."""
    return [(h.fake_launch_kernel(i).decode(), h.fake_launch_device(i))
            for i in range(h.fake_launches())]
