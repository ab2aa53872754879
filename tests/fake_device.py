"""The library's boundary on a stand-in for the device (fake_device.cc), for host tests."""

import ctypes
import os
import subprocess

from token_sparse_denoising_layer_b200 import abi, build

HERE = os.path.dirname(os.path.abspath(__file__))


def load(folder, monkeypatch):
    """Build api.cu with fake_device.cc in `folder` and have the binding use it."""
    api, fake, lib = (os.path.join(str(folder), n) for n in ("api.o", "fake.o", "libhsa_fake.so"))
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    for cmd in ([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                 "-c", os.path.join(build.CSRC, "api.cu"), "-o", api],
                ["g++", "-std=c++17", "-O1", "-fPIC", "-Wno-attributes", "-I", cuda, "-c",
                 os.path.join(HERE, "fake_device.cc"), "-o", fake],
                # its own names come first: the process may hold the real runtime too
                ["g++", "-shared", "-o", lib, api, fake, "-Wl,-Bsymbolic", "-Wl,-z,defs"]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{' '.join(cmd)}:\n{r.stderr[-4000:]}")
    monkeypatch.setattr(abi, "_lib", None)
    monkeypatch.setattr(abi, "LIB_PATH", lib)
    fake = abi.load()
    fake.fake_turns.restype = ctypes.POINTER(ctypes.c_uint64)
    return fake
