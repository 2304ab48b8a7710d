"""libdpclip's host side on a stand-in for the CUDA runtime (tests/native/fake_cudart.cpp): the binding's
functions then validate, plan and "launch" without a GPU, whatever machine the tests run on."""
import contextlib
import ctypes
import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "native", "fake_cudart.cpp")
OUT = os.path.join(HERE, "_build", "libdpclip_host.so")
STREAM = 4096   # a stream handle that is never followed
PTR = 1 << 20   # a device pointer that is never followed, on a 16-byte boundary


def _build():
    import __graft_entry__
    __graft_entry__.build()
    objs = sorted(glob.glob(os.path.join(ROOT, "_build", "dpclip", "*.o")))
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    if not os.path.exists(OUT) or any(os.path.getmtime(f) > os.path.getmtime(OUT) for f in objs + [SRC]):
        tmp = f"{OUT}.{os.getpid()}"
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I/usr/local/cuda/include",
                        SRC, *objs, "-o", tmp], check=True)
        os.replace(tmp, OUT)


class Host:
    """The package with its library replaced, and the stand-in's log."""

    def __init__(self):
        _build()
        import example_gradient_clipping_gb300 as dp
        self.dp, self.real = dp, dp._lib
        self.so = ctypes.CDLL(OUT)
        for name in vars(dp._lib):
            f = getattr(dp._lib, name)
            if name.startswith("dp_"):
                g = getattr(self.so, name)
                g.restype, g.argtypes = f.restype, f.argtypes
        self.so.fake_kernel.restype = ctypes.c_char_p
        self.so.fake_capture.argtypes = self.so.fake_join.argtypes = [ctypes.c_ulonglong] * 2
        self.hook_type = ctypes.CFUNCTYPE(None)

    @contextlib.contextmanager
    def installed(self):
        self.so.fake_clear()
        self.so.fake_device(0)
        self.dp._lib = self.dp.sequence._lib = self.so
        try:
            yield self
        finally:
            self.dp._lib = self.dp.sequence._lib = self.real

    def launches(self):
        """[(kernel, stream, device, starts under the launch before it, status)] since the last call."""
        out = []
        for i in range(self.so.fake_launches()):
            stream, dev, smem, status = ctypes.c_ulonglong(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
            early = self.so.fake_launch(i, ctypes.byref(stream), ctypes.byref(dev), ctypes.byref(smem),
                                        ctypes.byref(status))
            out.append((self.so.fake_kernel(i).decode(), stream.value, dev.value, bool(early), status.value))
        self.so.fake_clear()
        return out
