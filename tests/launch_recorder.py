"""What the entry points for the experts' rows launch, recorded without a device: the host
side of their sources, linked with a HIP runtime that only writes launches down."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import combine_ep_get_amd as ep
from combine_ep_get_amd import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = [s for s in libbuild.MORE_SRC if os.path.basename(s) in ("ep_ffn.hip", "ep_rowops.hip")]
NAMES = ("ep_ffn", "ep_ffn_backward", "ep_combine_backward", "ep_quantize_rows",
         "ep_integer_linear")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    return r.stdout


class Recorder:
    def __init__(self, folder):
        base = [libbuild.HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                "-fPIC", "-I", libbuild.INCLUDE]

        def compiled(src):
            obj = os.path.join(folder, os.path.basename(src) + ".o")
            _run([*base, *(["-x", "hip"] if src.endswith(".cpp") else []), "-c", src, "-o", obj])
            return obj

        with ThreadPoolExecutor(3) as pool:
            objs = list(pool.map(compiled, [*SOURCES, os.path.join(HERE, "c", "launch_recorder.cpp")]))
        # the device code that is not there
        absent = {w for o in objs for w in _run(["nm", "-u", o]).split() if "hip_fatbin" in w}
        lib = os.path.join(folder, "librecorder.so")
        _run(["g++", "-shared", "-Wl,-Bsymbolic", *[f"-Wl,--defsym={a}=0" for a in sorted(absent)],
              *objs, "-o", lib])
        self.lib = ctypes.CDLL(lib)
        self.lib.recorder_kernel.restype = self.lib.recorder_launch.restype = ctypes.c_char_p
        full = ep.lib()
        for name in NAMES:
            getattr(self.lib, name).argtypes = getattr(full, name).argtypes
        self.kernels = sorted(self.lib.recorder_kernel(i).decode()
                              for i in range(self.lib.recorder_kernels()))

    def call(self, name, *args):
        """[(kernel, grid, block)] of one call."""
        self.lib.recorder_clear()
        rc = getattr(self.lib, name)(*args, None)
        assert rc == ep.EP_OK, rc
        out = []
        for i in range(self.lib.recorder_launches()):
            sizes = (ctypes.c_uint32 * 6)()
            kernel = self.lib.recorder_launch(i, sizes).decode()
            out.append((kernel, tuple(sizes[:3]), tuple(sizes[3:])))
        return out

    # made-up addresses, far apart: nothing is read
    def rows(self, n, experts=0, sources=0, per_source=0, capacity=None):
        at = 1 << 44
        cap = capacity or max(n, experts * sources * per_source)
        if not experts:
            return ep.RowsDesc(None, None, cap, 1, 1, 0, n)
        return ep.RowsDesc(None if sources else at, at + (1 << 20), cap, experts, sources or 1,
                           per_source, n)

    def weight(self, i, int8):
        at = i << 44
        return ep.WeightDesc(at, at + (1 << 43) if int8 else None, None,
                             ep.EP_WEIGHT_INT8 if int8 else ep.EP_WEIGHT_BF16, 0)

    def ffn(self, rows, H, I, int8=False):
        a = ep.FfnArgs(2 << 44, self.weight(3, int8), self.weight(4, int8), 5 << 44, None, 6 << 44,
                       H, I)
        return self.call("ep_ffn", ctypes.byref(rows), ctypes.byref(a))

    def backward(self, rows, H, I):
        a = ep.FfnGradArgs(*[i << 44 for i in range(2, 11)], H, I)
        return self.call("ep_ffn_backward", ctypes.byref(rows), ctypes.byref(a))

    def integer(self, rows, C, O, codes=False):
        a = ep.Int8Args(2 << 44, 3 << 44 if codes else None, self.weight(4, True), 5 << 44,
                        6 << 44, C, O)
        return self.call("ep_integer_linear", ctypes.byref(rows), ctypes.byref(a))

    def combine(self, N, K, H, cap):
        p = ep.problem(N, H, K, 64, 1)
        return self.call("ep_combine_backward", ctypes.byref(p), *[i << 44 for i in range(2, 8)],
                         cap)

    def quantize(self, n, cols):
        return self.call("ep_quantize_rows", n, cols, 2 << 44, 3 << 44, 4 << 44)
