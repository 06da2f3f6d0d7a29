"""The library's host side without a GPU: its object files linked against the runtime of
tests/fake_cudart.cpp, which records allocations, clears and launches and runs nothing."""
import ctypes
import glob
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Fake:
    def __init__(self, folder):
        from dense_gemm_blackwell_02_gb300 import build
        build.build()
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
        so = os.path.join(str(folder), "libgemm_fake.so")
        pattern = os.path.join(build.BUILD_DIR, "*.cu.o")
        if len(glob.glob(pattern)) < len(build._sources()):  # (a library without its objects)
            build.build(force=True)
        objects = sorted(glob.glob(pattern))
        # (-Bsymbolic: the runtime of this file, whatever other one the process has loaded)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I",
                               os.path.join(cuda, "include"), "-o", so,
                               os.path.join(ROOT, "tests", "fake_cudart.cpp")] + objects)
        self.lib = ctypes.CDLL(so)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        self.lib.fake_journal.restype = ctypes.c_char_p
        self.lib.fake_fail.argtypes = [ctypes.c_char_p]
        self.lib.fake_largest.argtypes = [ctypes.c_size_t]
        self.lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
        self.lib.gemm_destroy.argtypes = [vp]
        self.lib.gemm_run.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
        self.lib.gemm_device_status.argtypes = [vp, vp, vp]

    def create(self):
        h = ctypes.c_void_p()
        assert self.lib.gemm_create(ctypes.byref(h)) == 0
        return h

    def journal(self, clear=True):
        """[(what, address, bytes, stream, name)] since the last time."""
        lines = self.lib.fake_journal().decode().splitlines()
        if clear:
            self.lib.fake_clear()
        rows = [line.split(" ", 4) for line in lines]
        return [(w, int(p, 16), int(n), int(s, 16), name) for w, p, n, s, name in rows]

    # Operands are addresses that nothing follows.
    def run(self, h, M, N, K, stream=0, dtype=1, out=1):
        return self.lib.gemm_run(h, 1 << 20, 2 << 20, 3 << 20, M, N, K, dtype, out, stream)

    def run_adapters(self, h, M, N, K, rank, count, stream=0, dtype=1, out=1):
        from dense_gemm_blackwell_02_gb300.binding import _ADAPTERS_CALL
        return self.lib.gemm_run_adapters_packed(_ADAPTERS_CALL.pack(
            h.value, 1 << 20, 2 << 20, 3 << 20, M, N, K, 4 << 20, stream, dtype, out, 5 << 20, 6 << 20,
            0, count, rank))

    def rotary(self, h, tokens, heads, dim, x, y, pairs=4, in_place=False, dtype=1):
        """x and y: (token stride, head stride) in elements."""
        from dense_gemm_blackwell_02_gb300.binding import _ROTARY_CALL
        return self.lib.gemm_rotary_packed(_ROTARY_CALL.pack(
            h.value, 1 << 20, 1 << 20 if in_place else 2 << 20, tokens, heads, dim, *x, *y, 0, 3 << 20,
            4 << 20, 5 << 20, 0, 100, 1, 2 * pairs, 0, 0, dtype, 0))
