"""Builds tests/product_forms.cu: the products' kernels with their form given.
Test infrastructure."""
import ctypes
import os
import subprocess

from allreduce_residual_rmsnorm_gb300 import build as BUILD

HERE = os.path.dirname(os.path.abspath(__file__))


def load(out_dir, wait_ns, alone=False):
    """The library's kernels and status words, the limit holding for lone_wait; or,
    `alone`, the kernels built anew with that limit for all of their waits."""
    BUILD.build()
    so = os.path.join(str(out_dir), "alone.so" if alone else "linked.so")
    where = os.path.dirname(BUILD.LIB)
    cmd = [BUILD.nvcc(), *BUILD.ARCH, *BUILD.NVCC_FLAGS, "-shared", "-cudart", "shared",
           "-Xlinker", f"-rpath,{BUILD.cuda_lib_dir()}", f"-DARF_WAIT_NS={wait_ns}ull", "-DARF_WAIT_TRIES=1u",
           '-DARF_WAIT_TRY="test_wait"', "-o", so,
           os.path.join(HERE, "product_forms.cu")]
    if alone:
        cmd += ["-Darf=arf_alone", "-DPRODUCT_FORMS_ALONE", "--threads", "0"]
        cmd += [os.path.join(BUILD.CSRC, f) for f in
                ("matmul_fp8.cu", "matmul_narrow.cu", "matmul_wide.cu")]
    else:
        cmd += ["-L", where, "-l:" + os.path.basename(BUILD.LIB), "-Xlinker", f"-rpath,{where}"]
    subprocess.run(cmd, check=True)
    L = ctypes.CDLL(so)
    p, i = ctypes.c_void_p, ctypes.c_int
    L.product_form.argtypes = [p, p, p, p, p, i, i, i, i, i, p, i, i, p]
    L.lone_wait.argtypes = [i, p]
    L.product_choice.argtypes = [i, i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.product_choice.restype = None
    L.ar_fusion_matmul_status.argtypes = [p, ctypes.POINTER(i)]
    return L


def status(L):
    """(status, detail) of the kernels behind L, cleared by the query."""
    d = ctypes.c_int(-1)
    return L.ar_fusion_matmul_status(None, ctypes.byref(d)), d.value


def choice(L, rows, cols, depth, experts=1, sms=152):
    """(tokens, split) of the form that a call of these sizes takes; (0, 0) is the
    kernel for many rows."""
    t, s = ctypes.c_int(-1), ctypes.c_int(-1)
    L.product_choice(experts, rows, cols, depth, sms, ctypes.byref(t), ctypes.byref(s))
    return t.value, s.value
