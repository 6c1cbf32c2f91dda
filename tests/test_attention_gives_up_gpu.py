"""Prompt kernels whose waits give up after a nanosecond do give up, in every form: what
test_attention_waits_gpu.py looks at (an answer that is right or reported) includes the reported one."""
import ctypes
import os
import subprocess

import pytest
import torch

import attention_ref as R
from allreduce_residual_rmsnorm_gb300 import binding as B
from allreduce_residual_rmsnorm_gb300 import build as BUILD

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def hasty(cuda_lib, tmp_path_factory):
    so = os.path.join(str(tmp_path_factory.mktemp("hasty")), "alone.so")
    cmd = [BUILD.nvcc(), *BUILD.ARCH, *BUILD.NVCC_FLAGS, "-shared", "-cudart", "shared", "-Xlinker",
           f"-rpath,{BUILD.cuda_lib_dir()}", "-DARF_WAIT_NS=1ull", "-DARF_WAIT_TRIES=1u",
           '-DARF_WAIT_TRY="test_wait"', "-Darf=arf_alone", "--threads", "0", "-o", so,
           os.path.join(HERE, "attention_alone.cu")]
    cmd += [os.path.join(BUILD.CSRC, f) for f in
            ("attention_api.cu", "rope_append.cu", "decode_attention.cu", "prompt_attention.cu",
             "matmul_fp8.cu", "matmul_narrow.cu", "matmul_wide.cu")]
    subprocess.run(cmd, check=True)
    L = ctypes.CDLL(so)
    L.ar_fusion_prompt_attention.argtypes = B.load().ar_fusion_prompt_attention.argtypes
    L.ar_fusion_attention_status.argtypes = B.load().ar_fusion_attention_status.argtypes
    return L


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
@pytest.mark.parametrize("workspace", [0, B.AR_ATTENTION_WORKSPACE_BYTES])
def test_a_wait_of_a_nanosecond_gives_up(hasty, cache, D, window, sinks, workspace):
    new, lengths, H, K = [300, 1, 40], [300, 500, 900], 8, 2
    pages = R.Pages(lengths, 64, K, D, cache, junk=False)
    T = sum(new)
    starts = torch.tensor([0, 300, 301, 341], dtype=torch.int32).cuda()
    q = torch.ones(T, H, D, dtype=torch.bfloat16, device="cuda")
    kc, vc, table, dev_lengths, kv_scale = pages.cuda()
    work = torch.empty(max(workspace, 1), dtype=torch.uint8, device="cuda")
    c = B._kv_cache(kc, vc, table, dev_lengths, kv_scale)
    details = set()
    for _ in range(10):
        out = torch.full((T + 8, H, D), 77.0, dtype=torch.bfloat16, device="cuda")
        rows = [B._HeadRows(t.data_ptr(), t.stride(0), t.stride(1)) for t in (q, out)]
        assert hasty.ar_fusion_prompt_attention(
            c, *rows, None, starts.data_ptr(), T, H, B.AR_DT_BF16, D ** -0.5, window, sinks,
            work.data_ptr() if workspace else None, workspace, B._stream(None)) == 0
        d = ctypes.c_int(-1)
        code = hasty.ar_fusion_attention_status(None, ctypes.byref(d))
        assert code in (B.AR_OK, B.AR_ERR_TIMEOUT) and bool((out[T:] == 77.0).all())
        if code == B.AR_ERR_TIMEOUT:
            details.add(d.value)
    assert details and details <= set(range(1, 11)), details
