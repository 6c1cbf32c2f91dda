"""The bounded waits of prompts' attention: kernels whose waits give up almost at once, with
copies and products in flight.  They answer right or report the wait; either way they
end, write nothing outside the output and leave the device usable."""
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


@pytest.fixture(scope="module", params=[1, 500, 3_000])
def hasty(cuda_lib, tmp_path_factory, request):
    """The kernels with waits that give up after that many nanoseconds."""
    so = os.path.join(str(tmp_path_factory.mktemp("hasty")), "alone.so")
    cmd = [BUILD.nvcc(), *BUILD.ARCH, *BUILD.NVCC_FLAGS, "-shared", "-cudart", "shared", "-Xlinker",
           f"-rpath,{BUILD.cuda_lib_dir()}", f"-DARF_WAIT_NS={request.param}ull", "-DARF_WAIT_TRIES=1u",
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


def status(L):
    d = ctypes.c_int(-1)
    return L.ar_fusion_attention_status(None, ctypes.byref(d)), d.value


@pytest.mark.parametrize("new,lengths,H,K,D,window,sinks", [
    ([300, 1, 40], [300, 500, 900], 8, 2, 128, 0, 0), ([700], [700], 64, 8, 128, 100, 5),
    ([5000], [5000], 32, 8, 64, 0, 0), ([4, 3], [3000, 2000], 8, 1, 64, 0, 0)])
@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_prompts_whose_waits_give_up_at_once(hasty, new, lengths, H, K, D, window, sinks, cache):
    pages = R.Pages(lengths, 64, K, D, cache, junk=False)
    T = sum(new)
    starts = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    g = torch.Generator()
    g.manual_seed(3)
    q = torch.randn(T, H, D, generator=g).to(torch.bfloat16).cuda()
    kc, vc, table, dev_lengths, kv_scale = pages.cuda()
    work = torch.empty(B.AR_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    want, want_lse = torch.empty_like(q), torch.empty(T, H, device="cuda")

    def call(L, out, lse):
        cache = B._kv_cache(kc, vc, table, dev_lengths, kv_scale)
        rows = [B._HeadRows(t.data_ptr(), t.stride(0), t.stride(1)) for t in (q, out)]
        assert L.ar_fusion_prompt_attention(
            cache, *rows, lse.data_ptr(), starts.data_ptr(), T, H, B.AR_DT_BF16, D ** -0.5, window,
            sinks, work.data_ptr(), work.numel(), B._stream(None)) == 0

    call(B.load(), want, want_lse)
    assert B.ar_fusion_attention_status() == (B.AR_OK, -1)
    gave_up = 0
    for _ in range(10):
        guard = torch.full((T + 8, H, D), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T + 8, H), 77.0, device="cuda")
        call(hasty, guard[:T], lse[:T])
        code, detail = status(hasty)
        assert bool((guard[T:] == 77.0).all()) and bool((lse[T:] == 77.0).all())
        if code == B.AR_OK:
            assert torch.equal(guard[:T], want) and torch.equal(lse[:T], want_lse)
        else:
            assert code == B.AR_ERR_TIMEOUT and detail in range(1, 11)
            gave_up += 1
        assert status(hasty) == (B.AR_OK, -1)
        again, again_lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
        call(B.load(), again, again_lse)
        assert B.ar_fusion_attention_status() == (B.AR_OK, -1)
        assert torch.equal(again, want) and torch.equal(again_lse, want_lse)
    print("gave up", gave_up, "of 10")
