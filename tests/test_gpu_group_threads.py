"""The expert products called from other host threads than the first, each with its own stream and
workspace: in a thread that has made no CUDA call before, and in several at once."""
import os
import shutil
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _calls(ft, E, stream):
    """Every product over E experts, few rows: the same kernels whatever E is."""
    P, N, K = 16, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(E)
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[1:] = torch.bincount(torch.randint(E, (P,), generator=gen, device="cuda"), minlength=E).cumsum(0)
    x, dy = (torch.randn((P, c), generator=gen, device="cuda").bfloat16() for c in (K, N))
    w = torch.randn((E, N, K), generator=gen, device="cuda").bfloat16()
    codes, scales = torch.full((P, K), 0x38, dtype=torch.uint8, device="cuda"), torch.ones((1, P), device="cuda")
    wq, wsc = w.float().to(torch.float8_e4m3fn), torch.ones((E, 1, 1), device="cuda")
    outs = [torch.empty(s, device="cuda") for s in ((P, N), (P, K), (E, N, K), (P, N))]
    ws = torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    calls = [
        lambda: ft.ft_moe_group_gemm(x, w, offs, outs[0], ws, stream=stream),
        lambda: ft.ft_moe_group_gemm_dgrad(dy, w, offs, outs[1], ws, stream=stream),
        lambda: ft.ft_moe_group_gemm_wgrad(dy, x, offs, outs[2], ws, stream=stream),
        lambda: ft.ft_moe_group_gemm_fp8(codes, scales, wq, wsc, offs, outs[3], ws, stream=stream),
    ]
    return calls, outs, ws


@pytest.mark.parametrize("which", range(4), ids=["forward", "dgrad", "wgrad", "fp8"])
def test_first_call_of_a_thread(ft, which):
    stream = torch.cuda.Stream()
    calls, outs, ws = _calls(ft, 5, stream)
    calls[which]()
    torch.cuda.synchronize()
    first, failed = outs[which].clone(), []
    outs[which].zero_()
    torch.cuda.synchronize()

    def work():
        try:
            calls[which]()
        except Exception as error:  # noqa: BLE001 - reported below, from the test's own thread
            failed.append(str(error))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert ft.ft_moe_read_status(ws) == 0 and torch.equal(outs[which], first)


def test_threads_with_unlike_numbers_of_experts(ft, tmp_path):
    """From C++, where nothing serialises the calls (gpu_probes/unlike_threads.cpp)."""
    here, lib = os.path.dirname(os.path.abspath(__file__)), os.path.abspath(ft.LIB_PATH)
    exe = str(tmp_path / "unlike_threads")
    subprocess.check_call([shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc", "-O2", "-std=c++17", "-I",
                           os.path.join(os.path.dirname(here), "include"), "-o", exe,
                           os.path.join(here, "gpu_probes", "unlike_threads.cpp"), lib, "-Xlinker",
                           "-rpath=" + os.path.dirname(lib)])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
