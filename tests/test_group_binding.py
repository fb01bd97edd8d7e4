"""Every tensor of an expert-product or row-kernel call lies on one device: the binding refuses a call
otherwise, before it reaches the library (no GPU needed: the library is a stand-in that counts
calls, and a tensor says that it is on the GPU)."""
import pytest
import torch

import nvfp4_quantized_moe_gb300 as ft


class OnGpu(torch.Tensor):
    """A CPU tensor that says it lies on the GPU with number `at`."""
    at = 0

    def get_device(self):
        return self.at


class OnOtherGpu(OnGpu):
    at = 1


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
E, P, N, K = 2, 8, 128, 64
OFFS, WS = ((E + 1,), I32), ((256,), U8)
# the operands of each call, in order
CALLS = {
    "ft_moe_group_gemm": [((P, K), BF), ((E, N, K), BF), OFFS, ((P, N), BF), WS],
    "ft_moe_group_gemm_dgrad": [((P, N), BF), ((E, N, K), BF), OFFS, ((P, K), F32), WS],
    "ft_moe_group_gemm_wgrad": [((P, N), BF), ((P, K), BF), OFFS, ((E, N, K), F32), WS],
    "ft_moe_group_gemm_fp8": [((P, K), U8), ((1, P), F32), ((E, N, K), U8), ((E, 1, 1), F32), OFFS, ((P, N), BF), WS],
    "ft_moe_quantize_fp8": [((P, K), BF), ((P, K), U8), ((1, P), F32)],
    "ft_moe_swiglu": [((P, 2 * K), BF), ((P,), F32), ((P, K), BF)],
    "ft_moe_swiglu_quantize_fp8": [((P, 2 * K), BF), ((P,), F32), ((P, K), U8), ((1, P), F32)],
    "ft_moe_swiglu_backward": [((P, 2 * K), BF), ((P,), F32), ((P, K), BF), ((P, 2 * K), BF), ((P,), F32)],
}


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(ft, "_lib", lib)
    return lib


def _tensors(name, kinds):
    return [torch.zeros(shape, dtype=dtype).as_subclass(kind) for (shape, dtype), kind in zip(CALLS[name], kinds)]


@pytest.mark.parametrize("name", list(CALLS))
def test_a_call_on_one_gpu_reaches_the_library(library, name):
    for kind in (OnGpu, OnOtherGpu):
        getattr(ft, name)(*_tensors(name, [kind] * len(CALLS[name])), stream=0)
    assert library.calls == [name, name]


@pytest.mark.parametrize("odd", [torch.Tensor, OnOtherGpu], ids=["cpu", "other gpu"])
@pytest.mark.parametrize("name,at", [(n, i) for n in CALLS for i in range(len(CALLS[n]))])
def test_one_operand_elsewhere_is_refused(library, name, at, odd):
    kinds = [OnGpu] * len(CALLS[name])
    kinds[at] = odd
    with pytest.raises(ValueError):
        getattr(ft, name)(*_tensors(name, kinds), stream=0)
    assert not library.calls


@pytest.mark.parametrize("name", [n for n in CALLS if CALLS[n][-1] == WS])
def test_a_workspace_with_gaps_is_refused(library, name):
    """Its size in bytes would not be what lies behind its address."""
    tensors = _tensors(name, [OnGpu] * len(CALLS[name]))
    tensors[-1] = torch.zeros(512, dtype=U8).as_subclass(OnGpu)[::2]
    with pytest.raises(ValueError):
        getattr(ft, name)(*tensors, stream=0)
    assert not library.calls
