"""Every tensor of a norm, sorting or MXFP4 call lies on one device, and that device is the current one: the binding
refuses a call otherwise, before it reaches the library (no GPU needed: the library is a stand-in that counts calls, and a
tensor says that it is on the GPU)."""
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
T, k, P, H, E, N, K = 4, 2, 8, 64, 2, 16, 64
# the tensors of each call by argument name, and its plain arguments
CALLS = {
    "ft_moe_rmsnorm": (dict(x=((T, H), BF), weight=((H,), BF), y=((T, H), BF), residual=((T, H), F32), total=((T, H), F32),
                            codes=((T, H), U8), scales=((1, T), F32), rstd=((T,), F32)), dict(eps=1e-6)),
    "ft_moe_rmsnorm_backward": (dict(dy=((T, H), BF), total=((T, H), BF), weight=((H,), F32), rstd=((T,), F32), dx=((T, H), BF),
                                     workspace=((4096,), U8), dw=((H,), F32), dtotal=((T, H), BF)), {}),
    "ft_moe_dispatch": (dict(x=((T, H), U8), slot=((P,), I32), out=((P, H), U8), x_scale=((1, T), F32), out_scale=((1, P), F32),
                             w=((T, k), F32), row_w=((P,), F32), pos=((T, k), I32), count=((1,), I32)), dict(k=k)),
    "ft_moe_dispatch_backward": (dict(dout=((P, H), BF), pos=((T, k), I32), dx=((T, H), BF), drow_w=((P,), F32), dw=((T, k), F32)), {}),
    "ft_moe_combine": (dict(y=((P, H), BF), pos=((T, k), I32), w=((T, k), F32), out=((T, H), F32), add=((T, H), F32)), {}),
    "ft_moe_combine_backward": (dict(dout=((T, H), F32), y=((P, H), BF), pos=((T, k), I32), w=((T, k), F32), dy=((P, H), BF),
                                     dw=((T, k), F32)), {}),
    "ft_moe_group_gemm_mxfp4": (dict(x=((P, K // 2), U8), x_scale=((1, P, 4), U8), w=((E, N, K // 2), U8),
                                     w_scale=((E, 1, 1, 512), U8), offs=((E + 1,), I32), y=((P, N), BF), workspace=((256,), U8)), {}),
    "ft_moe_quantize_mxfp4": (dict(src=((P, K), BF), codes=((P, K // 2), U8), scales=((1, P, 4), U8)), {}),
    "ft_moe_quantize_mxfp4_weights": (dict(src=((E, N, K), F32), codes=((E, N, K // 2), U8), tiles=((E, 1, 1, 512), U8)), {}),
    "ft_moe_pack_mxfp4_scales": (dict(src=((E, N, K // 32), U8), tiles=((E, 1, 1, 512), U8)), {}),
    "ft_moe_swiglu_quantize_mxfp4": (dict(gu=((P, 2 * K), BF), w=((P,), F32), codes=((P, K // 2), U8), scales=((1, P, 4), U8)), {}),
}


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(ft, "_lib", lib)
    return lib


def _call(name, kind, odd=None, odd_kind=None, **more):
    tensors, plain = CALLS[name]
    args = {n: torch.zeros(shape, dtype=dtype).as_subclass(odd_kind if n == odd else kind) for n, (shape, dtype) in tensors.items()}
    getattr(ft, name)(**args, **plain, **more)


@pytest.mark.parametrize("name", list(CALLS))
def test_a_call_on_one_gpu_reaches_the_library(library, name):
    for kind in (OnGpu, OnOtherGpu):
        _call(name, kind, stream=0)
    assert library.calls == [name, name]


@pytest.mark.parametrize("odd_kind", [torch.Tensor, OnOtherGpu], ids=["cpu", "other gpu"])
@pytest.mark.parametrize("name,odd", [(n, a) for n in CALLS for a in CALLS[n][0]])
def test_one_operand_elsewhere_is_refused(library, name, odd, odd_kind):
    with pytest.raises(ValueError):
        _call(name, OnGpu, odd, odd_kind, stream=0)
    assert not library.calls


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_on_another_device_than_the_current_one_are_refused(library, name, monkeypatch):
    """Without a stream: the default stream has the same handle on every device."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    _call(name, OnGpu)
    assert library.calls == [name]
    with pytest.raises(ValueError):
        _call(name, OnOtherGpu)
    assert library.calls == [name]


@pytest.mark.parametrize("name", ["ft_moe_rmsnorm_backward", "ft_moe_group_gemm_mxfp4"])
def test_a_workspace_with_gaps_is_refused(library, name):
    tensors, plain = CALLS[name]
    args = {n: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu) for n, (shape, dtype) in tensors.items()}
    args["workspace"] = torch.zeros(8192, dtype=U8).as_subclass(OnGpu)[::2]
    with pytest.raises(ValueError):
        getattr(ft, name)(**args, **plain, stream=0)
    assert not library.calls
