"""The library launches on the current device, so that the binding refuses tensors that lie on another one, and streams
of another one, whatever the call is given (no GPU needed: the library is a stand-in that counts calls, a tensor says on
which GPU it lies, and cuda:0 is said to be the current device)."""
import pytest
import torch

import nvfp4_quantized_moe_gb300 as ft
import test_group_binding as products
import test_layer_binding as layers

CALLS = [*products.CALLS, *layers.CALLS]


class Stream:
    """A stream of the GPU with number `at`; as on a GPU, a default stream's handle is 0."""

    def __init__(self, at):
        self.device_index, self.cuda_stream = at, 0


@pytest.fixture
def library(monkeypatch):
    lib = layers.Library()
    monkeypatch.setattr(ft, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return lib


def _call(name, kind, stream):
    if name in products.CALLS:
        getattr(ft, name)(*products._tensors(name, [kind] * len(products.CALLS[name])), stream=stream)
    else:
        layers._call(name, kind, stream=stream)


def _kind(name, at):
    module = products if name in products.CALLS else layers
    return (module.OnGpu, module.OnOtherGpu)[at]


@pytest.mark.parametrize("stream", [None, 0, 1234, Stream(0)], ids=["none", "zero", "handle", "stream"])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_device_is_taken(library, name, stream):
    _call(name, _kind(name, 0), stream)
    assert library.calls == [name]


@pytest.mark.parametrize("stream", [None, 0, 1234, Stream(0), Stream(1)], ids=["none", "zero", "handle", "stream", "theirs"])
@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(library, name, stream):
    with pytest.raises(ValueError, match="current device"):
        _call(name, _kind(name, 1), stream)
    assert not library.calls


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(library, name):
    with pytest.raises(ValueError, match="stream belongs to"):
        _call(name, _kind(name, 0), Stream(1))
    assert not library.calls


# The calls of the forward and in front of it: operands in order (a list: banks), by argument name; plain arguments.
T, k, E, H = 4, 2, 8, 64
U8, BF, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
CFG = ft.MoEConfig(128, 64, E, k, 16, 64, 0, 1)
BANKS = [((16,), U8)] * ft.FT_NBANKS
FORWARD = (dict(routed=BANKS, shared=BANKS, x=((T, H), BF), topk_ids=((T, k), I32), topk_w=((T, k), F32), out=((T, H), F32),
                workspace=((256,), U8)), dict(cfg=CFG))
OLDER = {
    "ft_moe_pack": (dict(banks=BANKS), dict(cfg=CFG, shared=0, pieces={})),
    "ft_moe_route": (dict(logits=((T, E), F32), topk_ids=((T, k), I32), topk_w=((T, k), F32)), dict(k=k)),
    "ft_moe_route_gemm": (dict(x=((T, H), BF), w_router=((E, H), BF), logits=((T, E), F32), topk_ids=((T, k), I32),
                               topk_w=((T, k), F32)), dict(k=k)),
    "ft_moe_forward": FORWARD,
    "ft_moe_forward_w4a4": FORWARD,
    "ft_moe_quantize_nvfp4": (dict(src=((T, H), BF), codes=((T, H // 2), U8), scales=((T, H // 16), U8), glob=((T,), F32)), {}),
    "ft_moe_align": (dict(topk_ids=((T, k), I32), sorted_slot=((T * k,), I32), block_expert=((T * k + 1,), I32),
                          expert_off=((E + 1,), I32), n_padded=((1,), I32), workspace=((256,), U8)), dict(E=E, block=1)),
    "ft_moe_dequant": (dict(banks=BANKS, out=((H,), F32)), dict(cfg=CFG, shared=0, which=0, expert=0)),
    "ft_moe_read_status": (dict(workspace=((256,), U8)), {}),
}


def _call_older(name, kind, stream, odd=None):
    """With every operand of `kind`, but the one that `odd` names (and the last of several banks) on the other device."""
    specs, plain = OLDER[name]

    def make(spec, kind):
        return torch.zeros(spec[0], dtype=spec[1]).as_subclass(kind)

    args = {}
    for n, spec in specs.items():
        this = layers.OnOtherGpu if n == odd else kind
        args[n] = [make(b, kind) for b in spec[:-1]] + [make(spec[-1], this)] if isinstance(spec, list) else make(spec, this)
    getattr(ft, name)(**args, **plain, stream=stream)


@pytest.mark.parametrize("stream", [None, 0, 1234, Stream(0)], ids=["none", "zero", "handle", "stream"])
@pytest.mark.parametrize("name", list(OLDER))
def test_the_current_device_is_taken_by_the_forward_calls(library, name, stream):
    _call_older(name, layers.OnGpu, stream)
    assert library.calls == [name]


@pytest.mark.parametrize("stream", [None, 0, 1234, Stream(0)], ids=["none", "zero", "handle", "stream"])
@pytest.mark.parametrize("name,odd", [(n, a) for n in OLDER for a in OLDER[n][0]])
def test_an_operand_of_another_device_is_refused_by_the_forward_calls(library, name, odd, stream):
    with pytest.raises(ValueError, match="current device"):
        _call_older(name, layers.OnGpu, stream, odd)
    assert not library.calls


@pytest.mark.parametrize("name", list(OLDER))
def test_a_stream_of_another_device_is_refused_by_the_forward_calls(library, name):
    with pytest.raises(ValueError, match="stream belongs to"):
        _call_older(name, layers.OnGpu, Stream(1))
    assert not library.calls
