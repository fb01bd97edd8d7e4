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
