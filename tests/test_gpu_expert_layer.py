"""The expert products, SwiGLU and the quantizer run together as a layer (examples/expert_layer.py):
the training step against torch's autograd in 64 bits, the 8-bit serving step against the oracle's
forward on the same fp8_block banks."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import synth
from moe_cases import GpuLayer, logits_for, oracle_banks

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 64, 8, 2), (37, 256, 64, 8, 2), (300, 128, 72, 16, 4), (700, 640, 512, 8, 2)])
def test_training_step_matches_autograd(layer, T, H, I, E, k):
    """Output and every gradient within a few bf16 roundings (2^-8) of the 64-bit ones: gu, h, dh and
    dgu are rounded to bf16 on the way, each adding at most 2^-8 relative in norm; 4 * 2^-8 = 1.6e-2."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5  # noqa: E731
    x = (mk(T, H) * H ** 0.5).bfloat16().requires_grad_()
    w = [mk(E, H).requires_grad_(), mk(E, 2 * I, H).bfloat16().requires_grad_(), mk(E, H, I).bfloat16().requires_grad_()]
    dout = torch.randn((T, H), generator=gen, device="cuda")
    out = layer.train_forward(x, *w, k)
    got = torch.autograd.grad((out * dout).sum(), [x, *w])

    x64, (r64, gu64, dn64) = x.detach().double().requires_grad_(), [a.detach().double().requires_grad_() for a in w]
    logits = x64 @ r64.t()
    ids, _ = layer.route((x.float() @ w[0].t()).detach().contiguous(), k)
    kept = torch.softmax(logits, 1).gather(1, ids.long())
    weights = kept / kept.sum(1, keepdim=True)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            g, u = (x64[t] @ gu64[e].t()).chunk(2, dim=1)
            ref = ref.index_add(0, t, weights[t, j, None] * (torch.nn.functional.silu(g) * u) @ dn64[e].t())
    want = torch.autograd.grad((ref * dout.double()).sum(), [x64, r64, gu64, dn64])
    assert _rel(out.detach(), ref.detach()) <= 1.6e-2
    for a, b in zip(got, want):
        assert _rel(a, b) <= 1.6e-2
    untouched = [e for e in range(E) if not (ids == e).any()]
    assert all(not got[2][e].any() and not got[3][e].any() for e in untouched)


def test_training_reduces_the_loss(layer):
    losses = layer.main(T=256, H=256, I=128, E=8, k=2, steps=4)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("name,T", [("mini_fp8", 1), ("mini_fp8", 64), ("mini_fp8", 700), ("qwen36_fp8", 16)])
def test_serving_step_matches_the_oracle(layer, name, T):
    """Against the forward on unquantized activations: x and h each carry an e4m3 rounding (at most
    2^-4, about 2^-5.3 = 2.6% in norm for smoothly distributed values), so 2 * 2.6% and the bf16 gu."""
    shape = synth.SHAPES[name]
    L = GpuLayer(name)
    x_bits = synth.make_activations(T, shape.hidden, seed=3)
    ids, w = L.route(logits_for(name, T, False, seed=3))
    x = torch.from_numpy(x_bits.view(np.int16)).cuda().view(torch.bfloat16)
    r = L.routed
    out = layer.serve_forward(x, ids, w, r[0], r[1], r[3], r[4])
    routed, _ = oracle_banks(name)
    ref = oracle.moe_forward(routed, None, shape.group, x_bits, ids.cpu().numpy(), w.cpu().numpy(),
                             nthreads=oracle.default_threads())
    assert _rel(out.cpu(), torch.from_numpy(np.asarray(ref))) <= 6e-2
