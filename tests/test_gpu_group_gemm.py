"""Grouped expert products (bf16 with gradients, 8-bit with block scales) against the formulas
in 64 bits, through the C ABI.

Tolerances come from the arithmetic: products of two bf16 (or e4m3) values are exact in fp32; a sum
of R of them in fp32, in any order and even with every addition truncated, is within R * 2^-23 of
sum |a b|; the store rounds once (2^-8 relative for bf16, 2^-24 for fp32). The 8-bit products add
two fp32 multiplications per block of 128 (2^-22 of the block).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _offs(sizes, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def _ws(ft, E, P, N, K):
    n = ft.ft_moe_group_workspace_size(E, P, N, K)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def _close(got, ref, mag, R, out, extra=0.0):
    err = (got.double() - ref).abs()
    tol = U[out] * ref.abs() + (R * 2.0 ** -23 + extra) * mag + 1e-30
    assert torch.isfinite(got).all()
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 1.0, worst


# ragged batches: empty experts, single rows, sizes around the 16-column step, the 32-, 64- and
# 256-row tiles, and a batch of several tiles
RAGGED = [0, 1, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 255, 256, 257, 600, 0]
BATCHES = {
    "one row": [0, 0, 1, 0],
    "single expert": [37],
    "all in one of eight": [0, 0, 0, 1000, 0, 0, 0, 0],
    "ragged": RAGGED,
    "a row each": [1] * 40,
    "few rows": [3, 0, 5, 2, 8, 16, 0, 1],
    "many experts": [(7 * i) % 23 for i in range(300)],
}
# (N, K): tile multiples; below, across and just past a 128-row tile; odd multiples of 8 on the
# contraction side (partial 64- and 16-steps)
SHAPES = [(256, 512), (128, 64), (8, 8), (640, 200), (136, 1032), (1000, 24)]


def _forms(ft, form, x, w, dy, offs, sizes, out, start=0):
    """The call's result, the 64-bit one and the sum of magnitudes."""
    E, N, K = w.shape
    P = x.shape[0]
    ws = _ws(ft, E, P, N, K)
    if form == "wgrad":
        got = torch.full((E, N, K), float("nan"), dtype=out, device="cuda")
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, got, ws)
        ref, mag = (torch.zeros((E, N, K), dtype=torch.float64, device="cuda") for _ in range(2))
    else:
        cols = N if form == "forward" else K
        got = torch.zeros((P, cols), dtype=out, device="cuda")
        if form == "forward":
            ft.ft_moe_group_gemm(x, w, offs, got, ws)
        else:
            ft.ft_moe_group_gemm_dgrad(dy, w, offs, got, ws)
        ref, mag = (torch.zeros((P, cols), dtype=torch.float64, device="cuda") for _ in range(2))
    assert ft.ft_moe_read_status(ws) == 0
    at = start
    for e, n in enumerate(sizes):
        r = slice(at, at + n)
        at += n
        if form == "wgrad":
            ref[e] = dy[r].double().t() @ x[r].double()
            mag[e] = dy[r].double().abs().t() @ x[r].double().abs()
        else:
            a, m = (x[r], w[e].t()) if form == "forward" else (dy[r], w[e])
            ref[r] = a.double() @ m.double()
            mag[r] = a.double().abs() @ m.double().abs()
    return got, ref, mag


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("batch", list(BATCHES))
def test_ragged_batches(ft, batch, form, out):
    sizes = BATCHES[batch]
    E, P = len(sizes), sum(sizes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for N, K in ((256, 512), (136, 264)):
        x, w, dy = _randn(gen, P, K), _randn(gen, E, N, K), _randn(gen, P, N)
        got, ref, mag = _forms(ft, form, x, w, dy, _offs(sizes), sizes, out)
        R = {"forward": K, "dgrad": N, "wgrad": max(sizes)}[form]
        _close(got, ref, mag, R, out)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("N,K", SHAPES)
def test_widths(ft, N, K, form):
    sizes = [5, 0, 70, 300, 1]
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, dy = _randn(gen, sum(sizes), K), _randn(gen, 5, N, K), _randn(gen, sum(sizes), N)
    got, ref, mag = _forms(ft, form, x, w, dy, _offs(sizes), sizes, torch.float32)
    _close(got, ref, mag, {"forward": K, "dgrad": N, "wgrad": 300}[form], torch.float32)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("P", [1, 2, 130, 2000])
def test_plain_product_without_offsets(ft, P, form):
    """offs = None: one expert owns every row."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    N, K = 384, 1024
    x, w, dy = _randn(gen, P, K), _randn(gen, 1, N, K), _randn(gen, P, N)
    got, ref, mag = _forms(ft, form, x, w, dy, None, [P], torch.bfloat16)
    _close(got, ref, mag, {"forward": K, "dgrad": N, "wgrad": P}[form], torch.bfloat16)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
def test_large_batches(ft, form):
    """Enough rows per expert for the widest tiles, several of them per expert."""
    sizes = [700, 1300, 0, 513, 256, 1025, 3, 900]
    gen = torch.Generator(device="cuda").manual_seed(4)
    N, K = 776, 520
    x, w, dy = _randn(gen, sum(sizes), K), _randn(gen, 8, N, K), _randn(gen, sum(sizes), N)
    for out in (torch.bfloat16, torch.float32):
        got, ref, mag = _forms(ft, form, x, w, dy, _offs(sizes), sizes, out)
        _close(got, ref, mag, {"forward": K, "dgrad": N, "wgrad": 1300}[form], out)


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_with_their_expert(ft, form, bad):
    """Rows of the experts on both sides are not finite: the experts between them must not notice."""
    sizes = [9, 3, 40, 77, 64, 21, 5]
    gen = torch.Generator(device="cuda").manual_seed(5)
    N, K = 200, 328
    x, w, dy = _randn(gen, sum(sizes), K), _randn(gen, 7, N, K), _randn(gen, sum(sizes), N)
    at = np.concatenate([[0], np.cumsum(sizes)])
    for e in range(0, 7, 2):
        for t in (x, dy):
            t[at[e]:at[e + 1]] = bad
        if form != "wgrad":
            w[e] = bad
    got, ref, mag = _forms(ft, form, x, w, dy, _offs(sizes), sizes, torch.float32)
    R = {"forward": K, "dgrad": N, "wgrad": 77}[form]
    for e in range(7):
        r = e if form == "wgrad" else slice(at[e], at[e + 1])
        if e % 2:
            _close(got[r], ref[r], mag[r], R, torch.float32)
        else:
            assert not torch.isfinite(got[r]).any()


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strided_rows_and_rows_of_no_expert(ft, form, out):
    """Rows inside wider buffers; rows before the first and after the last expert stay untouched."""
    sizes, lead, trail = [20, 0, 133, 18], 7, 11
    P, E, N, K = lead + sum(sizes) + trail, 4, 264, 136
    gen = torch.Generator(device="cuda").manual_seed(6)
    xb, dyb = _randn(gen, P, K + 24), _randn(gen, P, N + 8)
    x, dy, w = xb[:, 8:8 + K], dyb[:, :N], _randn(gen, E, N, K)
    x[:lead] = dy[:lead] = float("nan")
    x[P - trail:] = dy[P - trail:] = float("nan")
    offs = _offs(sizes, lead)
    cols = {"forward": N, "dgrad": K}.get(form)
    if form == "wgrad":
        got, ref, mag = _forms(ft, form, x, w, dy, offs, sizes, out, lead)
        _close(got, ref, mag, 133, out)
        return
    buf = torch.full((P, cols + 16), 7.0, dtype=out, device="cuda")
    y, ws = buf[:, 8:8 + cols], _ws(ft, E, P, N, K)
    if form == "forward":
        ft.ft_moe_group_gemm(x, w, offs, y, ws)
    else:
        ft.ft_moe_group_gemm_dgrad(dy, w, offs, y, ws)
    assert ft.ft_moe_read_status(ws) == 0
    _, ref, mag = _forms(ft, form, x, w, dy, offs, sizes, out, lead)
    own = slice(lead, P - trail)
    _close(y[own], ref[own], mag[own], K if form == "forward" else N, out)
    assert (buf[:lead] == 7).all() and (buf[P - trail:] == 7).all()
    assert (buf[:, :8] == 7).all() and (buf[:, 8 + cols:] == 7).all()


def test_wgrad_accumulates(ft):
    sizes = [30, 0, 200]
    gen = torch.Generator(device="cuda").manual_seed(7)
    N, K = 136, 256
    x, dy = _randn(gen, 230, K), _randn(gen, 230, N)
    base = torch.randn((3, N, K), generator=gen, device="cuda")
    dw = base.clone()
    ft.ft_moe_group_gemm_wgrad(dy, x, _offs(sizes), dw, _ws(ft, 3, 230, N, K), accumulate=True)
    _, ref, mag = _forms(ft, "wgrad", x, base.bfloat16(), dy, _offs(sizes), sizes, torch.float32)
    _close(dw, ref + base.double(), mag + base.double().abs(), 201, torch.float32)
    assert torch.equal(dw[1], base[1])


def test_gradients_match_differences(ft):
    """<dy, y(x + h) - y(x)> = <dx, h> and the same for w: the products are linear, so that the
    difference quotient is exact up to rounding."""
    sizes = [33, 0, 100, 7]
    P, E, N, K = 140, 4, 128, 192
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, w, dy = _randn(gen, P, K), _randn(gen, E, N, K), _randn(gen, P, N)
    offs = _offs(sizes)
    hx, hw = _randn(gen, P, K), _randn(gen, E, N, K)

    def y(a, b):
        out = torch.empty((P, N), device="cuda")
        ft.ft_moe_group_gemm(a, b, offs, out, _ws(ft, E, P, N, K))
        return out.double()

    dx = torch.empty((P, K), device="cuda")
    dw = torch.empty((E, N, K), device="cuda")
    ft.ft_moe_group_gemm_dgrad(dy, w, offs, dx, _ws(ft, E, P, N, K))
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, _ws(ft, E, P, N, K))
    for quotient, grad in (((dy.double() * y(hx, w)).sum(), (dx.double() * hx.double()).sum()),
                           ((dy.double() * y(x, hw)).sum(), (dw.double() * hw.double()).sum())):
        # both sides are sums of P N K products; each fp32 sum within its length * 2^-23 of the magnitudes
        mag = (dy.double().abs().sum() * 1.0) * K * 1.0
        assert abs(float(quotient - grad)) <= float(mag) * 400 * 2.0 ** -23


def test_runs_are_bitwise_equal_and_capture(ft):
    sizes = [300, 1, 0, 64, 500]
    gen = torch.Generator(device="cuda").manual_seed(9)
    P, E, N, K = sum(sizes), 5, 512, 384
    x, w, dy, offs = _randn(gen, P, K), _randn(gen, E, N, K), _randn(gen, P, N), _offs(sizes)
    ws = _ws(ft, E, P, N, K)
    y, dx, dw = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((P, N), (P, K), (E, N, K)))

    def step():
        ft.ft_moe_group_gemm(x, w, offs, y, ws)
        ft.ft_moe_group_gemm_dgrad(dy, w, offs, dx, ws)
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)

    step()
    first = [t.clone() for t in (y, dx, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))
    for t in (y, dx, dw):
        t.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))


@pytest.mark.parametrize("N,K", [(512, 512), (64, 1024)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_wgrad_of_many_units_is_bitwise_equal_and_captures(ft, out, N, K):
    """Enough units that they are handed out by a counter: which CTA computes a unit must not show."""
    sizes = [(37 * i) % 150 for i in range(200)] + [0, 900, 1, 2000]
    gen = torch.Generator(device="cuda").manual_seed(14)
    P, E = sum(sizes), len(sizes)
    x, dy, offs = _randn(gen, P, K), _randn(gen, P, N), _offs(sizes)
    got, ref, mag = _forms(ft, "wgrad", x, torch.empty((E, N, K), device="cuda"), dy, offs, sizes, out)
    _close(got, ref, mag, 2000, out)
    dw, ws = torch.empty((E, N, K), dtype=out, device="cuda"), _ws(ft, E, P, N, K)
    for _ in range(3):
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)
        assert torch.equal(dw, got)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)
    for _ in range(2):
        dw.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, got)


@pytest.mark.parametrize("out,accumulate", ((torch.bfloat16, False), (torch.float32, False), (torch.float32, True)))
@pytest.mark.parametrize("sizes,N,K", (([1000], 256, 200), ([4099], 40, 1000), ([2048], 256, 256), ([700, 0, 1], 128, 136),
                                       ([0, 64, 3000, 5], 64, 128)))
def test_wgrad_of_few_tiles_shares_the_rows(ft, sizes, N, K, accumulate, out):
    """Few tiles and many rows: several thread blocks share an expert's rows, some without any."""
    P, E = sum(sizes), len(sizes)
    gen = torch.Generator(device="cuda").manual_seed(15)
    x, dy, offs = _randn(gen, P, K), _randn(gen, P, N), _offs(sizes)
    base = torch.randn((E, N, K), generator=gen, device="cuda")
    _, ref, mag = _forms(ft, "wgrad", x, base.bfloat16(), dy, offs, sizes, torch.float32)
    dw, ws = base.to(out, copy=True), _ws(ft, E, P, N, K)
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws, accumulate=accumulate)
    if accumulate:
        ref, mag = ref + base.double(), mag + base.double().abs()
    _close(dw, ref, mag, max(sizes) + accumulate, out)
    again = base.to(out, copy=True)
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, again, ws, accumulate=accumulate)
    assert torch.equal(dw, again)


def test_wgrad_accumulates_over_many_units(ft):
    """Twice into the same dw, units handed out by a counter; values that are not finite stay."""
    sizes, N, K = [(37 * i) % 150 for i in range(200)] + [0, 900, 1, 2000], 200, 520
    P, E = sum(sizes), len(sizes)
    gen = torch.Generator(device="cuda").manual_seed(17)
    x, dy, offs = _randn(gen, P, K), _randn(gen, P, N), _offs(sizes)
    base = torch.randn((E, N, K), generator=gen, device="cuda")
    base[3, 5, 7], base[200, 0, 0] = float("inf"), float("nan")
    _, ref, mag = _forms(ft, "wgrad", x, base.bfloat16(), dy, offs, sizes, torch.float32)
    dw, ws = base.clone(), _ws(ft, E, P, N, K)
    for _ in range(2):
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws, accumulate=True)
    again = base.clone()
    for _ in range(2):
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, again, ws, accumulate=True)
    assert torch.equal(dw.view(torch.int32), again.view(torch.int32))
    assert torch.isinf(dw[3, 5, 7]) and torch.isnan(dw[200, 0, 0])
    ok = torch.isfinite(base)
    assert torch.equal(torch.isfinite(dw), ok)
    _close(dw[ok], (2 * ref + base.double())[ok], (2 * mag + base.double().abs())[ok], 2001, torch.float32)


def test_wgrad_shared_rows_keep_to_their_expert(ft):
    """Rows of the next expert that are not finite, behind a last stage that several blocks' parts end in."""
    sizes, N, K = [1003, 500], 64, 128
    gen = torch.Generator(device="cuda").manual_seed(16)
    x, dy = _randn(gen, 1503, K), _randn(gen, 1503, N)
    x[1003:], dy[1003:] = float("nan"), float("inf")
    dw = torch.empty((2, N, K), device="cuda")
    ft.ft_moe_group_gemm_wgrad(dy, x, _offs(sizes), dw, _ws(ft, 2, 1503, N, K))
    assert torch.isfinite(dw[0]).all() and not torch.isfinite(dw[1]).any()


def test_one_row_of_any_stride(ft):
    """A single row has no stride: one cut out of an odd-sized buffer is as good as any."""
    buf = torch.ones((3, 64 + 5), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((1, 128, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((1, 128), device="cuda")
    ft.ft_moe_group_gemm(buf[:1, :64], w, None, y, _ws(ft, 1, 1, 128, 64))
    assert (y == 64).all()


@pytest.mark.parametrize("offs", [[0, 5, 3, 12], [0, 4, 8, 99], [-2, 4, 8, 12]])
def test_bad_offsets_are_reported(ft, offs):
    """Offsets that decrease or leave [0, P]: reported, and nothing outside the output is touched."""
    P, N, K = 12, 64, 64
    x = torch.ones((P, K), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((3, N, K), dtype=torch.bfloat16, device="cuda")
    buf = torch.full((P + 20, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = _ws(ft, 3, P, N, K)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    ft.ft_moe_group_gemm(x, w, o, buf[:P], ws)
    assert ft.STATUS[ft.ft_moe_read_status(ws)] == "FT_ERR_INVALID_ROUTING"
    assert (buf[P:] == 7).all()
    dw = torch.empty((3, N, K), device="cuda")
    ft.ft_moe_group_gemm_wgrad(x, x, o, dw, ws)
    assert ft.STATUS[ft.ft_moe_read_status(ws)] == "FT_ERR_INVALID_ROUTING"
    good = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")
    ft.ft_moe_group_gemm(x, w, good, buf[:P], ws)
    assert ft.ft_moe_read_status(ws) == 0 and (buf[:P] == K).all()


def test_no_rows(ft):
    N, K = 64, 128
    w = torch.ones((2, N, K), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    offs, ws = _offs([0, 0]), _ws(ft, 2, 0, N, K)
    ft.ft_moe_group_gemm(x, w, offs, torch.empty((0, N), device="cuda"), ws)
    assert ft.ft_moe_read_status(ws) == 0
    dw = torch.full((2, N, K), 3.0, device="cuda")
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws, accumulate=True)
    assert (dw == 3).all()
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)
    assert (dw == 0).all() and ft.ft_moe_read_status(ws) == 0


@pytest.mark.parametrize("rows", [4, 2000])
def test_a_stalled_pipeline_reports_timeout_and_recovers(ft, rows):
    gen = torch.Generator(device="cuda").manual_seed(10)
    N, K, offs = 256, 512, _offs([rows, 0])
    x, w, dy = _randn(gen, rows, K), _randn(gen, 2, N, K), _randn(gen, rows, N)
    ws = _ws(ft, 2, rows, N, K)
    q, s = torch.empty((rows, K), dtype=torch.uint8, device="cuda"), torch.empty((K // 128, rows), device="cuda")
    ft.ft_moe_quantize_fp8(x, q, s)
    wq, wsc = torch.full((2, N, K), 0x38, dtype=torch.uint8, device="cuda"), torch.ones((2, 2, 4), device="cuda")
    outs = [torch.empty((rows, N), device="cuda"), torch.empty((rows, K), device="cuda"),
            torch.empty((2, N, K), device="cuda"), torch.empty((rows, N), device="cuda")]
    calls = [lambda: ft.ft_moe_group_gemm(x, w, offs, outs[0], ws),
             lambda: ft.ft_moe_group_gemm_dgrad(dy, w, offs, outs[1], ws),
             lambda: ft.ft_moe_group_gemm_wgrad(dy, x, offs, outs[2], ws),
             lambda: ft.ft_moe_group_gemm_fp8(q, s, wq, wsc, offs, outs[3], ws)]
    for call, out in zip(calls, outs):
        call()
        assert ft.ft_moe_read_status(ws) == 0
        good = out.clone()
        ft.ft_moe_debug_inject_stall(5_000_000, 1)
        call()
        assert ft.STATUS[ft.ft_moe_read_status(ws)] == "FT_ERR_TIMEOUT"
        call()
        assert ft.ft_moe_read_status(ws) == 0 and torch.equal(out, good)


# ---------------------------------------------------------------- 8-bit products


def _e4m3(gen, *shape):
    return (torch.randn(shape, generator=gen, device="cuda") * 32).clamp(-448, 448).to(torch.float8_e4m3fn)


def _spread(scale, N, K):
    return scale.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def _fp8_case(ft, sizes, N, K, out, seed=0, offs=True, strided=False):
    E, P = len(sizes), sum(sizes)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-K // 128)
    x, w = _e4m3(gen, P, K), _e4m3(gen, E, N, K)
    xs = torch.rand((nb, P), generator=gen, device="cuda") + 0.01
    wsc = torch.rand((E, -(-N // 128), nb), generator=gen, device="cuda") * 0.01
    xd = x.double() * xs.double().t().repeat_interleave(128, 1)[:, :K]
    wd = w.double() * _spread(wsc, N, K)
    ref = torch.zeros((P, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    at = 0
    for e, n in enumerate(sizes):
        ref[at:at + n] = xd[at:at + n] @ wd[e].t()
        mag[at:at + n] = xd[at:at + n].abs() @ wd[e].abs().t()
        at += n
    y = torch.zeros((P, N), dtype=out, device="cuda")
    if strided:
        xb = torch.zeros((P, K + 32), dtype=torch.uint8, device="cuda")
        xb[:, 16:16 + K] = x.view(torch.uint8)
        sb = torch.zeros((nb, P + 3), device="cuda")
        sb[:, 3:] = xs
        y = torch.zeros((P, N + 5), dtype=out, device="cuda")[:, :N]
        x, xs = xb[:, 16:16 + K], sb[:, 3:]
    ws = _ws(ft, E, P, N, K)
    ft.ft_moe_group_gemm_fp8(x, xs, w, wsc, _offs(sizes) if offs else None, y, ws)
    assert ft.ft_moe_read_status(ws) == 0
    _close(y, ref, mag, K, out, extra=4 * 2.0 ** -23)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch", list(BATCHES))
def test_fp8_ragged_batches(ft, batch, out):
    for N, K in ((256, 512), (200, 272)):
        _fp8_case(ft, BATCHES[batch], N, K, out)


@pytest.mark.parametrize("N,K", [(128, 128), (1, 16), (129, 144), (77, 2000), (300, 96), (1024, 2048), (513, 1040)])
def test_fp8_widths(ft, N, K):
    _fp8_case(ft, [5, 0, 70, 300, 1], N, K, torch.float32, seed=1)


@pytest.mark.parametrize("P", [1, 3, 16, 17, 129, 1000, 2500])
def test_fp8_plain_product(ft, P):
    _fp8_case(ft, [P], 640, 1024, torch.bfloat16, seed=2, offs=False)


def test_fp8_large_batches_and_strides(ft):
    _fp8_case(ft, [700, 1300, 0, 513, 256, 1025, 3, 900], 776, 528, torch.bfloat16, seed=3)
    _fp8_case(ft, [700, 1300, 0, 513], 771, 528, torch.bfloat16, seed=3, strided=True)
    _fp8_case(ft, [20, 0, 33], 130, 272, torch.float32, seed=4, strided=True)


def test_fp8_wide_tiles(ft):
    """Both output types, widths that end inside a tile, rows without 16-byte pieces."""
    sizes = [700, 1300, 0, 513, 256, 1025, 3, 900]
    for N, K, out, strided in ((1300, 272, torch.float32, False), (1024, 144, torch.float32, True),
                               (1101, 128, torch.bfloat16, False), (1040, 1040, torch.bfloat16, True)):
        _fp8_case(ft, sizes, N, K, out, seed=5, strided=strided)


@pytest.mark.parametrize("N", [256, 300, 200, 1000])
def test_fp8_remainders_of_wide_tiles(ft, N):
    """Remainders on both sides of half a tile (128 rows), of a CTA's share (64) and of a box (32)."""
    sizes = [256 + r for r in (0, 1, 31, 33, 64, 65, 127, 128, 129, 255)] + [512 + 100, 512 + 190, 40, 0, 130]
    sizes = sizes * 3 if N <= 300 else sizes
    _fp8_case(ft, sizes, N, 272, torch.float32, seed=6)
    _fp8_case(ft, sizes, N, 400, torch.bfloat16, seed=7)


def test_fp8_on_another_stream_and_captured(ft):
    gen = torch.Generator(device="cuda").manual_seed(12)
    P, N, K = 300, 256, 384
    x, w = _randn(gen, P, K), _e4m3(gen, 2, N, K)
    wsc, offs = torch.rand((2, 2, 3), generator=gen, device="cuda"), _offs([100, 200])
    codes, scales = torch.empty((P, K), dtype=torch.uint8, device="cuda"), torch.empty((3, P), device="cuda")
    y, ws = torch.empty((P, N), device="cuda"), _ws(ft, 2, P, N, K)

    def step():
        ft.ft_moe_quantize_fp8(x, codes, scales)
        ft.ft_moe_group_gemm_fp8(codes, scales, w, wsc, offs, y, ws)

    step()
    first = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.zero_()
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, first)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)


def test_offsets_beyond_32_bits(ft):
    """Outputs and weights of more than 2^31 elements: the last rows and the last expert are right."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    P, N, K = 1 << 18, 8448, 64  # 2.2e9 output elements
    x, w = _randn(gen, P, K), _randn(gen, 1, N, K)
    y = torch.empty((P, N), dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_group_gemm(x, w, None, y, _ws(ft, 1, P, N, K))
    xq, xs = torch.empty((P, K), dtype=torch.uint8, device="cuda"), torch.empty((1, P), device="cuda")
    ft.ft_moe_quantize_fp8(x, xq, xs)
    wq, wsc = w.float().to(torch.float8_e4m3fn), torch.ones((1, N // 128, 1), device="cuda")
    rows = slice(P - 300, P)
    ref = x[rows].double() @ w[0].double().t()
    mag = x[rows].double().abs() @ w[0].double().abs().t()
    _close(y[rows], ref, mag, K, torch.bfloat16)
    ft.ft_moe_group_gemm_fp8(xq, xs, wq, wsc, None, y, _ws(ft, 1, P, N, K))
    xd = xq[rows].view(torch.float8_e4m3fn).double() * xs[0, rows, None].double()
    _close(y[rows], xd @ wq[0].double().t(), xd.abs() @ wq[0].double().abs().t(), K, torch.bfloat16, extra=4 * 2.0 ** -23)
    del y
    E, N, K = 520, 2048, 2048    # 2.2e9 weights
    sizes = [0] * (E - 2) + [40, 25]
    x, dy = _randn(gen, 65, K), _randn(gen, 65, N)
    dw = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_group_gemm_wgrad(dy, x, _offs(sizes), dw, _ws(ft, E, 65, N, K))
    assert not dw[E - 3].any()
    for e, r in ((E - 2, slice(0, 40)), (E - 1, slice(40, 65))):
        ref = dy[r].double().t() @ x[r].double()
        _close(dw[e], ref, dy[r].double().abs().t() @ x[r].double().abs(), 40, torch.bfloat16)
    out = torch.empty((65, N), device="cuda")
    ft.ft_moe_group_gemm(x, dw, _offs(sizes), out, _ws(ft, E, 65, N, K))
    _close(out[40:], x[40:].double() @ dw[E - 1].double().t(), x[40:].double().abs() @ dw[E - 1].double().abs().t(), K,
           torch.float32)


def test_fp8_values_that_are_not_finite_stay_in_their_rows(ft):
    """0x7F is NaN; an infinite scale: only the rows that hold them notice."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    P, N, K = 60, 192, 256
    offs = _offs([30, 30])
    x, w = _e4m3(gen, P, K).view(torch.uint8), _e4m3(gen, 2, N, K)
    xs, wsc = torch.ones((2, P), device="cuda"), torch.ones((2, 2, 2), device="cuda")
    good = torch.empty((P, N), device="cuda")
    ft.ft_moe_group_gemm_fp8(x, xs, w, wsc, offs, good, _ws(ft, 2, P, N, K))
    x[7, 200] = 0x7F
    xs[1, 31] = float("inf")
    got = torch.empty((P, N), device="cuda")
    ft.ft_moe_group_gemm_fp8(x, xs, w, wsc, offs, got, _ws(ft, 2, P, N, K))
    keep = torch.ones(P, dtype=torch.bool, device="cuda")
    keep[7] = keep[31] = False
    assert torch.equal(got[keep], good[keep]) and not torch.isfinite(got[~keep]).any()
