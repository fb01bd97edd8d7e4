"""The residual RMS norm and its gradient, through the C ABI, against the formulas in 64 bits.

Tolerances. The total is one fp32 addition, rounded to bf16 where it is stored so (2^-8 relative, and 2^-24 of the
operands before). A sum of H squares in fp32 is off by at most H 2^-24 relative; in a tree of short chains it is
far less, and H 2^-24 is allowed. y takes three more roundings of 2^-24 and the store's 2^-8 (bf16).
e4m3 values are off by half a step: 2^-4 of the value, or 2^-10 of the block's scale near zero.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _rows(gen, rows, H, pad, dtype=BF, scale=1.0):
    """A [rows, H] view whose rows are H + pad elements apart."""
    return (torch.randn((rows, H + pad), generator=gen, device="cuda") * scale).to(dtype)[:, :H]


def _gap(t, rows, H, pad):
    """What lies between the rows of an output made by _out."""
    return t._base[:, H:] if pad else t.new_full((1,), 7.0)


def _out(rows, H, pad, dtype):
    return torch.full((rows, H + pad), 7.0, dtype=dtype, device="cuda")[:, :H]


# H: every kernel variant (threads per row) and its edges, odd widths, a single column; pad: rows not 16-byte aligned
CASES = [(1, 1, 0), (3, 8, 0), (5, 31, 0), (1, 256, 0), (130, 256, 0), (7, 264, 8), (4, 1024, 0), (1, 2048, 0), (301, 2048, 0),
         (9, 2049, 1), (3, 4096, 0), (2, 5000, 3), (2, 8192, 0), (5, 8200, 0), (2, 16384, 0), (3, 16383, 0), (4000, 64, 0),
         (1000, 640, 3)]


@pytest.mark.parametrize("res", ["none", "bf16", "f32", "in place"])
@pytest.mark.parametrize("rows,H,pad", CASES)
def test_forward(ft, rows, H, pad, res):
    gen = torch.Generator(device="cuda").manual_seed(rows + H)
    x = _rows(gen, rows, H, pad)
    w_dtype, offset = (F32, 1.0) if H % 3 == 0 else (BF, 0.0)
    w = (torch.randn(H, generator=gen, device="cuda") * 0.3 + 1 - offset).to(w_dtype)
    kind = F32 if res == "f32" else BF
    r = None if res == "none" else _rows(gen, rows, H, pad, kind, 3.0)
    want = x.double() if r is None else x.double() + r.double()
    total = None if r is None else (r if res == "in place" else _out(rows, H, pad, kind))
    y, rstd = _out(rows, H, pad, BF), torch.full((rows,), -1.0, device="cuda")
    rc = None if r is None else r.double()
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=r, total=total, rstd=rstd, weight_offset=offset)
    if r is not None:
        step = 2.0 ** -24 if kind == F32 else 2.0 ** -8
        assert ((total.double() - want).abs() <= step * 1.001 * want.abs() + 2.0 ** -24 * (x.double().abs() + rc.abs())).all()
        want = total.double()
    mean = want.pow(2).mean(1)
    ref = (mean + EPS).rsqrt()
    assert ((rstd.double() - ref).abs() <= (H + 4) * 2.0 ** -24 * ref).all()
    yref = want * ref[:, None] * (w.double() + offset)
    bound = (2.0 ** -8 + (H + 8) * 2.0 ** -24) * want.abs() * ref[:, None] * (w.double().abs() + offset) + 1e-38
    assert ((y.double() - yref).abs() <= bound).all()
    assert (_gap(y, rows, H, pad) == 7).all()


@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("rows,H,pad", [(1, 16, 0), (1, 2048, 0), (65, 144, 0), (9, 2000, 16), (33, 4096, 0), (4, 16384, 0), (3, 272, 3)])
def test_forward_in_8_bits(ft, rows, H, pad, res):
    """Codes and scales of y by the quantizer's rule; with both outputs, y as without the codes. `pad` 3: rows of x that
    are not 16-byte aligned."""
    gen = torch.Generator(device="cuda").manual_seed(rows * 3 + H)
    x = _rows(gen, rows, H, pad)
    r = None if res is None else _rows(gen, rows, H, pad, res, 2.0)
    w = torch.randn(H, generator=gen, device="cuda").bfloat16()
    total = None if r is None else torch.empty((rows, H), dtype=res, device="cuda")
    codes = torch.full((rows, H + 16), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full(((H + 127) // 128, rows + 3), -1.0, device="cuda")
    y, alone = torch.empty((rows, H), dtype=BF, device="cuda"), torch.empty((rows, H), dtype=BF, device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=r, total=total, codes=codes[:, :H], scales=scales[:, :rows])
    assert (codes[:, H:] == 0xAA).all() and (scales[:, rows:] == -1).all()
    ft.ft_moe_rmsnorm(x, w, EPS, y=alone, residual=r, total=total)
    assert torch.equal(y, alone)
    again, sc2 = torch.empty((rows, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(scales)[:, :rows]
    ft.ft_moe_rmsnorm(x, w, EPS, residual=r, total=total, codes=again, scales=sc2)
    assert torch.equal(again.view(torch.uint8), codes[:, :H]) and torch.equal(sc2, scales[:, :rows])
    t = x.double() if r is None else total.double()
    ref = t * (t.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * w.double()
    nb = scales.shape[0]
    amax = torch.nn.functional.pad(ref, (0, nb * 128 - H)).view(rows, nb, 128).abs().amax(2).t()
    fine = (H + 8) * 2.0 ** -24
    assert ((scales[:, :rows].double() - amax / 448).abs() <= fine * amax / 448 + 2.0 ** -126).all()
    s = scales[:, :rows].double().t().repeat_interleave(128, 1)[:, :H]
    value = codes[:, :H].contiguous().view(torch.float8_e4m3fn).double() * s
    assert ((value - ref).abs() <= (2.0 ** -4 + 2 * fine) * ref.abs() + 2.0 ** -10 * 1.01 * s).all()


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("past", [False, True, "in place"])
@pytest.mark.parametrize("rows,H,pad", CASES)
def test_backward(ft, rows, H, pad, past, kind):
    """dx within the store's rounding and fp32 sums of magnitudes, dw within sums over the rows; twice the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(rows + 2 * H)
    total = _rows(gen, rows, H, pad, kind, 3.0)
    dy = _rows(gen, rows, H, pad, BF, 0.1)
    w_dtype, offset = (F32, 1.0) if H % 3 == 0 else (BF, 0.0)
    w = (torch.randn(H, generator=gen, device="cuda") * 0.3 + 1 - offset).to(w_dtype)
    rstd = (total.double().pow(2).mean(1) + EPS).rsqrt().float()
    ds = _rows(gen, rows, H, pad, kind, 0.1) if past else None
    ds64 = ds.double() if past else torch.zeros((rows, H), dtype=torch.float64, device="cuda")
    dx = ds if past == "in place" else _out(rows, H, pad, kind)
    ws = torch.full((ft.ft_moe_rmsnorm_workspace_size(rows, H),), 0xFF, dtype=torch.uint8, device="cuda")
    dw = torch.full((H,), float("nan"), device="cuda")
    keep = ds.clone() if past == "in place" else ds
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx, ws, dw=dw, dtotal=ds, weight_offset=offset)
    n, g = total.double() * rstd.double()[:, None], dy.double() * (w.double() + offset)
    c = (g * n).mean(1, keepdim=True)
    ref = ds64 + rstd.double()[:, None] * (g - n * c)
    mag = rstd.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    step = 2.0 ** -24 if kind == F32 else 2.0 ** -8
    assert ((dx.double() - ref).abs() <= step * 1.01 * ref.abs() + (H + 8) * 2.0 ** -24 * mag + 2.0 ** -23 * ds64.abs() + 1e-38).all()
    if past != "in place":
        assert (_gap(dx, rows, H, pad) == 7).all()
    dref, dmag = (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)
    assert ((dw.double() - dref).abs() <= (rows + 8) * 2.0 ** -24 * dmag + 1e-38).all()
    dx2, dw2 = torch.empty((rows, H), dtype=kind, device="cuda"), dw.clone()
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx2, ws, dw=dw2, dtotal=keep, weight_offset=offset, accumulate=True)
    assert torch.equal(dx2, dx)
    assert ((dw2.double() - 2 * dw.double()).abs() <= 2.0 ** -24 * 1.01 * (2 * dw.double()).abs()).all()
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx2, ws, dw=dw2, dtotal=keep, weight_offset=offset)
    assert torch.equal(dw2, dw)
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx2, dtotal=keep, weight_offset=offset)  # no dw, no workspace
    assert torch.equal(dx2, dx)


def test_backward_matches_differences(ft):
    """Central differences of the forward formula in 64 bits (step 1e-5: error ~ step^2)."""
    rows, H = 3, 40
    gen = torch.Generator(device="cuda").manual_seed(5)
    total = _rows(gen, rows, H, 0, F32)
    dy, w = _rows(gen, rows, H, 0), torch.randn(H, generator=gen, device="cuda")
    rstd = (total.double().pow(2).mean(1) + EPS).rsqrt().float()
    dx, dw = torch.empty((rows, H), device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(ft.ft_moe_rmsnorm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx, ws, dw=dw)

    def loss(t, g):
        return (dy.double() * t * (t.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * g).sum()

    t64, w64, h = total.double(), w.double(), 1e-5
    for at in range(0, rows * H, 7):
        e = torch.zeros_like(t64)
        e.view(-1)[at] = h
        d = (loss(t64 + e, w64) - loss(t64 - e, w64)) / (2 * h)
        assert abs(float(dx.view(-1)[at]) - float(d)) <= 1e-5 * (1 + abs(float(d)))
    for at in range(H):
        e = torch.zeros_like(w64)
        e[at] = h
        d = (loss(t64, w64 + e) - loss(t64, w64 - e)) / (2 * h)
        assert abs(float(dw[at]) - float(d)) <= 1e-5 * (1 + abs(float(d)))


def test_rows_stay_apart(ft):
    """A row that is not finite, an all-zero row (eps alone) and large values leave their neighbours as they are."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = _rows(gen, 12, 256, 0)
    x[1, 5], x[4, 0], x[6] = float("inf"), float("nan"), 0.0
    w = torch.ones(256, device="cuda")
    y, codes = torch.empty((12, 256), dtype=BF, device="cuda"), torch.empty((12, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((2, 12), device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, codes=codes, scales=scales)
    fine = [i for i in range(12) if i not in (1, 4)]
    ref = x.double()[fine] * (x.double()[fine].pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    assert ((y[fine].double() - ref).abs() <= 2.0 ** -8 * ref.abs()).all()
    assert not y[6].any() and torch.isfinite(scales[:, fine]).all()
    assert torch.isnan(y[4]).all() and torch.isnan(y[1, 5])


def test_no_rows(ft):
    x, w = torch.empty((0, 64), dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=x)
    dw = torch.ones(64, device="cuda")
    rstd, ws = torch.empty(0, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    ft.ft_moe_rmsnorm_backward(x, x, w, rstd, x, ws, dw=dw, accumulate=True)
    assert (dw == 1).all()
    ft.ft_moe_rmsnorm_backward(x, x, w, rstd, x, ws, dw=dw)
    assert (dw == 0).all()


def test_streams_and_replays(ft):
    """On a stream of its own, and captured into two graphs with a workspace each that are replayed at once after the inputs
    changed: the results of calls on the new inputs."""
    rows, H = 700, 640
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, r, dy = _rows(gen, rows, H, 0), _rows(gen, rows, H, 0), _rows(gen, rows, H, 0)
    w = torch.randn(H, generator=gen, device="cuda")

    class Run:
        def __init__(self):
            self.total, self.y, self.dx = (torch.zeros((rows, H), dtype=BF, device="cuda") for _ in range(3))
            self.rstd, self.dw = torch.zeros(rows, device="cuda"), torch.zeros(H, device="cuda")
            self.ws = torch.zeros(ft.ft_moe_rmsnorm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")

        def __call__(self, stream=None):
            ft.ft_moe_rmsnorm(x, w, EPS, y=self.y, residual=r, total=self.total, rstd=self.rstd, stream=stream)
            ft.ft_moe_rmsnorm_backward(dy, self.total, w, self.rstd, self.dx, self.ws, dw=self.dw, stream=stream)

        def same(self, other):
            return all(torch.equal(getattr(self, n), getattr(other, n)) for n in ("total", "y", "dx", "rstd", "dw"))

    plain, aside, side = Run(), Run(), torch.cuda.Stream()
    plain()
    torch.cuda.synchronize()
    aside(side)
    side.synchronize()
    assert aside.same(plain)
    runs, graphs = [Run(), Run()], []
    for run in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for t in (x, r, dy):
        t.copy_(_rows(gen, rows, H, 0))
    plain()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(run.same(plain) for run in runs)


def test_more_than_2_31_elements(ft):
    """Rows behind 2^31 elements: the last rows come out as the first ones."""
    rows, H = (1 << 31) // 16384 + 8, 16384
    x = torch.zeros((rows, H), dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(8)
    x[-8:] = x[:8] = _rows(gen, 8, H, 0)
    w = torch.ones(H, device="cuda")
    total, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    codes, scales = torch.empty((rows, H), dtype=torch.uint8, device="cuda"), torch.empty((128, rows), device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=x, total=total, codes=codes, scales=scales, rstd=rstd)
    for t in (total, y, codes):
        assert torch.equal(t[-8:], t[:8]) and t[:8].any()
    assert torch.equal(scales[:, -8:], scales[:, :8])
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(ft.ft_moe_rmsnorm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    ft.ft_moe_rmsnorm_backward(x, total, w, rstd, dx, ws, dw=dw, dtotal=x)
    assert torch.equal(dx[-8:], dx[:8]) and dx[:8].any()
