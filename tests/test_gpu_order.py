"""Tokens sorted by expert and back, through the C ABI: copies and positions bit for bit, sums against 64 bits.

A weighted sum of k rows in fp32 takes k fused multiply-adds (and the addition of `add`): off by (k + 1) 2^-24 of the
terms' magnitudes; the bf16 store by 2^-8. A dot product over H takes at most H + 5 additions of 2^-24.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _align(ft, ids, E, block=1):
    """sorted_slot, offsets and count of ft_moe_align."""
    T, k = ids.shape
    n = T * k + min(E, T * k) * (block - 1)
    slot = torch.full((n,), -5, dtype=I32, device="cuda")
    blocks, offs = torch.empty(n // block + 1, dtype=I32, device="cuda"), torch.empty(E + 1, dtype=I32, device="cuda")
    count = torch.empty(1, dtype=I32, device="cuda")
    ws = torch.empty(ft.ft_moe_align_workspace_size(T, k, E), dtype=U8, device="cuda")
    ft.ft_moe_align(ids, E, block, slot, blocks, offs, count, ws)
    return slot, offs, count


def _ids(gen, T, k, E):
    return torch.rand((T, E), generator=gen, device="cuda").topk(k, 1).indices.int()


def _order(gen, T, k, E):
    flat = _ids(gen, T, k, E).reshape(-1)
    slot = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(slot)
    pos[slot] = torch.arange(slot.numel(), device="cuda")
    return slot.int(), pos.view(T, k).int()


# rows of 16-byte pieces and not, one column, several warps a row; slots on both sides of the one-CTA limit
@pytest.mark.parametrize("dtype", [BF, F32, U8])
@pytest.mark.parametrize("T,k,E,H,pad", [(1, 1, 1, 16, 0), (1, 8, 16, 2048, 0), (37, 2, 8, 34, 2), (300, 8, 60, 640, 0), (700, 8, 256, 72, 8),
                                         (513, 8, 8, 130, 0), (5, 32, 64, 5000, 0), (900, 4, 8, 8, 0), (2000, 2, 8, 2, 0),
                                         (33, 3, 8, 128, 0), (70, 8, 16, 30, 6)])
def test_dispatch(ft, T, k, E, H, pad, dtype):
    gen = _gen(T + H)
    x = (torch.randn((T, H + pad), generator=gen, device="cuda") * 50).to(dtype)[:, :H]
    ids = _ids(gen, T, k, E)
    slot, offs, count = _align(ft, ids, E)
    w = torch.rand((T, k), generator=gen, device="cuda")
    out = torch.full((T * k, H + pad), 3, dtype=dtype, device="cuda")
    row_w, pos = torch.empty(T * k, device="cuda"), torch.full((T, k), 77, dtype=I32, device="cuda")
    ft.ft_moe_dispatch(x, slot, k, out[:, :H], w=w, row_w=row_w, pos=pos, count=count)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(slot.long(), order)
    assert torch.equal(out[:, :H], x[order // k])
    assert (out[:, H:] == 3).all()
    assert torch.equal(row_w, w.reshape(-1)[order])
    assert torch.equal(pos.reshape(-1)[order].long(), torch.arange(T * k, device="cuda"))
    plain = torch.empty((T * k, H), dtype=dtype, device="cuda")
    ft.ft_moe_dispatch(x, slot, k, plain)  # rows alone
    assert torch.equal(plain, out[:, :H])


@pytest.mark.parametrize("T,k,E,H", [(1, 8, 16, 2048), (64, 8, 256, 2048), (1000, 6, 60, 640), (3, 2, 4, 160)])
def test_dispatch_with_scales(ft, T, k, E, H):
    gen = _gen(T)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    slot, pos = _order(gen, T, k, E)
    token, nb, P = slot.long() // k, (H + 127) // 128, T * k
    codes, scales = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((nb, T), device="cuda")
    ft.ft_moe_quantize_fp8(x, codes, scales)
    out, os_ = torch.empty((P, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.full((nb, P + 5), -1.0, device="cuda")
    ft.ft_moe_dispatch(codes, slot, k, out, x_scale=scales, out_scale=os_[:, :P])
    assert torch.equal(out.view(U8), codes.view(U8)[token]) and torch.equal(os_[:, :P], scales[:, token]) and (os_[:, P:] == -1).all()
    c4, s4 = torch.empty((T, H // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(T, H)
    ft.ft_moe_quantize_mxfp4(x, c4, s4)
    out4, os4 = torch.empty((P, H // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(P, H)
    ft.ft_moe_dispatch(c4, slot, k, out4, x_scale=s4, out_scale=os4)
    assert torch.equal(out4, c4[token]) and torch.equal(os4, s4[:, token])


@pytest.mark.parametrize("T,k,E,block,H", [(40, 2, 8, 16, 64), (700, 8, 60, 8, 48)])
def test_padding_and_invalid_ids(ft, T, k, E, block, H):
    """Rows that hold no slot are zeros, rows behind the count stay as they were, slots without a row get position -1, and
    nothing of theirs is added."""
    gen = _gen(T * k)
    ids = _ids(gen, T, k, E)
    ids[3, 0], ids[5, 1] = E + 4, -1
    slot, offs, count = _align(ft, ids, E, block)
    n, P = int(count), slot.numel()
    x, w = torch.randn((T, H), generator=gen, device="cuda"), torch.rand((T, k), generator=gen, device="cuda")
    scales = torch.rand((1, T), generator=gen, device="cuda")
    out, row_w, pos = torch.full((P, H), 9.0, device="cuda"), torch.full((P,), 9.0, device="cuda"), torch.zeros((T, k), dtype=I32, device="cuda")
    os_ = torch.full((1, P), 9.0, device="cuda")
    ft.ft_moe_dispatch(x, slot, k, out, x_scale=scales, out_scale=os_, w=w, row_w=row_w, pos=pos, count=count)
    s = slot[:n].long()
    real = s < T * k
    assert real.sum() == T * k - 2 and not real.all()
    assert torch.equal(out[:n][real], x[s[real] // k]) and torch.equal(row_w[:n][real], w.reshape(-1)[s[real]])
    assert torch.equal(os_[0, :n][real], scales[0, s[real] // k])
    assert not out[:n][~real].any() and not row_w[:n][~real].any() and not os_[0, :n][~real].any()
    assert (out[n:] == 9).all() and (row_w[n:] == 9).all() and (os_[0, n:] == 9).all()
    flat = pos.reshape(-1)
    assert flat[3 * k] == -1 and flat[5 * k + 1] == -1 and (flat == -1).sum() == 2
    assert torch.equal(flat[s[real]].long(), real.nonzero()[:, 0])
    y = torch.randn((P, H), generator=gen, device="cuda")
    y[n:] = float("nan")
    got = torch.empty((T, H), device="cuda")
    ft.ft_moe_combine(y, pos, w, got)
    ref = torch.where(flat[:, None] >= 0, y[flat.clamp(min=0).long()].double() * w.reshape(-1, 1).double(), 0.0).view(T, k, H).sum(1)
    assert ((got.double() - ref).abs() <= (k + 1) * 2.0 ** -24 * 8 * k).all()
    dout = torch.randn((T, H), generator=gen, device="cuda")
    dy, dw = torch.full((P, H), 9.0, dtype=BF, device="cuda"), torch.empty((T, k), device="cuda")
    ft.ft_moe_combine_backward(dout, y, pos, w, dy, dw=dw)
    assert dw[3, 0] == 0 and dw[5, 1] == 0 and torch.isfinite(dw).all()
    free = torch.ones(P, dtype=torch.bool, device="cuda")
    free[flat[flat >= 0].long()] = False
    assert (dy[free] == 9).all() and torch.isfinite(dy[~free]).all()


def test_positions_out_of_range_reach_nothing(ft):
    T, k, P, H = 6, 3, 7, 64
    big = 2 ** 31 - 1
    pos = torch.tensor([[-1, 7, 0], [big, -big, 1], [2, 3, 4], [5, 6, 9], [8, 100, -9], [7, 7, 7]], dtype=I32, device="cuda")
    y = torch.randn((P, H), device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    live = (pos >= 0) & (pos < P)
    w[live] = 0.5
    out = torch.empty((T, H), device="cuda")
    ft.ft_moe_combine(y, pos, w, out)
    ref = torch.where(live[:, :, None], 0.5 * y[pos.clamp(0, P - 1).long()], 0.0).sum(1)
    assert torch.allclose(out, ref, rtol=1e-6, atol=1e-6) and not out[4].any() and not out[5].any()
    slot = torch.tensor([0, -3, big, 17, 18, -big, 2], dtype=I32, device="cuda")
    xs = torch.full((7, H), 9.0, device="cuda")
    ft.ft_moe_dispatch(y[:6], slot, 3, xs)
    assert torch.equal(xs[[0, 3, 6]], y[[0, 5, 0]]) and not xs[[1, 2, 4, 5]].any()


def test_a_slot_in_two_rows_counts_for_the_last(ft):
    for T, extra in ((4, 0), (3000, 3000)):
        slot = torch.arange(T, dtype=I32, device="cuda").repeat(2)
        pos = torch.empty((T, 1), dtype=I32, device="cuda")
        x = torch.zeros((T, 8), device="cuda")
        ft.ft_moe_dispatch(x, slot, 1, torch.empty((2 * T, 8), device="cuda"), pos=pos)
        assert torch.equal(pos[:, 0].long(), torch.arange(T, 2 * T, device="cuda"))


SUMS = [(1, 8, 16, 2048, 0), (1, 1, 1, 1, 0), (100, 32, 64, 8, 0), (777, 4, 8, 16, 0), (50, 9, 16, 2, 0), (300, 8, 60, 2056, 0),
        (40, 8, 60, 1025, 0), (300, 8, 60, 640, 0), (64, 6, 8, 33, 1), (17, 32, 64, 4100, 0), (1000, 2, 8, 264, 8)]


@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("T,k,E,H,pad", SUMS)
def test_combine(ft, T, k, E, H, pad, yt, ot):
    gen = _gen(T + k)
    slot, pos = _order(gen, T, k, E)
    y = torch.randn((T * k, H + pad), generator=gen, device="cuda").to(yt)[:, :H]
    w = torch.rand((T, k), generator=gen, device="cuda")
    add = torch.randn((T, H + pad), generator=gen, device="cuda").to(ot)[:, :H]
    step = 2.0 ** -24 if ot == F32 else 2.0 ** -8
    rows = y.double()[pos.long()]
    for weights, extra in ((w, None), (None, None), (w, add), (w, "in place")):
        out = torch.full((T, H + pad), 7.0, dtype=ot, device="cuda")[:, :H]
        terms = rows if weights is None else rows * weights.double()[:, :, None]
        ref, mag = terms.sum(1), terms.abs().sum(1)
        if extra is not None:
            ref, mag = ref + add.double(), mag + add.double().abs()
        if isinstance(extra, str):
            out.copy_(add)
            extra = out
        ft.ft_moe_combine(y, pos, weights, out, add=extra)
        assert ((out.double() - ref).abs() <= step * 1.01 * ref.abs() + (k + 2) * 2.0 ** -24 * mag + 1e-38).all()
        if pad:
            assert (out._base[:, H:] == 7).all()


@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("T,k,E,H,pad", SUMS)
def test_dispatch_backward(ft, T, k, E, H, pad, yt):
    gen = _gen(T + 2 * k)
    slot, pos = _order(gen, T, k, E)
    d = torch.randn((T * k, H + pad), generator=gen, device="cuda").to(yt)[:, :H]
    drow = torch.randn(T * k, generator=gen, device="cuda")
    for ot in (BF, F32):
        dx, dw = torch.empty((T, H), dtype=ot, device="cuda"), torch.empty((T, k), device="cuda")
        ft.ft_moe_dispatch_backward(d, pos, dx, drow_w=drow, dw=dw)
        ref, mag = d.double()[pos.long()].sum(1), d.double()[pos.long()].abs().sum(1)
        step = 2.0 ** -24 if ot == F32 else 2.0 ** -8
        assert ((dx.double() - ref).abs() <= step * 1.01 * ref.abs() + (k + 1) * 2.0 ** -24 * mag + 1e-38).all()
        assert torch.equal(dw, drow[pos.long()])
        again = torch.empty_like(dx)
        ft.ft_moe_dispatch_backward(d, pos, again)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,E,H,pad", SUMS)
def test_combine_backward(ft, T, k, E, H, pad, yt, dt):
    gen = _gen(T + 3 * k)
    slot, pos = _order(gen, T, k, E)
    y = torch.randn((T * k, H + pad), generator=gen, device="cuda").to(yt)[:, :H]
    dout = torch.randn((T, H + pad), generator=gen, device="cuda").to(dt)[:, :H]
    w = torch.rand((T, k), generator=gen, device="cuda")
    dy = torch.full((T * k, H + pad), 7.0, dtype=BF, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    ft.ft_moe_combine_backward(dout, y, pos, w, dy[:, :H], dw=dw)
    token = slot.long() // k
    ref = dout.double()[token] * w.double().reshape(-1)[slot.long()][:, None]
    assert ((dy[:, :H].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs() + 1e-38).all()
    assert (dy[:, H:] == 7).all()
    prod = dout.double()[:, None] * y.double()[pos.long()]
    assert ((dw.double() - prod.sum(2)).abs() <= (H + 8) * 2.0 ** -24 * prod.abs().sum(2) + 1e-38).all()
    again, dw2 = torch.empty((T * k, H), dtype=BF, device="cuda"), torch.empty((T, k), device="cuda")
    ft.ft_moe_combine_backward(dout, y, pos, w, again, dw=dw2)
    assert torch.equal(again, dy[:, :H]) and torch.equal(dw2, dw)
    ft.ft_moe_combine_backward(dout, None, pos, None, again)
    assert torch.equal(again, dout[token].bfloat16())


def test_nothing_to_do(ft):
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    ft.ft_moe_dispatch(z(0, 8), z(0, dtype=I32), 2, z(0, 8), pos=z(0, 2, dtype=I32))
    pos = z(3, 2, dtype=I32)
    ft.ft_moe_dispatch(z(3, 8), z(0, dtype=I32), 2, z(0, 8), pos=pos)
    assert (pos == -1).all()
    out = z(3, 8) + 5
    ft.ft_moe_combine(z(0, 8), pos, z(3, 2), out, add=out)
    assert (out == 5).all()
    ft.ft_moe_combine(z(0, 8), pos, None, out)
    assert (out == 0).all()
    dw = z(3, 2) + 1
    ft.ft_moe_combine_backward(z(3, 8), z(0, 8), pos, None, z(0, 8, dtype=BF), dw=dw)
    assert (dw == 0).all()
    rows = z(4, 8) + 1
    ft.ft_moe_dispatch(z(0, 8), z(4, dtype=I32), 2, rows)  # no token: every slot is out of range
    assert (rows == 0).all()


@pytest.mark.parametrize("T", [100, 1500])  # positions by one CTA, and cleared before the launch
def test_streams_and_replays(ft, T):
    """On a stream of its own, and captured and replayed after the routing changed: the results of calls on the new one."""
    k, E, H = 4, 16, 520
    gen = _gen(T)
    x, dout = torch.randn((T, H), generator=gen, device="cuda").bfloat16(), torch.randn((T, H), generator=gen, device="cuda")
    w = torch.rand((T, k), generator=gen, device="cuda")
    slot, _ = _order(gen, T, k, E)

    class Run:
        def __init__(self):
            self.xs, self.dy = (torch.zeros((T * k, H), dtype=BF, device="cuda") for _ in range(2))
            self.pos, self.row_w = torch.zeros((T, k), dtype=I32, device="cuda"), torch.zeros(T * k, device="cuda")
            self.out, self.dx = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), dtype=BF, device="cuda")
            self.dw, self.dw2 = torch.zeros((T, k), device="cuda"), torch.zeros((T, k), device="cuda")

        def __call__(self, stream=None):
            ft.ft_moe_dispatch(x, slot, k, self.xs, w=w, row_w=self.row_w, pos=self.pos, stream=stream)
            ft.ft_moe_combine(self.xs, self.pos, w, self.out, stream=stream)
            ft.ft_moe_combine_backward(dout, self.xs, self.pos, w, self.dy, dw=self.dw, stream=stream)
            ft.ft_moe_dispatch_backward(self.dy, self.pos, self.dx, drow_w=self.row_w, dw=self.dw2, stream=stream)

        def same(self, other):
            return all(torch.equal(a, b) for a, b in zip(vars(self).values(), vars(other).values()))

    plain, aside, side = Run(), Run(), torch.cuda.Stream()
    plain()
    torch.cuda.synchronize()
    aside(side)
    side.synchronize()
    assert aside.same(plain)
    run, g = Run(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    slot.copy_(_order(gen, T, k, E)[0])
    plain()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert run.same(plain)


def test_more_than_2_31_elements(ft):
    """The sorted rows behind 2^31 elements of a wide batch, there and back."""
    T, k, H = (1 << 20) // 8 + 16, 8, 2048
    gen = _gen(3)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    slot = torch.randperm(T * k, generator=gen, device="cuda").int()
    xs, pos = torch.empty((T * k, H), dtype=BF, device="cuda"), torch.empty((T, k), dtype=I32, device="cuda")
    ft.ft_moe_dispatch(x, slot, k, xs, pos=pos)
    for a in (0, T * k // 2, T * k - 1000):
        assert torch.equal(xs[a:a + 1000], x[slot[a:a + 1000].long() // k])
    w = torch.full((T, k), 0.125, device="cuda")
    out = torch.empty_like(x)
    ft.ft_moe_combine(xs, pos, w, out)
    assert torch.equal(out, x)
    dy, dw = torch.empty_like(xs), torch.empty((T, k), device="cuda")
    ft.ft_moe_combine_backward(x, xs, pos, None, dy, dw=dw)
    assert torch.equal(dy[-1000:], x[slot[-1000:].long() // k])
    ref = x[-100:].double().pow(2).sum(1)
    assert ((dw[-100:].double() - ref[:, None]).abs() <= 1e-4 * ref[:, None]).all()
