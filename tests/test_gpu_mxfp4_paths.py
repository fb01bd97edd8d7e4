"""Every kernel variant of the MXFP4 product, named: each case states the variant that its sizes are meant for and checks
that the dispatch takes it (ft_moe_debug_group_plan), then checks results against 64 bits, repeats, streams, replays and
threads to the bit, a stalled pipeline, and the largest sizes. Tolerances as in the product's other tests: exact terms,
(K / 64 + 8) additions of 2^-22 of the magnitudes, one rounding at the store.
"""
import threading

import pytest
import torch

from mxfp4_cases import decode, random_weights, row_scales, tiles_of

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
SOME = [(53 * i) % 500 for i in range(60)]                        # 60 experts, 225 rows each
LARGE = [700, 1300, 0, 513, 256, 1025, 3, 900]
SMALL = [3, 0, 17, 40, 1, 0, 33, 16]
MANY = [(37 * i) % 41 for i in range(1000)] + [0] * 24            # 1024 experts, 20 rows each

# (CTAs per tile, tile extent, contraction shared)
CASES = {
    "pairs, bf16": (LARGE, 1504, 544, BF, (2, 256, False)),
    "pairs, fp32": (LARGE, 1540, 2336, F32, (2, 256, False)),
    "pairs, odd rows of y": (SOME, 1001, 96, BF, (2, 256, False)),
    "pairs, short contraction": (SOME, 1000, 32, F32, (2, 256, False)),
    "128 rows, bf16": (SOME, 192, 544, BF, (1, 128, False)),
    "128 rows, fp32": (SOME, 131, 2400, F32, (1, 128, False)),
    "128 rows, shared": ([3000], 256, 2048, BF, (1, 128, True)),
    "128 rows, shared, fp32": ([1600], 510, 4128, F32, (1, 128, True)),
    "32 rows, fp32": (SMALL, 4099, 160, F32, (1, 32, False)),
    "32 rows, bf16": (MANY, 136, 288, BF, (1, 32, False)),
    "32 rows, shared": (SMALL, 130, 2080, BF, (1, 32, True)),
    "32 rows, shared, fp32": ([5], 640, 8192, F32, (1, 32, True)),
}


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


class Case:
    def __init__(self, ft, name):
        self.ft = ft
        self.sizes, self.N, self.K, self.out, want = CASES[name]
        self.E, self.P = len(self.sizes), sum(self.sizes)
        ctas, tile, split, counted = ft.ft_moe_debug_group_plan(ft.FT_GROUP_MXFP4, self.E, self.P, self.N, self.K, self.out)
        assert (ctas, tile, split > 1, counted) == (*want, 0)
        self.gen = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn((self.P, self.K), generator=self.gen, device="cuda")
        self.codes, self.xs = torch.empty((self.P, self.K // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(self.P, self.K)
        ft.ft_moe_quantize_mxfp4(x, self.codes, self.xs)
        self.w, self.ws = random_weights(self.gen, self.E, self.N, self.K, 2)
        self.tiles = tiles_of(self.ws)
        self.offs = torch.tensor([0, *self.sizes], device="cuda").cumsum(0).int()
        self.work = torch.zeros(256, dtype=U8, device="cuda")

    def empty(self):
        return torch.full((self.P, self.N), 7.0, dtype=self.out, device="cuda")

    def run(self, y, work=None, stream=None):
        self.ft.ft_moe_group_gemm_mxfp4(self.codes, self.xs, self.w, self.tiles, self.offs, y, self.work if work is None else work,
                                        stream=stream)
        return y

    def check(self, y):
        assert self.ft.ft_moe_read_status(self.work) == 0
        x64, at = decode(self.codes, row_scales(self.xs, self.K)), 0
        store = 2.0 ** -8 if self.out == BF else 2.0 ** -24
        for e, n in enumerate(self.sizes):
            if n == 0 or (self.E > 100 and e % 7):
                at += n
                continue
            w64, rows = decode(self.w[e], self.ws[e]), x64[at:at + n]
            ref, mag = rows @ w64.t(), rows.abs() @ w64.abs().t()
            err = (y[at:at + n].double() - ref).abs()
            assert (err <= store * 1.01 * ref.abs() + (self.K / 64 + 8) * 2.0 ** -22 * mag).all(), e
            at += n


@pytest.mark.parametrize("name", list(CASES))
def test_results(ft, name):
    c = Case(ft, name)
    y = c.run(c.empty())
    c.check(y)
    for _ in range(3):
        assert torch.equal(c.run(c.empty()), y)


@pytest.mark.parametrize("name", list(CASES))
def test_other_streams_and_replays(ft, name):
    """On a stream of its own, and captured twice into graphs with a workspace each, replayed on two streams at once after
    the inputs changed: the results of calls on the new inputs."""
    c = Case(ft, name)
    side = torch.cuda.Stream()
    first = c.run(c.empty())
    torch.cuda.synchronize()
    y = c.empty()
    torch.cuda.synchronize()
    c.run(y, stream=side)
    side.synchronize()
    assert torch.equal(y, first)
    ys, works, graphs = [c.empty(), c.empty()], [torch.zeros(256, dtype=U8, device="cuda") for _ in range(2)], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(ys[i], works[i])
        graphs.append(g)
    c.codes.copy_(torch.randint(0, 256, c.codes.shape, generator=c.gen, device="cuda", dtype=U8))
    c.xs.copy_(torch.randint(125, 130, c.xs.shape, generator=c.gen, device="cuda", dtype=U8))
    if c.K % 128:
        c.xs[-1, :, c.K % 128 // 32:] = 0
    want = c.run(c.empty())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)
    assert all(ft.ft_moe_read_status(w) == 0 for w in works)
    c.check(want)


@pytest.mark.parametrize("name", list(CASES))
def test_a_stalled_pipeline_ends_with_an_error(ft, name):
    c = Case(ft, name)
    want = c.run(c.empty())
    ft.ft_moe_debug_inject_stall(5_000_000, 1)
    c.run(c.empty())
    assert ft.STATUS[ft.ft_moe_read_status(c.work)] == "FT_ERR_TIMEOUT"
    assert torch.equal(c.run(c.empty()), want) and ft.ft_moe_read_status(c.work) == 0


@pytest.mark.parametrize("name", list(CASES))
def test_bad_offsets_compute_nothing(ft, name):
    """Ranges that overlap, decrease or leave the rows: reported, y left as it was, and the next call is right."""
    c = Case(ft, name)
    y = torch.full_like(c.empty(), 7.0)
    good, E, P = c.offs, c.E, c.P
    swing = torch.tensor([0, P] * E, dtype=torch.int32, device="cuda")[:E + 1]  # 0, P, 0, P, ...
    if E > 1:
        bad = [swing, torch.cat([good[:-1], good[-1:] + 1]), torch.cat([good[:1] - 1, good[1:]])]
    else:
        bad = [torch.tensor([0, P + 1], dtype=torch.int32, device="cuda"), torch.tensor([P, 0], dtype=torch.int32, device="cuda")]
    for offs in bad:
        c.offs = offs
        c.run(y)
        assert ft.STATUS[ft.ft_moe_read_status(c.work)] == "FT_ERR_INVALID_ROUTING"
        assert (y == 7).all()
    c.offs = good
    c.run(y)
    assert ft.ft_moe_read_status(c.work) == 0
    c.check(y)


@pytest.mark.parametrize("name", ["pairs, bf16", "32 rows, fp32"])
def test_first_call_of_a_thread(ft, name):
    c = Case(ft, name)
    want, y, failed = c.run(c.empty()), c.empty(), []
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        try:
            c.run(y, stream=stream)
        except Exception as error:  # noqa: BLE001 - reported below, from the test's own thread
            failed.append(str(error))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert torch.equal(y, want)


@pytest.mark.parametrize("P,N,dtype", [(40000, 65536, BF), (35000, 65535, F32)])
def test_more_than_2_31_elements(ft, P, N, dtype):
    """Outputs behind 2^31 elements, of the widest matrix."""
    K, E = 64, 3
    gen = torch.Generator(device="cuda").manual_seed(2)
    sizes = [P - 7, 0, 7]
    codes = torch.randint(0, 256, (P, K // 2), generator=gen, device="cuda", dtype=U8)
    xs = ft.alloc_mxfp4_scales(P, K)
    xs.fill_(0)
    xs[:, :, :2] = torch.randint(126, 129, (1, P, 2), generator=gen, device="cuda", dtype=U8)
    w, ws = random_weights(gen, E, N, K)
    y, work = torch.empty((P, N), dtype=dtype, device="cuda"), torch.zeros(256, dtype=U8, device="cuda")
    offs = torch.tensor([0, *sizes], device="cuda").cumsum(0).int()
    ft.ft_moe_group_gemm_mxfp4(codes, xs, w, tiles_of(ws), offs, y, work)
    assert ft.ft_moe_read_status(work) == 0
    for a, b, e in ((0, 40, 0), (P - 60, P - 7, 0), (P - 7, P, 2)):
        x64, w64 = decode(codes[a:b], row_scales(xs[:, a:b], K)), decode(w[e], ws[e])
        ref = x64 @ w64.t()
        assert ((y[a:b].double() - ref).abs() <= 2.0 ** -8 * ref.abs()).all()


def test_long_contractions(ft):
    """65536 steps: fp32 sums come from parts, and lose less than the products of one sign would in one accumulation."""
    K, N = 65536, 130
    gen = torch.Generator(device="cuda").manual_seed(3)
    for P in (3, 100, 3000):
        codes = torch.randint(0, 8, (P, K // 2), generator=gen, device="cuda", dtype=U8) | 0x20  # positive values
        xs = ft.alloc_mxfp4_scales(P, K)
        xs.copy_(torch.randint(126, 129, xs.shape, generator=gen, device="cuda", dtype=U8))
        w = torch.randint(0, 8, (1, N, K // 2), generator=gen, device="cuda", dtype=U8) | 0x30
        ws = torch.randint(126, 129, (1, N, K // 32), generator=gen, device="cuda", dtype=U8)
        y, work = torch.empty((P, N), device="cuda"), torch.zeros(256, dtype=U8, device="cuda")
        ft.ft_moe_group_gemm_mxfp4(codes, xs, w, tiles_of(ws), None, y, work)
        ref = decode(codes, row_scales(xs, K)) @ decode(w[0], ws[0]).t()
        # 32 truncations of at most 2^-22 in a part, 32 additions of 2^-24 of parts
        assert ((y.double() - ref).abs() <= (32 * 2.0 ** -22 + 32 * 2.0 ** -24) * ref).all()


def test_strided_rows(ft):
    """Codes, scales and results with gaps between their rows, which stay as they were."""
    for P, N, K in ((10, 200, 160), (400, 200, 288), (3000, 1008, 96)):
        gen = torch.Generator(device="cuda").manual_seed(P)
        codes = torch.randint(0, 256, (P, K // 2 + 48), generator=gen, device="cuda", dtype=U8)
        kt = (K + 127) // 128
        xs = torch.full((kt, P // 4 * 4 + 12, 4), 255, dtype=U8, device="cuda")
        xs[:, :P] = torch.randint(125, 130, (kt, P, 4), generator=gen, device="cuda", dtype=U8)
        if K % 128:
            xs[-1, :P, K % 128 // 32:] = 0
        w, ws = random_weights(gen, 1, N, K)
        y, work = torch.full((P, N + 24), 7.0, device="cuda"), torch.zeros(256, dtype=U8, device="cuda")
        ft.ft_moe_group_gemm_mxfp4(codes[:, :K // 2], xs[:, :P], w, tiles_of(ws), None, y[:, :N], work)
        ref = decode(codes[:, :K // 2], row_scales(xs[:, :P], K)) @ decode(w[0], ws[0]).t()
        mag = decode(codes[:, :K // 2], row_scales(xs[:, :P], K)).abs() @ decode(w[0], ws[0]).abs().t()
        assert ((y[:, :N].double() - ref).abs() <= 2.0 ** -24 * ref.abs() + (K / 64 + 8) * 2.0 ** -22 * mag).all()
        assert (y[:, N:] == 7).all()
