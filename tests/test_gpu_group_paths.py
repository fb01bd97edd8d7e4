"""Every kernel variant of the expert products, named: each case states the variant that its sizes are
meant for and checks that the dispatch takes it (ft_moe_debug_group_plan), then checks the results
against 64 bits, repeats and replays to the bit, values that are not finite beside finite ones, and
a pipeline that stalls.

Tolerances as the arithmetic gives them: products are exact in fp32, a sum of R of them is within
R * 2^-23 of the magnitudes, the 8-bit products add 2^-21 of them for the scales, the store rounds once.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FORWARD, DGRAD, WGRAD, FP8 = range(4)

MANY = [(37 * i) % 400 for i in range(200)] + [0, 900, 1, 2000]   # 204 experts, 214 rows each on average
SOME = [(53 * i) % 500 for i in range(60)]                        # 60 experts, 225 rows each
LARGE = [700, 1300, 0, 513, 256, 1025, 3, 900]
SMALL = [3, 0, 17, 40, 1, 0, 33, 16]

# (CTAs per tile, tile extent, contraction shared, counted)
CASES = {
    "wgrad, pairs, counted, bf16": (WGRAD, MANY, 512, 512, BF, False, (2, 256, False, True)),
    "wgrad, pairs, counted, fp32": (WGRAD, MANY, 512, 512, F32, False, (2, 256, False, True)),
    "wgrad, pairs, counted, added": (WGRAD, MANY, 512, 512, F32, True, (2, 256, False, True)),
    "wgrad, pairs, counted, bf16, odd": (WGRAD, MANY, 264, 328, BF, False, (2, 256, False, True)),
    "wgrad, pairs, counted, added, odd": (WGRAD, MANY, 328, 264, F32, True, (2, 256, False, True)),
    "wgrad, pairs, in turn, bf16": (WGRAD, SOME, 256, 256, BF, False, (2, 256, False, False)),
    "wgrad, pairs, in turn, fp32": (WGRAD, SOME, 200, 264, F32, False, (2, 256, False, False)),
    "wgrad, pairs, in turn, added": (WGRAD, SOME, 256, 200, F32, True, (2, 256, False, False)),
    "wgrad, single, bf16": (WGRAD, SOME, 304, 128, BF, False, (1, 256, False, False)),
    "wgrad, single, added": (WGRAD, SMALL, 136, 520, F32, True, (1, 256, False, False)),
    "wgrad, shared, bf16": (WGRAD, LARGE, 64, 128, BF, False, (1, 256, True, False)),
    "wgrad, shared, fp32": (WGRAD, LARGE, 128, 200, F32, False, (1, 256, True, False)),
    "wgrad, shared, added": (WGRAD, LARGE, 136, 264, F32, True, (1, 256, True, False)),
    "forward, pairs, bf16": (FORWARD, LARGE, 776, 520, BF, False, (2, 256, False, False)),
    "forward, pairs, fp32": (FORWARD, LARGE, 776, 1032, F32, False, (2, 256, False, False)),
    "forward, 128 rows, bf16": (FORWARD, LARGE, 128, 520, BF, False, (1, 128, None, False)),
    "forward, 32 rows, fp32": (FORWARD, SMALL, 4096, 72, F32, False, (1, 32, False, False)),
    "forward, 32 rows, shared": (FORWARD, SMALL, 136, 1032, BF, False, (1, 32, True, False)),
    "dgrad, pairs, bf16": (DGRAD, LARGE, 520, 776, BF, False, (2, 256, False, False)),
    "dgrad, pairs, fp32": (DGRAD, LARGE, 1032, 776, F32, False, (2, 256, False, False)),
    "dgrad, 128 rows, fp32": (DGRAD, LARGE, 520, 128, F32, False, (1, 128, None, False)),
    "dgrad, 32 rows, bf16": (DGRAD, SMALL, 72, 4096, BF, False, (1, 32, False, False)),
    "dgrad, 32 rows, shared": (DGRAD, SMALL, 1032, 136, F32, False, (1, 32, True, False)),
    "8-bit, pairs, bf16": (FP8, LARGE, 1300, 272, BF, False, (2, 256, False, False)),
    "8-bit, pairs, fp32": (FP8, LARGE, 1027, 400, F32, False, (2, 256, False, False)),
    "8-bit, 128 rows, bf16": (FP8, SOME, 128, 400, BF, False, (1, 128, False, False)),
    "8-bit, 32 rows, fp32": (FP8, SMALL, 4099, 144, F32, False, (1, 32, False, False)),
    "8-bit, 32 rows, shared": (FP8, SMALL, 130, 1040, BF, False, (1, 32, True, False)),
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
        self.product, self.sizes, self.N, self.K, self.out, self.accumulate, want = CASES[name]
        self.E, self.P = len(self.sizes), sum(self.sizes)
        ctas, tile, split, counted = ft.ft_moe_debug_group_plan(self.product, self.E, self.P, self.N, self.K, self.out,
                                                                self.accumulate)
        assert (ctas, tile, None if want[2] is None else split > 1, bool(counted)) == want
        E, P, N, K = self.E, self.P, self.N, self.K
        self.gen = torch.Generator(device="cuda").manual_seed(1)
        self.at = [0]
        for n in self.sizes:
            self.at.append(self.at[-1] + n)
        self.offs = torch.tensor(self.at, dtype=torch.int32, device="cuda")
        self.ws = torch.full((ft.ft_moe_group_workspace_size(E, P, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
        nb, f8 = -(-K // 128), torch.float8_e4m3fn
        if self.product == FP8:
            self.x, self.w = ((self.randn(*s) * 32).clamp(-448, 448).to(f8) for s in ((P, K), (E, N, K)))
            self.xs = torch.rand((nb, P), generator=self.gen, device="cuda") + 0.01
            self.wsc = (torch.rand((E, -(-N // 128), nb), generator=self.gen, device="cuda") + 0.1) * 0.01
        else:
            self.x, self.dy = self.randn(P, K).bfloat16(), self.randn(P, N).bfloat16()
            self.w = self.randn(E, N, K).bfloat16() if self.product != WGRAD else None
        shape = {FORWARD: (P, N), DGRAD: (P, K), WGRAD: (E, N, K), FP8: (P, N)}[self.product]
        self.base = self.randn(*shape).to(self.out)   # what an accumulating call finds, and garbage for the others

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def spoil(self, e):
        """The rows of expert e become values that are not finite."""
        rows = slice(self.at[e], self.at[e + 1])
        if self.product == FP8:
            self.x.view(torch.uint8)[rows] = 0x7F
        else:
            self.x[rows], self.dy[rows] = float("nan"), float("inf")

    def run(self, out):
        ft = self.ft
        if self.product == FORWARD:
            ft.ft_moe_group_gemm(self.x, self.w, self.offs, out, self.ws)
        elif self.product == DGRAD:
            ft.ft_moe_group_gemm_dgrad(self.dy, self.w, self.offs, out, self.ws)
        elif self.product == WGRAD:
            ft.ft_moe_group_gemm_wgrad(self.dy, self.x, self.offs, out, self.ws, accumulate=self.accumulate)
        else:
            ft.ft_moe_group_gemm_fp8(self.x, self.xs, self.w, self.wsc, self.offs, out, self.ws)
        return out

    def status(self):
        return self.ft.STATUS[self.ft.ft_moe_read_status(self.ws)]

    def expert(self, e):
        """Where expert e's results are, the 64-bit ones, the sum of magnitudes and its length."""
        rows = slice(self.at[e], self.at[e + 1])
        if self.product == FP8:
            N, K = self.N, self.K
            a = self.x[rows].double() * self.xs[:, rows].double().t().repeat_interleave(128, 1)[:, :K]
            b = self.w[e].double() * self.wsc[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
            return rows, a @ b.t(), a.abs() @ b.abs().t(), K + 4
        if self.product == WGRAD:
            a, b, at, length = self.dy[rows].double().t(), self.x[rows].double(), e, self.sizes[e]
        elif self.product == FORWARD:
            a, b, at, length = self.x[rows].double(), self.w[e].double().t(), rows, self.K
        else:
            a, b, at, length = self.dy[rows].double(), self.w[e].double(), rows, self.N
        ref, mag = a @ b, a.abs() @ b.abs()
        if self.accumulate:
            ref, mag, length = ref + self.base[e].double(), mag + self.base[e].double().abs(), length + 1
        return at, ref, mag, length

    def check(self, out, spoiled=()):
        for e, n in enumerate(self.sizes):
            at, ref, mag, length = self.expert(e)
            if e in spoiled and n:
                assert not torch.isfinite(out[at]).any(), e
            else:
                assert ((out[at].double() - ref).abs() <= U[self.out] * ref.abs() + length * 2.0 ** -23 * mag + 1e-30).all(), e


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF else torch.int32)


@pytest.mark.parametrize("name", list(CASES))
def test_results_repeats_and_replays(ft, name):
    case = Case(ft, name)
    out = case.run(case.base.clone())
    assert case.status() == "FT_OK"
    case.check(out)
    for _ in range(3):
        assert torch.equal(_bits(case.run(case.base.clone())), _bits(out))
    again = case.base.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.run(again)
    for _ in range(2):
        again.copy_(case.base)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(_bits(again), _bits(out))


@pytest.mark.parametrize("name", list(CASES))
def test_values_that_are_not_finite_stay_with_their_expert(ft, name):
    case = Case(ft, name)
    spoiled = set(range(0, case.E, 3))
    for e in spoiled:
        case.spoil(e)
    out = case.run(case.base.clone())
    assert case.status() == "FT_OK"
    case.check(out, spoiled)


@pytest.mark.parametrize("name", list(CASES))
def test_a_stalled_pipeline_reports_timeout_and_recovers(ft, name):
    case = Case(ft, name)
    good = case.run(case.base.clone())
    assert case.status() == "FT_OK"
    ft.ft_moe_debug_inject_stall(5_000_000, 1)
    case.run(case.base.clone())
    assert case.status() == "FT_ERR_TIMEOUT"
    again = case.run(case.base.clone())
    assert case.status() == "FT_OK" and torch.equal(_bits(again), _bits(good))


@pytest.mark.parametrize("out,accumulate", ((BF, False), (F32, False), (F32, True)))
def test_the_counter_runs_where_the_plan_says(ft, out, accumulate):
    """A counted call leaves the number of units it handed out in the workspace; another one leaves it alone."""
    for sizes, N, K, counted in ((MANY, 512, 512, True), (SOME, 256, 256, False)):
        E, P = len(sizes), sum(sizes)
        assert bool(ft.ft_moe_debug_group_plan(WGRAD, E, P, N, K, out, accumulate)[3]) == counted
        x, dy = torch.zeros((P, K), dtype=BF, device="cuda"), torch.zeros((P, N), dtype=BF, device="cuda")
        offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offs[1:] = torch.tensor(sizes).cumsum(0)
        ws = torch.full((ft.ft_moe_group_workspace_size(E, P, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
        ft.ft_moe_group_gemm_wgrad(dy, x, offs, torch.empty((E, N, K), dtype=out, device="cuda"), ws, accumulate=accumulate)
        assert ft.ft_moe_read_status(ws) == 0
        left = int(ws[64:68].view(torch.int32)[0])
        units = E * ((N + 255) // 256) * ((K + 255) // 256)
        assert left == -1 if not counted else units - 100 <= left <= units


@pytest.mark.parametrize("name", list(CASES))
def test_rows_of_no_expert(ft, name):
    """Every expert is empty although there are rows: nothing is written but the zeros of a weight gradient."""
    case = Case(ft, name)
    case.offs.fill_(case.P // 2)
    out = case.run(case.base.clone())
    assert case.status() == "FT_OK"
    if case.product == WGRAD and not case.accumulate:
        assert not out.any()
    else:
        assert torch.equal(_bits(out), _bits(case.base))
