"""MXFP4 rows on the test side: the quantization rule, decoding, and scale layouts, in plain torch."""
import torch

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = torch.cat([VALUES, -VALUES])


def codes_of(codes):
    """Codes [..., K] (0..15) of packed bytes [..., K / 2]."""
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def decode(codes, scales):
    """Values in 64 bits of packed codes [..., K / 2] and scale bytes [..., K / 32]."""
    s = scales.view(torch.uint8).double() - 127.0
    factor = torch.where(s == 128.0, torch.full_like(s, float("nan")), torch.exp2(s))
    return TABLE.to(codes.device).double()[codes_of(codes).int()] * factor.repeat_interleave(32, -1)


def row_scales(words, K):
    """Scale bytes [rows, K / 32] of words [ceil(K / 128), rows, 4]."""
    return words.permute(1, 0, 2).reshape(words.shape[1], -1)[:, :K // 32]


def words_of(scales):
    """Words [ceil(K / 128), rows, 4] of scale bytes [rows, K / 32] (zeros beyond K)."""
    rows, nb = scales.shape
    kt = (nb + 3) // 4
    t = torch.zeros((rows, kt * 4), dtype=torch.uint8, device=scales.device)
    t[:, :nb] = scales
    return t.view(rows, kt, 4).permute(1, 0, 2)


def tiles_of(scales):
    """Tiles [E, ceil(N / 128), ceil(K / 128), 512] of scale bytes [E, N, K / 32], a word at a time."""
    E, N, nb = scales.shape
    nt, kt = (N + 127) // 128, (nb + 3) // 4
    full = torch.zeros((E, nt * 128, kt * 4), dtype=torch.uint8, device=scales.device)
    full[:, :N, :nb] = scales
    out = torch.zeros((E, nt, kt, 128, 4), dtype=torch.uint8, device=scales.device)
    for n in range(128):
        out[:, :, :, 4 * (n % 32) + n // 32] = full.view(E, nt, 128, kt, 4)[:, :, n]
    return out.view(E, nt, kt, 512)


def rule(v):
    """Codes [rows, K] (0..15) and scale bytes [rows, K / 32] of fp32 rows, by the definition, in 64 bits."""
    b = v.double().view(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    finite = torch.isfinite(v).view(b.shape).all(2)
    s = torch.full(amax.shape, -127.0, dtype=torch.float64, device=v.device)
    for e in range(-126, 127):  # the smallest power that holds the block
        s = torch.where(amax > 6.0 * 2.0 ** (e - 1), torch.full_like(s, float(e)), s)
    x = torch.where(finite[:, :, None], b, 0.0) * torch.exp2(-s)[:, :, None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=v.device)
    a = x.abs()
    code = torch.zeros(a.shape, dtype=torch.int32, device=v.device)
    for i, m in enumerate(mids):  # above a midpoint, or on one whose lower neighbour is odd
        code = torch.where((a > m) | ((a == m) & (i % 2 == 1)), i + 1, code)
    code = code + 8 * torch.signbit(x).int()
    byte = torch.where(finite, s + 127.0, 255.0).to(torch.uint8)
    return code.view(v.shape), byte


def random_weights(gen, E, N, K, spread=1):
    """Codes [E, N, K / 2] and scale bytes [E, N, K / 32] around 2^0 +- spread."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(127 - spread, 128 + spread, (E, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales
