"""Plain 64-bit reference of 4-bit storage, on the CPU with torch: scales by comparison, codes by
distance to the grid."""
import torch

GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def up(n, m):
    return -(-n // m) * m


def code_values():
    """fp64 values of the 16 codes."""
    return torch.cat([GRID, -GRID])


def quantise(x):
    """(codes 0 .. 15, scale bytes [R][blocks]) of x [R][C]."""
    x = x.double()
    R, C = x.shape
    p = torch.zeros((R, up(C, 32)), dtype=torch.float64)
    p[:, :C] = x
    p = p.reshape(R, -1, 32)
    bad = ~torch.isfinite(p).all(2)
    a = torch.where(torch.isfinite(p), p.abs(), 0.0).amax(2)
    m, e = torch.frexp(a)  # 6 is 0.75 * 2^3
    b = torch.where(a > 0, e - 3 + (m > 0.75) + 127, 17).clamp(17, 252).long()
    v = (p / torch.ldexp(torch.ones_like(a), b - 127)[..., None]).abs().clamp(max=6)
    v = torch.where(torch.isfinite(p), v, 0.0)
    d = (v[..., None] - GRID).abs()
    near = d.amin(-1, keepdim=True)
    # the two nearest of a tie are neighbours: the even code of them
    tie = (d == near)
    code = torch.where(tie & (torch.arange(8) % 2 == 0), 1, 0).argmax(-1)
    code = torch.where((tie & (torch.arange(8) % 2 == 0)).any(-1), code, tie.int().argmax(-1))
    code = code + 8 * torch.signbit(p).long()
    code = torch.where(bad[..., None], 0, code)
    b = torch.where(bad, 255, b)
    return code.reshape(R, -1)[:, :C], b


def values(code, b):
    """fp64 values of codes [R][C] under scale bytes [R][blocks]."""
    s = torch.ldexp(torch.ones(b.shape, dtype=torch.float64), b - 127)
    s = torch.where(b == 255, torch.nan, s)
    return code_values()[code] * s.repeat_interleave(32, 1)[:, :code.shape[1]]
