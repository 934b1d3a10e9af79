"""Plain 64-bit reference of the 8-bit training calls, on the CPU with torch: the stored form
by its definition (largest finite magnitude, least power-of-two scale, rounding on the
format's grid), sums and activations in fp64."""
import math

import torch

FORMATS = {"e4m3": (4, 3, 7, 0.875, 9), "e5m2": (5, 2, 15, 0.875, 16)}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def up(n, m):
    return -(-n // m) * m


def code_values(fmt):
    """fp64 values of the 256 codes."""
    ebits, mbits, bias, _, _ = FORMATS[fmt]
    out = []
    for c in range(256):
        e, m = (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        v = math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp((1 << mbits) + m, e - bias - mbits)
        if fmt == "e4m3" and e == 15 and m == 7:
            v = math.nan
        if fmt == "e5m2" and e == 31:
            v = math.nan if m else math.inf
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


def block_max(x, square):
    """Largest finite magnitude of every block, [row blocks][column blocks], fp64."""
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    br = 128 if square else 1
    R, C = up(max(x.shape[0], 1), br), up(max(x.shape[1], 1), 128)
    p = torch.zeros((R, C), dtype=torch.float64)
    p[:x.shape[0], :x.shape[1]] = a
    return p.reshape(R // br, br, C // 128, 128).amax(dim=(1, 3))


def scale_bytes(a, fmt):
    """Bytes b of the least 2^(b - 127) with a <= MAX 2^(b - 127), MAX = 0.875 * 2^top."""
    _, _, _, top_m, top_e = FORMATS[fmt]
    m, e = torch.frexp(a)
    return torch.where(a > 0, e - top_e + (m > top_m) + 127, 17).clamp(min=17).to(torch.int64)


def spread(b, R, C, square):
    """2^(b - 127) for every element, fp64, from bytes [row blocks][column blocks]."""
    f = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    if square:
        f = f.repeat_interleave(128, 0)
    return f.repeat_interleave(128, 1)[:R, :C]


def quantise(x, fmt, square=False):
    """(values of the codes in fp64, scale bytes [row blocks][column blocks])."""
    x = x.double()
    b = scale_bytes(block_max(x, square), fmt)
    v = x / spread(b, *x.shape, square)
    ebits, mbits, bias, _, _ = FORMATS[fmt]
    e = torch.frexp(v.abs().clamp(min=2.0 ** (1 - bias)))[1] - 1
    step = torch.ldexp(torch.ones_like(v), e - mbits)
    q = torch.round(v / step) * step
    q = torch.where(torch.isfinite(x), q, x)
    if fmt == "e4m3":
        q = torch.where(torch.isinf(x), torch.full_like(q, math.nan), q)
    return q, b


def act(g, kind):
    """act(g), act'(g) in fp64."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if kind == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    z = 2 * k * (g + 0.044715 * g ** 3)
    s, r = torch.sigmoid(z), torch.sigmoid(-z)  # (1 + tanh(z / 2)) / 2 and its complement
    return g * s, s + g * s * r * 2 * k * (1 + 0.134145 * g * g)
