"""Measured cases of the 8-bit training operators: storage in 8 bits with a scale for each
block of 128, the block-scaled matrix product, the weight gradient from an 8-bit checkpoint
and the (gated) activation with its gradient.

An 8-bit matrix is held as `q` [rows][ld] codes (e4m3 or e5m2) and `scale` [ceil(cols / 128)]
[lds] exponent bytes, 2^(b - 127): one for 128 elements of a row, or one for 128 x 128
(weights, lds over the blocks of rows).  Codes come back as torch's 8-bit floating types and
scales as torch.float8_e8m0fnu, both without a copy.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
BIAS = {"e4m3": 8, "e5m2": 15}
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token through a projection: the weights are read once, latency counts
        dict(name="gemm_one_token", op="gemm", M=1, N=4096, K=4096, a="e4m3", out="bf16"),
        # a few tokens, not a multiple of anything
        dict(name="gemm_few_tokens", op="gemm", M=37, N=4096, K=1024, a="e4m3", out="f16"),
        # input gradient of a ragged layer: e5m2 gradients, fp32 result
        dict(name="gemm_ragged", op="gemm", M=5001, N=1000, K=4100, a="e5m2", out="f32"),
        # a long batch through a wide layer
        dict(name="gemm_large", op="gemm", M=16384, N=8192, K=4096, a="e4m3", out="bf16"),
        # weight gradient of a short batch: few output tiles, a long sum
        dict(name="wgrad_small", op="wgrad", M=2048, N=1024, K=512, dy="bf16", x="e4m3", acc=False),
        # ragged, gradients in 8 bits, added to an earlier micro-batch's
        dict(name="wgrad_ragged", op="wgrad", M=5001, N=1000, K=2050, dy="e5m2", x="e4m3", acc=True),
        dict(name="wgrad_large", op="wgrad", M=16384, N=4096, K=4096, dy="bf16", x="e4m3",
             acc=False),
        # a checkpoint written, and read back by the backward pass
        dict(name="save_large", op="save", M=16384, K=8192, t="bf16", q="e4m3"),
        dict(name="load_ragged", op="load", M=5001, K=1000, t="f32", q="e5m2"),
        # a layer's weights, laid out for both directions after an update
        dict(name="weight", op="weight", N=8192, K=4096, t="bf16", q="e4m3"),
        # the feed-forward activation of a long batch, and a plain ragged one's gradient
        dict(name="glu_forward", op="glu", M=8192, F=8192, act="silu", gated=True, t="bf16",
             q="e4m3"),
        dict(name="glu_backward", op="glu_grad", M=8192, F=8192, act="silu", gated=True, t="bf16",
             q="e4m3", dq="e5m2"),
    ]


def _size(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice([1, 1, 2, 16, 128])  # odd sizes as often as even ones
    return min(hi, max(lo, v // step * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "wgrad", "wgrad", "save", "load", "weight", "glu", "glu_grad"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    q = rng.choice(["e4m3", "e4m3", "e5m2"])
    M = _size(rng, 1, 16384)
    if op == "gemm":
        return dict(op=op, M=M, N=_size(rng, 64, 8192), K=_size(rng, 64, 4096), a=q, out=t)
    if op == "wgrad":
        return dict(op=op, M=M, N=_size(rng, 64, 4096), K=_size(rng, 64, 4096),
                    dy=rng.choice(["bf16", "e4m3", "e5m2"]), x="e4m3",
                    acc=rng.random() < 0.5)
    if op in ("save", "load"):
        return dict(op=op, M=M, K=_size(rng, 64, 8192), t=t, q=q)
    if op == "weight":
        return dict(op=op, N=_size(rng, 64, 8192), K=_size(rng, 64, 4096), t=t, q="e4m3")
    c = dict(op=op, M=min(M, 8192), F=_size(rng, 64, 8192),
             act=rng.choice(["silu", "gelu", "gelu_tanh"]), gated=rng.random() < 0.7, t=t, q="e4m3")
    if op == "glu_grad":
        c["dq"] = rng.choice(["e4m3", "e5m2"])
    return c


def _up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------------------------------
# plain form


def _blocked(x, by_rows):
    """fp32 view [row blocks][br][column blocks][128] of x, padded with zeros."""
    R, C = x.shape
    br = 128 if by_rows else 1
    x = torch.nn.functional.pad(x, (0, _up(C, 128) - C, 0, _up(R, br) - R))
    return x.reshape(x.shape[0] // br, br, x.shape[1] // 128, 128)


def _exponents(x, fmt, by_rows):
    """Scale bytes [column blocks][row blocks]: the least power of two that keeps the block's
    largest finite magnitude within the format, and no less than 2^-110."""
    b = _blocked(torch.where(torch.isfinite(x), x.abs(), torch.zeros((), device=x.device)), by_rows)
    bits = b.amax(dim=(1, 3)).view(torch.int32)
    return (((bits + 0x1FFFFF) >> 23) - BIAS[fmt]).clamp(min=17).t().to(torch.uint8)


def _spread(scale, R, C, by_rows):
    """fp32 factors [R][C] of scale bytes [column blocks][row blocks]."""
    f = (scale.to(torch.int32) << 23).view(torch.float32).t()
    if by_rows:
        f = f.repeat_interleave(128, 0)
    return f.repeat_interleave(128, 1)[:R, :C]


def _quantise(x, fmt, by_rows=False):
    """(codes [R][C] in the 8-bit type, scale bytes [column blocks][row blocks])."""
    x = x.float()
    s = _exponents(x, fmt, by_rows)
    inv = _spread(254 - s, *x.shape, by_rows)
    return (x * inv).to(F8[fmt]), s


def _values(q, scale, R, C, fmt, by_rows=False):
    """fp32 values of a stored matrix (its rows and columns without padding)."""
    br = _up(R, 128) // 128 if by_rows else R
    return q[:R, :C].view(F8[fmt]).float() * _spread(scale[:, :br], R, C, by_rows)


def _act(g, act):
    """act(g) and its derivative in fp32."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g)


# ---------------------------------------------------------------------------------------
# inputs


def _store(x, fmt, by_rows=False):
    """A stored 8-bit matrix: rows and scale rows padded to 16 bytes, as programs keep them."""
    q, s = _quantise(x, fmt, by_rows)
    qb = torch.zeros((x.shape[0], _up(x.shape[1], 16)), dtype=torch.uint8, device=DEV)
    qb[:, :x.shape[1]] = q.view(torch.uint8)
    sb = torch.zeros((s.shape[0], _up(s.shape[1], 16)), dtype=torch.uint8, device=DEV)
    sb[:, :s.shape[1]] = s
    return qb, sb


def _draw(gen, R, C, t, std=1.0):
    """Activations with a few strong columns, rows padded to 16 bytes; the [R][C] view."""
    dt = T[t]
    x = torch.zeros((R, _up(C, 16)), dtype=dt, device=DEV)
    strong = 1 + 7 * (torch.rand(C, generator=gen, device=DEV) < 0.01)
    x[:, :C] = (torch.randn((R, C), generator=gen, device=DEV) * (std * strong)).to(dt)
    return x[:, :C]


def _space(R, C, by_rows=False):
    """Room for a stored matrix."""
    br = _up(R, 128) // 128 if by_rows else R
    return (torch.zeros((R, _up(C, 16)), dtype=torch.uint8, device=DEV),
            torch.zeros((_up(C, 128) // 128, _up(br, 16)), dtype=torch.uint8, device=DEV))


def _room(R, C, t):
    return torch.zeros((R, _up(C, 16)), dtype=T[t], device=DEV)[:, :C]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s, op = case, {"case": case}, case["op"]
    if op == "gemm":
        s["a"] = _store(_draw(gen, c["M"], c["K"], "f32", 1e-3 if c["a"] == "e5m2" else 1.0), c["a"])
        s["b"] = _store(_draw(gen, c["N"], c["K"], "f32", c["K"] ** -0.5), "e4m3", True)
        s["c"] = _room(c["M"], c["N"], c["out"])
    elif op == "wgrad":
        dy = _draw(gen, c["M"], c["N"], "bf16", 1e-3)
        s["dy"] = dy if c["dy"] == "bf16" else _store(dy.float(), c["dy"])
        s["x"] = _store(_draw(gen, c["M"], c["K"], "f32"), c["x"])
        s["dw"] = torch.zeros((c["N"], c["K"]), device=DEV)
        if c["acc"]:
            s["dw0"] = torch.randn((c["N"], c["K"]), generator=gen, device=DEV) * 1e-2
    elif op == "save":
        s["x"] = _draw(gen, c["M"], c["K"], c["t"])
        s["q"] = _space(c["M"], c["K"])
    elif op == "load":
        s["q"] = _store(_draw(gen, c["M"], c["K"], "f32"), c["q"])
        s["x"] = _room(c["M"], c["K"], c["t"])
    elif op == "weight":
        s["x"] = _draw(gen, c["N"], c["K"], c["t"], c["K"] ** -0.5)
        s["q"], s["qt"] = _space(c["N"], c["K"], True), _space(c["K"], c["N"], True)
    elif op == "glu":
        s["g"] = _draw(gen, c["M"], c["F"], c["t"])
        s["u"] = _draw(gen, c["M"], c["F"], c["t"]) if c["gated"] else None
        s["gq"], s["yq"] = _space(c["M"], c["F"]), _space(c["M"], c["F"])
        s["uq"] = _space(c["M"], c["F"]) if c["gated"] else None
    else:
        s["g"] = _store(_draw(gen, c["M"], c["F"], "f32"), c["q"])
        s["u"] = _store(_draw(gen, c["M"], c["F"], "f32"), c["q"]) if c["gated"] else None
        s["dy"] = _draw(gen, c["M"], c["F"], c["t"], 1e-3)
        s["dgq"] = _space(c["M"], c["F"])
        s["duq"] = _space(c["M"], c["F"]) if c["gated"] else None
    if own:  # the descriptors and the workspace that a program makes once
        _handles(s)
    return s


def _handles(s):
    import count_sketch_aggregation_amd as s2r
    c, op = s["case"], s["case"]["op"]

    def q8(pair, fmt):
        return None if pair is None else s2r.q8_mat(pair[0], pair[1], fmt)

    def mat(x):
        return None if x is None else s2r.mat(x)

    s["s2r"] = s2r
    if op == "gemm":
        s["h"] = (q8(s["a"], c["a"]), q8(s["b"], "e4m3"), mat(s["c"]))
        need = s2r.s2r_q8_gemm_workspace_bytes(c["M"], c["N"], c["K"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    elif op == "wgrad":
        s["h"] = (mat(s["dy"]) if c["dy"] == "bf16" else q8(s["dy"], c["dy"]), q8(s["x"], c["x"]))
        need = s2r.s2r_q8_wgrad_workspace_bytes(c["M"], c["N"], c["K"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    elif op in ("save", "load"):
        s["h"] = (mat(s["x"]), q8(s["q"], c["q"]))
    elif op == "weight":
        s["h"] = (mat(s["x"]), q8(s["q"], c["q"]), q8(s["qt"], c["q"]))
    elif op == "glu":
        s["h"] = (mat(s["g"]), mat(s["u"]), q8(s["gq"], c["q"]), q8(s["uq"], c["q"]),
                  q8(s["yq"], c["q"]))
    else:
        s["h"] = (q8(s["g"], c["q"]), q8(s["u"], c["q"]), mat(s["dy"]), q8(s["dgq"], c["dq"]),
                  q8(s["duq"], c["dq"]))


# ---------------------------------------------------------------------------------------
# one pass


def _stored(pair, R, C, fmt, by_rows=False):
    br = _up(R, 128) // 128 if by_rows else R
    return [pair[0][:R, :C].view(F8[fmt]), pair[1][:, :br].view(torch.float8_e8m0fnu)]


def _plain_stored(x, fmt, by_rows=False):
    q, s = _quantise(x, fmt, by_rows)
    return [q, s.view(torch.float8_e8m0fnu)]


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, op, s2r, h = s["case"], s["case"]["op"], s["s2r"], s["h"]
    if op == "gemm":
        s2r.s2r_q8_gemm(c["M"], c["N"], c["K"], h[0], h[1], h[2], workspace=s["ws"])
        return s["c"]
    if op == "wgrad":
        if c["acc"]:
            s["dw"].copy_(s["dw0"])
        s2r.s2r_q8_wgrad(c["M"], c["N"], c["K"], h[0], h[1], s["dw"], c["K"], accumulate=c["acc"],
                         workspace=s["ws"])
        return s["dw"]
    if op == "save":
        s2r.s2r_q8_save(c["M"], c["K"], h[0], h[1])
        return _stored(s["q"], c["M"], c["K"], c["q"])
    if op == "load":
        s2r.s2r_q8_load(c["M"], c["K"], h[1], h[0])
        return s["x"]
    if op == "weight":
        s2r.s2r_q8_weight(c["N"], c["K"], h[0], h[1], h[2])
        return _stored(s["q"], c["N"], c["K"], c["q"], True) + \
            _stored(s["qt"], c["K"], c["N"], c["q"], True)
    if op == "glu":
        s2r.s2r_q8_glu(c["M"], c["F"], c["act"], h[0], h[1], gq=h[2], uq=h[3], yq=h[4])
        keep = [s["gq"], s["yq"]] + ([s["uq"]] if c["gated"] else [])
        return [_stored(p, c["M"], c["F"], c["q"]) for p in keep]
    s2r.s2r_q8_glu_grad(c["M"], c["F"], c["act"], h[0], h[1], h[2], dgq=h[3], duq=h[4])
    keep = [s["dgq"]] + ([s["duq"]] if c["gated"] else [])
    return [_stored(p, c["M"], c["F"], c["dq"]) for p in keep]


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "gemm":
        a = _values(*s["a"], c["M"], c["K"], c["a"])
        b = _values(*s["b"], c["N"], c["K"], "e4m3", True)
        return (a @ b.t()).to(T[c["out"]])
    if op == "wgrad":
        dy = s["dy"].float() if c["dy"] == "bf16" else _values(*s["dy"], c["M"], c["N"], c["dy"])
        dw = dy.t() @ _values(*s["x"], c["M"], c["K"], c["x"])
        return s["dw0"] + dw if c["acc"] else dw
    if op == "save":
        return _plain_stored(s["x"], c["q"])
    if op == "load":
        return _values(*s["q"], c["M"], c["K"], c["q"]).to(T[c["t"]])
    if op == "weight":
        q = _plain_stored(s["x"], c["q"], True)
        return q + [x.view(torch.uint8).t().contiguous().view(x.dtype) for x in q]
    if op == "glu":
        y, _ = _act(s["g"].float(), c["act"])
        if c["gated"]:
            y = y * s["u"].float()
        keep = [s["g"], y] + ([s["u"]] if c["gated"] else [])
        return [_plain_stored(x, c["q"]) for x in keep]
    a, da = _act(_values(*s["g"], c["M"], c["F"], c["q"]), c["act"])
    dy = s["dy"].float()
    if not c["gated"]:
        return [_plain_stored(dy * da, c["dq"])]
    u = _values(*s["u"], c["M"], c["F"], c["q"])
    return [_plain_stored(dy * u * da, c["dq"]), _plain_stored(dy * a, c["dq"])]


# ---------------------------------------------------------------------------------------
# the definition in 64 bits


def _table(fmt):
    """Values of the 256 codes from the formats' definitions."""
    ebits, mbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    out = []
    for code in range(256):
        e, m = (code >> mbits) & (2 ** ebits - 1), code & (2 ** mbits - 1)
        v = 2.0 ** (1 - bias) * m / 2 ** mbits if e == 0 else 2.0 ** (e - bias) * (1 + m / 2 ** mbits)
        if fmt == "e4m3" and (e, m) == (15, 7):
            v = math.nan
        if fmt == "e5m2" and e == 31:
            v = math.inf if m == 0 else math.nan
        out.append(-v if code >= 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _two_to(e):
    """2^e in 64 bits, to the bit."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(pair, R, C, fmt, block_rows=1):
    v = _table(fmt)[pair[0][:R, :C].int()]
    r = torch.arange(R, device=DEV) // block_rows
    for k in range(0, C, 128):
        v[:, k:k + 128] *= _two_to(pair[1][k // 128].int() - 127)[r][:, None]
    return v


def _exact_stored(x, fmt, block_rows=1):
    """[code values, scales] in 64 bits: the scale by comparison, the rounding on the grid."""
    R, C = x.shape
    nk, nr = -(-C // 128), -(-R // block_rows)
    scale = torch.empty((nk, nr), dtype=torch.float64, device=DEV)
    code = torch.empty((R, C), dtype=torch.float64, device=DEV)
    low, mbits, top = (-6, 3, 9) if fmt == "e4m3" else (-14, 2, 16)
    r = torch.arange(R, device=DEV) // block_rows
    for k in range(nk):
        part = x[:, k * 128:(k + 1) * 128]
        most = torch.zeros(nr, dtype=torch.float64, device=DEV)
        most.scatter_reduce_(0, r, part.abs().amax(1), "amax")
        m, e = torch.frexp(most)  # the formats' largest values are 0.875 * 2^top
        e = torch.where(most > 0, e - top + (m > 0.875), -110).clamp(min=-110)
        scale[k] = _two_to(e)
        v = part / scale[k][r][:, None]
        step = _two_to(torch.frexp(v.abs().clamp(min=2.0 ** low))[1] - 1 - mbits)
        code[:, k * 128:(k + 1) * 128] = torch.round(v / step) * step
    return [code, scale]


def _exact_act(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))  # (1 + tanh z) / 2 = sigmoid(2 z)
    return g * s, s + g * s * (1 - s) * 2 * k * (1 + 0.134145 * g * g)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op == "gemm":
        return _exact_values(s["a"], c["M"], c["K"], c["a"]) @ \
            _exact_values(s["b"], c["N"], c["K"], "e4m3", 128).t()
    if op == "wgrad":
        dy = s["dy"].double() if c["dy"] == "bf16" else _exact_values(s["dy"], c["M"], c["N"], c["dy"])
        dw = dy.t() @ _exact_values(s["x"], c["M"], c["K"], c["x"])
        return s["dw0"].double() + dw if c["acc"] else dw
    if op == "save":
        return _exact_stored(s["x"].double(), c["q"])
    if op == "load":
        return _exact_values(s["q"], c["M"], c["K"], c["q"])
    if op == "weight":
        q = _exact_stored(s["x"].double(), c["q"], 128)
        return q + [x.t().contiguous() for x in q]
    if op == "glu":
        y, _ = _exact_act(s["g"].double(), c["act"])
        if c["gated"]:
            y = y * s["u"].double()
        keep = [s["g"].double(), y] + ([s["u"].double()] if c["gated"] else [])
        return [_exact_stored(x, c["q"]) for x in keep]
    a, da = _exact_act(_exact_values(s["g"], c["M"], c["F"], c["q"]), c["act"])
    dy = s["dy"].double()
    if not c["gated"]:
        return [_exact_stored(dy * da, c["dq"])]
    u = _exact_values(s["u"], c["M"], c["F"], c["q"])
    return [_exact_stored(dy * u * da, c["dq"]), _exact_stored(dy * a, c["dq"])]


def work(case):
    c, op = case, case["op"]
    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    if op == "wgrad":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * N * (2 if c["dy"] == "bf16" else 1) + M * K + N * K * (8 if c["acc"] else 4),
                "flops": 2 * M * N * K}
    if op in ("save", "load"):
        return {"bytes": c["M"] * c["K"] * (SIZE[c["t"]] + 1), "flops": 0}
    if op == "weight":
        return {"bytes": c["N"] * c["K"] * (SIZE[c["t"]] + 2), "flops": 0}
    n, k = c["M"] * c["F"], 2 if c["gated"] else 1
    if op == "glu":
        return {"bytes": n * (SIZE[c["t"]] * k + k + 1), "flops": 0}
    return {"bytes": n * (k + SIZE[c["t"]] + k), "flops": 0}
