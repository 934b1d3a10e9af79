"""Measured cases of layers of experts and of 4-bit matrices: tokens sorted by expert and back
with their weights and gradients, the experts' products and weight gradients in 8 bits, and
microscaled 4-bit storage with its product.

A token t chooses K experts, `expert` [T][K] (-1: none).  The rows of an expert lie together, in
the order of the choices: expert e has rows[e] rows from first[e] on, which is a multiple of 4, and
choice (t, k) has row place[t][k] (-1: none).  Rows that no choice has are left as they were.

8-bit matrices are as in operators.py: `q` [rows][ld] codes and `scale` [ceil(cols / 128)][lds]
exponent bytes, 2^(b - 127), for 128 elements of a row or, for weights, 128 x 128.  A 4-bit
matrix (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) is `q` [rows][ld bytes], two codes to a
byte, the even column's in the low half, and `scale` [rows][lds], a byte for 32 elements of a row.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BIAS = {"e4m3": 8, "e5m2": 15}
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # a few tokens of a serving step to their experts: launches and latency
        dict(name="dispatch_few", op="dispatch", T=24, K=8, E=64, D=2048, x="bf16", q=""),
        # a long batch, stored in 8 bits on its way to the experts
        dict(name="dispatch_large", op="dispatch", T=16384, K=4, E=64, D=4096, x="bf16", q="e4m3"),
        # the experts' results of a ragged batch, weighted and added
        dict(name="combine_ragged", op="combine", T=1001, K=6, E=48, D=1000, x="f16", y="f32"),
        # the same of a training step, with the gradients of rows, weights and tokens
        dict(name="combine_train", op="combine_train", T=8192, K=4, E=32, D=4096, x="bf16", q="e5m2"),
        # experts' layer outputs of a few tokens: the weights of the chosen experts are read once
        dict(name="experts_few", op="gemm", T=16, K=4, E=32, N=2048, D=1024, a="e4m3", out="bf16"),
        # a long batch through experts of which some are chosen far more often
        dict(name="experts_large", op="gemm", T=8192, K=4, E=16, N=4096, D=2048, a="e4m3", out="bf16"),
        # weight gradients of ragged experts, added to an earlier micro-batch's
        dict(name="wgrad_ragged", op="wgrad", T=1501, K=2, E=8, N=1000, D=516, dy="e5m2", acc=True),
        dict(name="wgrad_large", op="wgrad", T=8192, K=4, E=16, N=2048, D=2048, dy="bf16", acc=False),
        # a ragged matrix to 4 bits and back
        dict(name="q4_store_ragged", op="q4_store", R=1001, C=1000, x="f32", both=False),
        # a layer's weights or a long batch, for the products along either side
        dict(name="q4_store_large", op="q4_store", R=8192, C=8192, x="bf16", both=True),
        # one token through a projection: the weights are read once
        dict(name="q4_one_token", op="q4_gemm", M=1, N=8192, K=4096, out="bf16"),
        # a long batch through a wide layer
        dict(name="q4_large", op="q4_gemm", M=16384, N=8192, K=4096, out="bf16"),
    ]


def _size(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice([1, 1, 2, 16, 128])  # odd sizes as often as even ones
    return min(hi, max(lo, v // step * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_train", "gemm", "gemm", "wgrad", "q4_store", "q4_gemm", "q4_gemm"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "q4_store":
        return dict(op=op, R=_size(rng, 1, 8192), C=_size(rng, 32, 8192), x=t, both=rng.random() < 0.5)
    if op == "q4_gemm":
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 64, 8192), K=_size(rng, 64, 4096), out=t)
    E = _size(rng, 1, 64)
    c = dict(op=op, T=_size(rng, 1, 8192), K=min(E, rng.choice([1, 2, 4, 6, 8])), E=E)
    if op == "dispatch":
        return dict(c, D=_size(rng, 64, 4096), x=t, q=rng.choice(["", "e4m3", "e5m2"]))
    if op == "combine":
        return dict(c, D=_size(rng, 64, 4096), x=t, y=rng.choice(["bf16", "f16", "f32"]))
    if op == "combine_train":
        return dict(c, T=min(c["T"], 4096), D=_size(rng, 64, 4096), x=t, q=rng.choice(["e4m3", "e5m2"]))
    c["T"] = min(c["T"], 32768 // c["K"])
    c["E"] = min(c["E"], 32)
    c["K"] = min(c["K"], c["E"])
    if op == "gemm":
        return dict(c, N=_size(rng, 64, 4096), D=_size(rng, 64, 2048), a=rng.choice(["e4m3", "e5m2"]), out=t)
    return dict(c, N=_size(rng, 64, 2048), D=_size(rng, 64, 2048), dy=rng.choice(["bf16", "e4m3", "e5m2"]),
                acc=rng.random() < 0.5)


def _up(n, m):
    return -(-n // m) * m


def _most_rows(c):
    """Rows that the sorted matrices of a case may need: a multiple of 4 for every chosen expert."""
    A = c["T"] * c["K"]
    return (A + 3 * min(c["E"], A)) // 4 * 4


# ---------------------------------------------------------------------------------------
# plain form: 8 bits


def _quantise(x, fmt):
    """(codes [R][C] in the 8-bit type, scale bytes [column blocks][R]) of fp32 rows: the least power of
    two that keeps the block's largest finite magnitude within the format, no less than 2^-110."""
    R, C = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros((), device=x.device))
    a = torch.nn.functional.pad(a, (0, _up(C, 128) - C)).reshape(R, -1, 128).amax(2)
    b = (((a.view(torch.int32) + 0x1FFFFF) >> 23) - BIAS[fmt]).clamp(min=17)
    inv = ((254 - b) << 23).view(torch.float32).repeat_interleave(128, 1)[:, :C]
    return (x * inv).to(F8[fmt]), b.t().to(torch.uint8)


def _values(q, scale, R, C, fmt):
    """fp32 values of a matrix stored in row blocks."""
    f = (scale[:, :R].to(torch.int32) << 23).view(torch.float32).t()
    return q[:R, :C].view(F8[fmt]).float() * f.repeat_interleave(128, 1)[:, :C]


def _weights(q, scale, E, N, C):
    """fp32 values [E][N][C] of the experts' weights, stacked with NS rows each, in square blocks."""
    NS = _up(N, 128)
    f = (scale[:, :E * NS // 128].to(torch.int32) << 23).view(torch.float32).t()
    f = f.repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :C]
    return (q[:, :C].view(F8["e4m3"]).float() * f).view(E, NS, C)[:, :N]


# ---------------------------------------------------------------------------------------
# plain form: experts


def _route(expert, E):
    """first [E], rows [E] and place [T][K] of the choices."""
    flat = expert.reshape(-1).to(torch.int64)
    A = flat.numel()
    key, order = torch.sort(torch.where((flat >= 0) & (flat < E), flat, E), stable=True)
    rows = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    up = (rows + 3) // 4 * 4
    first = up.cumsum(0) - up
    row = first[key] + torch.arange(A, device=DEV) - (rows.cumsum(0) - rows)[key]
    place = torch.empty_like(row).scatter_(0, order, torch.where(key < E, row, -1))
    return first[:E].int(), rows[:E].int(), place.view_as(expert).int()


def _by_row(values, place, into):
    """into[place[t][k]] = values[t][k], [T][K][...]; the other rows stay."""
    R = into.shape[0]
    out = torch.cat([into, into.new_zeros((1,) + into.shape[1:])])
    at = place.reshape(-1).long()
    out[torch.where(at < 0, R, at)] = values.reshape((at.numel(),) + into.shape[1:])
    return out[:R]


def _by_token(rows, place):
    """fp32 [T][K][D] rows of the choices, zeros where there is none."""
    r = torch.cat([rows.float(), torch.zeros((1, rows.shape[1]), device=DEV)])
    return r[torch.where(place < 0, rows.shape[0], place).long()]


def _grouped(m, s):
    """fp32 [E][most][cols] of the rows of each expert, zeros behind them."""
    at = s["first"][:, None].long() + torch.arange(s["most"], device=DEV)[None]
    there = torch.arange(s["most"], device=DEV)[None] < s["rows"][:, None]
    return torch.where(there[..., None], m[at.clamp(max=m.shape[0] - 1)], torch.zeros((), device=DEV))


def _ungrouped(g, s, into):
    """The rows of each expert back to theirs; the other rows stay."""
    at = s["first"][:, None].long() + torch.arange(s["most"], device=DEV)[None]
    there = torch.arange(s["most"], device=DEV)[None] < s["rows"][:, None]
    R = into.shape[0]
    out = torch.cat([into, into.new_zeros((1, into.shape[1]))])
    out[torch.where(there, at, R)] = g.to(into.dtype)
    return out[:R]


# ---------------------------------------------------------------------------------------
# plain form: 4 bits


def _q4_quantise(x):
    """(code values as fp32 [R][C], scale bytes [R][blocks of 32]): the least power of two that keeps
    the block's largest magnitude within 6, 2^-110 to 2^125; to nearest, ties to even codes."""
    R, C = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, _up(C, 32) - C)).reshape(R, -1, 32).amax(2)
    b = (((a.view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp(min=17, max=252)
    v = x * ((254 - b) << 23).view(torch.float32).repeat_interleave(32, 1)[:, :C]
    m = v.abs().clamp(max=6)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.round(m / step) * step * torch.sign(v), b.to(torch.uint8)


def _q4_spread(b, C):
    return (b.to(torch.int32) << 23).view(torch.float32).repeat_interleave(32, 1)[:, :C]


def _q4_pack(v, s, C):
    """Stored form of code values and scale bytes, rows padded as programs keep them."""
    R = v.shape[0]
    a = v.abs()
    code = (a >= 0.5).int() + (a >= 1) + (a >= 1.5) + (a >= 2) + (a >= 3) + (a >= 4) + (a >= 6)
    code = (code + 8 * (v < 0)).to(torch.uint8)
    p = torch.zeros((R, _up(C, 32)), dtype=torch.uint8, device=DEV)
    p[:, :C] = code
    sb = torch.zeros((R, _up(s.shape[1], 8)), dtype=torch.uint8, device=DEV)
    sb[:, :s.shape[1]] = s
    return (p[:, 0::2] | (p[:, 1::2] << 4)).contiguous(), sb


def _q4_values(q, s, C):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    code = torch.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)[:, :C]
    return table[code.int()] * _q4_spread(s[:, :_up(C, 32) // 32], C)


# ---------------------------------------------------------------------------------------
# inputs


def _draw(gen, R, C, t, std=1.0):
    """Activations with a few strong columns, rows padded to 16 bytes; the [R][C] view."""
    x = torch.zeros((R, _up(C, 16)), dtype=T[t], device=DEV)
    strong = 1 + 7 * (torch.rand(C, generator=gen, device=DEV) < 0.01)
    x[:, :C] = (torch.randn((R, C), generator=gen, device=DEV) * (std * strong)).to(T[t])
    return x[:, :C]


def _room(R, C, t):
    return torch.zeros((R, _up(C, 16)), dtype=T[t], device=DEV)[:, :C]


def _space(R, C):
    """Room for row blocks of 8 bits."""
    return (torch.zeros((R, _up(C, 16)), dtype=torch.uint8, device=DEV),
            torch.zeros((_up(C, 128) // 128, _up(R, 16)), dtype=torch.uint8, device=DEV))


def _q4_space(R, C):
    return (torch.zeros((R, _up(C, 32) // 2), dtype=torch.uint8, device=DEV),
            torch.zeros((R, _up(_up(C, 32) // 32, 8)), dtype=torch.uint8, device=DEV))


def _store(x, fmt):
    """Row blocks, rows and scale rows padded as programs keep them."""
    q, s = _quantise(x.float(), fmt)
    qb, sb = _space(*x.shape)
    qb[:, :x.shape[1]] = q.view(torch.uint8)
    sb[:, :s.shape[1]] = s
    return qb, sb


def _store_weights(gen, E, N, C):
    """The experts' weights, stacked with a multiple of 128 rows each, in square blocks."""
    NS, CS = _up(N, 128), _up(C, 128)
    w = torch.zeros((E, NS, CS), device=DEV)
    w[:, :N, :C] = torch.randn((E, N, C), generator=gen, device=DEV) * C ** -0.5
    a = w.view(E * NS // 128, 128, CS // 128, 128).abs().amax((1, 3))
    b = (((a.view(torch.int32) + 0x1FFFFF) >> 23) - BIAS["e4m3"]).clamp(min=17)
    inv = ((254 - b) << 23).view(torch.float32).repeat_interleave(128, 0).repeat_interleave(128, 1)
    q = (w.view(E * NS, CS) * inv).to(F8["e4m3"]).view(torch.uint8)[:, :_up(C, 16)].contiguous()
    sb = torch.zeros((CS // 128, _up(E * NS // 128, 16)), dtype=torch.uint8, device=DEV)
    sb[:, :E * NS // 128] = b.t()
    return q, sb


def _choices(gen, c):
    """expert [T][K]: different experts for a token, some experts chosen far more often; a few
    choices are dropped."""
    liking = torch.randn((1, c["E"]), generator=gen, device=DEV)
    score = liking - torch.log(-torch.log(torch.rand((c["T"], c["E"]), generator=gen, device=DEV).clamp(1e-9, 1 - 1e-6)))
    expert = score.topk(c["K"], dim=1).indices.int()
    drop = torch.rand((c["T"], c["K"]), generator=gen, device=DEV) < 0.01
    return torch.where(drop, torch.full_like(expert, -1), expert).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s, op = case, {"case": case}, case["op"]
    if op == "q4_store":
        s["x"] = _draw(gen, c["R"], c["C"], c["x"])
        s["q"], s["y"] = _q4_space(c["R"], c["C"]), _room(c["R"], c["C"], "bf16")
        if c["both"]:
            s["qt"], s["yt"] = _q4_space(c["C"], c["R"]), _room(c["C"], c["R"], "bf16")
    elif op == "q4_gemm":
        s["a"] = _q4_pack(*_q4_quantise(_draw(gen, c["M"], c["K"], "f32")), c["K"])
        s["b"] = _q4_pack(*_q4_quantise(_draw(gen, c["N"], c["K"], "f32", c["K"] ** -0.5)), c["K"])
        s["c"] = _room(c["M"], c["N"], c["out"])
    else:
        R = _most_rows(c)
        expert = _choices(gen, c)
        s["first"], s["rows"], s["place"] = _route(expert, c["E"])
        if op == "dispatch":
            s["expert"] = expert
            s["x"] = _draw(gen, c["T"], c["D"], c["x"])
            s["out"] = _space(R, c["D"]) if c["q"] else _room(R, c["D"], c["x"])
            s["first"], s["rows"] = torch.empty_like(s["first"]), torch.empty_like(s["rows"])
            s["place"] = torch.empty_like(s["place"])
        elif op in ("combine", "combine_train"):
            s["sorted"] = _draw(gen, R, c["D"], c["x"])
            s["w"] = torch.rand((c["T"], c["K"]), generator=gen, device=DEV)
            s["w"] /= s["w"].sum(1, keepdim=True)
            s["y"] = _room(c["T"], c["D"], c["y"] if op == "combine" else c["x"])
            if op == "combine_train":
                s["dy"] = _draw(gen, c["T"], c["D"], c["x"], 1e-3)
                s["dsorted"], s["dx"] = _space(R, c["D"]), _room(c["T"], c["D"], c["x"])
                s["din"] = _draw(gen, R, c["D"], c["x"], 1e-3)  # what comes back through the experts
                s["dw"] = torch.zeros((c["T"], c["K"]), device=DEV)
        else:
            s["most"] = max(1, int(s["rows"].max()))
            if op == "gemm":
                s["a"] = _store(_draw(gen, R, c["D"], "f32", 1e-3 if c["a"] == "e5m2" else 1.0), c["a"])
                s["b"] = _store_weights(gen, c["E"], c["N"], c["D"])
                s["c"] = _room(R, c["N"], c["out"])
            else:
                dy = _draw(gen, R, c["N"], "bf16", 1e-3)
                s["dy"] = dy if c["dy"] == "bf16" else _store(dy, c["dy"])
                s["x"] = _store(_draw(gen, R, c["D"], "f32"), "e4m3")
                s["dw"] = torch.zeros((c["E"], c["N"], c["D"]), device=DEV)
                if c["acc"]:
                    s["dw0"] = torch.randn((c["E"], c["N"], c["D"]), generator=gen, device=DEV) * 1e-2
    if own:  # the descriptors and the workspace that a program makes once
        _handles(s)
    return s


def _handles(s):
    import count_sketch_aggregation_amd as s2r
    c, op = s["case"], s["case"]["op"]
    s["s2r"] = s2r
    room = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    if op == "q4_store":
        s["h"] = [s2r.mat(s["x"]), s2r.q4_mat(*s["q"]), s2r.mat(s["y"])]
        s["h"] += [s2r.q4_mat(*s["qt"]), s2r.mat(s["yt"])] if c["both"] else [None, None]
        return
    if op == "q4_gemm":
        s["h"] = [s2r.q4_mat(*s["a"]), s2r.q4_mat(*s["b"]), s2r.mat(s["c"])]
        s["ws"] = room(s2r.s2r_q4_gemm_workspace_bytes(c["M"], c["N"], c["K"]))
        return
    s["R"] = _most_rows(c)
    if op == "dispatch":
        s["h"] = [s2r.mat(s["x"]), None if c["q"] else s2r.mat(s["out"]),
                  s2r.q8_mat(*s["out"], c["q"]) if c["q"] else None]
        s["ws"] = room(s2r.s2r_moe_route_workspace_bytes(c["T"], c["K"], c["E"]))
    elif op == "combine":
        s["h"] = [s2r.mat(s["sorted"]), s2r.mat(s["y"])]
    elif op == "combine_train":
        s["h"] = [s2r.mat(s["sorted"]), s2r.mat(s["y"]), s2r.mat(s["dy"]), s2r.q8_mat(*s["dsorted"], c["q"]),
                  s2r.mat(s["din"]), s2r.mat(s["dx"])]
    else:
        s["e"] = s2r.experts(s["first"], s["rows"])
        if op == "gemm":
            s["h"] = [s2r.q8_mat(*s["a"], c["a"]), s2r.q8_mat(*s["b"]), s2r.mat(s["c"])]
        else:
            s["h"] = [s2r.mat(s["dy"]) if c["dy"] == "bf16" else s2r.q8_mat(*s["dy"], c["dy"]), s2r.q8_mat(*s["x"])]


# ---------------------------------------------------------------------------------------
# one pass


def _stored(pair, R, C, fmt):
    return [pair[0][:R, :C].view(F8[fmt]), pair[1][:, :R].view(torch.float8_e8m0fnu)]


def _q4_scales(pair, C):
    return pair[1][:, :_up(C, 32) // 32].view(torch.float8_e8m0fnu)


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, op, s2r, h = s["case"], s["case"]["op"], s["s2r"], s["h"]
    if op == "dispatch":
        s2r.s2r_moe_route(c["T"], c["K"], c["E"], s["expert"], s["first"], s["rows"], s["place"], workspace=s["ws"])
        s2r.s2r_moe_gather(c["T"], c["K"], c["D"], h[0], s["place"], s["R"], out=h[1], outq=h[2])
        out = _stored(s["out"], s["R"], c["D"], c["q"]) if c["q"] else [s["out"]]
        return [s["first"], s["rows"], s["place"]] + out
    if op == "combine":
        s2r.s2r_moe_combine(c["T"], c["K"], c["D"], h[0], s["R"], s["place"], s["w"], h[1])
        return s["y"]
    if op == "combine_train":
        s2r.s2r_moe_combine(c["T"], c["K"], c["D"], h[0], s["R"], s["place"], s["w"], h[1])
        s2r.s2r_moe_combine_grad(c["T"], c["K"], c["D"], h[2], s["place"], s["R"], weight=s["w"], rows=h[0],
                                 drowsq=h[3], dweight=s["dw"])
        s2r.s2r_moe_combine(c["T"], c["K"], c["D"], h[4], s["R"], s["place"], None, h[5])
        return [s["y"], s["dw"], s["dx"]] + _stored(s["dsorted"], s["R"], c["D"], c["q"])
    if op == "gemm":
        NS = _up(c["N"], 128)
        s2r.s2r_q8_gemm_experts(s["R"], c["N"], c["D"], s["e"], h[0], h[1], NS * h[1].ld, NS // 128, h[2])
        return s["c"]
    if op == "wgrad":
        if c["acc"]:
            s["dw"].copy_(s["dw0"])
        s2r.s2r_q8_wgrad_experts(s["R"], c["N"], c["D"], s["e"], h[0], h[1], s["dw"], c["D"], c["N"] * c["D"],
                                 accumulate=c["acc"])
        return s["dw"]
    if op == "q4_store":
        s2r.s2r_q4_save(c["R"], c["C"], h[0], h[1], h[3])
        s2r.s2r_q4_load(c["R"], c["C"], h[1], h[2])
        out = [s["y"], _q4_scales(s["q"], c["C"])]
        if c["both"]:
            s2r.s2r_q4_load(c["C"], c["R"], h[3], h[4])
            out += [s["yt"], _q4_scales(s["qt"], c["R"])]
        return out
    s2r.s2r_q4_gemm(c["M"], c["N"], c["K"], h[0], h[1], h[2], workspace=s["ws"])
    return s["c"]


def _q4_stored(x):
    v, b = _q4_quantise(x)
    return [(v * _q4_spread(b, x.shape[1])).to(torch.bfloat16), b.view(torch.float8_e8m0fnu)]


def _run_plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        first, rows, place = _route(s["expert"], c["E"])
        if not c["q"]:
            x = s["x"][:, None].expand(c["T"], c["K"], c["D"])
            return [first, rows, place, _by_row(x, place, s["out"])]
        q, b = _quantise(s["x"].float(), c["q"])
        q = q.view(torch.uint8)[:, None].expand(c["T"], c["K"], c["D"])
        b = b.t()[:, None].expand(c["T"], c["K"], b.shape[0])
        R = _most_rows(c)
        q = _by_row(q, place, s["out"][0][:, :c["D"]])
        b = _by_row(b, place, s["out"][1][:, :R].t()).t().contiguous()
        return [first, rows, place, q.view(F8[c["q"]]), b.view(torch.float8_e8m0fnu)]
    if op in ("combine", "combine_train"):
        r = _by_token(s["sorted"], s["place"])
        y = (s["w"][..., None] * r).sum(1).to(s["y"].dtype)
        if op == "combine":
            return y
        dy = s["dy"].float()
        dw = (r * dy[:, None]).sum(2)
        q, b = _quantise((s["w"][..., None] * dy[:, None]).reshape(-1, c["D"]), c["q"])
        R = _most_rows(c)
        q = _by_row(q.view(torch.uint8), s["place"], s["dsorted"][0][:, :c["D"]])
        b = _by_row(b.t(), s["place"], s["dsorted"][1][:, :R].t()).t().contiguous()
        dx = _by_token(s["din"], s["place"]).sum(1).to(s["dx"].dtype)
        return [y, dw, dx, q.view(F8[c["q"]]), b.view(torch.float8_e8m0fnu)]
    if op == "gemm":
        a = _grouped(_values(*s["a"], _most_rows(c), c["D"], c["a"]), s)
        w = _weights(*s["b"], c["E"], c["N"], c["D"])
        return _ungrouped(torch.bmm(a, w.transpose(1, 2).contiguous()), s, s["c"])
    if op == "wgrad":
        R = _most_rows(c)
        dy = s["dy"].float() if c["dy"] == "bf16" else _values(*s["dy"], R, c["N"], c["dy"])
        x = _grouped(_values(*s["x"], R, c["D"], "e4m3"), s)
        dw = torch.bmm(_grouped(dy, s).transpose(1, 2).contiguous(), x)
        return s["dw0"] + dw if c["acc"] else dw
    if op == "q4_store":
        x = s["x"].float()
        return _q4_stored(x) + (_q4_stored(x.t().contiguous()) if c["both"] else [])
    return (_q4_values(*s["a"], c["K"]) @ _q4_values(*s["b"], c["K"]).t()).to(T[c["out"]])


# ---------------------------------------------------------------------------------------
# the definition in 64 bits


def _grid(fmt, codes):
    """Values of a format's codes from its definition."""
    ebits, mbits, bias = {"e4m3": (4, 3, 7), "e5m2": (5, 2, 15), "e2m1": (2, 1, 1)}[fmt]
    out = []
    for code in range(codes):
        e, m = (code >> mbits) & (2 ** ebits - 1), code & (2 ** mbits - 1)
        v = 2.0 ** (1 - bias) * m / 2 ** mbits if e == 0 else 2.0 ** (e - bias) * (1 + m / 2 ** mbits)
        out.append(-v if code >= codes // 2 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _two_to(e):
    """2^e in 64 bits, to the bit."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(pair, R, C, fmt):
    v = _grid(fmt, 256)[pair[0][:R, :C].int()]
    for k in range(0, C, 128):
        v[:, k:k + 128] *= _two_to(pair[1][k // 128, :R].int() - 127)[:, None]
    return v


def _exact_q4(pair, C):
    code = torch.empty((pair[0].shape[0], 2 * pair[0].shape[1]), dtype=torch.uint8, device=DEV)
    code[:, 0::2], code[:, 1::2] = pair[0] & 15, pair[0] >> 4
    v = _grid("e2m1", 16)[code.int()][:, :C]
    for k in range(0, C, 32):
        v[:, k:k + 32] *= _two_to(pair[1][:, k // 32].int() - 127)[:, None]
    return v


def _exact_stored(x, fmt, block, low, mbits, top, most):
    """(code values, scales) in 64 bits: the scale by comparison, the rounding on the format's grid.
    The format's largest value is most * 2^top, its least normal 2^low."""
    R, C = x.shape
    n = -(-C // block)
    scale = torch.empty((R, n), dtype=torch.float64, device=DEV)
    code = torch.empty((R, C), dtype=torch.float64, device=DEV)
    for k in range(n):
        part = x[:, k * block:(k + 1) * block]
        m, e = torch.frexp(part.abs().amax(1))
        e = torch.where(m > 0, e - top + (m > most), -110).clamp(min=-110)
        scale[:, k] = _two_to(e)
        v = part / scale[:, k:k + 1]
        step = _two_to(torch.frexp(v.abs().clamp(min=2.0 ** low))[1] - 1 - mbits)
        code[:, k * block:(k + 1) * block] = torch.round(v / step) * step
    return code, scale


def _exact_q8(x, fmt):
    return _exact_stored(x, fmt, 128, *((-6, 3, 9, 0.875) if fmt == "e4m3" else (-14, 2, 16, 0.875)))


def _exact_route(expert, E):
    """place as lists, by going through the choices."""
    flat = expert.reshape(-1).tolist()
    rows = [0] * E
    for e in flat:
        if 0 <= e < E:
            rows[e] += 1
    first = [sum((r + 3) // 4 * 4 for r in rows[:e]) for e in range(E)]
    nxt, place = list(first), []
    for e in flat:
        place.append(nxt[e] if 0 <= e < E else -1)
        if 0 <= e < E:
            nxt[e] += 1
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    return as_int(first), as_int(rows), as_int(place).view(expert.shape)


def _exact_rows(pair, place, R, K):
    """Code values and scales of rows [T * K] or [T], of their choices' places; zeros elsewhere."""
    code, scale = pair
    at = place.reshape(-1).long()
    some = at >= 0
    of = torch.arange(at.numel(), device=DEV) // (at.numel() // code.shape[0])
    q = torch.zeros((R, code.shape[1]), dtype=torch.float64, device=DEV)
    b = torch.full((R, scale.shape[1]), 2.0 ** -127, dtype=torch.float64, device=DEV)
    q[at[some]], b[at[some]] = code[of[some]], scale[of[some]]
    return [q, b.t().contiguous()]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op == "q4_store":
        x, out = s["x"].double(), []
        for v in [x, x.t()] if c["both"] else [x]:
            code, scale = _exact_stored(v, "e2m1", 32, 0, 1, 3, 0.75)
            out += [code * scale.repeat_interleave(32, 1)[:, :v.shape[1]], scale]
        return out
    if op == "q4_gemm":
        return _exact_q4(s["a"], c["K"]) @ _exact_q4(s["b"], c["K"]).t()
    R, D = _most_rows(c), c["D"]
    if op == "dispatch":
        first, rows, place = _exact_route(s["expert"], c["E"])
        x = s["x"].double()
        if c["q"]:
            return [first, rows, place] + _exact_rows(_exact_q8(x, c["q"]), place, R, c["K"])
        out = torch.zeros((R, D), dtype=torch.float64, device=DEV)
        for k in range(c["K"]):
            some = place[:, k] >= 0
            out[place[some, k].long()] = x[some]
        return [first, rows, place, out]
    if op in ("combine", "combine_train"):
        def added(rows, w):
            y = torch.zeros((c["T"], D), dtype=torch.float64, device=DEV)
            for k in range(c["K"]):
                some = s["place"][:, k] >= 0
                y[some] += rows[s["place"][some, k].long()].double() * (1 if w is None else w[some, k, None].double())
            return y
        y = added(s["sorted"], s["w"])
        if op == "combine":
            return y
        dy = s["dy"].double()
        dw = torch.zeros((c["T"], c["K"]), dtype=torch.float64, device=DEV)
        for k in range(c["K"]):
            some = s["place"][:, k] >= 0
            dw[some, k] = (s["sorted"][s["place"][some, k].long()].double() * dy[some]).sum(1)
        # the operator stores products rounded to 32 bits
        dr = (s["w"][..., None].double() * dy[:, None]).float().double().reshape(-1, D)
        return [y, dw, added(s["din"], None)] + _exact_rows(_exact_q8(dr, c["q"]), s["place"], R, c["K"])
    first, rows = s["first"].tolist(), s["rows"].tolist()
    if op == "gemm":
        a, NS = _exact_values(s["a"], R, D, c["a"]), _up(c["N"], 128)
        out = torch.zeros((R, c["N"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            w = _grid("e4m3", 256)[s["b"][0][e * NS:e * NS + c["N"], :D].int()]
            for k in range(0, D, 128):
                w[:, k:k + 128] *= _two_to(s["b"][1][k // 128, e * NS // 128:(e + 1) * NS // 128].int() - 127) \
                    .repeat_interleave(128)[:c["N"], None]
            out[first[e]:first[e] + rows[e]] = a[first[e]:first[e] + rows[e]] @ w.t()
        return out
    dy = s["dy"].double() if c["dy"] == "bf16" else _exact_values(s["dy"], R, c["N"], c["dy"])
    x = _exact_values(s["x"], R, D, "e4m3")
    dw = torch.stack([dy[f:f + r].t() @ x[f:f + r] for f, r in zip(first, rows)])
    return s["dw0"].double() + dw if c["acc"] else dw


def work(case):
    c, op = case, case["op"]
    if op == "q4_store":  # x read; codes and scales written, and read to be returned as values
        n = c["R"] * c["C"]
        return {"bytes": n * SIZE[c["x"]] + (2 if c["both"] else 1) * (n * 17 // 16 + 2 * n), "flops": 0}
    if op == "q4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K * 17 // 32 + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    A, D = c["T"] * c["K"], c["D"]
    if op == "dispatch":
        row = D * 129 // 128 if c["q"] else D * SIZE[c["x"]]
        return {"bytes": 8 * A + 8 * c["E"] + c["T"] * D * SIZE[c["x"]] + A * row, "flops": 0}
    if op == "combine":
        return {"bytes": A * (D * SIZE[c["x"]] + 8) + c["T"] * D * SIZE[c["y"]], "flops": 2 * A * D}
    if op == "combine_train":  # y from the rows; their gradients and the weights'; dx from what comes back
        t = D * SIZE[c["x"]]
        return {"bytes": 2 * A * t + 2 * c["T"] * t + A * t + c["T"] * t + A * D * 129 // 128 + 20 * A, "flops": 6 * A * D}
    if op == "gemm":
        weights = min(c["E"], A) * c["N"] * D
        return {"bytes": A * D + weights + A * c["N"] * SIZE[c["out"]], "flops": 2 * A * c["N"] * D}
    return {"bytes": A * c["N"] * (2 if c["dy"] == "bf16" else 1) + A * D + c["E"] * c["N"] * D * (8 if c["acc"] else 4),
            "flops": 2 * A * c["N"] * D}
