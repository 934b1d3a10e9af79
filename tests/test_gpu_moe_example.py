"""The example of a layer of experts: its gradients against torch's in 64 bits, eager and from replays of a
graph whose tokens choose other experts each time, on several streams and threads."""
import importlib.util
import os
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

gp = pytest.importorskip("gpu_path")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "q8_experts.py")
    spec = importlib.util.spec_from_file_location("q8_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, x, out_grad):
    """out and the gradients of Wg over Wu, Wd, the router and, through the experts alone, x, in 64 bits, with the layer's
    choices."""
    T, D, F, E, K = layer.sizes
    w = [t.double().cpu().requires_grad_() for t in (layer.wgu, layer.wd, layer.router)]
    xd = x.double().cpu()
    xe = xd.clone().requires_grad_()
    expert = layer.expert.long().cpu()
    weight = (xd @ w[2].t()).gather(1, expert).softmax(1)
    out = torch.zeros((T, D), dtype=torch.float64)
    for e in range(E):
        t, k = (expert == e).nonzero(as_tuple=True)
        gu = xe[t] @ w[0][e].t()
        y = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ w[1][e].t()
        out = out.index_add(0, t, y * weight[t, k, None])
    out.backward(out_grad.double().cpu())
    return out.detach(), [t.grad for t in w], xe.grad


@pytest.mark.parametrize("tokens,width,hidden,experts,choices", [(300, 128, 256, 8, 2), (40, 256, 128, 16, 4), (700, 128, 128, 3, 1)])
def test_gradients(example, tokens, width, hidden, experts, choices):
    """What differs is the storage in 8 bits: independent roundings of at most 2^-4 (e4m3) or 2^-3 (e5m2) of
    a value, on average below half of that.  A gradient passes at most eight of e4m3 (token, gate and
    up weights, gate, up, activation, down weight, result) and two of e5m2: in the root of the
    sum of squares below sqrt(8 * 2^-10 + 2 * 2^-8) = 0.125."""
    gp.say(f"experts example gradients {tokens}x{choices} of {experts}, {width}x{hidden}")
    torch.manual_seed(1)
    layer = example.ExpertLayer(tokens, width, hidden, experts, choices)
    layer.weights_to_8_bits()
    x, d = (example.q8_training.matrix(tokens, width) for _ in range(2))
    x.normal_()
    d.normal_(0, 1e-3)
    row = torch.full((layer.n,), 7.0, device="cuda")
    out = layer.forward(x).double().cpu()
    dx = layer.backward(d, row).double().cpu()
    want, grads, want_dx = reference(layer, x, d)
    assert (out - want).norm() < 0.125 * want.norm()
    for got, g in zip(layer.views(row), grads):
        if choices == 1 and g.shape == layer.router.shape:
            assert bool((got == 0).all())  # the softmax of one score is 1
        else:
            assert (got.double().cpu() - g).norm() < 0.125 * g.norm()
    assert (dx - want_dx).norm() < 0.125 * want_dx.norm()
    for e in range(experts):
        if not bool((layer.expert == e).any()):
            assert bool((layer.views(row)[0][e] == 0).all()) and bool((layer.views(row)[1][e] == 0).all())


def everything(layer, x, d, row):
    layer.forward(x)
    layer.backward(d, row)
    return [t.clone() for t in (layer.out, layer.dx, layer.dweight, row, layer.place, layer.first, layer.rows)]


def test_graph_replays_of_other_choices(example):
    """One captured pass serves every routing: nothing in it goes by how many rows an expert has."""
    gp.say("experts example, graph")
    torch.manual_seed(2)
    T, D = 600, 128
    layer = example.ExpertLayer(T, D, 128, 8, 2)
    layer.weights_to_8_bits()
    x, d = example.q8_training.matrix(T, D), example.q8_training.matrix(T, D).normal_(0, 1e-3)
    row = torch.zeros(layer.n, device="cuda")
    inputs = [torch.randn((T, D), device="cuda") + shift for shift in (0, 1, -2)]
    want = []
    for v in inputs:
        x.copy_(v)
        want.append(everything(layer, x, d, row))
    assert not torch.equal(want[0][4], want[1][4])
    graph = torch.cuda.CUDAGraph()
    e = layer.sizes[3]
    scores = torch.randn((T, e), device="cuda")
    # the router's own torch operations stay outside
    weight, expert = torch.rand((T, 2), device="cuda"), torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    s2r = example.s2r

    def library(layer):
        T, D, F, E, K = layer.sizes
        s2r.s2r_moe_route(T, K, E, expert, layer.first, layer.rows, layer.place, workspace=layer.ws)
        s2r.s2r_moe_gather(T, K, D, s2r.mat(x), layer.place, layer.R, outq=layer.x8)
        s2r.s2r_q8_gemm_experts(layer.R, 2 * F, D, layer.experts, layer.x8, layer.wgu8, 2 * F * layer.wgu8.ld, 2 * F // 128,
                                s2r.mat(layer.gu))
        s2r.s2r_q8_wgrad_experts(layer.R, D, D, layer.experts, s2r.mat(layer.gu[:, :D]), layer.x8, row, D, D * D)
        s2r.s2r_moe_combine(T, K, D, s2r.mat(layer.gu[:, :D]), layer.R, layer.place, weight, s2r.mat(layer.out))
        s2r.s2r_moe_combine_grad(T, K, D, s2r.mat(d), layer.place, layer.R, weight=weight, rows=s2r.mat(layer.gu[:, :D]),
                                 drowsq=layer.drows8, dweight=layer.dweight)

    used = lambda: [t.clone() for t in (layer.out, layer.dweight, row[:e * D * D], layer.place, layer.first, layer.rows)]
    with torch.cuda.graph(graph):
        library(layer)
    for rep in range(4):
        expert.copy_((scores + (rep % 3) * torch.arange(e, device="cuda")).topk(2, dim=1).indices)
        if rep == 2:
            expert.fill_(-1)
        library(layer)
        eager = used()
        for t in (layer.out, layer.dweight, row, layer.place, layer.first, layer.rows):
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(used(), eager)), rep
        x.copy_(inputs[rep % 3])


def test_the_same_bits_on_streams_and_threads(example):
    gp.say("experts example, threads")
    torch.manual_seed(3)
    layers, rows, ins = [], [], []
    for i in range(3):
        layer = example.ExpertLayer(500, 128, 128, 6, 2)
        layer.weights_to_8_bits()
        layers.append(layer)
        rows.append(torch.zeros(layer.n, device="cuda"))
        ins.append((example.q8_training.matrix(500, 128).normal_(), example.q8_training.matrix(500, 128).normal_(0, 1e-3)))
    want = [everything(l, x, d, r) for l, (x, d), r in zip(layers, ins, rows)]
    torch.cuda.synchronize()
    got, errors = [None] * 3, []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(3):
                    got[i] = everything(layers[i], *ins[i], rows[i])
            stream.synchronize()
        except Exception as e:  # surfaced below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        # the router's own gradient is torch's
        n = layers[0].n - layers[0].router.numel()
        assert all(torch.equal(u[:n] if i == 3 else u, v[:n] if i == 3 else v) for i, (u, v) in enumerate(zip(a, b)))


def test_training_runs(example):
    gp.say("experts example, training")
    losses = example.train(steps=4, log=None)
    assert len(losses) == 4 and all(l == l and l < float("inf") for l in losses)
