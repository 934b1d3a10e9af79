"""Data-parallel training of a layer of gated experts in 8 bits, end to end through libs2r:

    out[t] = sum over the K chosen experts e of weight[t][e] * (silu(x Wg_e^T) * (x Wu_e^T)) Wd_e^T

The router's K largest scores choose a token's experts, and their softmax weighs them.  Each of W
workers (buffers of one GPU) sorts its tokens by expert, runs every expert's rows through 8-bit products in
one launch each and writes all weight gradients straight into its row of the gradient matrix (include/s2r_moe.h),
which block-wise Top-K, sketch and bitmap then aggregate as in q8_training.py: an expert that
no token chose has a gradient of zeros.  The target is a fixed layer of the same shape.

    python examples/q8_experts.py [--steps 40] [--workers 2] [--tokens 512] [--experts 8] [--choices 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import q8_training  # noqa: E402  (finds the package, too)
import count_sketch_aggregation_amd as s2r  # noqa: E402


def columns(m, first, cols):
    """Columns first .. first + cols - 1 of an 8-bit matrix in row blocks; multiples of 128."""
    fmt = "e4m3" if m.format == s2r.S2R_E4M3 else "e5m2"
    return s2r.q8_mat(m.codes[:, first:first + cols], m.scales[first // 128:(first + cols) // 128], fmt)


class ExpertLayer:
    """E experts on `tokens` tokens of K choices; width and hidden are multiples of 128.  `flat` holds, one after the
    other in fp32, every expert's Wg over Wu [2 hidden][width], every expert's Wd [width][hidden]
    and the router [E][width].  Gate and up projections are one product, their results side by side."""

    def __init__(self, tokens, width, hidden, experts, choices, dev="cuda"):
        T, D, F, E, K = self.sizes = tokens, width, hidden, experts, choices
        assert D % 128 == 0 and F % 128 == 0
        self.R = R = s2r.s2r_moe_rows(T, K, E)
        self.n = 3 * E * D * F + E * D
        self.flat = torch.empty(self.n, device=dev)
        self.wgu, self.wd, self.router = self.views(self.flat)
        for w in (self.wgu, self.wd, self.router):
            w.normal_(0, w.shape[-1] ** -0.5)
        q = lambda rows, cols, fmt="e4m3", **k: s2r.alloc_q8(rows, cols, fmt, device=dev, **k)
        # weights of all experts in square blocks, stacked; the transposed copies lie side by side
        self.wgu8, self.wgu8t = q(E * 2 * F, D, square=True), q(D, E * 2 * F, square=True)
        self.wd8, self.wd8t = q(E * D, F, square=True), q(F, E * D, square=True)
        # which rows
        self.first, self.rows = (torch.empty(E, dtype=torch.int32, device=dev) for _ in range(2))
        self.place = torch.empty((T, K), dtype=torch.int32, device=dev)
        self.experts = s2r.experts(self.first, self.rows)
        self.ws = q8_training._workspace(s2r.s2r_moe_route_workspace_bytes(T, K, E), dev)
        # sorted rows: checkpoints, gradients in 8 bits, and what is not kept
        self.x8, self.gu8, self.y8 = q(R, D), q(R, 2 * F), q(R, F)
        self.drows8, self.dgu8 = q(R, D, "e5m2"), q(R, 2 * F, "e5m2")
        self.gu, self.dy, self.expert_out, self.dx_rows = (q8_training.matrix(R, c, dev) for c in (2 * F, F, D, D))
        self.out, self.dx = q8_training.matrix(T, D, dev), q8_training.matrix(T, D, dev)
        self.dweight = torch.empty((T, K), device=dev)

    def views(self, row):
        """The weights, or their gradients, in a row of n floats."""
        T, D, F, E, K = self.sizes
        gu, d, r = row[:self.n].split([2 * E * D * F, E * D * F, E * D])
        return gu.view(E, 2 * F, D), d.view(E, D, F), r.view(E, D)

    def weights_to_8_bits(self):
        """After an update, once for all workers."""
        T, D, F, E, K = self.sizes
        s2r.s2r_q8_weight(E * 2 * F, D, s2r.mat(self.wgu.view(-1, D)), self.wgu8, self.wgu8t)
        s2r.s2r_q8_weight(E * D, F, s2r.mat(self.wd.view(-1, F)), self.wd8, self.wd8t)

    def forward(self, x):
        T, D, F, E, K = self.sizes
        self.x = x.float()
        self.scores = (self.x @ self.router.t()).requires_grad_()
        best, expert = self.scores.topk(K, dim=1)
        self.weight = best.softmax(1)
        self.expert = expert.int()
        s2r.s2r_moe_route(T, K, E, self.expert, self.first, self.rows, self.place, workspace=self.ws)
        s2r.s2r_moe_gather(T, K, D, s2r.mat(x), self.place, self.R, outq=self.x8)
        s2r.s2r_q8_gemm_experts(self.R, 2 * F, D, self.experts, self.x8, self.wgu8, 2 * F * self.wgu8.ld, 2 * F // 128,
                                s2r.mat(self.gu))
        s2r.s2r_q8_glu(self.R, F, "silu", s2r.mat(self.gu[:, :F]), s2r.mat(self.gu[:, F:]), gq=columns(self.gu8, 0, F),
                       uq=columns(self.gu8, F, F), yq=self.y8)
        s2r.s2r_q8_gemm_experts(self.R, D, F, self.experts, self.y8, self.wd8, D * self.wd8.ld, D // 128,
                                s2r.mat(self.expert_out))
        s2r.s2r_moe_combine(T, K, D, s2r.mat(self.expert_out), self.R, self.place, self.weight.detach(), s2r.mat(self.out))
        return self.out

    def backward(self, out_grad, row):
        """The weights' gradients into `row`, a worker's row of the gradient matrix; returns x's through the
        experts (the router's part is left to whoever needs it)."""
        T, D, F, E, K = self.sizes
        dwgu, dwd, drouter = self.views(row)
        s2r.s2r_moe_combine_grad(T, K, D, s2r.mat(out_grad), self.place, self.R, weight=self.weight.detach(),
                                 rows=s2r.mat(self.expert_out), drowsq=self.drows8, dweight=self.dweight)
        s2r.s2r_q8_wgrad_experts(self.R, D, F, self.experts, self.drows8, self.y8, dwd, F, D * F)
        s2r.s2r_q8_gemm_experts(self.R, F, D, self.experts, self.drows8, self.wd8t, D, D // 128 * self.wd8t.lds,
                                s2r.mat(self.dy))
        s2r.s2r_q8_glu_grad(self.R, F, "silu", columns(self.gu8, 0, F), columns(self.gu8, F, F), s2r.mat(self.dy),
                            dgq=columns(self.dgu8, 0, F), duq=columns(self.dgu8, F, F))
        s2r.s2r_q8_wgrad_experts(self.R, 2 * F, D, self.experts, self.dgu8, self.x8, dwgu, D, 2 * F * D)
        s2r.s2r_q8_gemm_experts(self.R, D, 2 * F, self.experts, self.dgu8, self.wgu8t, 2 * F, 2 * F // 128 * self.wgu8t.lds,
                                s2r.mat(self.dx_rows))
        s2r.s2r_moe_combine(T, K, D, s2r.mat(self.dx_rows), self.R, self.place, None, s2r.mat(self.dx))
        dscores, = torch.autograd.grad(self.weight, self.scores, self.dweight)
        drouter.copy_(dscores.t() @ self.x)
        return self.dx


def train(steps=40, workers=2, tokens=512, width=128, hidden=256, experts=8, choices=2, lr=40.0, dev="cuda", log=print):
    """The loss of every step."""
    torch.manual_seed(0)
    layer, goal = (ExpertLayer(tokens, width, hidden, experts, choices, dev) for _ in range(2))
    goal.weights_to_8_bits()
    aggregate = q8_training.Aggregation(workers, layer.n, dev=dev)
    x = [q8_training.matrix(tokens, width, dev).normal_() for _ in range(workers)]
    out_grad = q8_training.matrix(tokens, width, dev)
    target = [goal.forward(b).float().clone() for b in x]
    losses = []
    for step in range(steps):
        layer.weights_to_8_bits()
        loss = torch.zeros((), device=dev)
        for k in range(workers):
            diff = layer.forward(x[k]).float() - target[k]
            loss += diff.square().mean() / workers
            layer.backward(out_grad.copy_(diff * (2 / diff.numel())), aggregate.grads[k])
        layer.flat.add_(aggregate(), alpha=-lr / workers)
        losses.append(float(loss))
        if log and (step % 5 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {losses[-1]:.5f}", flush=True)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in [("steps", 40), ("workers", 2), ("tokens", 512), ("experts", 8), ("choices", 2)]:
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    train(a.steps, a.workers, a.tokens, experts=a.experts, choices=a.choices)


if __name__ == "__main__":
    main()
