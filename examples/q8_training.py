"""Data-parallel training of a gated feed-forward layer in 8 bits, end to end through libs2r:

    out = (silu(x Wg^T) * (x Wu^T)) Wd^T

Each of W workers (buffers of one GPU) runs the layer on its own batch with 8-bit products and
8-bit checkpoints (include/s2r_q8.h) and writes its weight gradients in fp32 straight into its
row of the gradient matrix; block-wise Top-K with error feedback makes the rows sparse, and
encode, reduce and decode aggregate them (include/s2r.h).  The target is a fixed layer of the
same shape.

    python examples/q8_training.py [--steps 40] [--workers 4] [--tokens 512] [--fast]

--fast takes the products at the 8-bit matrix rate, which cuts them short (include/s2r_q8.h).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import count_sketch_aggregation_amd as s2r  # noqa: E402


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def matrix(rows, cols, dev="cuda"):
    """A bf16 matrix with its rows padded to 16 bytes, as the calls need them."""
    return torch.zeros((rows, -(-cols // 8) * 8), dtype=torch.bfloat16, device=dev)[:, :cols]


class FeedForward:
    """The layer's fp32 weights, one after the other in `flat`, their 8-bit copies, and the
    buffers of one pass over `tokens` rows; width and hidden are multiples of 4."""

    def __init__(self, tokens, width, hidden, dev="cuda", fast=False):
        self.gemm = s2r.s2r_q8_gemm_fast if fast else s2r.s2r_q8_gemm
        self.M, self.D, self.F = tokens, width, hidden
        M, D, F = tokens, width, hidden
        self.n = 3 * D * F
        self.flat = torch.empty(self.n, device=dev)
        self.wg, self.wu, self.wd = self.views(self.flat)
        for w in (self.wg, self.wu, self.wd):
            w.normal_(0, w.shape[1] ** -0.5)
        # weights: square blocks; the transposed copy of Wd carries the gradient back
        self.wg8, self.wu8 = (s2r.alloc_q8(F, D, square=True, device=dev) for _ in range(2))
        self.wd8 = s2r.alloc_q8(D, F, square=True, device=dev)
        self.wd8t = s2r.alloc_q8(F, D, square=True, device=dev)
        # checkpoints of the forward pass and gradients of the backward pass
        self.x8, self.out_grad8 = s2r.alloc_q8(M, D, device=dev), s2r.alloc_q8(M, D, "e5m2", device=dev)
        self.g8, self.u8, self.y8 = (s2r.alloc_q8(M, F, device=dev) for _ in range(3))
        self.dg8, self.du8 = (s2r.alloc_q8(M, F, "e5m2", device=dev) for _ in range(2))
        self.g, self.u, self.dy, self.out = (matrix(M, c, dev) for c in (F, F, F, D))
        need = max(s2r.s2r_q8_gemm_workspace_bytes(M, F, D), s2r.s2r_q8_gemm_workspace_bytes(M, D, F),
                   s2r.s2r_q8_wgrad_workspace_bytes(M, F, D), s2r.s2r_q8_wgrad_workspace_bytes(M, D, F))
        self.ws = _workspace(need, dev)

    def views(self, row):
        """Wg, Wu and Wd, or their gradients, in a row of n floats."""
        g, u, d = row[:self.n].split(self.D * self.F)
        return g.view(self.F, self.D), u.view(self.F, self.D), d.view(self.D, self.F)

    def weights_to_8_bits(self):
        """After an update, once for all workers."""
        s2r.s2r_q8_weight(self.F, self.D, s2r.mat(self.wg), self.wg8)
        s2r.s2r_q8_weight(self.F, self.D, s2r.mat(self.wu), self.wu8)
        s2r.s2r_q8_weight(self.D, self.F, s2r.mat(self.wd), self.wd8, self.wd8t)

    def forward(self, x):
        M, D, F = self.M, self.D, self.F
        s2r.s2r_q8_save(M, D, s2r.mat(x), self.x8)
        self.gemm(M, F, D, self.x8, self.wg8, s2r.mat(self.g), workspace=self.ws)
        self.gemm(M, F, D, self.x8, self.wu8, s2r.mat(self.u), workspace=self.ws)
        s2r.s2r_q8_glu(M, F, "silu", s2r.mat(self.g), s2r.mat(self.u), gq=self.g8, uq=self.u8, yq=self.y8)
        self.gemm(M, D, F, self.y8, self.wd8, s2r.mat(self.out), workspace=self.ws)
        return self.out

    def backward(self, out_grad, row):
        """The weights' gradients into `row`, a worker's row of the gradient matrix."""
        M, D, F = self.M, self.D, self.F
        dwg, dwu, dwd = self.views(row)
        s2r.s2r_q8_wgrad(M, D, F, s2r.mat(out_grad), self.y8, dwd, F, workspace=self.ws)
        s2r.s2r_q8_save(M, D, s2r.mat(out_grad), self.out_grad8)
        self.gemm(M, F, D, self.out_grad8, self.wd8t, s2r.mat(self.dy), workspace=self.ws)
        s2r.s2r_q8_glu_grad(M, F, "silu", self.g8, self.u8, s2r.mat(self.dy), dgq=self.dg8, duq=self.du8)
        s2r.s2r_q8_wgrad(M, F, D, self.dg8, self.x8, dwg, D, workspace=self.ws)
        s2r.s2r_q8_wgrad(M, F, D, self.du8, self.x8, dwu, D, workspace=self.ws)


class Aggregation:
    """W gradient rows of n floats to their summed Top-K parts, by sketch and bitmap."""

    def __init__(self, W, n, keep=0.125, block=256, dev="cuda"):
        self.W, self.n, self.block = W, n, block
        self.ld = -(-n // 4) * 4
        self.K = max(1, int(-(-n // block) * keep))
        kept = min(n, W * self.K * block)
        self.p = s2r.s2r_params_from_seed(1234, 5, s2r.s2r_log2_w_for_lambda(5, kept, 1.0))
        rows = lambda: torch.zeros((W, self.ld), device=dev)
        self.grads, self.residual, self.sparse = rows(), rows(), rows()
        self.topk_ws = _workspace(s2r.s2r_topk_workspace_bytes(W, n, block), dev)
        self.cap = self.K * block
        self.buf = s2r.alloc_encode_buffers(self.p, W, n, self.cap, dev)
        self.bitmap = torch.empty(s2r.s2r_bitmap_words(n), dtype=torch.int64, device=dev)
        self.sketch = torch.empty((self.p.d, 1 << self.p.log2_w), device=dev)
        self.decode_ws = s2r.alloc_decode_workspace(self.p, n, kept, dev)
        self.kept = kept
        self.sum = torch.empty(n, device=dev)

    def __call__(self):
        b, W, n = self.buf, self.W, self.n
        s2r.s2r_topk_ef(W, self.grads, self.residual, n, self.ld, self.block, self.K, self.sparse, None,
                        self.topk_ws)
        s2r.s2r_encode(self.p, W, self.sparse, n, self.ld, b["bitmaps"], b["sketches"], b["idx"], b["val"],
                       self.cap, b["nnz"], b["workspace"])
        s2r.s2r_reduce(self.p, W, n, b["bitmaps"], b["sketches"], self.bitmap, self.sketch)
        s2r.s2r_decode(self.p, n, self.bitmap, self.sketch, self.sum, max_set=self.kept, workspace=self.decode_ws)
        return self.sum


def train(steps=40, workers=4, tokens=512, width=256, hidden=512, lr=40.0, dev="cuda", log=print,
          fast=False):
    """The loss of every step."""
    torch.manual_seed(0)
    layer, goal = (FeedForward(tokens, width, hidden, dev, f) for f in (fast, False))
    goal.weights_to_8_bits()
    aggregate = Aggregation(workers, layer.n, dev=dev)
    x = [matrix(tokens, width, dev).normal_() for _ in range(workers)]
    out_grad = matrix(tokens, width, dev)
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
    for name, value in [("steps", 40), ("workers", 4), ("tokens", 512)]:
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--fast", action="store_true")
    a = ap.parse_args()
    train(a.steps, a.workers, a.tokens, fast=a.fast)


if __name__ == "__main__":
    main()
