"""Train linear layers in 8 bits: quantise, the three products, the update.

``scaled_linear(x, weight)`` is ``x @ weight.T`` with both operands in e4m3 and
a scale per 128 elements of K, and its gradients from the same two operators:

    forward             Y  = X W^T      X by rows,   W by 128 x 128 blocks
    input gradient      dX = dY W       dY by rows,  W^T from the same pass
    weight gradient     dW = dY^T X     dY^T and X^T along the tokens, fp32 out

Each tensor is read once by ``quantize``, which writes both directions (the columns
only where a gradient reads them).
``OrthogonalMomentum`` updates the weights with ``orthogonalize`` of their
momentum.  ``python -m dense_gemm_blackwell_03_gb300.linear_training`` fits a
small two-layer network to a teacher and prints the loss.
"""
from __future__ import annotations

import argparse

import torch

from . import binding


class _ScaledLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, of_x, of_weight):
        xq, xs, *xt = binding.quantize(x, transposed=of_weight)
        wq, ws, *wt = binding.quantize(weight, blocks="square", transposed=of_x)
        ctx.save_for_backward(*xt, *wt)
        ctx.weight_dtype = weight.dtype
        return binding.gemm_scaled(xq, xs, wq, ws, out_dtype=x.dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable  # computed outside the graph: a second derivative raises
    def backward(ctx, dy):
        of_x, of_weight = ctx.needs_input_grad[:2]
        # quantize reads rows on 16-byte boundaries; autograd may hand in any layout
        dyq, dys, *dyt = binding.quantize(_aligned_rows(dy), transposed=of_weight)
        dx = dw = None
        saved = list(ctx.saved_tensors)
        if of_weight:
            xtq, xts = saved[:2]
            dw = binding.gemm_scaled(*dyt, xtq, xts, out_dtype=torch.float32).to(ctx.weight_dtype)
        if of_x:
            wtq, wts = saved[-2:]
            dx = binding.gemm_scaled(dyq, dys, wtq, wts, out_dtype=dy.dtype)
        return dx, dw, None, None


def _aligned_rows(t):
    """t, or a copy of it, in rows as `quantize` reads them: apart from each other (the
    gradient of a sum over rows is one row expanded) and on 16-byte boundaries."""
    per = 16 // t.element_size()
    rows, cols = t.shape
    if t.stride(1) == 1 and t.stride(0) >= cols and t.stride(0) % per == 0 and t.data_ptr() % 16 == 0:
        return t
    wide = torch.empty((rows, -(-cols // per) * per), dtype=t.dtype, device=t.device)
    wide[:, :cols] = t
    return wide[:, :cols]


def scaled_linear(x, weight):
    """``x @ weight.T`` of CUDA matrices x (tokens x K) and weight (N x K), computed in 8 bits;
    differentiable in both, once."""
    grad = torch.is_grad_enabled()
    return _ScaledLinear.apply(_aligned_rows(x), _aligned_rows(weight), grad and x.requires_grad, grad and weight.requires_grad)


class OrthogonalMomentum:
    """Momentum whose update is its orthogonalised direction (Muon): per weight

        m = beta m + g;   w -= lr * sqrt(max(1, rows / cols)) * orthogonalize(g + beta m)
    """

    def __init__(self, weights, lr=0.02, beta=0.95, steps=5):
        self.weights = list(weights)
        self.lr, self.beta, self.steps = lr, beta, steps
        self.momentum = [torch.zeros_like(w, dtype=torch.float32) for w in self.weights]

    @torch.no_grad()
    def step(self):
        for w, m in zip(self.weights, self.momentum):
            if w.grad is None:  # not part of this step's loss
                continue
            g = w.grad.float()
            m.mul_(self.beta).add_(g)
            rows, cols = w.shape
            update = binding.orthogonalize(g + self.beta * m, steps=self.steps,
                                           scale=self.lr * max(1.0, rows / cols) ** 0.5)
            w.sub_(update.to(w.dtype))
            w.grad = None


def train(tokens=512, inner=256, hidden=640, outer=128, steps=60, seed=0, device="cuda:0"):
    """Fit hidden(relu) and output layers to a random teacher; returns the losses."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    teacher = draw(outer, inner) / inner ** 0.5
    w1 = (draw(hidden, inner) / inner ** 0.5).requires_grad_()
    w2 = (draw(outer, hidden) / hidden ** 0.5).requires_grad_()
    opt = OrthogonalMomentum([w1, w2])
    losses = []
    for _ in range(steps):
        x = draw(tokens, inner)
        y = scaled_linear(torch.relu(scaled_linear(x, w1)), w2)
        loss = (y - x @ teacher.t()).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    losses = train(steps=a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
