"""Train a small two-layer network whose products run in 4 bits, with the
gradients clipped to a largest global norm, then serve it token by token from
weights kept in 4 bits.

  training   Fp4Linear forward and backward of both layers (x, W and dY
             quantised with their transposed copies, y, dX and dW in 4 bits),
             clip_grad_norm over both weight gradients into fp32, and a plain
             SGD step on fp32 master weights
  serving    each weight quantised once (Fp4Tensor), then fp4_linear for
             every token: one launch quantises it and multiplies

Run on a GB300:  python examples/fp4_train_and_serve.py [--fmt nv|mx]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantised_gemm_gb300 as q  # noqa: E402


class Network:
    """y = relu(x W1^T) W2^T with fp32 master weights and bf16 copies."""

    def __init__(self, tokens: int, d_in: int, d_hidden: int, d_out: int, fmt: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.fmt = fmt
        self.sizes = ((d_in, d_hidden), (d_hidden, d_out))
        self.master = [torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
                       for k, n in self.sizes]
        self.weights = [w.to(torch.bfloat16) for w in self.master]
        self.layers = [q.Fp4Linear(tokens, k, n, fmt=fmt) for k, n in self.sizes]
        self.grads = [torch.empty_like(w) for w in self.master]
        self.norm = torch.empty(1, device="cuda")
        self.ws = q.Workspace()

    def step(self, x: torch.Tensor, target: torch.Tensor, lr: float, max_norm: float):
        """One training step; returns the loss (a device tensor)."""
        l1, l2 = self.layers
        h = l1.forward(x, self.weights[0]).relu()
        y = l2.forward(h, self.weights[1])
        diff = y.float() - target
        dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        dh, dw2 = l2.backward(dy)
        _, dw1 = l1.backward(dh * (h > 0), need_dx=False)
        q.clip_grad_norm([dw1, dw2], max_norm, self.norm, self.ws, outs=self.grads)
        for master, weight, grad in zip(self.master, self.weights, self.grads):
            master.add_(grad, alpha=-lr)
            weight.copy_(master)
        return diff.square().mean()


class Server:
    """The trained weights in 4 bits, and the buffers of a batch of tokens."""

    def __init__(self, net: Network, batch: int):
        self.ws = q.Workspace()
        self.layers = []
        for (k, n), w in zip(net.sizes, net.weights):
            w4 = q.Fp4Tensor(n, k, net.fmt)
            q.fp4_quantise(w, w4, None, self.ws)
            self.layers.append((q.Fp4Tensor(batch, k, net.fmt), w4,
                                torch.empty((batch, n), dtype=torch.bfloat16, device="cuda")))

    def __call__(self, tokens: torch.Tensor) -> torch.Tensor:
        (x1, w1, h), (x2, w2, y) = self.layers
        q.fp4_linear(tokens, x1, w1, h, self.ws)
        return q.fp4_linear(h.relu_(), x2, w2, y, self.ws)


def main(fmt: int = q.NVFP4, tokens: int = 512, d_in: int = 256, d_hidden: int = 1024,
         d_out: int = 192, steps: int = 100, lr: float = 2.0, max_norm: float = 0.5, say=print):
    """Returns (first loss, last loss, relative difference of serving and training outputs)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, d_in), generator=g, device="cuda").to(torch.bfloat16)
    teacher = torch.randn((d_out, d_in), generator=g, device="cuda") * d_in ** -0.5
    target = (x.float() @ teacher.t()).relu()
    net = Network(tokens, d_in, d_hidden, d_out, fmt)
    losses = []
    for i in range(steps):
        losses.append(net.step(x, target, lr, max_norm))
        if i % 10 == 0 or i == steps - 1:
            say("step %3d  loss %.4f  gradient norm %.4f" % (i, float(losses[-1]), float(net.norm)))
    for layer in net.layers:
        q.check(layer.ws)
    l1, l2 = net.layers
    want = l2.forward(l1.forward(x, net.weights[0]).relu(), net.weights[1]).float()
    serve = Server(net, 1)
    got = torch.cat([serve(x[i:i + 1]).clone() for i in range(16)]).float()
    far = float((got - want[:16]).norm() / want[:16].norm())
    say("serving one token at a time is %.3f (relative) from the training forward" % far)
    return float(losses[0]), float(losses[-1]), far


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fmt", choices=("nv", "mx"), default="nv")
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    main(q.NVFP4 if a.fmt == "nv" else q.MXFP4, steps=a.steps)
