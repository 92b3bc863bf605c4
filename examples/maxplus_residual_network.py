"""Train a deep residual network of max-plus layers, its activations kept in 8 bits.

    h = x W_in^T,  y = pre norm of h
    for each block:
        u = y (x) W            max-plus product, argmax kept
        v = layer norm of u    u is defined up to the constants added to W
        h = h + gate v,  y = rms norm of h
    loss = cross entropy of y over `labels` classes (W_out), the logits never kept

Between two blocks one call does the norm, gate, sum and norm; what it leaves
for the backward are u and h in 8 bits and the rows' statistics.  A max-plus
product needs only its argmax, the linear layer its input, in 8 bits too.  torch
holds the memory, draws the random numbers and multiplies x by W_in.

Usage: python examples/maxplus_residual_network.py [--steps 100] [--full]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from tropical_semiring_tensor_amd import binding as tb  # noqa: E402


class MaxPlusResidualNetwork:
    """hold: activations for the backward in 8 bits, else as they are."""

    def __init__(self, features, hidden, labels, blocks, seed=0, hold=True, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        def ones():
            return torch.ones(hidden, device=device)

        def zeros():
            return torch.zeros(hidden, device=device)

        self.hold, self.blocks = hold, blocks
        self.w_in = randn(hidden, features) / features ** 0.5
        self.first_gamma = ones()
        self.w = [randn(hidden, hidden) for _ in range(blocks)]
        self.post_gamma = [ones() for _ in range(blocks)]
        self.post_beta = [zeros() for _ in range(blocks)]
        self.gate = [0.5 * ones() for _ in range(blocks)]
        self.pre_gamma = [ones() for _ in range(blocks)]
        self.w_out = randn(labels, hidden) / hidden ** 0.5
        self.params = [self.w_in, self.first_gamma, *self.w, *self.post_gamma, *self.post_beta, *self.gate,
                       *self.pre_gamma, self.w_out]
        count = [-(-p.numel() // tb.ADAMW_BLOCK) for p in self.params]
        self.m = [torch.zeros(p.shape, dtype=torch.int8, device=device) for p in self.params]
        self.v = [torch.zeros(p.shape, dtype=torch.uint8, device=device) for p in self.params]
        self.m_scale = [torch.zeros(n, device=device) for n in count]
        self.v_scale = [torch.zeros(n, device=device) for n in count]
        self.step_count = 0

    def _between(self, i):
        """Weights of the call after block i."""
        return dict(gate=self.gate[i], post="layer", post_gamma=self.post_gamma[i], post_beta=self.post_beta[i],
                    pre="rms", pre_gamma=self.pre_gamma[i])

    def forward(self, x, target):
        """(per-token loss, what the backward needs)."""
        tokens, hidden = x.shape[0], self.w_in.shape[0]
        h = x @ self.w_in.t()
        # (without a gate or a residual the first norm's input is the call's u)
        first = tb.tropical_residual_norm_forward(h, pre="rms", pre_gamma=self.first_gamma, h=None, hold_u=self.hold)
        first_kept = (first.u8 if self.hold else h, first.pre_rstd)
        blocks, y = [], first.y
        for i in range(self.blocks):
            u = torch.empty(1, tokens, hidden, device=x.device)
            winner = torch.empty(1, tokens, hidden, dtype=torch.int32, device=x.device)
            tb.tropical_gemm_strided_batched("max_plus", y, self.w[i], u, winner)
            f = tb.tropical_residual_norm_forward(u[0], h, hold_u=self.hold, hold_h=self.hold, **self._between(i))
            statistics = dict(post_mean=f.post_mean, post_rstd=f.post_rstd, pre_rstd=f.pre_rstd)
            blocks.append((winner, f.u8 if self.hold else u[0], f.h8 if self.hold else f.h, statistics))
            h, y = f.h, f.y
        loss, lse = tb.tropical_linear_cross_entropy_forward(y, self.w_out, target)
        return loss, (tb.tropical_act8_pack(x), first_kept, blocks, y, lse)

    def gradients(self, target, kept, grad_loss):
        """Gradients of sum(grad_loss * loss) for the parameters, in order."""
        x8, (first_h, first_rstd), blocks, y, lse = kept
        dy, dw_out = tb.tropical_linear_cross_entropy_backward(y, self.w_out, target, lse, grad_loss)
        dh, grads = None, []
        for i in reversed(range(self.blocks)):
            winner, u, h, statistics = blocks[i]
            g = tb.tropical_residual_norm_backward(dy, dh, u, h, **statistics, **self._between(i))
            da, dw = tb.tropical_gemm_backward("max_plus", winner, g.u.unsqueeze(0), k=self.w[i].shape[0])
            dy, dh = da[0], g.r
            grads.append((dw[0], g.post_gamma, g.post_beta, g.gate, g.pre_gamma))
        g = tb.tropical_residual_norm_backward(dy, dh, None, first_h, pre="rms", pre_rstd=first_rstd,
                                               pre_gamma=self.first_gamma, dr=None)
        dw_in = tb.tropical_act8_linear_grad_w(g.u, x8)
        return [dw_in, g.pre_gamma, *(t for column in zip(*reversed(grads)) for t in column), dw_out]

    def step(self, x, target, lr=1e-2, weight_decay=1e-4):
        """One training step on a batch; returns the mean loss (a device scalar)."""
        loss, kept = self.forward(x, target)
        counted = (target >= 0).sum().clamp(min=1)
        grads = self.gradients(target, kept, 1.0 / counted.float())
        self.step_count += 1
        tb.tropical_adamw8_step(self.params, grads, self.m, self.m_scale, self.v, self.v_scale, lr=lr, beta1=0.9,
                                beta2=0.99, weight_decay=weight_decay, step=self.step_count)
        return loss.sum() / counted


def train(steps=100, tokens=1024, features=64, hidden=128, labels=50, blocks=3, hold=True, seed=1):
    """Losses of `steps` training steps (a list of floats), on random inputs
    whose label is the place of their largest element."""
    model = MaxPlusResidualNetwork(features, hidden, labels, blocks, seed=seed, hold=hold)
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, features, generator=g, device="cuda:0")
        losses.append(model.step(x, x[:, :labels].argmax(1)))
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--full", action="store_true", help="keep the activations as they are")
    args = ap.parse_args()
    out = train(args.steps, hold=not args.full)
    for i in range(0, len(out), max(1, len(out) // 10)):
        print(f"step {i}: loss {out[i]:.4f}")
    print(f"last: loss {out[-1]:.4f}")
