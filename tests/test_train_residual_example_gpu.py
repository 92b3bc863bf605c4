"""The residual network of examples/: the 8-bit activations, the norms between
its blocks, the weight gradient, the max-plus products, the cross entropy and
the optimiser together.  Its gradients against torch autograd in 64 bits on the
CPU, with activations as they are; with activations in 8 bits, the same bits as
from their values."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("maxplus_residual_network",
                                                  os.path.join(ROOT, "examples", "maxplus_residual_network.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()


def problem(example, tokens, hold):
    model = example.MaxPlusResidualNetwork(24, 40, 30, blocks=3, seed=4, hold=hold)
    g = torch.Generator(device="cuda:0").manual_seed(5)
    # codes of one block step apart: packing x is exact, and so is W_in's gradient
    x = torch.randint(-127, 128, (tokens, 24), generator=g, device="cuda:0") / 64.0
    x[:, 0] = 127 / 64
    target = torch.randint(0, 30, (tokens,), generator=g, device="cuda:0")
    target[::7] = -100
    return model, x, target, torch.rand(tokens, generator=g, device="cuda:0")


@pytest.mark.parametrize("tokens", [7, 300])
def test_gradients(example, tokens):
    """Float32 sums of up to 300 terms through four norms (rstd below 4): each
    of about a dozen steps adds a few hundred roundings of 2^-24, relative, to
    a gradient tensor's norm: below 1e-4 with room for the norms'
    amplification.  Winners of the max-plus products are taken from the run
    (a tie within a rounding may go either way)."""
    model, x, target, weight = problem(example, tokens, hold=False)
    loss, kept = model.forward(x, target)
    grads = model.gradients(target, kept, weight)
    params = [p.detach().cpu().double().requires_grad_() for p in model.params]
    n = model.blocks
    w_in, first_gamma, rest, w_out = params[0], params[1], params[2:-1], params[-1]
    w, post_gamma, post_beta, gate, pre_gamma = (rest[i * n:(i + 1) * n] for i in range(5))

    def rms(h, gamma):
        return h / (h * h).mean(1, keepdim=True).add(1e-5).sqrt() * gamma

    h = x.cpu().double() @ w_in.t()
    y = rms(h, first_gamma)
    for i in range(n):
        winner = kept[2][i][0][0].cpu().long()
        u = y.gather(1, winner) + w[i].gather(0, winner)
        v = torch.nn.functional.layer_norm(u, (40,), post_gamma[i], post_beta[i], 1e-5)
        h = h + gate[i] * v
        y = rms(h, pre_gamma[i])
    per = torch.nn.functional.cross_entropy(y @ w_out.t(), target.cpu(), ignore_index=-100, reduction="none")
    (per * weight.cpu().double()).sum().backward()
    assert torch.allclose(loss.cpu().double(), per.detach(), rtol=1e-4, atol=1e-4)
    for k, (got, want) in enumerate(zip(grads, params)):
        err = (got.cpu().double() - want.grad).norm() / want.grad.norm()
        assert err < 1e-4, (k, float(err))


def test_held_activations(example):
    """From 8-bit activations: what their values, kept as they are, give."""
    import tropical_semiring_tensor_amd.binding as tb
    model, x, target, weight = problem(example, 200, hold=True)
    loss, kept = model.forward(x, target)
    held = model.gradients(target, kept, weight)
    x8, (first, rstd), blocks, y, lse = kept
    values = [(winner, tb.tropical_act8_unpack(u), tb.tropical_act8_unpack(h), st) for winner, u, h, st in blocks]
    plain = model.gradients(target, (x8, (tb.tropical_act8_unpack(first), rstd), values, y, lse), weight)
    assert all(torch.equal(a, b) for a, b in zip(held, plain))


@pytest.mark.parametrize("hold", [True, False])
def test_training_runs(example, hold):
    losses = example.train(steps=8, tokens=256, features=32, hidden=64, labels=20, blocks=2, hold=hold)
    assert len(losses) == 8 and all(v == v and v < 100 for v in losses)
