"""The max-plus classifier of examples/: its gradients against torch autograd
in 64 bits on the CPU, and that training lowers the loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("maxplus_classifier",
                                                  os.path.join(ROOT, "examples", "maxplus_classifier.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens", [7, 300])
def test_gradients(example, tokens):
    """Float32 products over 40 terms and sums over up to 300 tokens: relative
    errors stay below 2^-24 times a few hundred roundings, 2e-5 of a gradient
    tensor's norm with room for the layer norm's amplification (rstd near 1)."""
    teacher = example.MaxPlusClassifier(24, 40, 60, seed=3)
    model = example.MaxPlusClassifier(24, 40, 60, seed=4)
    g = torch.Generator(device="cuda:0").manual_seed(5)
    x, target = example.batch(teacher, tokens, 24, g)
    loss, kept = model.forward(x, target)
    weight = torch.rand(tokens, generator=g, device="cuda:0")
    grads = model.gradients(target, kept, weight)

    params = [p.detach().cpu().double().requires_grad_() for p in model.params]
    w1, gamma, beta, w2 = params
    t = target.cpu()
    h = (x.cpu().double()[:, :, None] + w1[None]).max(1).values
    z = torch.nn.functional.layer_norm(h, (40,), gamma, beta, 1e-5)
    per = torch.nn.functional.cross_entropy(z @ w2.t(), t, ignore_index=-100, reduction="none")
    (per * weight.cpu().double()).sum().backward()
    assert torch.allclose(loss.cpu().double(), per.detach(), rtol=1e-5, atol=1e-5)
    for got, want in zip(grads, params):
        err = (got.cpu().double() - want.grad).norm() / want.grad.norm()
        assert err < 2e-5, float(err)


@pytest.mark.parametrize("state8", [False, True])
def test_training_lowers_the_loss(example, state8):
    losses = example.train(steps=60, tokens=1024, features=32, hidden=64, labels=20, state8=state8)
    assert all(v == v for v in losses)
    assert sum(losses[-10:]) < 0.75 * sum(losses[:10]), losses
