"""examples/feed_forward.py: the operators together, as a program uses them.
One training step's outputs against plain float64 arithmetic, the loss going
down over a few steps, and a captured decoding step against the eager one.

The chain rounds h, dh and the gradients to bf16 (half-step 2^-8 each), and
the backward pass starts from a dy rounded once: 2-norms within 4 such steps
cover them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _near(got, want):
    return float((got.double() - want).norm() / want.norm()) <= 4 * 2.0 ** -8


@pytest.mark.parametrize("M,K,F", [(300, 256, 520), (1, 128, 72)])
def test_step_against_float64(ex, M, K, F):
    b = ex.Block(K, F, seed=3)
    x = torch.randn((M, K), device="cuda").bfloat16()
    dy = torch.randn((M, K), device="cuda").bfloat16()
    y, h, saved = b.forward(x, save=True)
    dx = b.backward(dy, x, h, saved)
    X, Wgu, Wd, D = (t.double().requires_grad_() for t in (x, b.w_gu, b.w_down, dy))
    gu = X @ Wgu.t()
    H = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
    Y = X + H @ Wd.t()
    gx, ggu, gd = torch.autograd.grad(Y, (X, Wgu, Wd), D)
    for got, want in ((y, Y.detach()), (dx, gx), (b.grads[0], ggu), (b.grads[1], gd)):
        assert _near(got, want)


def test_training_and_decoding(ex):
    losses = ex.main(["--tokens", "256", "--hidden", "128", "--width", "352", "--steps", "8"])
    assert losses[-1] < losses[0]
    b = ex.Block(256, 520)
    for rows in (1, 7, 40):
        x = torch.randn((rows, 256), device="cuda").bfloat16()
        graph, y = ex.decode_graph(b, x)
        for _ in range(3):
            x.copy_(torch.randn((rows, 256), device="cuda").bfloat16())
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, b.forward(x))
        assert graph.handle.status() == 0
