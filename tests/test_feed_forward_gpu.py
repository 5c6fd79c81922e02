"""The feed-forward example: its operators and products together, forward, backward, a few steps of training and
decoding with 4-bit weights."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(w1, w2, norm, x, r):
    h = x + r
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * norm
    g, u = (y @ w1.t()).chunk(2, 1)
    return torch.nn.functional.silu(g) * u @ w2.t()


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("tokens,hidden,inner", [(256, 256, 512), (200, 544, 320)])
def test_forward_and_gradients(ff, tokens, hidden, inner):
    block = ff.FeedForward(tokens, hidden, inner, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, r, dout, dh = (torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16() for _ in range(4))
    out = block.forward(x, r)
    dx = block.backward(dout, dh)
    torch.cuda.synchronize()
    leaves = [t.double().requires_grad_() for t in (block.w1, block.w2, block.norm, x, r)]
    want = reference(*leaves)
    dw1, dw2, dnorm, dx_want, dr_want = torch.autograd.grad(want, leaves, dout.double())
    # An e4m3 operand is off by at most 2^-4 per element and about 2.7 % in the root mean square; each result
    # passes four such roundings (two operands of each product, or the checkpoint's), in quadrature 5.4 %, and at most twice
    # that where one of them enters more than once.
    for name, got, ref in (("out", out, want), ("dw1", block.dw1, dw1), ("dw2", block.dw2, dw2), ("dnorm", block.dnorm, dnorm),
                           ("dx", dx, dx_want + dh.double())):
        assert rel(got, ref.detach()) < 0.11, name
    assert torch.equal(dx_want, dr_want)
    block.close()


def test_training_reduces_the_loss_and_decoding_agrees(ff):
    block, losses, x, r = ff.train(tokens=256, hidden=256, inner=512, steps=12, report=lambda _: None)
    assert losses[-1] < 0.7 * losses[0]
    out = block.forward(x, r)
    for m in (1, 3, 16):
        few, h = ff.Decoder(block)(x[:m].contiguous(), r[:m].contiguous())
        assert torch.equal(h, block.h[:m])
        # weights in 4 bits: steps of a quarter to a half, about 10 % in the root mean square, in each of two products
        assert rel(few, out[:m]) < 0.25
    block.close()
