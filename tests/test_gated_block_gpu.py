"""The feed-forward example with its products and gated unit in one kernel: forward, gradients, clipping and decoding together,
eager and from a captured graph."""
import pytest

from tests import opsref as ref
from tests.test_feed_forward_gpu import ff, reference, rel  # noqa: F401  (ff: a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def data(tokens, hidden, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16() for _ in range(4)]


def grads(block):
    return [block.dw1, block.dw2, block.dnorm]


@pytest.mark.parametrize("tokens,hidden,inner", [(256, 256, 512), (200, 544, 320), (1, 288, 1056)])
def test_forward_and_gradients(ff, tokens, hidden, inner):  # noqa: F811
    if tokens % 8:
        tokens_, tokens = tokens, 8                     # the products by the weights take rows of 16 bytes: a padded batch
    else:
        tokens_ = tokens
    x, r, dout, dh = data(tokens, hidden, 4)
    for t in (x, r, dout, dh):
        t[tokens_:] = 0
    block = ff.FeedForward(tokens, hidden, inner, seed=3, fused=True)
    out = block.forward(x, r)
    dx = block.backward(dout, dh)
    torch.cuda.synchronize()
    leaves = [t.double().requires_grad_() for t in (block.w1, block.w2, block.norm, x, r)]
    want = reference(*leaves)
    dw1, dw2, dnorm, dx_want, _ = torch.autograd.grad(want, leaves, dout.double())
    # An e4m3 operand is off by at most 2^-4 per element and about 2.7 % in the root mean square; each result
    # passes four such roundings (two operands of each product, or the checkpoint's), in quadrature 5.4 %, and at most twice
    # that where one of them enters more than once.
    for name, got, exact in (("out", out, want), ("dw1", block.dw1, dw1), ("dw2", block.dw2, dw2), ("dnorm", block.dnorm, dnorm),
                             ("dx", dx, dx_want + dh.double())):
        assert rel(got, exact.detach()) < 0.11, name
    assert not out[tokens_:].any() and not dx[tokens_:].any()
    block.close()


def test_the_fused_block_agrees_with_the_separate_operators(ff):  # noqa: F811
    """Both from the same operands: they differ by the roundings of z and da to bf16, which the fused form has not."""
    x, r, dout, dh = data(512, 544, 5)
    one, two = (ff.FeedForward(512, 544, 800, seed=6, fused=f) for f in (True, False))
    got, want = one.forward(x, r), two.forward(x, r)
    dg, dw = one.backward(dout, dh), two.backward(dout, dh)
    torch.cuda.synchronize()
    assert torch.equal(one.y, two.y) and torch.equal(one.h, two.h)
    # z off by 2^-9 in the root mean square moves about one e4m3 rounding in 20 (2^-9 of a step of 2^-3 to 2^-4) by a step of
    # 2^-4 at most: 2^-4 / sqrt(20) = 1.4 % of the e4m3 values in the root mean square, of a and of the checkpoint alike, and two
    # such factors meet in a gradient; twice that as the bound
    assert rel(got, want) < 0.03 and rel(dg, dw) < 0.06
    for a, b in zip(grads(one), grads(two)):
        assert rel(a, b) < 0.06
    one.close()
    two.close()


def test_a_captured_step_replays_on_new_inputs(ff):  # noqa: F811
    """Forward, backward and clipping in one graph: each replay gives the eager call's bits for the inputs of that moment."""
    tokens, hidden, inner, limit = 256, 288, 544, 3.0
    block = ff.FeedForward(tokens, hidden, inner, seed=7, fused=True)
    static = data(tokens, hidden, 8)

    def step():
        out = block.forward(static[0], static[1])
        dx = block.backward(static[2], static[3])
        block.clip(limit)
        return out, dx

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (block.out, block.dx, block.total, block.ck, *grads(block))]

    step()                                             # once before the capture: kernels loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (9, 10):
        for t, n in zip(static, data(tokens, hidden, seed)):
            t.copy_(n)
        graph.replay()
        replayed = results()
        step()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(replayed, results()))
    assert block.up.last_status() == 0 and block.d_down.last_status() == 0
    block.close()


@pytest.mark.parametrize("limit", [0.5, 1e6])
def test_clipping_the_step(ff, limit):  # noqa: F811
    block = ff.FeedForward(200, 288, 544, seed=11, fused=True)
    x, r, dout, dh = data(200, 288, 12)
    block.forward(x, r)
    block.backward(dout, dh)
    torch.cuda.synchronize()
    before = [t.double() for t in grads(block)]
    weights = [t.double() for t in (block.w1, block.w2, block.norm)]
    norm = float(torch.cat([t.flatten() for t in before]).norm())
    block.step(0.25, limit)
    torch.cuda.synchronize()
    # the norm's own error is a few fp32 roundings, and the factor, the product and the update add one each
    assert abs(float(block.total) - norm) <= 8 * ref.U * norm
    factor = min(1.0, limit / norm)
    assert (factor == 1.0) == (limit == 1e6)
    for g, was, w, now in zip(grads(block), before, weights, (block.w1, block.w2, block.norm)):
        want = was * factor
        assert ((g.double() - want).abs() <= 12 * ref.U * want.abs() + 2.0 ** -149).all()
        assert ((now.double() - (w - 0.25 * want)).abs() <= 16 * ref.U * (w.abs() + want.abs())).all()
    block.close()


@pytest.mark.parametrize("m", [1, 2, 3, 8, 9, 16])
def test_decoding_on_the_blocks_own_weights(ff, m):  # noqa: F811
    block = ff.FeedForward(16, 544, 1056, seed=13, fused=True)
    x, r, _, _ = data(m, 544, 14)
    decoder = ff.Decoder(block)
    out, h = decoder(x, r)
    torch.cuda.synchronize()
    w1 = block.w1_q.view(torch.float8_e4m3fn).double() * torch.exp2(block.sf1.double() - 127).repeat_interleave(32, 1)
    codes = torch.stack([decoder.w2 & 15, decoder.w2 >> 4], 2).flatten(1).long()
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    w2 = torch.cat([table, -table])[codes] * decoder.sf2.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    want = reference(w1, w2, block.norm.double(), (h.double()), torch.zeros_like(h, dtype=torch.float64))
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    # y, a and out are each rounded to bf16, by at most 2^-8; y enters g and u, and silu's slope is at most 1.1: 4.1 halves of
    # a step as norms (the products of random weights keep a relative error's size)
    assert rel(out, want) < 4.1 * 2.0 ** -8
    block.close()


def test_two_blocks_on_two_streams(ff):  # noqa: F811
    """Steps and decoded tokens of two blocks at once, nothing waited for in between: the bits of each block alone."""
    def make(k):
        block = ff.FeedForward(200 + 56 * k, 288, 544, seed=20 + k, fused=True)
        return block, data(200 + 56 * k, 288, 30 + k), ff.Decoder(block)

    def run(block, t, decoder, n):
        kept = []
        for i in range(n):
            block.forward(t[0], t[1])
            block.backward(t[2], t[3])
            block.clip(2.0 + i)
            few, _ = decoder(t[0][:3 + i], t[1][:3 + i])
            kept += [block.out.clone(), block.dx.clone(), block.total.clone(), few, *(g.clone() for g in grads(block))]
        return kept

    made = [make(k) for k in range(2)]
    alone = [run(*m, 6) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                both[k] = run(*made[k], 6)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    for block, _, _ in made:
        assert block.up.last_status() == 0 and block.d_down.last_status() == 0
        block.close()


def test_two_graphs_of_one_block(ff):  # noqa: F811
    """Two graphs of the same plans and buffers, replayed one behind the other in either order, and eager calls between them."""
    block = ff.FeedForward(200, 544, 320, seed=40, fused=True)
    inputs = [data(200, 544, 41 + k) for k in range(2)]

    def run(t):
        block.forward(t[0], t[1])
        block.backward(t[2], t[3])
        block.clip(1.0)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (block.out, block.dx, block.total, *grads(block))]

    eager = []
    for t in inputs:
        run(t)
        eager.append(results())
    graphs = []
    for t in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(t)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0)):
        for k in order:
            graphs[k].replay()
            got = results()
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, eager[k]))
        run(inputs[order[0]])
        graphs[order[1]].replay()
        got = results()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, eager[order[1]]))
    block.close()
