"""The example's blocks in 8 bits: their autograd functions refuse a second derivative (without a
GPU), give the gradients of what they compute, and train and serve."""
import pytest
import torch

from gated_delta_rule_52_gb300 import block, fp8, kda, rms_norm

BF, F = torch.bfloat16, torch.float32
N = lambda *s: torch.randn(s, requires_grad=True)  # noqa: E731


def test_second_derivative_is_refused(monkeypatch):
    monkeypatch.setattr(rms_norm, "rms_norm_fwd", lambda *a, **k: None)
    monkeypatch.setattr(rms_norm, "rms_norm_bwd", lambda dout, x, w, r: {"dx": torch.ones_like(x), "dweight": torch.ones_like(w)})
    monkeypatch.setattr(fp8, "quantize", lambda *a, **k: None)
    monkeypatch.setattr(fp8, "matmul", lambda a, s, b, t, out, add=None: out.fill_(1))
    for f, inputs in ((block.RmsNorm, (N(3, 8), N(8))), (block.Linear, (N(3, 8), N(8, 5), None)), (block.Linear, (N(3, 8), N(8, 5), N(3, 5)))):
        out = f.apply(*inputs)
        leaves = [t for t in inputs if t is not None]
        first = torch.autograd.grad(out.sum(), leaves, create_graph=True, retain_graph=True)
        for got, t in zip(first, leaves):
            assert torch.equal(got, torch.ones_like(t))
        with pytest.raises(RuntimeError, match="first derivative"):
            torch.autograd.grad((first[0].square() + leaves[0].square()).sum(), leaves[0])


def test_rows_that_are_not_contiguous_are_laid_out(monkeypatch):
    """What autograd hands over (an expanded gradient, a transposed tensor) is quantised from contiguous rows."""
    seen = []
    monkeypatch.setattr(fp8, "quantize", lambda x, *a, **k: seen.append(x))
    for t in (torch.ones(()).expand(4, 8), torch.arange(32.).view(8, 4).T, torch.arange(12.)[:, None].expand(2, 12, 8), torch.arange(64.).view(4, 16)[:, ::2]):
        block.eight_bits(t)
        assert seen[-1].stride(-1) == 1 and torch.equal(seen[-1], t.reshape(-1, t.shape[-1]))
    t = torch.arange(64.).view(4, 16)
    block.eight_bits(t[:, 3:11])             # rows of a wider tensor are read where they are
    assert seen[-1].data_ptr() == t[:, 3:].data_ptr()


def _whole(gen, *shape):
    """Whole numbers that 8 bits hold exactly, whatever their neighbours are: 0 to 3 in magnitude."""
    return torch.randint(-3, 4, shape, generator=gen).to(BF).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,N_,add", [((2, 70), 129, True), ((1, 1), 64, False), ((3, 200), 300, True)])
def test_linear_and_its_gradients(shape, N_, add):
    """On whole numbers every product and sum is exact (|sum| < 2^24, out < 2^8 or checked in its own
    rounding): outputs, gradients by the formula, and differences of the outputs."""
    gen = torch.Generator().manual_seed(N_)
    K = 136
    x, w, dy = _whole(gen, *shape, K).requires_grad_(), _whole(gen, K, N_).requires_grad_(), _whole(gen, *shape, N_)
    a = _whole(gen, *shape, N_).requires_grad_() if add else None
    out = block.Linear.apply(x, w, a)
    exact = x.double() @ w.double() + (0 if a is None else a.double())
    assert torch.equal(out, exact.to(BF))
    got = torch.autograd.grad(out, [x, w] + ([a] if add else []), dy)
    flat = lambda t: t.detach().double().flatten(0, -2)  # noqa: E731
    assert torch.equal(got[0], (dy.double() @ w.double().T).to(BF))
    assert torch.equal(got[1], (flat(x).T @ flat(dy)).to(F).to(BF))
    if add:
        assert torch.equal(got[2], dy)
    # differences of the loss sum(out * dy) along a step of one element, 32-bit outputs
    step = torch.zeros_like(x)
    step[..., 5] = 1

    def loss(t):
        q, s, _, _ = block.eight_bits(t.detach(), turned=False)
        _, _, wt, wts = block.eight_bits(w.detach(), tile=True, rows=False)
        y = torch.empty(t[..., 0].numel(), N_, device="cuda")
        fp8.matmul(q, s, wt, wts, y)
        return float((y.double() * flat(dy)).sum())

    clamped = torch.where(x.detach() == 3, x.detach() - 1, x.detach())     # so that x + 1 is still among them
    assert loss(clamped + step) - loss(clamped) == float((flat(dy) @ w.double().T)[:, 5].sum())
    assert kda.get_device_status() == kda.KDA_OK


@pytest.mark.gpu
def test_block_in_eight_bits_trains_and_serves():
    gen = torch.Generator().manual_seed(0)
    blocks = [block.Block(kind, 128, gen, eight=True) for kind in ("glr", "kda")]
    losses = block.train(blocks, 3, 2, 200, gen)
    assert all(l == l and l < float("inf") for l in losses)
    u = torch.randn(2, 90, 128, generator=gen).to("cuda", BF)
    before = u.clone()
    whole, stepped = block.serve(blocks, u, 90), block.serve(blocks, u, 70)
    assert torch.equal(u, before)
    assert kda.get_device_status() == kda.KDA_OK
    # Sums in another order round to another bf16 now and then, and the rounding to 8 bits behind
    # makes a difference of up to 2^-8 a whole step, 2^-3 or 2^-4 of the value, in about one element
    # of 16: 2^-2 * 0.09 = 0.02 in the mean square, at each of the stack's 4 quantisations 0.045.
    assert float((whole.float() - stepped.float()).norm()) <= 2.0 ** -4 * float(whole.float().norm())
    h = u
    for b in blocks:
        h = b.train(h)
    assert float((whole.float() - h.float()).norm()) <= 2.0 ** -4 * float(whole.float().norm())


@pytest.mark.gpu
def test_gradient_of_a_sum():
    """An expanded gradient, and an addend that is one: exact on whole numbers."""
    gen = torch.Generator().manual_seed(5)
    x, w = _whole(gen, 6, 40).requires_grad_(), _whole(gen, 40, 24).requires_grad_()
    a = torch.ones((), dtype=BF, device="cuda").expand(6, 24)
    out = block.Linear.apply(x, w, a)
    assert torch.equal(out, (x.double() @ w.double() + 1).to(BF))
    dx, dw = torch.autograd.grad(out.sum(), [x, w])
    assert torch.equal(dx, w.detach().double().sum(1).expand(6, 40).to(BF)) and torch.equal(dw, x.detach().double().sum(0)[:, None].expand(40, 24).to(BF))


@pytest.mark.gpu
def test_serving_reads_the_weights_as_they_are_at_its_start():
    gen = torch.Generator().manual_seed(7)
    b = block.Block("glr", 128, gen, eight=True)
    u = torch.randn(2, 9, 128, generator=gen).to("cuda", BF)
    first = block.serve([b], u, 5)
    with torch.no_grad():
        b.p["w_out"].zero_()
    assert torch.equal(block.serve([b], u, 5), u)        # the block adds nothing
    assert not torch.equal(first, u)
