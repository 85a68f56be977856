"""The example token model: the operators together, as a training loop uses them."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_training_lowers_the_losses(gpu_lib):
    from examples import token_model
    losses, margins, rewards = token_model.train(steps=30)
    assert abs(losses[0] - math.log(2)) < 1e-3           # every margin starts at zero
    assert losses[-1] < 0.5 * losses[0]
    assert min(margins) > 0
    assert sum(rewards[-5:]) / 5 > sum(rewards[:5]) / 5 + 0.2


def test_one_step_is_the_autograd_step(gpu_lib):
    """The weights after one preference step against FP64 autograd of the same model.  The
    step's own 16-bit rounding of activations and gradients, 2^-8 each over about eight
    roundings in a row, bounds the difference relative to the update."""
    from examples import token_model
    vocab, dim, experts, pairs, length, eta = 200, 64, 3, 4, 10, 0.25
    rows = 2 * pairs * length
    m = token_model.TokenModel(vocab, dim, experts, rows, pairs, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    targets[5] = -100
    seq = torch.arange(0, rows + 1, length, dtype=torch.int32, device="cuda")
    ref = torch.randn(2 * pairs, generator=g, device="cuda") - 55
    before = [t.double().clone().requires_grad_() for t in (m.table, m.w32, m.u32)]
    E, W, U = before
    h = E[tokens] * m.scale
    z = h + torch.einsum("tij,tj->ti", W[tokens % experts], h)
    lp = torch.log_softmax(z @ U[0].T, 1).gather(1, targets.clamp(min=0)[:, None])[:, 0]
    lp = torch.where(targets >= 0, lp, 0.0).view(2 * pairs, length).sum(1)
    margin = 0.1 * ((lp - ref)[0::2] - (lp - ref)[1::2])
    loss = torch.nn.functional.softplus(-margin).mean()
    grads = torch.autograd.grad(loss, before)
    got = m.preference_step(tokens, targets, seq, ref, eta)
    m.check()
    assert abs(float(got) - loss.item()) < 0.02 * loss.item()
    for new, old, grad in zip((m.table, m.w32, m.u32), before, grads):
        want = -eta * grad
        err = (new.double() - old.detach() - want).norm() / want.norm()
        assert err < 8 * 2.0 ** -8, float(err)
