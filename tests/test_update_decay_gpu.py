"""The weights' update where little is taken from a parameter at a time: weight decay at the rates of fine-tuning,
updates of tiny moments, rates that vanish."""
import math

import numpy as np
import pytest

from oracle import optim_oracle as O
from train_helpers import EPS32, TORCH, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _optim(*a, **kw):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    return DominoAdamW(*a, **kw)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("fp32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("rate", [1e-6, 3e-6, 1e-5])
def test_decay_of_small_rates(bits, dtype, master, rate):
    """A thousand steps with and without decay on equal gradients: the means differ by (1 - rate decay)^1000.  The
    steps themselves, of several fp32 places, carry what is below one."""
    n, steps, decay = 1 << 24, 1000, 0.01
    torch.manual_seed(0)
    start = torch.rand(n, device="cuda").add_(1.0).mul_(torch.randn(n, device="cuda").sign()).to(TORCH[dtype])
    p = [start.clone(), start.clone()]
    opts = [_optim([t], lr=rate, weight_decay=d, state_bits=bits, master=master) for t, d in zip(p, (decay, 0.0))]
    g = torch.empty_like(start)
    for _ in range(steps):
        g.normal_()
        for opt in opts:
            opt.step(grads=[g])
    end = [opt.state["master"] if master else t for opt, t in zip(opts, p)]
    got = ((end[0].double() - end[1].double()) * start.double().sign()).mean().item()
    want = start.double().abs().mean().item() * math.expm1(steps * math.log1p(-rate * decay))
    # the first steps are of one size everywhere, so that their roundings (half of 2^-23 below 2) may share a sign: five
    # of them in each run.  Later ones are spread over several places: deviations of 2^-23 / sqrt(12).
    tol = 5 * 2.0 ** -23 + 6 * 2.0 ** -23 * math.sqrt(2 * steps / 12 / n) + 1e-5 * abs(want)
    if dtype == "bf16" and not master:
        # each step goes to one of two neighbours, 2^-7 apart, with a variance of at most 2^-7 times its size, 1.2 rate;
        # six deviations of the mean's difference
        tol += 6 * math.sqrt(2 * steps * 2.0 ** -7 * 1.2 * rate / n)
    assert abs(got - want) <= tol, (got, want, tol)


@pytest.mark.parametrize("eps", [1e-16, 1e-8, 1.0])
@pytest.mark.parametrize("lr", [1e3, 1e-3, 1e-12, 1e-25])
@pytest.mark.parametrize("beta1", [0.0, 0.9])
def test_values_of_updates_of_any_moments(eps, lr, beta1):
    """Gradients from 1e-22 to 1e15: what is taken from a parameter that is 0, relative to itself."""
    g = (10.0 ** torch.arange(-22, 16, device="cuda", dtype=torch.float64)).float()
    p = torch.zeros_like(g)
    opt = _optim([p], lr=lr, eps=eps, betas=(beta1, 0.999), weight_decay=0.0)
    for t in range(1, 4):
        p.zero_()
        m0, v0 = (wide(a) for a in opt.moments(0))
        opt.step(grads=[g])
        m, v = (a.astype(np.float64) for a in O.moments32(m0, v0, wide(g), 1.0, beta1, 0.999))
        v = np.where(v < 2.0 ** -126, 0.0, v)  # whose root counts as 0
        want = -lr / (1 - beta1 ** t) * m / (np.sqrt(v) / math.sqrt(1 - 0.999 ** t) + eps)
        # the two bias corrections (a logarithm, a product and expm1f each: 4), the root, the quotient, the sum's and
        # the products' roundings; results below 2^-126 may be 0 (factors of 2^-126 times m's are)
        tol = 40 * EPS32 * np.abs(want) + 2.0 ** -126 * (1 + np.abs(m))
        assert (np.abs(wide(p) - want) <= tol).all(), (t, np.argwhere(np.abs(wide(p) - want) > tol)[:4])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("factor", [0.0, 1e-45, 1e-38, 1e-30])
def test_a_rate_that_vanishes(bits, factor):
    """Nothing is left of an update and of the decay; the moments go on."""
    p = torch.randn(1000, device="cuda")
    opt = _optim([p], lr=1e-3, weight_decay=0.1, state_bits=bits)
    start, g = p.clone(), torch.randn(1000, device="cuda") * torch.logspace(-18, 15, 1000, device="cuda")
    g[::7] = 0.0
    f = torch.tensor(factor, device="cuda", dtype=torch.float32)
    for _ in range(3):
        opt.step(grads=[g], lr_factor=f)
    assert torch.equal(p, start) and opt.steps() == 3
    assert (opt.moments(0)[1][g.abs() > 1e-10] > 0).all() or bits == 8
