"""The gradients' norm where the order of its sums would show."""
import math

import numpy as np
import pytest

from train_helpers import EPS32, TORCH, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _norm(grads, most=1e9):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    opt = DominoAdamW([torch.zeros_like(t) for t in grads], state_bits=8)
    return opt.grad_norm(most, grads=grads)


def _check(grads):
    want = math.sqrt(math.fsum(float((wide(t) ** 2).sum()) for t in grads))
    norm, scale = _norm(grads, most=0.5)
    # two roundings of every square on its way, of which the sums' are twice as exact, half of them in the root, and the
    # result's
    assert abs(norm.item() - want) <= 2 * EPS32 * want, (norm.item() / want - 1) / EPS32
    assert abs(scale.item() - min(1.0, 0.5 / (want + 1e-6))) <= 3 * EPS32 * scale.item()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("period", [2, 8, 16, 256, 4096])
@pytest.mark.parametrize("place", [0, 1, 15])
def test_one_large_element_among_small_ones(dtype, period, place):
    """Squares just below half of the large one's last place: a plain sum that meets the large one first drops them all."""
    n = 16 * 4096 + 7
    for small in (2.0 ** -12 * 255 / 256, 2.0 ** -12 * 257 / 256 if dtype == "fp32" else 2.0 ** -12 * 129 / 128):
        g = torch.full((n,), small, dtype=torch.float32)
        g[place % period::period] = 1.0
        _check([g.to(TORCH[dtype]).cuda()])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["up", "down"])
def test_elements_of_all_sizes(dtype, order):
    g = np.random.default_rng(0).permutation(np.logspace(-18, 18, 30001))
    g = np.sort(g) if order == "up" else np.sort(g)[::-1].copy()
    _check([torch.as_tensor(g).float().to(TORCH[dtype]).cuda()])


def test_ends_of_the_range():
    """Infinite sums, NaN beside them, and nothing but what is too small."""
    for values, check in (([1e19] * 40, lambda x: x == math.inf), ([3e38], lambda x: x == math.inf),
                          ([math.inf, 1.0], lambda x: x == math.inf), ([-math.inf], lambda x: x == math.inf),
                          ([math.inf, math.nan], math.isnan), ([math.nan] * 20, math.isnan),
                          ([1e19, 1e10, 1.0], lambda x: abs(x / 1e19 - 1) < 1e-6), ([1e-24] * 100, lambda x: x < 1e-22),
                          ([0.0] * 50, lambda x: x == 0)):
        for at in (0, 7, 16, 4097):
            g = torch.zeros(5000)
            g[at:at + len(values)] = torch.tensor(values, dtype=torch.float64).float()
            norm, scale = _norm([g.cuda()])
            assert check(norm.item()), (values[:2], at, norm.item())
            if math.isfinite(norm.item()):  # the norm's rounding and the scale's
                want = min(1.0, 1e9 / (norm.item() + 1e-6))
                assert abs(scale.item() - want) <= 3 * EPS32 * want
            else:
                assert math.isnan(scale.item())
