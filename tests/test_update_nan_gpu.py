"""Elements that are not numbers beside others of their thread, block and warp."""
import pytest

from train_helpers import TORCH

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _optim(*a, **kw):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    return DominoAdamW(*a, **kw)


@pytest.mark.parametrize("dtype,master", [("bf16", False), ("bf16", True), ("fp32", False)])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_a_gradient_that_is_none_spoils_its_block_of_8_bit_moments_alone(dtype, master, grad):
    """In the step itself its own parameter alone: the others of the block are updated from exact moments."""
    n = 128 * 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    g = torch.randn(n, device="cuda", generator=gen).to(TORCH[grad])
    start = torch.randn(n, device="cuda", generator=gen).to(TORCH[dtype])
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[torch.randint(0, n, (40,), device="cuda", generator=gen)] = True
    block = bad.view(-1, 128).any(1).repeat_interleave(128)
    h = g.clone()
    h[bad] = float("nan")
    p, q = start.clone(), start.clone()
    a, b = (_optim([t], state_bits=8, master=master, seed=3) for t in (p, q))
    a.step(grads=[g])
    b.step(grads=[h])
    assert torch.isnan(q[bad]).all() and torch.equal(q[~bad], p[~bad])
    for x, y in zip(a.moments(0), b.moments(0)):
        assert torch.equal(x[~block], y[~block]) and torch.isnan(y[block]).all()
