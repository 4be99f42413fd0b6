"""Elements that are not numbers beside others of their thread, block and warp."""
import pytest

from train_helpers import TORCH

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _optim(*a, **kw):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    return DominoAdamW(*a, **kw)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("bf16", False), ("bf16", True), ("fp32", False)])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 3])
def test_parameters_that_are_not_numbers(bits, dtype, master, grad, shift):
    """NaN stays where it was, infinite ones stay infinite; all else, the moments too, as if they had been 0."""
    n = 20011
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.randn(n, device="cuda", generator=gen).to(TORCH[grad])
    clean = torch.randn(n + shift, device="cuda", generator=gen).to(TORCH[dtype])[shift:]
    u = torch.rand(n, device="cuda", generator=gen)
    # one in a thousand, whole blocks of every second, and a run over threads' ends
    nan = (u < 0.001) | ((torch.arange(n, device="cuda") // 128 == 9) & (u < 0.5))
    nan[5000:5021] = True
    inf = (u > 0.999) & ~nan
    clean[nan | inf] = 0.0
    odd = torch.zeros(n + shift, device="cuda", dtype=TORCH[dtype])[shift:]
    odd.copy_(clean)
    odd[nan] = float("nan")
    odd[inf] = float("inf")
    opts = [_optim([p], state_bits=bits, master=master, seed=3) for p in (clean, odd)]
    for _ in range(2):
        for opt in opts:
            opt.step(grads=[g])
    assert torch.isnan(odd[nan]).all() and (odd[inf] == float("inf")).all()
    rest = ~(nan | inf)
    assert torch.equal(odd[rest], clean[rest]) and torch.isfinite(clean).all()
    for name in opts[0].state:
        if name != "master":
            a, b = (opt.state[name].view(torch.uint8) for opt in opts)
            assert torch.equal(a, b), name


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
