"""The autograd lookup of more tokens than one table gradient takes."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, rows, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,most", [(64, 64), (65, 64), (200, 64), (200, 1), (1, 1), (0, 0)])
def test_more_tokens_than_one_call_takes(dtype, n, most):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, embedding
    V, E = 50, 24
    g = np.random.default_rng(n + most)
    scale = float(np.float32(0.3))
    tr = DominoTrain(V, E=E, max_tokens=most, dtype=dtype)
    W = rows(g.normal(0, 1, (V, E)), TORCH[dtype]).contiguous().requires_grad_()
    tok = g.integers(-1, V, n).astype(np.int32)
    d = torch.as_tensor(g.normal(0, 1, (n, E)).astype(np.float32)).to(TORCH[dtype]).cuda()
    y = embedding(tr, W, torch.as_tensor(tok).cuda(), scale)
    y.backward(d)
    want, terms, count = O.embed_grad(wide(d), tok, V, scale)
    # an addition and a product per token at most, and the output's rounding
    tol = (2 * count[:, None] + 3) * EPS32 * terms + OUT_EPS[TORCH[dtype]] * 1.01 * np.abs(want)
    assert W.grad.dtype is TORCH[dtype] and (np.abs(wide(W.grad) - want) <= tol).all()
    assert tr.status() == 0


def test_no_gradient_without_a_workspace():
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, embedding
    tr = DominoTrain(20, E=8, dtype="fp32")
    W = torch.zeros(20, 8, device="cuda", requires_grad=True)
    y = embedding(tr, W, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="max_tokens"):
        y.sum().backward()
