"""Records of the longest rows: on both sides of the lengths from which an fp32
row takes two CTAs, and four."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,K", [(327616, 64), (327617, 64), (229312, 8192), (229313, 8192), (524288, 1), (524287, 2048), (524288, 8192)])
@pytest.mark.parametrize("pad", [0, 3])
def test_longest_rows(dtype, V, K, pad):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    g = np.random.default_rng(V + K)
    x = g.normal(0, 2, (3, V))
    x[1] = g.integers(-3, 4, V)
    x[2, np.arange(V) % 3 == 0] = -np.inf
    t = rows(x, TORCH[dtype], pad)
    ids, top, rest = DominoTrain(V).top_logits(t, K, 1.5)
    torch.cuda.synchronize()
    oi, ot, orest = O.top_logits(wide(t), K, 1.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    np.testing.assert_array_equal(wide(top) + 0.0, ot + 0.0)
    tol = 2 * sum_error(V) + 4 * EPS32 * (np.abs(orest) + 20.0)
    assert (np.abs(wide(rest) - orest) <= tol).all()
