"""The loss of rows far from zero: what all logits of a row share takes no part."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _losses(x, ids, top, rest, T):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    tr = DominoTrain(x.shape[1], dtype="bf16" if x.dtype == torch.bfloat16 else "fp32")
    i, t = torch.as_tensor(ids).cuda(), torch.as_tensor(top).cuda()
    r = None if rest is None else torch.as_tensor(rest).cuda()
    forward, _ = tr.distill_forward(x, i, t, r, T)
    step, grad = tr.distill_step(x, i, t, r, torch.ones(x.shape[0], device="cuda"), T)
    torch.cuda.synchronize()
    assert torch.isfinite(grad).all()
    return {"forward": wide(forward), "step": wide(step)}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,K", [(640, 8), (640, 300), (30011, 40)])
@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("with_rest", [False, True])
def test_a_row_of_the_lowest_value(dtype, V, K, T, with_rest):
    """A student whose every logit is masked by the type's lowest value is uniform: q = 1 / V."""
    g = np.random.default_rng(K)
    x = rows(np.full((2, V), float(torch.finfo(TORCH[dtype]).min)), TORCH[dtype])
    ids = np.stack([g.permutation(V)[:K] for _ in range(2)]).astype(np.int32)
    top = g.normal(0, 2, (2, K)).astype(np.float32)
    rest = np.asarray([0.5, -1.0], np.float32) if with_rest else None
    want, _, _ = O.distill(np.zeros((2, V)), ids, top.astype(np.float64), None if rest is None else rest.astype(np.float64), T)
    # sums of at most ten: logs of V, of the record's mass, and the weighted differences of the tops (three roundings each)
    tol = 4 * sum_error(V) + 16 * EPS32 * (np.log(V) + np.abs(top).max() / T * 2 + 10.0)
    for route, loss in _losses(x, ids, top, rest, T).items():
        assert (np.abs(loss - want) <= tol).all(), (route, loss, want)


@pytest.mark.parametrize("student,teacher", [(4096.0, 0.0), (-4096.0, 0.0), (0.0, 4096.0), (1024.0, -512.0)])
def test_shifted_rows(student, teacher):
    """Logits that are multiples of 1/64 stay exact under these shifts, and so does the loss but for its own roundings."""
    g = np.random.default_rng(5)
    N, V, K, T = 3, 5003, 60, 1.0
    x = np.round(g.normal(0, 2, (N, V)) * 64) / 64
    ids = np.stack([g.permutation(V)[:K] for _ in range(N)]).astype(np.int32)
    top = (np.round(g.normal(3, 2, (N, K)) * 64) / 64).astype(np.float32)
    want, _, parts = O.distill(x, ids, top.astype(np.float64), None, T)
    tol = (4 * sum_error(V) + 8 * EPS32) * (1.0 + parts["loss"])
    for route, loss in _losses(rows(x + student, torch.float32), ids, top + np.float32(teacher), None, T).items():
        assert (np.abs(loss - want) <= tol).all(), (route, np.abs(loss - want), tol)
    # with a rest, which is one rounded number beside the tops
    rest = (top.max(1) - 1.0).astype(np.float32)
    want, _, parts = O.distill(x, ids, top.astype(np.float64), rest.astype(np.float64), T)
    tol = (4 * sum_error(V) + 8 * EPS32) * (1.0 + parts["loss"])
    got = _losses(rows(x + student, torch.float32), ids, top + np.float32(teacher), rest + np.float32(teacher), T)
    for route, loss in got.items():
        assert (np.abs(loss - want) <= tol).all(), (route, np.abs(loss - want), tol)
