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


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("with_rest", [False, True])
def test_a_student_without_any_logit(dtype, with_rest):
    """All logits -inf: no q.  NaN with a target, 0 without one; the rows beside it are untouched by it."""
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    g = np.random.default_rng(6)
    V, K = 700, 9
    xv = g.normal(0, 2, (4, V))
    xv[[0, 2]] = -np.inf
    x = rows(xv, TORCH[dtype])
    ids = np.stack([g.permutation(V)[:K] for _ in range(4)]).astype(np.int32)
    ids[2] = -1
    top = g.normal(0, 2, (4, K)).astype(np.float32)
    rest = np.asarray([0.5, 0.5, -np.inf, 0.5], np.float32) if with_rest else None
    tr = DominoTrain(V, dtype=dtype)
    i, t, r = torch.as_tensor(ids).cuda(), torch.as_tensor(top).cuda(), None if rest is None else torch.as_tensor(rest).cuda()
    want, _, parts = O.distill(wide(x), ids, top.astype(np.float64), None if rest is None else rest.astype(np.float64), 1.0)
    tol = (4 * sum_error(V) + 8 * EPS32) * (1.0 + parts["loss"])
    loss, stats = tr.distill_forward(x, i, t, r)
    w = torch.ones(4, device="cuda")
    grad = tr.distill_backward(x, i, t, r, stats, w)
    both = tr.distill_step(x, i, t, r, w)
    torch.cuda.synchronize()
    for l, d in ((loss, grad), both):
        assert np.isnan(wide(l)[0]) and wide(l)[2] == 0 and not d[2].any()
        assert (np.abs(wide(l) - want)[[1, 3]] <= tol[[1, 3]]).all() and torch.isfinite(d[[1, 3]]).all()
