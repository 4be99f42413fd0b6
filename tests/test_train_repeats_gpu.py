"""Records in which ids occur more than once: only the first place counts, and
the time stays that of a walk over the record, not of its square."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

N = 5


def _ids(kind, g, V, K):
    some = g.permutation(V)
    if kind == "one":          # a single repeat, of the first id, at the end
        ids = some[np.arange(K) % V].copy()
        ids[-1] = ids[0]
    elif kind == "halves":     # each twice
        ids = some[np.arange(K) % (K // 2) % V]
    elif kind == "neighbours":
        ids = some[np.arange(K) // 2 % V]
    elif kind == "same":
        ids = np.full(K, some[0])
    else:                      # any, and padding
        ids = g.integers(-1, V, K)
    return ids.astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["one", "halves", "neighbours", "same", "any"])
@pytest.mark.parametrize("V,K", [(64, 33), (64, 700), (4097, 31), (4097, 8192), (60001, 300), (60001, 8192), (151936, 2048)])
def test_first_places(dtype, kind, V, K):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    g = np.random.default_rng(V + K)
    T = 1.3
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype], 3)
    ids = np.stack([_ids(kind, g, V, K) for _ in range(N)])
    ids[3] = _ids("any", g, V, K)
    top = g.normal(3, 2, (N, K)).astype(np.float32)
    rest = (top.max(1) / T + g.normal(-1, 1, N)).astype(np.float32)
    w = g.normal(0, 1, N).astype(np.float32)
    tr = DominoTrain(V, dtype=dtype)
    i, t, r, wt = (torch.as_tensor(a).cuda() for a in (ids, top, rest, w))
    xs = wide(x)
    o_loss, o_grad, parts = O.distill(xs, ids, top.astype(np.float64), rest.astype(np.float64), T)
    e, span = sum_error(V), ((xs.max(1) - xs.min(1)) / T)[:, None]
    w64 = w.astype(np.float64)[:, None]
    # as for records without repeats; a CTA's warp may sum all of a record alone: K / 32 additions in a row
    e = e + K / 32 * EPS32
    tol = (2 * e + 8 * EPS32 + 6 * EPS32 * span) * parts["grad"] * np.abs(w64) + OUT_EPS[x.dtype] * 1.01 * np.abs(o_grad * w64) + 1e-36
    tol_l = (4 * e + 8 * EPS32) * (1.0 + parts["loss"])
    loss, stats = tr.distill_forward(x, i, t, r, T)
    pair = tr.distill_backward(x, i, t, r, stats, wt, T)
    both, grad = tr.distill_step(x, i, t, r, wt, T)
    torch.cuda.synchronize()
    for route, l, d in (("pair", loss, pair), ("step", both, grad)):
        finite = np.isfinite(o_loss)  # a record of the whole vocabulary with a rest: no student mass outside, +inf
        assert (wide(l)[~finite] == o_loss[~finite]).all(), route
        assert (np.abs(wide(l)[finite] - o_loss[finite]) <= tol_l[finite]).all(), route
        assert (np.abs(wide(d) - o_grad * w64) <= tol).all(), route
    again = tr.distill_step(x, i, t, r, wt, T)
    assert torch.equal(again[0], both) and torch.equal(again[1], grad)
    assert tr.status() == 0


@pytest.mark.parametrize("V", [9001, 151936])
def test_a_repeat_does_not_square_the_time(V):
    """The longest record with each id twice: a walk of one warp over 8192 entries is some 256 steps of two memory
    latencies, under half a millisecond; a scan of all earlier entries for each is about 16 M loads."""
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    K = 8192
    g = np.random.default_rng(0)
    x = torch.randn(1, V, device="cuda")
    ids = torch.as_tensor(_ids("halves", g, V, K)[None]).cuda()
    top, w = torch.randn(1, K, device="cuda"), torch.ones(1, device="cuda")
    tr = DominoTrain(V, dtype="fp32")
    loss, stats = tr.distill_forward(x, ids, top)
    calls = {"step": lambda: tr.distill_step(x, ids, top, None, w), "forward": lambda: tr.distill_forward(x, ids, top),
             "backward": lambda: tr.distill_backward(x, ids, top, None, stats, w)}
    for name, call in calls.items():
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        assert best < 1.0, (name, best)
