"""Distillation at sizes where the kernels reach their steady state: a cluster
of the step takes several rows in turn, of different kinds, and the rings of
forward and backward run round.  A sample of the rows against the fp64 oracle."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ("plain", "skipped", "skipped_nan", "repeated", "no_target", "no_rest", "padded", "plain")


def _case(N, V, K, T, dtype, pad, seed):
    """Rows of logits (stride V + pad), records, rests and weights on the GPU; the kinds alternate without a period
    that a number of clusters could share."""
    g = np.random.default_rng(seed)
    kind = np.asarray(KINDS)[g.integers(0, len(KINDS), N)]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, V + pad, device="cuda", generator=gen).mul_(2.0).to(TORCH[dtype])[:, :V]
    ids = np.stack([g.choice(V, K, replace=False) if K * 4 > V else _distinct(g, V, K) for _ in range(N)]).astype(np.int32)
    top = g.normal(3, 2, (N, K)).astype(np.float32)
    rest = (top.max(1) / T + g.normal(-1, 1, N)).astype(np.float32)
    w = g.normal(0, 1, N).astype(np.float32)
    for n in range(N):
        if kind[n].startswith("skipped"):
            w[n] = 0.0
        if kind[n] == "repeated" and K > 1:
            ids[n, K // 2:] = ids[n, : K - K // 2]
        if kind[n] == "no_target":
            ids[n], rest[n] = -1, -np.inf
        if kind[n] == "no_rest":
            rest[n] = -np.inf
        if kind[n] == "padded":
            ids[n, g.random(K) < 0.5] = -1
    x[torch.as_tensor(kind == "skipped_nan").cuda()] = float("nan")
    return kind, x, ids, top, rest, w


def _distinct(g, V, K):
    """K ids of different K-ths of the vocabulary, in any order."""
    edge = np.arange(K + 1) * V // K
    return g.permutation(edge[:-1] + (g.random(K) * (edge[1:] - edge[:-1])).astype(np.int64))


def _check(kind, x, ids, top, rest, w, T, route, loss, grad, sample):
    N, V = x.shape
    xs = wide(x[sample])
    o_loss, o_grad, parts = O.distill(xs, ids[sample], top[sample].astype(np.float64), rest[sample].astype(np.float64), T)
    w64 = w[sample].astype(np.float64)[:, None]
    o_grad[w[sample] == 0] = 0.0
    parts["grad"][w[sample] == 0] = 0.0
    want = o_grad * w64
    span = np.where(np.isfinite(xs), xs, 0.0)
    span = np.minimum((span.max(1) - span.min(1)) / T, 100.0)[:, None]
    e = sum_error(V)
    # q and p: two sums, an exponential with three roundings of its argument, up to eight roundings of factors;
    # the output's rounding; results that the hardware's exponential flushes to zero
    tol = (2 * e + 8 * EPS32 + 6 * EPS32 * span) * parts["grad"] * np.abs(w64) + OUT_EPS[x.dtype] * 1.01 * np.abs(want) + 1e-36
    bad = ~(np.abs(wide(grad[sample]) - want) <= tol)
    assert not bad.any(), (route, kind[sample][np.argwhere(bad)[:5, 0]], np.argwhere(bad)[:5])
    got = wide(loss[sample])
    skip = kind[sample] == "skipped_nan"
    if route == "step":
        skip = w[sample] == 0
        assert (got[skip] == 0).all()
    tol_l = (4 * e + 8 * EPS32) * (1.0 + parts["loss"])
    d = np.abs(got - o_loss)[~skip]
    assert (d <= tol_l[~skip]).all(), (route, kind[sample][~skip][~(d <= tol_l[~skip])])


def _run(N, V, K, T, dtype, pad, out_pad, routes, samples):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    kind, x, ids, top, rest, w = _case(N, V, K, T, dtype, pad, N + V + K)
    tr = DominoTrain(V, dtype=dtype)
    i, t, r, wt = (torch.as_tensor(a).cuda() for a in (ids, top, rest, w))
    sample = np.unique(np.linspace(0, N - 1, samples).round().astype(np.int64))
    for route in routes:
        buf = torch.full((N, V + out_pad), 7.0, dtype=x.dtype, device="cuda")
        grad = buf[:, :V]
        if route == "step":
            loss, _ = tr.distill_step(x, i, t, r, wt, T, out=(torch.full((N,), 7.0, device="cuda"), grad))
        else:
            loss, stats = tr.distill_forward(x, i, t, r, T)
            tr.distill_backward(x, i, t, r, stats, wt, T, out=grad)
        torch.cuda.synchronize()
        assert (buf[:, V:] == 7.0).all()
        assert not (grad[torch.as_tensor(w == 0).cuda()] != 0).any()
        assert not grad.isnan().any()
        _check(kind, x, ids, top, rest, w, T, route, loss, grad, sample)
        # every row written: a row with weight and a target has a gradient
        some = torch.as_tensor((w != 0) & (kind != "no_target")).cuda()
        assert (grad[some] != 0).any(1).all()
        if route == "pair":
            continue
        again = torch.full_like(buf, 3.0)
        tr.distill_step(x, i, t, r, wt, T, out=(loss, again[:, :V]))
        assert torch.equal(again[:, :V], grad)
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,K,T,pad,out_pad", [(5000, 257, 40, 1.0, 0, 0), (3000, 1003, 300, 1.5, 5, 5), (3000, 520, 128, 0.7, 0, 1),
                                                 (1200, 9001, 700, 1.0, 0, 0), (400, 20011, 300, 2.0, 3, 3),
                                                 (400, 40000, 64, 1.0, 8, 8), (330, 151936, 64, 1.0, 0, 0),
                                                 (250, 151935, 1000, 1.0, 1, 0)])
def test_rows_in_turn(dtype, N, V, K, T, pad, out_pad):
    _run(N, V, K, T, dtype, pad, out_pad, ("step",), 2000 if V < 2000 else 60)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,K,T,pad,out_pad", [(700, 20011, 40, 1.0, 0, 0), (700, 60001, 300, 1.5, 7, 7), (640, 80000, 64, 1.0, 0, 0),
                                                 (640, 151936, 256, 2.0, 0, 0), (620, 70003, 64, 1.0, 2, 1)])
def test_rings_run_round(dtype, N, V, K, T, pad, out_pad):
    _run(N, V, K, T, dtype, pad, out_pad, ("pair",), 60)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_hard_label_is_cross_entropy(dtype):
    """K = 1 without a rest: the usual cross entropy and its gradient; -1 is an ignored position."""
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, distill_loss
    N, V = 40, 5003
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(N, V, device="cuda", generator=g).mul_(3.0).to(TORCH[dtype])
    label = torch.randint(0, V, (N,), device="cuda", generator=g)
    label[::7] = -1
    d = x.double().requires_grad_()
    want = torch.nn.functional.cross_entropy(d, label, ignore_index=-1, reduction="none")
    want.sum().backward()
    x.requires_grad_()
    loss = distill_loss(DominoTrain(V, dtype=dtype), x, label.to(torch.int32)[:, None], torch.zeros(N, 1, device="cuda"))
    loss.sum().backward()
    # log q and the label's logit: the sum's error, three roundings of the terms
    tol = 2 * sum_error(V) + 4 * EPS32 * (want.detach().abs() + 2 * d.detach().abs().max())
    assert ((loss.detach().double() - want.detach()).abs() <= tol).all()
    span = 6 * EPS32 * 40.0  # the exponentials' arguments
    assert ((x.grad.double() - d.grad).abs() <= (2 * sum_error(V) + 8 * EPS32 + span) * (d.grad.abs() + (d.grad < 0) * 2.0)
            + OUT_EPS[x.dtype] * 1.01 * d.grad.abs() + 1e-36).all()
