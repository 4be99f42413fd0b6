"""Distillation loss and gradient against the fp64 oracle, on both routes
(forward then backward, and the one-call step)."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _train(V, dtype):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, dtype=dtype)


def _dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


def _record(g, N, V, K, T):
    ids = np.stack([g.permutation(V)[:K] for _ in range(N)]).astype(np.int32)
    top = g.normal(3, 2, (N, K)).astype(np.float32)
    rest = (top.max(1) / T + g.normal(-1, 1, N)).astype(np.float32)
    return ids, top, rest


def run_both(tr, x, ids, top, rest, w, T, out_pad=0, out_shift=0):
    """{route: (loss, grad)} as device tensors."""
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), None if rest is None else _dev(rest, torch.float32)
    wt = _dev(w, torch.float32)
    N, V = x.shape
    res = {}
    for route in ("pair", "step"):
        grad = rows(np.full((N, V), 7.0), x.dtype, out_pad, out_shift)
        if route == "pair":
            loss, stats = tr.distill_forward(x, i, t, r, T)
            tr.distill_backward(x, i, t, r, stats, wt, T, out=grad)
        else:
            loss = torch.full((N,), 7.0, device="cuda")
            tr.distill_step(x, i, t, r, wt, T, out=(loss, grad))
        torch.cuda.synchronize()
        res[route] = (loss, grad)
    return res


def check(tr, x, ids, top, rest, w, T, **kw):
    o_loss, o_grad, parts = O.distill(wide(x), ids, top.astype(np.float64),
                                      None if rest is None else rest.astype(np.float64), T)
    V = x.shape[1]
    e = sum_error(V)
    xw = wide(x)
    span = np.where(np.isfinite(xw), xw, 0.0)
    span = np.minimum((span.max(1) - span.min(1)) / T, 100.0)[:, None]
    w64 = w.astype(np.float64)[:, None]
    want = o_grad * w64
    # q and p: two sums, an exponential with three roundings of its argument, and
    # up to eight roundings of factors; then the output's rounding, and results
    # that the hardware's exponential flushes to zero
    tol = (2 * e + 8 * EPS32 + 6 * EPS32 * span) * parts["grad"] * np.abs(w64) + OUT_EPS[x.dtype] * 1.01 * np.abs(want)
    tol = tol + 1e-36
    tol_l = (4 * e + 8 * EPS32) * (1.0 + parts["loss"])
    for route, (loss, grad) in run_both(tr, x, ids, top, rest, w, T, **kw).items():
        l, g = wide(loss), wide(grad)
        skip = (w == 0) & (route == "step")
        assert (l[skip] == 0).all()
        d = np.abs(np.where(l == o_loss, 0.0, l - np.where(np.isfinite(o_loss), o_loss, 1e300)))[~skip]
        assert (d <= tol_l[~skip]).all(), (route, d.max(), tol_l[~skip][d.argmax()])
        bad = ~(np.abs(g - want) <= tol)
        assert not bad.any(), (route, np.argwhere(bad)[:5], np.abs(g - want)[bad][:5], tol[bad][:5])
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,K,T", [(1, 2, 1, 1.0), (1, 2, 2, 1.0), (3, 31, 7, 0.7), (2, 33, 32, 2.0), (5, 1000, 1, 1.0),
                                     (4, 4097, 300, 1.5), (3, 9001, 8192, 1.0), (2, 20011, 64, 4.0),
                                     (2, 151936, 64, 1.0), (1, 151935, 2048, 2.0)])
def test_random_rows(dtype, N, V, K, T):
    g = np.random.default_rng(N + V + K)
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype])
    ids, top, rest = _record(g, N, V, K, T)
    check(_train(V, dtype), x, ids, top, rest, g.normal(0, 1, N).astype(np.float32), T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift,out_pad,out_shift", [(0, 1, 0, 1), (1, 0, 0, 0), (3, 5, 3, 5), (8, 8, 16, 8),
                                                         (0, 0, 0, 3), (2, 4, 7, 1)])
def test_strides_and_alignment(dtype, pad, shift, out_pad, out_shift):
    N, V, K = 6, 2503, 40
    g = np.random.default_rng(pad + 10 * shift + out_pad)
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype], pad, shift)
    ids, top, rest = _record(g, N, V, K, 1.0)
    check(_train(V, dtype), x, ids, top, rest, np.ones(N, np.float32), 1.0, out_pad=out_pad, out_shift=out_shift)


def test_writes_stay_inside_the_rows():
    N, V, K = 4, 1001, 10
    g = np.random.default_rng(0)
    tr = _train(V, "bf16")
    x = rows(g.normal(0, 2, (N, V)), torch.bfloat16)
    ids, top, rest = _record(g, N, V, K, 1.0)
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), _dev(rest, torch.float32)
    buf = torch.full((3 + N * (V + 5) + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    grad = buf[3:3 + N * (V + 5)].view(N, V + 5)[:, :V]
    tr.distill_step(x, i, t, r, torch.ones(N, device="cuda"), out=(torch.empty(N, device="cuda"), grad))
    torch.cuda.synchronize()
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[3:3 + N * (V + 5)].view(N, V + 5)[:, :V] = False
    assert (buf[mask] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rest_kind", ["none", "minus_inf", "tiny", "dominant"])
def test_rest(dtype, rest_kind):
    N, V, K = 5, 1500, 30
    g = np.random.default_rng(7)
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype])
    ids, top, rest = _record(g, N, V, K, 1.0)
    rest = {"none": None, "minus_inf": np.full(N, -np.inf, np.float32), "tiny": rest - 40.0,
            "dominant": rest + 60.0}[rest_kind]
    check(_train(V, dtype), x, ids, top, rest, np.ones(N, np.float32), 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_repeats_order_and_empty_rows(dtype):
    N, V, K = 8, 777, 24
    g = np.random.default_rng(8)
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype])
    ids, top, rest = _record(g, N, V, K, 1.0)
    ids[0, 10:] = -1
    ids[1, ::3] = -1
    ids[2] = ids[2, 0]                       # one id throughout
    ids[3, 12:] = ids[3, :12]                # each twice
    ids[4] = -1                              # empty, mass in the rest only
    ids[5] = -1
    rest[5] = -np.inf                        # no target
    top[6, 5:] = -np.inf                     # entries without mass
    top[7] = -np.inf
    rest[7] = -np.inf                        # a record without mass: no target
    w = np.full(N, 0.5, np.float32)
    check(_train(V, dtype), x, ids, top, rest, w, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_students(dtype):
    """-inf and the lowest value where a grammar forbids tokens, outside the record."""
    N, V, K = 4, 1200, 16
    g = np.random.default_rng(9)
    xv = g.normal(0, 2, (N, V))
    ids, top, rest = _record(g, N, V, K, 1.0)
    lowest = float(torch.finfo(TORCH[dtype]).min)
    for n, m in enumerate((-np.inf, lowest, -np.inf, lowest)):
        keep = np.zeros(V, bool)
        keep[ids[n]] = True
        if n < 2:
            keep[: V // 2] = True
        xv[n, ~keep] = m
    rest[2:] = -np.inf                       # nothing outside on either side
    check(_train(V, dtype), rows(xv, TORCH[dtype]), ids, top, rest, np.ones(N, np.float32), 1.0)


def test_a_row_of_the_lowest_value_is_uniform():
    V, K = 640, 8
    tr = _train(V, "bf16")
    lowest = float(torch.finfo(torch.bfloat16).min)
    x = rows(np.full((1, V), lowest), torch.bfloat16)
    ids = np.arange(K, dtype=np.int32)[None]
    top = np.zeros((1, K), np.float32)
    for loss, grad in run_both(tr, x, ids, top, None, np.ones(1, np.float32), 1.0).values():
        want = np.where(np.arange(V) < K, 1 / V - 1 / K, 1 / V)
        np.testing.assert_allclose(wide(grad)[0], want, rtol=2 ** -8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unreachable_targets_and_nan(dtype):
    """A record on a forbidden token, a rest with no student mass, NaN and +inf logits."""
    N, V, K = 6, 500, 6
    g = np.random.default_rng(10)
    xv = g.normal(0, 2, (N, V))
    ids, top, rest = _record(g, N, V, K, 1.0)
    xv[0, ids[0, 2]] = -np.inf               # loss +inf, gradient finite
    keep = np.zeros(V, bool)
    keep[ids[1]] = True
    xv[1, ~keep] = -np.inf                   # q_r = 0 < p_r: loss +inf
    xv[2, 17] = np.nan                       # NaN
    top[3, 1] = np.nan                       # NaN
    xv[4, :] = np.nan                        # weight 0: skipped
    w = np.array([1, 1, 1, 1, 0, 1], np.float32)
    x = rows(xv, TORCH[dtype])
    o_loss, o_grad, _ = O.distill(wide(x), ids, top.astype(np.float64), rest.astype(np.float64), 1.0)
    for route, (loss, grad) in run_both(_train(V, dtype), x, ids, top, rest, w, 1.0).items():
        l, gr = wide(loss), wide(grad)
        assert l[0] == np.inf and l[1] == np.inf and np.isnan(l[2]) and np.isnan(l[3])
        np.testing.assert_allclose(gr[0], o_grad[0], rtol=0.01, atol=1e-5)
        np.testing.assert_allclose(gr[1], o_grad[1], rtol=0.01, atol=1e-5)
        assert np.isnan(gr[2]).any() and np.isnan(gr[3]).any()
        assert (gr[4] == 0).all()
        np.testing.assert_allclose(gr[5], o_grad[5], rtol=0.01, atol=1e-5)


def test_no_target_rows_ignore_their_logits():
    V = 300
    tr = _train(V, "fp32")
    x = rows(np.full((2, V), np.nan), torch.float32)
    ids = np.full((2, 3), -1, np.int32)
    for loss, grad in run_both(tr, x, ids, np.zeros((2, 3), np.float32), None, np.ones(2, np.float32), 1.0).values():
        assert (wide(loss) == 0).all() and (wide(grad) == 0).all()


def test_outside_far_below_the_record():
    """The outside's share of the student underflows next to the record, but the
    teacher's rest does not vanish."""
    V, K = 900, 4
    g = np.random.default_rng(11)
    ids, top, rest = _record(g, 2, V, K, 1.0)
    xv = g.normal(-120, 1, (2, V))
    for n in range(2):
        xv[n, ids[n]] = g.normal(0, 1, K)
    check(_train(V, "fp32"), rows(xv, torch.float32), ids, top, rest, np.ones(2, np.float32), 1.0)


def test_bad_ids_are_reported_and_ignored():
    from speculative_decoding_draft_lm_gb300 import rollout as R
    V = 100
    g = np.random.default_rng(12)
    tr = _train(V, "fp32")
    x = rows(g.normal(0, 2, (1, V)), torch.float32)
    ids = np.array([[5, 100, -2, 7, 2 ** 31 - 1]], np.int32)
    top = np.array([[1, 9, 9, 2, 9]], np.float32)
    i, t = _dev(ids, torch.int32), _dev(top, torch.float32)
    loss, _ = tr.distill_forward(x, i, t)
    assert tr.status() == R.DOMINO_ERR_BAD_TOKEN
    assert tr.status() == 0
    want, _, _ = O.distill(wide(x), ids, top.astype(np.float64), None, 1.0)
    assert abs(wide(loss)[0] - want[0]) < 1e-5


def test_gradient_matches_differences_of_the_loss():
    """Along random directions: central differences of the fp32 loss (error h^2/6
    of the third derivative, and the loss's rounding over h)."""
    N, V, K, T, h = 4, 400, 12, 1.3, 2e-2
    g = np.random.default_rng(13)
    tr = _train(V, "fp32")
    x = g.normal(0, 2, (N, V)).astype(np.float32)
    ids, top, rest = _record(g, N, V, K, T)
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), _dev(rest, torch.float32)
    w = torch.ones(N, device="cuda")
    _, grad = tr.distill_step(rows(x, torch.float32), i, t, r, w, T)
    for _ in range(4):
        d = g.normal(0, 1, (N, V)).astype(np.float32)
        lp = wide(tr.distill_forward(rows(x + h * d, torch.float32), i, t, r, T)[0])
        lm = wide(tr.distill_forward(rows(x - h * d, torch.float32), i, t, r, T)[0])
        slope = (wide(grad) * d).sum(1)
        assert (np.abs((lp - lm) / (2 * h) - slope) <= 2e-3).all()


def test_repeated_calls_streams_and_graph_give_equal_bits():
    N, V, K = 33, 5003, 20
    g = np.random.default_rng(14)
    tr = _train(V, "bf16")
    x = rows(g.normal(0, 2, (N, V)), torch.bfloat16)
    ids, top, rest = _record(g, N, V, K, 1.0)
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), _dev(rest, torch.float32)
    w = torch.rand(N, device="cuda")
    loss, grad = tr.distill_step(x, i, t, r, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss2, grad2 = tr.distill_step(x, i, t, r, w)
        f, stats = tr.distill_forward(x, i, t, r)
        b = tr.distill_backward(x, i, t, r, stats, w)
    s.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)
    out = (torch.empty_like(loss), torch.empty_like(grad))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.distill_step(x, i, t, r, w, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], loss) and torch.equal(out[1], grad)


def test_rows_beyond_32_bit_offsets():
    V, ld, N, K = 1003, 2 ** 30 + 7, 3, 9
    g = np.random.default_rng(15)
    tr = _train(V, "bf16")
    mk = lambda: torch.empty(ld * (N - 1) + V, dtype=torch.bfloat16, device="cuda").as_strided((N, V), (ld, 1))
    x, grad = mk(), mk()
    x.copy_(torch.as_tensor(g.normal(0, 2, (N, V))).to(torch.bfloat16))
    ids, top, rest = _record(g, N, V, K, 1.0)
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), _dev(rest, torch.float32)
    near = tr.distill_step(x.contiguous(), i, t, r, torch.ones(N, device="cuda"))
    far = tr.distill_step(x, i, t, r, torch.ones(N, device="cuda"), out=(torch.empty(N, device="cuda"), grad))
    torch.cuda.synchronize()
    np.testing.assert_allclose(wide(far[0]), wide(near[0]), rtol=1e-5)
    np.testing.assert_allclose(wide(far[1]), wide(near[1]), rtol=2 ** -7, atol=1e-9)


def test_autograd_function():
    from speculative_decoding_draft_lm_gb300.train import distill_loss
    N, V, K = 5, 600, 7
    g = np.random.default_rng(16)
    tr = _train(V, "fp32")
    x = rows(g.normal(0, 2, (N, V)), torch.float32).contiguous().requires_grad_()
    ids, top, rest = _record(g, N, V, K, 1.0)
    i, t, r = _dev(ids, torch.int32), _dev(top, torch.float32), _dev(rest, torch.float32)
    (distill_loss(tr, x, i, t, r).mean() * 3.0).backward()
    _, o_grad, _ = O.distill(wide(x), ids, top.astype(np.float64), rest.astype(np.float64), 1.0)
    np.testing.assert_allclose(wide(x.grad), o_grad * 3.0 / N, rtol=1e-4, atol=1e-7)


def test_refusals():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    V, N, K = 64, 3, 4
    tr = _train(V, "fp32")
    x = torch.zeros(N, V, device="cuda")
    i = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    t, r, w = torch.zeros(N, K, device="cuda"), torch.zeros(N, device="cuda"), torch.ones(N, device="cuda")
    for bad in (dict(x=x.to(torch.bfloat16)), dict(x=x[:, :-1]), dict(x=x.t()), dict(x=x.cpu()), dict(i=i.long()),
                dict(i=i[:, :-1]), dict(t=t.double()), dict(r=r[:-1]), dict(w=w.double()), dict(w=w[:-1])):
        a = dict(x=x, i=i, t=t, r=r, w=w)
        a.update(bad)
        with pytest.raises(ValueError):
            tr.distill_step(a["x"], a["i"], a["t"], a["r"], a["w"])
    for T in (0.0, float("nan"), -2.0, 1e4):
        with pytest.raises(DominoError):
            tr.distill_step(x, i, t, r, w, T)
    with pytest.raises(DominoError):  # in place
        tr.distill_step(x, i, t, r, w, out=(torch.empty(N, device="cuda"), x))
    with pytest.raises(DominoError):
        tr.distill_forward(x, i[:, :0], t[:, :0], r)
    with pytest.raises(ValueError):
        tr.distill_forward(x, i, t, r, out=(torch.empty(N, device="cuda"), torch.empty(N, 4, device="cuda")))
    loss, grad = tr.distill_step(x[:0], i[:0], t[:0], r[:0], w[:0])
    assert loss.shape == (0,) and grad.shape == (0, V)
