"""Scores of rows of logits and their gradient against the fp64 oracle, on both
routes (forward then backward, and the one-call step)."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _train(V, dtype):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, dtype=dtype)


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype or torch.float32).cuda()


def tolerances(x, T, terms):
    """(of a log probability whose (x - max) / T is d: a + b |d|), of the entropy), per row.

    log s: the sum's relative error, and two roundings of the logarithm.  d: a
    difference and a quotient.  The entropy's t = sum e d: each term has the
    exponential's error (2 ulp, 3 |d| roundings from its argument) and 3 roundings of d and of the
    product, on |d|; the sums and the quotient as above."""
    e = sum_error(x.shape[1])
    log_s = np.abs(terms["log_s"])
    a = e + 4 * EPS32 * (log_s + 1)
    h = a + terms["a1"] * (2 * e + 16 * EPS32) + 5 * EPS32 * terms["a2"] + 8 * EPS32 * (log_s + terms["a1"])
    return a, 4 * EPS32, h


def close(got, want, tol, what):
    with np.errstate(all="ignore"):  # what fp32 cannot hold is infinite
        want = np.asarray(want, dtype=np.float32).astype(np.float64) if np.abs(want).max(initial=0) > 3e38 else want
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def check_forward(tr, x, tok, T, k, stats=None):
    out = tr.logprobs_forward(x, _dev(tok, torch.int32), T, alternatives=k, stats=stats)
    torch.cuda.synchronize()
    xw = wide(x)
    lp, H, ids, alt, terms = O.logprobs(xw, tok, T, k)
    a, b, h = tolerances(xw, T, terms)
    close(wide(out[0]), lp, a + b * np.where(np.isfinite(lp), np.abs(lp), 0), "logprob")
    close(wide(out[1]), H, h, "entropy")
    if k:
        assert (out[2].cpu().numpy() == ids).all(), (out[2].cpu().numpy()[ids != out[2].cpu().numpy()][:5])
        close(wide(out[3]), alt, a[:, None] + b * np.where(np.isfinite(alt), np.abs(alt), 0), "alternatives")
    return out


def check_gradient(tr, x, tok, T, g, h, out_pad=0, out_shift=0):
    """Both routes; g, h: arrays or None."""
    N, V = x.shape
    z = np.zeros(N, np.float32)
    t = _dev(tok, torch.int32)
    g64, h64 = (z if g is None else g).astype(np.float64), (z if h is None else h).astype(np.float64)
    xw = wide(x)
    want, q, l = O.logprobs_grad(xw, tok, T, g64, h64)
    lp, H, _, _, terms = O.logprobs(xw, tok, T)
    a, b, th = tolerances(xw, T, terms)
    e = sum_error(V)
    d = np.where(q > 0, np.abs(l) + np.abs(terms["log_s"] - H)[:, None] + np.abs(terms["log_s"])[:, None], 0)
    hot = np.zeros((N, V))
    hot[np.arange(N), np.clip(tok, 0, V - 1)] = 1
    rq = e + (12 + 5 * d) * EPS32  # q: the sum, the exponential and its argument, factors
    tol = np.abs(g64)[:, None] * (q * rq + 4 * EPS32 * (hot + q))
    tol += np.abs(h64)[:, None] * q * (np.abs(l) * (rq + 6 * EPS32) + th[:, None] + a[:, None] + 8 * EPS32 * (d + np.abs(H)[:, None]))
    tol = tol / T * (1 + OUT_EPS[x.dtype]) + OUT_EPS[x.dtype] * 1.01 * np.abs(want) + 1e-36
    gd, hd = None if g is None else _dev(g), None if h is None else _dev(h)
    res = {}
    for route in ("pair", "step"):
        grad = rows(np.full((N, V), 7.0), x.dtype, out_pad, out_shift)
        if route == "pair":
            *_, stats = tr.logprobs_forward(x, t, T, stats=True)
            tr.logprobs_backward(x, t, stats, gd, hd, T, out=grad)
        else:
            got_lp, got_H, grad = tr.logprobs_step(x, t, gd, hd, T, out=(torch.empty(N, device="cuda"),
                                                                        torch.empty(N, device="cuda"), grad))
            off = (g64 == 0) & (h64 == 0)
            close(wide(got_lp), np.where(off, 0, lp), a + b * np.where(np.isfinite(lp), np.abs(lp), 0), "logprob")
            close(wide(got_H), np.where(off, 0, H), th, "entropy")
        torch.cuda.synchronize()
        got = wide(grad)
        close(got, want, tol, route)
        if out_pad and N > 1:  # what is not the rows' stays
            between = grad.as_strided((N - 1, out_pad), (V + out_pad, 1), grad.storage_offset() + V)
            assert torch.isnan(between).all()
        res[route] = grad
    return res


SHAPES = [(1, 2), (3, 7), (2, 33), (5, 257), (4, 1000), (3, 4099), (700, 64), (2, 20011), (3, 79999), (2, 151936),
          (1, 151935)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V", SHAPES)
@pytest.mark.parametrize("T,k", [(1.0, 20), (0.75, 1), (2.0, 32)])
def test_random_rows(dtype, N, V, T, k):
    g = np.random.default_rng(N + V)
    x = rows(g.normal(0, 2, (N, V)), TORCH[dtype], pad=3, shift=1)
    tok = g.integers(0, V, N).astype(np.int32)
    tr = _train(V, dtype)
    check_forward(tr, x, tok, T, min(k, V))
    adv, bonus = g.normal(0, 1, N).astype(np.float32), g.random(N).astype(np.float32)
    check_gradient(tr, x, tok, T, adv, bonus, out_pad=5, out_shift=2)
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("which", ["g", "h"])
@pytest.mark.parametrize("N,V", [(4, 1000), (2, 20011)])
def test_one_gradient_alone(dtype, which, N, V):
    g = np.random.default_rng(3)
    x = rows(g.normal(0, 3, (N, V)), TORCH[dtype], pad=8)
    tok = g.integers(0, V, N).astype(np.int32)
    w = g.normal(0, 1, N).astype(np.float32)
    check_gradient(_train(V, dtype), x, tok, 1.5, w if which == "g" else None, w if which == "h" else None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [40, 1000, 30011])
def test_masks(dtype, V):
    """-inf over parts of rows, over all of one, all but one logit, the type's lowest value; masked tokens; padding."""
    g = np.random.default_rng(V)
    low = float(torch.finfo(TORCH[dtype]).min)
    v = g.normal(0, 2, (10, V))
    v[0, : V // 2] = -np.inf
    v[1, V // 3:] = -np.inf
    v[2] = -np.inf
    v[3] = -np.inf
    v[3, V - 1] = 1.5
    v[4, : V // 2] = low
    v[5] = low
    v[6, 1::2] = -np.inf
    v[7] = 3.25          # all equal: ties go by the id
    v[8] = np.round(v[8])  # many ties
    tok = np.asarray([V - 1, V - 1, 3, V - 1, 0, 5, 2, 7, -1, 1], np.int32)  # row 1's and row 4's are masked
    x = rows(v, TORCH[dtype], pad=1)
    tr = _train(V, dtype)
    for T in (0.5, 1.0, 2.0):
        for k in (0, 1, 20, 32):
            check_forward(tr, x, tok, T, k)
        adv, bonus = g.normal(0, 1, 10).astype(np.float32), g.random(10).astype(np.float32)
        adv[9] = bonus[9] = 0
        check_gradient(tr, x, tok, T, adv, bonus)
        check_gradient(tr, x, tok, T, adv, None)
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.001, 1000.0])
def test_far_values(dtype, T):
    """Logits of any size, all far from zero, or far apart, at the ends of the temperature."""
    g = np.random.default_rng(5)
    V = 5000
    v = g.normal(0, 1, (6, V))
    v[0] += 3e4
    v[1] -= 3e4
    v[2] *= 1e30
    v[3] *= 1e-30
    v[4] = v[4] * 1e29 - 2e38
    v[5, ::7] = float(torch.finfo(torch.bfloat16).max)
    x = rows(v, TORCH[dtype])
    tok = g.integers(0, V, 6).astype(np.int32)
    tr = _train(V, dtype)
    out = tr.logprobs_forward(x, _dev(tok, torch.int32), T, alternatives=32, stats=True)
    lp, H, ids, alt, terms = O.logprobs(wide(x), tok, T, 32)
    # T is rounded to fp32 on its way: a relative 2^-24 of every d
    a, b, h = tolerances(wide(x), T, terms)
    close(wide(out[0]), lp, a + (b + EPS32) * np.where(np.isfinite(lp), np.abs(lp), 0), "logprob")
    close(wide(out[1]), H, h + EPS32 * (terms["a1"] + terms["a2"]), "entropy")
    assert (out[2].cpu().numpy() == ids).all()
    grad = tr.logprobs_backward(x, _dev(tok, torch.int32), out[4], _dev(np.ones(6)), _dev(np.ones(6)), T)
    assert torch.isfinite(grad).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_not_numbers(dtype):
    """A NaN or +inf logit makes its row's floats NaN, and no other's; ids still come in order."""
    g = np.random.default_rng(6)
    V = 3000
    v = g.normal(0, 1, (5, V))
    v[1, 700] = np.nan
    v[2, 2999] = np.inf
    v[3, 5] = v[3, 6] = np.nan
    v[3, 900:] = -np.inf
    x = rows(v, TORCH[dtype])
    tok = np.asarray([1, 2, 3, 4, -1], np.int32)
    tr = _train(V, dtype)
    out = check_forward(tr, x, tok, 1.0, 8, stats=True)
    grad = tr.logprobs_backward(x, _dev(tok, torch.int32), out[4], _dev(np.ones(5)), None)
    lp, H, step = tr.logprobs_step(x, _dev(tok, torch.int32), _dev(np.ones(5)))
    torch.cuda.synchronize()
    for d in (grad, step):
        assert torch.isfinite(d[0]).all() and torch.isnan(d[1:4]).all() and (d[4] == 0).all()
    assert torch.isnan(lp[1:4]).all() and torch.isnan(H[1:4]).all()


def test_rows_that_take_no_part_are_not_read():
    """Padding, and weights of 0, give zeros whatever the logits hold."""
    V = 700
    x = torch.full((4, V), float("nan"), device="cuda", dtype=torch.bfloat16)
    x[0] = torch.randn(V, device="cuda").to(torch.bfloat16)
    tok = torch.tensor([3, -1, 5, 6], dtype=torch.int32, device="cuda")
    tr = _train(V, "bf16")
    lp, H, grad = tr.logprobs_step(x, tok, _dev([1.0, 1.0, 0.0, 0.0]), _dev([0.5, 1.0, 0.0, 0.0]))
    assert (grad[1:] == 0).all() and (lp[1:] == 0).all() and (H[1:] == 0).all()
    lp, H, ids, alt, stats = tr.logprobs_forward(x, tok, alternatives=4, stats=True)
    assert lp[1] == 0 and H[1] == 0 and (ids[1] == -1).all() and (alt[1] == float("-inf")).all()
    assert torch.isnan(lp[2:]).all()
    grad = tr.logprobs_backward(x, tok, stats, _dev([1.0, 1.0, 0.0, 0.0]), _dev([0.0, 1.0, 0.0, 0.0]))
    assert (grad[1:] == 0).all() and torch.isfinite(grad[0]).all() and (grad[0] != 0).any()


def test_tokens_out_of_range():
    from speculative_decoding_draft_lm_gb300.rollout import DOMINO_ERR_BAD_TOKEN
    V = 500
    x = torch.randn(4, V, device="cuda")
    tr = _train(V, "fp32")
    for tok in ([0, V, 1, 2], [0, -2, 1, 2], [0, 2 ** 31 - 1, 1, 2]):
        t = torch.tensor(tok, dtype=torch.int32, device="cuda")
        lp, H, ids, alt = tr.logprobs_forward(x, t, alternatives=3)
        assert tr.status() == DOMINO_ERR_BAD_TOKEN and tr.status() == 0
        assert lp[1] == 0 and (ids[1] == -1).all() and (lp[[0, 2, 3]] < 0).all()
        lp, H, grad = tr.logprobs_step(x, t, torch.ones(4, device="cuda"))
        assert tr.status() == DOMINO_ERR_BAD_TOKEN
        assert (grad[1] == 0).all() and (grad[0] != 0).all()


def test_a_teachers_type_is_its_own():
    """The forward takes either type, whatever the context's."""
    g = np.random.default_rng(1)
    tok = g.integers(0, 900, 3).astype(np.int32)
    for ours, theirs in (("bf16", "fp32"), ("fp32", "bf16")):
        check_forward(_train(900, ours), rows(g.normal(0, 2, (3, 900)), TORCH[theirs], pad=1), tok, 1.0, 5)


@pytest.mark.parametrize("n", [1, 30, 1000])
def test_repeated_calls_and_graphs(n):
    """Equal bits on every call, on another stream and from a replayed graph; two graphs of one context in turn."""
    V = 20011
    tr = _train(V, "bf16")
    x = torch.randn(n, V, device="cuda").to(torch.bfloat16)
    tok = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    w = torch.randn(n, device="cuda")

    def calls(out):
        *out[:5], = tr.logprobs_forward(x, tok, 1.5, alternatives=20, stats=True)
        out[5] = tr.logprobs_backward(x, tok, out[4], w, w, 1.5)
        out[6:] = tr.logprobs_step(x, tok, w, w, 1.5)
        return out

    want = calls([None] * 6)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = calls([None] * 6)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(calls([None] * 6))
    for _ in range(3):
        for out in outs:
            for t in out:
                t.fill_(7)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in (again, *outs):
            for a, b in zip(want, out):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd(dtype):
    """The loss of a policy step with an entropy bonus, through torch; only one of the two used; neither."""
    from speculative_decoding_draft_lm_gb300.train import token_logprobs
    V, N, T = 700, 5, 1.5
    tr = _train(V, dtype)
    x = torch.randn(N, V, device="cuda").to(TORCH[dtype]).requires_grad_()
    tok = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    adv = torch.randn(N, device="cuda")
    lp, H, ids, alt = token_logprobs(tr, x, tok, T, alternatives=4)
    assert not ids.requires_grad and not alt.requires_grad
    (adv * lp + 0.1 * H).sum().backward()
    d = x.detach().double().requires_grad_()
    log_q = torch.log_softmax(d / T, 1)
    ref_lp, ref_H = log_q.gather(1, tok.long()[:, None])[:, 0], -(log_q.exp() * log_q).sum(1)
    (adv * ref_lp + 0.1 * ref_H).sum().backward()
    # the output's rounding, element by element, and 1e-5 of the row's largest for what was summed
    tol = OUT_EPS[TORCH[dtype]] * 1.01 * d.grad.abs() + 1e-5 * d.grad.abs().max(1, keepdim=True).values
    assert ((x.grad.double() - d.grad).abs() <= tol).all()
    for use in (0, 1):
        x.grad = d.grad = None
        token_logprobs(tr, x, tok, T)[use].sum().backward()
        log_q = torch.log_softmax(d / T, 1)
        (log_q.gather(1, tok.long()[:, None])[:, 0], -(log_q.exp() * log_q).sum(1))[use].sum().backward()
        tol = OUT_EPS[TORCH[dtype]] * 1.01 * d.grad.abs() + 1e-5 * d.grad.abs().max(1, keepdim=True).values
        assert ((x.grad.double() - d.grad).abs() <= tol).all()


def test_gradient_against_differences():
    """fp32 gradient of g logprob + h entropy against central differences of the oracle."""
    g = np.random.default_rng(2)
    V, T = 40, 0.75
    x = rows(g.normal(0, 1.5, (1, V)), torch.float32)
    tok, a, b = np.asarray([7], np.int32), 0.8, -0.6
    _, _, grad = _train(V, "fp32").logprobs_step(x, _dev(tok, torch.int32), _dev([a]), _dev([b]), T)
    v = wide(x)

    def value(u):
        lp, H, *_ = O.logprobs(u, tok, T)
        return a * lp[0] + b * H[0]

    eps = 1e-5
    for i in range(V):
        e = np.zeros_like(v)
        e[0, i] = eps
        slope = (value(v + e) - value(v - e)) / (2 * eps)
        # differences: eps^2 times third derivatives of about 1 / T^3, and 1e-16 / eps
        assert abs(slope - wide(grad)[0, i]) < 1e-9 + 20 * EPS32


def test_long_rows():
    """Rows that start beyond 2^31 elements, and the largest vocabulary."""
    V, N = 524288, 4100
    tr = _train(V, "bf16")
    x = torch.zeros(N, V, device="cuda", dtype=torch.bfloat16)
    x[N - 1] = torch.randn(V, device="cuda").to(torch.bfloat16)
    tok = torch.full((N,), -1, device="cuda", dtype=torch.int32)
    tok[N - 1] = V - 1
    lp, H, ids, alt, stats = tr.logprobs_forward(x, tok, alternatives=20, stats=True)
    want = torch.topk(x[N - 1].double(), 20)
    log_q = torch.log_softmax(x[N - 1].double(), 0)
    assert (lp[:-1] == 0).all() and abs(lp[-1].item() - log_q[-1].item()) < 1e-5
    assert torch.equal(x[N - 1].double()[ids[-1].long()], want.values)
    grad = tr.logprobs_backward(x, tok, stats, torch.ones(N, device="cuda"), out=x.new_full((N, V), 3.0))
    assert (grad[:-1] == 0).all() and (grad[N - 1] != 0).any()
    assert abs(grad[N - 1, V - 1].item() - (1 - log_q[-1].exp().item())) < 0.01
