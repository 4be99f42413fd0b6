"""CPU pins of the training operators' oracle: torch's double-precision
autograd, finite differences and hand-made cases."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import train_oracle as O


def _case(seed, N=4, V=23, K=5, T=1.3):
    g = np.random.default_rng(seed)
    x = g.normal(0, 2, (N, V))
    ids = np.stack([g.permutation(V)[:K] for _ in range(N)]).astype(np.int32)
    return x, ids, g.normal(2, 2, (N, K)), g.normal(1, 1, N), T


@pytest.mark.parametrize("with_rest", [True, False])
def test_distill_matches_torch_kl(with_rest):
    """A distribution over K + 1 buckets: torch's kl_div and its autograd."""
    x, ids, top, rest, T = _case(0)
    N, V = x.shape
    rest = rest if with_rest else None
    loss, grad, _ = O.distill(x, ids, top, rest, T)
    for n in range(N):
        xt = torch.tensor(x[n], requires_grad=True)
        logq = torch.log_softmax(xt / T, 0)
        out = np.setdiff1d(np.arange(V), ids[n])
        q = torch.cat([logq[torch.tensor(ids[n]).long()], torch.logsumexp(logq[torch.tensor(out)], 0)[None]])
        t = np.append(top[n] / T, rest[n] if with_rest else -np.inf)
        p = torch.softmax(torch.tensor(t), 0)
        kl = torch.nn.functional.kl_div(q, p, reduction="sum")
        kl.backward()
        assert abs(kl.item() - loss[n]) < 1e-12
        np.testing.assert_allclose(grad[n], xt.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_distill_gradient_matches_differences():
    x, ids, top, rest, T = _case(1, N=2, V=9, K=3)
    _, grad, _ = O.distill(x, ids, top, rest, T)
    h = 1e-5
    for n in range(2):
        for v in range(9):
            xp, xm = x.copy(), x.copy()
            xp[n, v] += h
            xm[n, v] -= h
            d = (O.distill(xp, ids, top, rest, T)[0][n] - O.distill(xm, ids, top, rest, T)[0][n]) / (2 * h)
            assert abs(d - grad[n, v]) < 1e-8


def test_distill_full_record_is_plain_kl():
    """K = V without a rest: the usual divergence of two softmaxes; zero at the teacher."""
    x, _, _, _, T = _case(2, N=1, V=7)
    ids = np.arange(7, dtype=np.int32)[None]
    t = np.random.default_rng(3).normal(0, 1, (1, 7))
    loss, _, _ = O.distill(x, ids, t, None, T)
    lp, lq = torch.log_softmax(torch.tensor(t / T), 1), torch.log_softmax(torch.tensor(x / T), 1)
    assert abs(loss[0] - (lp.exp() * (lp - lq)).sum().item()) < 1e-12
    loss, grad, _ = O.distill(t, ids, t, None, T)
    assert abs(loss[0]) < 1e-12 and np.abs(grad).max() < 1e-12


def test_distill_record_of_the_student_itself_is_zero():
    """Record and rest taken from the student's own logits: loss and gradient 0."""
    x, _, _, _, T = _case(4, N=3, V=50)
    ids, top, rest = O.top_logits(x, 8, T)
    loss, grad, _ = O.distill(x, ids, top, rest, T)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12


def test_distill_padding_repeats_and_empty_rows():
    x, ids, top, rest, T = _case(5, N=1, V=11, K=4)
    a = O.distill(x, ids, top, rest, T)
    more = np.array([[ids[0, 0], -1, ids[0, 1], ids[0, 0], ids[0, 2], 99, ids[0, 3]]], dtype=np.int32)
    tops = np.array([[top[0, 0], 5.0, top[0, 1], 7.0, top[0, 2], 1.0, top[0, 3]]])
    b = O.distill(x, more, tops, rest, T)
    assert abs(a[0][0] - b[0][0]) < 1e-12
    np.testing.assert_allclose(a[1], b[1], atol=1e-14)
    empty = np.full((1, 3), -1, dtype=np.int32)
    loss, grad, _ = O.distill(x, empty, np.zeros((1, 3)), None, T)
    assert loss[0] == 0 and not grad.any()


def test_top_logits_small_cases():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 3.0, 0.0], [np.nan, 1.0, np.inf, 1.0, -0.0, 0.0]])
    ids, top, rest = O.top_logits(x, 2, 1.0)
    assert ids.tolist() == [[1, 2], [0, 2]]
    assert top[0].tolist() == [3.0, 3.0]
    assert abs(rest[0] - np.log(np.exp(1) + np.exp(3) + 1)) < 1e-12
    ids, _, _ = O.top_logits(x, 5, 1.0)
    assert ids.tolist() == [[0, 1, 2, 4, 5], [0, 1, 2, 3, 4]]  # the tied zeros: the lower id
    _, _, rest = O.top_logits(x[:1], 6, 1.0)
    assert rest[0] == -np.inf


def test_embed_grad_is_the_transpose_of_embed():
    g = np.random.default_rng(6)
    V, E, N = 13, 5, 40
    tok = g.integers(-1, V + 1, N).astype(np.int32)
    W, d = g.normal(size=(V, E)), g.normal(size=(N, E))
    y = O.embed(W, tok, 1.7)
    dW, _, count = O.embed_grad(d, tok, V, 1.7)
    assert abs((y * d).sum() - (W * dW).sum()) < 1e-10
    assert count.sum() == ((tok >= 0) & (tok < V)).sum()
    t = torch.tensor(W, requires_grad=True)
    ok = (tok >= 0) & (tok < V)
    (torch.nn.functional.embedding(torch.tensor(tok[ok]).long(), t) * 1.7 * torch.tensor(d[ok])).sum().backward()
    np.testing.assert_allclose(dW, t.grad.numpy(), atol=1e-12)
