"""Scaled embedding lookup and its gradient against the fp64 oracle."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, OUT_EPS, TORCH, rows, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _train(V, E, n=0, dtype="bf16"):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, E=E, max_tokens=n, dtype=dtype)


def _tok(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _tokens(g, kind, n, V):
    return {"uniform": lambda: g.integers(0, V, n), "one": lambda: np.full(n, V - 1),
            "frequent": lambda: np.minimum((g.random(n) ** 8 * V).astype(np.int64), V - 1) * 37 % V,
            "sorted": lambda: np.sort(g.integers(0, V, n)), "two": lambda: np.where(np.arange(n) % 2 == 0, 0, V - 1),
            "padded": lambda: np.where(g.random(n) < 0.4, -1, g.integers(0, V, n)),
            "none": lambda: np.full(n, -1)}[kind]().astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V,E,pad,shift", [(1, 2, 1, 0, 0), (3, 10, 7, 0, 0), (16, 1000, 40, 0, 0), (5, 100, 1024, 8, 8),
                                             (33, 500, 1536, 0, 1), (7, 300, 129, 3, 2), (300, 4096, 128, 0, 0)])
def test_embed(dtype, n, V, E, pad, shift):
    g = np.random.default_rng(n + E)
    W = rows(g.normal(0, 0.02, (V, E)), TORCH[dtype], 0, 0)
    tok = _tokens(g, "padded", n, V)
    tr = _train(V, E, dtype=dtype)
    out = rows(np.full((n, E), 7.0), TORCH[dtype], pad, shift)
    tr.embed(W, _tok(tok), 3.7, out=out)
    torch.cuda.synchronize()
    want = O.embed(wide(W), tok, float(np.float32(3.7)))
    assert (np.abs(wide(out) - want) <= (OUT_EPS[TORCH[dtype]] * 1.01 + 2 * EPS32) * np.abs(want)).all()
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_embed_unaligned_table(dtype):
    g = np.random.default_rng(0)
    V, E, n = 50, 64, 20
    W = rows(g.normal(0, 1, (V, E)), TORCH[dtype], 0, 1)
    tok = _tokens(g, "uniform", n, V)
    out = _train(V, E, dtype=dtype).embed(W, _tok(tok), 1.0)
    assert torch.equal(out, W[_tok(tok).long()])


def check_grad(n, V, E, kind, dtype, gdtype, accumulate=False, pad=0, shift=0, seed=0):
    g = np.random.default_rng(seed + n + E)
    d = rows(g.normal(0, 1, (n, E)), TORCH[dtype], pad, shift)
    tok = _tokens(g, kind, n, V)
    tr = _train(V, E, max(n, 1), dtype)
    start = g.normal(0, 1, (V, E))
    out = rows(start, TORCH[gdtype])
    before = wide(out)
    scale = float(np.float32(0.3))
    tr.embed_grad(d, _tok(tok), scale, out=out, accumulate=accumulate)
    torch.cuda.synchronize()
    want, terms, count = O.embed_grad(wide(d), tok, V, scale)
    if accumulate:
        want, terms = want + before, terms + np.abs(before)
        assert (wide(out)[count == 0] == before[count == 0]).all()
    else:
        assert (wide(out)[count == 0] == 0).all()
    tol = (count[:, None] + 3) * EPS32 * terms + OUT_EPS[TORCH[gdtype]] * 1.01 * np.abs(want)
    assert (np.abs(wide(out) - want) <= tol).all()
    assert tr.status() == 0
    return d, tok, tr, scale, out


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,V,E,kind", [(1, 2, 1, "uniform"), (3, 10, 7, "one"), (16, 1000, 40, "uniform"),
                                        (100, 1000, 129, "frequent"), (700, 50, 64, "padded"), (513, 300, 72, "sorted"),
                                        (64, 100, 1024, "two"), (40, 64, 33, "none")])
def test_embed_grad(dtype, gdtype, accumulate, n, V, E, kind):
    check_grad(n, V, E, kind, dtype, gdtype, accumulate)


@pytest.mark.parametrize("n", [4095, 4096, 4097, 9000, 20000])
@pytest.mark.parametrize("kind", ["uniform", "frequent", "one", "two"])
def test_embed_grad_many_tokens(n, kind):
    check_grad(n, 3000, 24, kind, "bf16", "fp32")


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16385, 40000, 131072, 131073, 140001])
@pytest.mark.parametrize("kind", ["uniform", "frequent", "padded"])
def test_embed_grad_tile_edges(n, kind):
    """Token counts at and beside the sort's tiles and the most that one cluster sorts."""
    check_grad(n, 5000, 8, kind, "bf16", "fp32")


@pytest.mark.parametrize("V", [2, 3, 255, 256, 257, 1023, 1024, 1025, 65535, 65536, 151936, 524288])
def test_embed_grad_vocabulary_edges(V):
    """The sort's digits: vocabularies at and beside powers of two, first and last ids."""
    n, E = 300, 8
    g = np.random.default_rng(V)
    tok = np.concatenate([[0, V - 1, V - 1, 0, -1], g.integers(0, V, n - 5)]).astype(np.int32)
    d = rows(g.normal(0, 1, (n, E)), torch.float32)
    tr = _train(V, E, n, "fp32")
    out = tr.embed_grad(d, _tok(tok), 1.0)
    want, terms, count = O.embed_grad(wide(d), tok, V, 1.0)
    assert (np.abs(wide(out) - want) <= (count[:, None] + 3) * EPS32 * terms).all()


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_embed_grad_strides(pad, shift, dtype):
    check_grad(200, 90, 136, "frequent", dtype, "fp32", pad=pad, shift=shift)


def test_embed_grad_unaligned_table():
    g = np.random.default_rng(3)
    V, E, n = 40, 24, 100
    tok = _tokens(g, "uniform", n, V)
    d = rows(g.normal(0, 1, (n, E)), torch.bfloat16)
    out = rows(np.full((V, E), 7.0), torch.float32, 0, 1)
    _train(V, E, n).embed_grad(d, _tok(tok), 1.0, out=out)
    want, terms, count = O.embed_grad(wide(d), tok, V, 1.0)
    assert (np.abs(wide(out) - want) <= (count[:, None] + 3) * EPS32 * terms).all()


def test_embed_grad_nan_stays_in_its_row():
    g = np.random.default_rng(4)
    V, E, n = 30, 16, 50
    tok = np.arange(n, dtype=np.int32) % 20
    dv = g.normal(0, 1, (n, E))
    dv[3] = np.nan
    tok[7] = -1
    dv[7] = np.nan  # a padding position's gradient is not read
    out = wide(_train(V, E, n).embed_grad(rows(dv, torch.bfloat16), _tok(tok), 1.0))
    assert np.isnan(out[3]).all()
    assert np.isfinite(np.delete(out, 3, 0)).all()


def test_repeated_calls_sizes_and_streams():
    """One context over calls of several sizes; equal bits on a second stream and in a graph."""
    g = np.random.default_rng(5)
    V, E, n = 500, 96, 9000
    tr = _train(V, E, n)
    for m in (9000, 1, 0, 4097, 30):
        tok = _tok(_tokens(g, "frequent", m, V))
        d = rows(g.normal(0, 1, (m, E)), torch.bfloat16) if m else torch.empty(0, E, dtype=torch.bfloat16, device="cuda")
        a = tr.embed_grad(d, tok, 2.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            b = tr.embed_grad(d, tok, 2.0)
        s.synchronize()
        assert torch.equal(a, b)
        want, terms, count = O.embed_grad(wide(d), tok.cpu().numpy(), V, 2.0)
        assert (np.abs(wide(a) - want) <= (count[:, None] + 3) * EPS32 * terms).all()
    tok, d = _tok(_tokens(g, "frequent", n, V)), rows(g.normal(0, 1, (n, E)), torch.bfloat16)
    a, b = tr.embed_grad(d, tok), torch.empty(V, E, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.embed_grad(d, tok, out=b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_table_beyond_32_bit_offsets():
    V, E, n = 300000, 8192, 64  # 2.4 G elements
    g = np.random.default_rng(6)
    tok = np.concatenate([[V - 1, V - 2, 0, V - 1], g.integers(V - 1000, V, n - 4)]).astype(np.int32)
    tr = _train(V, E, n)
    W = torch.zeros(V, E, dtype=torch.bfloat16, device="cuda")
    W[V - 1000:] = torch.randn(1000, E, device="cuda").to(torch.bfloat16)
    out = tr.embed(W, _tok(tok), 1.0)
    assert torch.equal(out, W[_tok(tok).long()])
    d = torch.randn(n, E, device="cuda").to(torch.bfloat16)
    dW = tr.embed_grad(d, _tok(tok), 1.0, grad_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    ref = torch.zeros(1000, E, dtype=torch.float64, device="cuda")
    late = _tok(tok).long() >= V - 1000
    ref.index_add_(0, _tok(tok).long()[late] - (V - 1000), d[late].double())
    assert ((dW[V - 1000:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5).all()
    assert not dW[1:V - 1000].any()


def test_bad_tokens_are_reported_and_ignored():
    from speculative_decoding_draft_lm_gb300 import rollout as R
    V, E = 20, 8
    tr = _train(V, E, 4, "fp32")
    W = torch.ones(V, E, device="cuda")
    tok = _tok([3, 20, -5, 2 ** 31 - 1])
    out = tr.embed(W, tok)
    assert tr.status() == R.DOMINO_ERR_BAD_TOKEN and tr.status() == 0
    assert (out[0] == 1).all() and (out[1:] == 0).all()
    g = tr.embed_grad(torch.ones(4, E, device="cuda"), tok)
    assert tr.status() == R.DOMINO_ERR_BAD_TOKEN
    assert (g[3] == 1).all() and g.sum() == E
    tr.embed(W, _tok([-1, 2]))
    assert tr.status() == 0


def test_gradient_is_the_transpose_of_the_lookup():
    """<embed(W), d> = <W, embed_grad(d)>, and differences of the lookup along one weight."""
    g = np.random.default_rng(7)
    V, E, n, h = 60, 16, 200, 0.5
    tr = _train(V, E, n, "fp32")
    W, d = rows(g.normal(0, 1, (V, E)), torch.float32), rows(g.normal(0, 1, (n, E)), torch.float32)
    tok = _tok(_tokens(g, "frequent", n, V))
    dW = tr.embed_grad(d, tok, 1.5)
    a, b = (tr.embed(W, tok, 1.5).double() * d.double()).sum(), (W.double() * dW.double()).sum()
    assert abs(a - b) <= 1e-4
    v, e = int(tok[0]), 5
    up, dn = W.clone(), W.clone()
    up[v, e] += h
    dn[v, e] -= h
    slope = ((tr.embed(up, tok, 1.5).double() - tr.embed(dn, tok, 1.5).double()) * d.double()).sum() / (2 * h)
    assert abs(slope - dW[v, e].double()) <= 1e-4


def test_autograd_function():
    from speculative_decoding_draft_lm_gb300.train import embedding
    V, E, n = 30, 12, 40
    tr = _train(V, E, n, "fp32")
    W = torch.randn(V, E, device="cuda", requires_grad=True)
    tok = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    y = embedding(tr, W, tok, 2.0)
    (y ** 2).sum().backward()
    W2 = W.detach().clone().requires_grad_()
    ((2.0 * W2[tok.long()]) ** 2).sum().backward()
    torch.testing.assert_close(W.grad, W2.grad, rtol=1e-5, atol=1e-4)


def test_refusals():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    V, E, n = 20, 8, 6
    tr = _train(V, E, n, "fp32")
    W, tok, d = torch.zeros(V, E, device="cuda"), _tok([0] * n), torch.zeros(n, E, device="cuda")
    for bad in (W[:-1], W.double(), W.cpu(), W.t(), torch.zeros(V, 2 * E, device="cuda")[:, :E]):
        with pytest.raises(ValueError):
            tr.embed(bad, tok)
    with pytest.raises(ValueError):
        tr.embed(W, tok.long())
    with pytest.raises(ValueError):
        tr.embed_grad(d[:-1], tok)
    with pytest.raises(ValueError):
        tr.embed_grad(d, tok, accumulate=True)
    with pytest.raises(ValueError):
        tr.embed_grad(d, tok, out=torch.zeros(V, E, device="cuda", dtype=torch.float16))
    with pytest.raises(DominoError):  # more than max_tokens
        tr.embed_grad(torch.zeros(n + 1, E, device="cuda"), _tok([0] * (n + 1)))
    with pytest.raises(DominoError):  # no embedding in this context
        _train(V, 0, n, "fp32").embed(torch.zeros(V, 0, device="cuda"), tok)
    assert tr.embed(W, tok[:0]).shape == (0, E)
