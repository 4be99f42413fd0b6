"""Record of a teacher's logits against the fp64 oracle: ids and logits equal,
the rest within the sums' rounding."""
import numpy as np
import pytest

from oracle import train_oracle as O
from train_helpers import EPS32, TORCH, rows, sum_error, wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _train(V, **kw):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, **kw)


def check(x, K, T, got=None, tr=None):
    """x: device rows [N, V]."""
    tr = tr or _train(x.shape[1])
    ids, top, rest = got or tr.top_logits(x, K, T)
    torch.cuda.synchronize()
    xw = wide(x)
    oi, ot, orest = O.top_logits(xw, K, T)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    np.testing.assert_array_equal(wide(top) + 0.0, ot + 0.0)
    r = wide(rest)
    bad = ~np.isfinite(orest)
    np.testing.assert_array_equal(r[bad], orest[bad])
    m = np.abs(xw[np.isfinite(xw)]).max(initial=0.0) / T
    tol = 2 * sum_error(x.shape[1]) + 4 * EPS32 * (np.abs(orest[~bad]) + min(m, 1e3))
    d = np.abs(r[~bad] - orest[~bad])
    assert (d <= tol).all(), (d.max(), tol.min())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,K", [(1, 2, 1), (1, 2, 2), (3, 31, 7), (2, 33, 33), (5, 1000, 1), (4, 1001, 100),
                                   (3, 4097, 2048), (2, 9000, 8192), (2, 20011, 64), (1, 151936, 64),
                                   (2, 151935, 2048)])
def test_random_rows(dtype, N, V, K):
    g = np.random.default_rng(N + V + K)
    check(rows(g.normal(0, 2, (N, V)), TORCH[dtype]), K, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (16, 2)])
def test_strides_and_alignment(dtype, pad, shift):
    g = np.random.default_rng(pad * 10 + shift)
    check(rows(g.normal(0, 2, (7, 2503)), TORCH[dtype], pad, shift), 40, 0.7)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["equal", "two_values", "ascending", "descending", "one_spike", "zeros", "blocks"])
@pytest.mark.parametrize("K", [1, 64, 700])
def test_ties_and_orders(dtype, kind, K):
    V = 6007
    g = np.random.default_rng(K)
    x = {"equal": np.full(V, 1.5), "two_values": g.integers(0, 2, V) * 1.0, "ascending": np.arange(V) / 64.0,
         "descending": -np.arange(V) / 64.0, "one_spike": np.where(np.arange(V) == 4321, 100.0, 0.0),
         "zeros": np.where(g.random(V) < 0.5, 0.0, -0.0),
         "blocks": np.floor(np.arange(V) / 1000.0)}[kind]
    check(rows(np.stack([x, x[::-1]]), TORCH[dtype]), K, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks_infinities_and_nan(dtype):
    V, K = 3001, 50
    g = np.random.default_rng(1)
    lowest = float(torch.finfo(TORCH[dtype]).min)
    x = g.normal(0, 2, (9, V))
    x[0, 40:] = -np.inf                   # fewer finite logits than K
    x[1, :] = -np.inf                     # nothing left
    x[2, :] = lowest
    x[3, 7:] = lowest
    x[4, [5, 17]] = np.inf
    x[5, [100, 3]] = np.nan
    x[6, : V // 2] = np.nan               # more than K
    x[7, 200:400] = np.inf                # more than K
    x[8, ::2] = -np.inf
    t = rows(x, TORCH[dtype])
    ids, top, rest = _train(V).top_logits(t, K, 1.0)
    torch.cuda.synchronize()
    oi, ot, orest = O.top_logits(wide(t), K, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    np.testing.assert_array_equal(wide(top), ot)
    r = wide(rest)
    for n in range(9):
        if np.isfinite(orest[n]):
            tol = 2 * sum_error(V) + 8 * EPS32 * abs(orest[n])
            assert abs(r[n] - orest[n]) <= tol, n
        else:
            np.testing.assert_array_equal(r[n], orest[n])


def test_rest_of_a_peaked_row_is_not_a_difference():
    """The others hold e^-60 of the mass: far below the whole's rounding."""
    g = np.random.default_rng(2)
    x = g.normal(0, 1, (2, 5000))
    x[:, [3, 4000]] += 60.0
    check(rows(x, torch.float32), 2, 1.0)


def test_temperatures_and_no_rows():
    g = np.random.default_rng(3)
    x = rows(g.normal(0, 2, (3, 1000)), torch.float32)
    tr = _train(1000)
    for T in (1e-3, 0.1, 3.0, 1e3):
        check(x, 10, T, tr=tr)
    ids, top, rest = tr.top_logits(x[:0], 10)
    assert ids.shape == (0, 10) and rest.shape == (0,)
    assert tr.status() == 0


def test_many_rows_repeat_bits_and_other_streams():
    g = np.random.default_rng(4)
    x = rows(g.normal(0, 2, (700, 3000)), torch.bfloat16)
    tr = _train(3000)
    a = tr.top_logits(x, 33, 2.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = tr.top_logits(x, 33, 2.0)
    s.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    check(x[::97].contiguous(), 33, 2.0)


def test_rows_beyond_32_bit_offsets():
    V, ld, N = 1003, 2 ** 30 + 7, 3  # the last row starts 4 GiB in
    g = np.random.default_rng(5)
    buf = torch.empty(ld * (N - 1) + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((N, V), (ld, 1))
    x.copy_(torch.as_tensor(g.normal(0, 2, (N, V))).to(torch.bfloat16))
    check(x, 20, 1.0)


def test_refusals():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    tr = _train(100)
    x = torch.zeros(4, 100, device="cuda")
    for K in (0, -1, 101):
        with pytest.raises((DominoError, ValueError, RuntimeError)):
            tr.top_logits(x, K)
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-4):
        with pytest.raises(DominoError):
            tr.top_logits(x, 3, T)
    for bad in (x[:, :99], x.double(), x.cpu(), x.t(), x[0], torch.zeros(4, 200, device="cuda")[:, ::2],
                x[:1].expand(4, 100)):
        with pytest.raises(ValueError):
            tr.top_logits(bad, 3)
    with pytest.raises(ValueError):
        tr.top_logits(x, 3, out=(torch.empty(4, 3, device="cuda", dtype=torch.int64), torch.empty(4, 3, device="cuda"),
                                 torch.empty(4, device="cuda")))
    with pytest.raises(DominoError):
        _train(100000).top_logits(torch.zeros(1, 100000, device="cuda"), 8193)
    with pytest.raises(ValueError):
        _train(100, dtype="fp16")
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [5, 64, 300, 700])
def test_ties_at_every_level(dtype, K):
    """Few distinct logits, of either sign, so that the cut falls inside large
    groups of equal ones; and masks that leave whole slices of a row empty."""
    g = np.random.default_rng(K)
    V = 40000
    x = np.stack([g.integers(-3, 4, V) * 1.0, -g.integers(1, 4, V) * 0.5, np.where(g.random(V) < 0.01, 2.0, -1.5),
                  np.where(g.random(V) < 0.9, -np.inf, g.normal(0, 1, V)), np.where(np.arange(V) < 39000, -np.inf, 1.0),
                  np.where(np.arange(V) > 200, -np.inf, g.normal(0, 1, V)), np.full(V, -np.inf),
                  np.where(g.random(V) < 0.5, np.nan, 3.0)])
    for rows_at_once in (x, x[4:5]):  # one CTA a row or a few, and a cluster a row
        check(rows(rows_at_once, TORCH[dtype], 1), K, 1.0)
        check(rows(rows_at_once, TORCH[dtype], 0), K, 1.0)
    check(rows(np.repeat(x, 60, 0), TORCH[dtype], 3), K, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_clustered_candidates(dtype):
    """The best logits all in one place, or all a vector apart: more words than the buffer holds."""
    g = np.random.default_rng(9)
    V = 70001
    a, b = g.normal(0, 1, V), g.normal(0, 1, V)
    a[30000:36000] += 20.0
    b[::8] += 20.0
    x = np.stack([a, b, np.sort(a), -np.sort(a)])
    for K in (1, 50, 400, 3000):
        check(rows(x, TORCH[dtype]), K, 1.0)
    check(rows(np.repeat(x, 100, 0), TORCH[dtype]), 50, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,K", [(19, 12064, 1888), (400, 9001, 380), (400, 12063, 4000), (3, 30000, 8192), (700, 2500, 700)])
def test_records_of_much_of_a_row(dtype, N, V, K):
    """K near the number of vectors, or above it; plain rows, few distinct logits, masked ones and sorted ones."""
    g = np.random.default_rng(V + K)
    x = g.normal(0, 2, (N, V))
    x[1 % N] = g.integers(-2, 3, V)
    x[2 % N, K // 2:] = -np.inf
    x[0] = np.sort(x[0])
    check(rows(x, TORCH[dtype], 3, 1), K, 1.0)


@pytest.mark.parametrize("K", [1, 64, 700, 8192])
def test_rows_longer_than_a_block_holds(K):
    """fp32 rows whose groups are spread over several blocks: ties, masks that leave slices empty, all in one slice."""
    V = 500003
    g = np.random.default_rng(K)
    x = np.stack([g.normal(0, 2, V), g.integers(-3, 4, V) * 1.0, np.where(np.arange(V) < V - 100, -np.inf, 1.0),
                  np.where(np.arange(V) > 9000, -np.inf, g.normal(0, 1, V)), np.full(V, -np.inf), np.sort(g.normal(0, 1, V)),
                  np.where(g.random(V) < 0.01, np.nan, 3.0)])
    check(rows(x, torch.float32, 1), K, 1.0)
