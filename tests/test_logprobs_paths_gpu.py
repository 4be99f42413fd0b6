"""Alternatives and sums where the kernels take another way: few places hold all
allowed ids, whole warps' places are poor, rows for one CTA each."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _train(V, dtype):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, dtype=dtype)


def check(x, k, T=1.0):
    """Ids by a stable sort, scores and entropies in 64 bits, on the GPU."""
    N, V = x.shape
    tr = _train(V, "bf16" if x.dtype == torch.bfloat16 else "fp32")
    tok = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    lp, H, ids, alt = tr.logprobs_forward(x, tok, T, alternatives=k)
    for n in range(N):
        row = x[n].double()
        order = torch.sort(x[n], descending=True, stable=True).indices[:k]
        real = x[n][order] > float("-inf")
        assert torch.equal(ids[n].long(), torch.where(real, order, -1)), n
        q = torch.softmax(row / T, 0)
        log_q = torch.log_softmax(row / T, 0)
        want = torch.where(real, log_q[order], float("-inf"))
        # the sum (V / 128 sequential additions and an exponential of 2 ulp), its logarithm, and d's two roundings
        tol = (V / 128 + 60) * 2.0 ** -24 + 4 * 2.0 ** -24 * log_q[order].abs().nan_to_num(posinf=0.0)
        assert ((alt[n].double() == want) | ((alt[n].double() - want).abs() <= tol)).all(), n
        entropy = -torch.special.xlogy(q, q).sum()
        assert abs(H[n].double() - entropy) <= (V / 128 + 60) * 2.0 ** -24 * (2 + 2 * entropy), n
        # the token's is d - log s like the alternatives': two roundings of d, on whose size (6e30 for some rows) they
        # lie, and the difference's
        said = log_q[tok[n].long()]
        tol = (V / 128 + 60) * 2.0 ** -24 + 4 * 2.0 ** -24 * said.abs()
        assert lp[n].double() == said or abs(lp[n].double() - said) <= tol, n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 160])  # rows spread over a cluster, and one CTA each
@pytest.mark.parametrize("k", [1, 8, 32])
def test_allowed_ids_in_few_places(dtype, N, k):
    V = 151936 if dtype == "bf16" else 80000
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.full((N, V), float("-inf"), device="cuda")
    for n in range(N):
        first = (n * 977) % (V - 3000)
        width = [3, 40, 700, 2500][n % 4]
        x[n, first:first + width] = torch.randn(width, device="cuda", generator=g)
    check(x.to(TORCH[dtype]), k)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 160])
@pytest.mark.parametrize("warp", [0, 7])
def test_a_warps_places_are_poor(dtype, N, warp):
    """64-byte groups go to the threads in turn: one warp's all lie far below the others'."""
    V = 151936 if dtype == "bf16" else 80000
    per = 32 if dtype == "bf16" else 16
    x = torch.randn(N, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) + 10
    place = torch.arange(V, device="cuda") // per % 256 // 32
    x[:, place == warp] -= 50
    check(x.to(TORCH[dtype]), 20)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [0.0, -3.5, 7.0])
@pytest.mark.parametrize("N", [1, 200])
def test_equal_logits_everywhere(dtype, value, N):
    """Ties go by the id: the first ones, also among many equal best below a few better."""
    V = 20011
    x = torch.full((N, V), value, device="cuda")
    x[:, 19000] = value + 1
    x[:, 5] = value - 1
    check(x.to(TORCH[dtype]), 32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [32, 100, 1000, 5000])
def test_rows_of_one_cta(dtype, V):
    """As many rows as there are SMs and more, short ones, in every state: masked in part and whole, by the type's
    lowest value, far values, ties; the rows start anywhere modulo 16 bytes."""
    N = 400
    g = torch.Generator(device="cuda").manual_seed(V)
    buf = torch.full((N * (V + 5) + 3,), float("nan"), device="cuda", dtype=TORCH[dtype])
    x = buf[3:].view(N, V + 5)[:, :V]
    x.copy_(torch.randn(N, V, device="cuda", generator=g) * 3)
    low = torch.finfo(TORCH[dtype]).min
    x[0::10, : V // 2] = float("-inf")
    x[1::10, 1:] = float("-inf")
    x[2::10] = low
    x[3::10, V // 3:] = low
    x[4::10] += 1e4
    x[5::10] = x[5::10].round()
    x[6::10] *= 1e30
    x[7::10, ::2] = float("-inf")
    check(x, min(V, 32))
    empty = torch.full((N, V), float("-inf"), device="cuda", dtype=TORCH[dtype])
    tr = _train(V, dtype)
    tok = torch.zeros(N, device="cuda", dtype=torch.int32)
    lp, H, ids, alt = tr.logprobs_forward(empty, tok, alternatives=5)
    assert (lp == float("-inf")).all() and (H == 0).all() and (ids == -1).all() and (alt == float("-inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_step_takes_many_rows_in_turn(dtype):
    """More rows than clusters fit the GPU, rows that take no part between them, against forward and backward."""
    V, N = 9001, 3000
    tr = _train(V, dtype)
    x = (torch.randn(N, V, device="cuda") * 2).to(TORCH[dtype])
    x[::7, :4000] = float("-inf")
    x[5] = float("-inf")
    tok = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    tok[::11] = -1
    w, h = torch.randn(N, device="cuda"), torch.rand(N, device="cuda")
    w[::13] = h[::13] = 0
    lp, H, grad = tr.logprobs_step(x, tok, w, h, 1.5)
    lp2, H2, stats = tr.logprobs_forward(x, tok, 1.5, stats=True)
    grad2 = tr.logprobs_backward(x, tok, stats, w, h, 1.5)
    off = torch.zeros(N, dtype=torch.bool, device="cuda")
    off[::13] = True
    assert (lp[off] == 0).all() and (H[off] == 0).all()
    # two orders of the sums: each within the sum's error of the exact one
    for a, b in ((lp, lp2), (H, H2)):
        same = (a == b) | ((a - b).abs() <= 4 * (V / 128 + 60) * 2.0 ** -24 * (1 + b.abs()))
        assert same[~off].all()
    a, b = grad.float(), grad2.float()
    rounding = 2.0 ** -7 if dtype == "bf16" else 0.0  # a step of bf16, where the two fall on its two sides
    tol = rounding * b.abs() + 4 * (V / 128 + 60) * 2.0 ** -24 * b.abs().amax(1, keepdim=True)
    assert ((a - b).abs() <= tol).all()
    assert tr.status() == 0
