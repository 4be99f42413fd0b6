"""Calls of the scores and the update that their interface allows: nothing to do,
explicit streams, the largest vocabulary, several captured graphs of one context,
buffers that are not aligned."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _train(V, dtype):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, dtype=dtype)


def _optim(*a, **kw):
    from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
    return DominoAdamW(*a, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows(dtype):
    tr = _train(100, "bf16" if dtype == torch.bfloat16 else "fp32")
    x, tok = torch.empty(0, 100, device="cuda", dtype=dtype), torch.empty(0, device="cuda", dtype=torch.int32)
    w = torch.empty(0, device="cuda")
    lp, H, ids, alt, stats = tr.logprobs_forward(x, tok, alternatives=5, stats=True)
    assert lp.shape == H.shape == (0,) and ids.shape == alt.shape == (0, 5) and stats.shape == (0, 4)
    assert tr.logprobs_backward(x, tok, stats, w).shape == (0, 100)
    assert tr.logprobs_step(x, tok, w, w)[2].shape == (0, 100)
    assert tr.last_launch_count() == 0 and tr.status() == 0


def test_refusals():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    V = 100
    tr = _train(V, "bf16")
    x = torch.randn(3, V, device="cuda").to(torch.bfloat16)
    tok, w = torch.zeros(3, device="cuda", dtype=torch.int32), torch.ones(3, device="cuda")
    *_, stats = tr.logprobs_forward(x, tok, stats=True)
    for call in (lambda: tr.logprobs_forward(x, tok, alternatives=33), lambda: tr.logprobs_forward(x, tok, alternatives=-1),
                 lambda: tr.logprobs_forward(x, tok, 0.0), lambda: tr.logprobs_forward(x, tok, float("nan")),
                 lambda: tr.logprobs_backward(x, tok, stats, None, None), lambda: tr.logprobs_step(x, tok, None, None),
                 lambda: tr.logprobs_backward(x, tok, stats, w, out=x), lambda: tr.logprobs_step(x, tok, w, temperature=2e3)):
        with pytest.raises(DominoError):
            call()
    small = _train(10, "bf16")
    with pytest.raises(DominoError):
        small.logprobs_forward(x[:, :10], tok, alternatives=11)
    for call in (lambda: tr.logprobs_forward(x.half(), tok), lambda: tr.logprobs_forward(x[:, :99], tok),
                 lambda: tr.logprobs_forward(x.t(), tok), lambda: tr.logprobs_forward(x, tok.long()),
                 lambda: tr.logprobs_forward(x, tok[:2]), lambda: tr.logprobs_forward(x, tok.cpu()),
                 lambda: tr.logprobs_forward(x, tok, stats=torch.empty(3, 3, device="cuda")),
                 lambda: tr.logprobs_forward(x, tok, alternatives=2, out=(w, w)),
                 lambda: tr.logprobs_backward(x.float(), tok, stats, w), lambda: tr.logprobs_backward(x, tok, stats[:2], w),
                 lambda: tr.logprobs_backward(x, tok, stats, w[:2]), lambda: tr.logprobs_step(x, tok, w.double()),
                 lambda: tr.logprobs_step(x, tok, w, out=(w, w, x.float()))):
        with pytest.raises(ValueError):
            call()
    assert tr.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 170])
def test_largest_vocabulary(dtype, N):
    V = 524288
    tr = _train(V, dtype)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (torch.randn(N, V, device="cuda") * 2).to(td)
    tok = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    w = torch.randn(N, device="cuda")
    lp, H, ids, alt, stats = tr.logprobs_forward(x, tok, alternatives=32, stats=True)
    lp2, H2, grad2 = tr.logprobs_step(x, tok, w, w)
    grad = tr.logprobs_backward(x, tok, stats, w, w)
    for n in (0, N - 1):
        order = torch.sort(x[n], descending=True, stable=True).indices[:32]
        assert torch.equal(ids[n].long(), order)
        log_q = torch.log_softmax(x[n].double(), 0)
        q = log_q.exp()
        entropy = -(q * log_q).sum()
        # sums of V / 128 additions in a row, log q of at most 30
        tol = (V / 128 + 60) * 2.0 ** -24 * 2 + 30 * 4 * 2.0 ** -24
        assert (alt[n].double() - log_q[order]).abs().max() < tol
        for a, b in ((lp, log_q[tok[n].long()]), (lp2, log_q[tok[n].long()])):
            assert abs(a[n].double() - b) < tol
        assert abs(H[n].double() - entropy) < tol * 15 and abs(H2[n].double() - entropy) < tol * 15
        hot = torch.zeros_like(q)
        hot[tok[n].long()] = 1
        want = w[n].double() * (hot - q) - w[n].double() * q * (log_q + entropy)
        rounding = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * 1.01
        for g in (grad, grad2):
            most = rounding * want.abs() + 30 * tol * w[n].abs() * (q * 20 + hot * 2.0 ** -20) + 1e-30
            assert ((g[n].double() - want).abs() <= most).all()


def test_explicit_streams():
    """A stream object and a raw handle, with outputs given."""
    V, N = 5000, 40
    tr = _train(V, "fp32")
    x = torch.randn(N, V, device="cuda")
    tok, w = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32), torch.randn(N, device="cuda")
    want = tr.logprobs_forward(x, tok, alternatives=4, stats=True)
    want_grad = tr.logprobs_step(x, tok, w, w)[2]
    p, q = torch.randn(5000, device="cuda"), None
    q = p.clone()
    g = torch.randn_like(p)
    a, b = _optim([p]), _optim([q])
    norm = a.grad_norm(1.0, grads=[g])
    a.step(grads=[g], scale=norm[1])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out = [torch.empty_like(t) for t in want]
        grad = torch.empty_like(x)
        more = [torch.empty(N, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        tr.logprobs_forward(x, tok, alternatives=4, stats=out[4], out=out[:4], stream=stream)
        tr.logprobs_step(x, tok, w, w, out=(*more, grad), stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, want)) and torch.equal(grad, want_grad)
        assert tr.status(stream=stream) == 0
    out = torch.empty((), device="cuda"), torch.empty((), device="cuda")
    torch.cuda.synchronize()
    b.grad_norm(1.0, grads=[g], out=out, stream=side)
    b.step(grads=[g], scale=out[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[0], norm[0]) and torch.equal(p, q)


@pytest.mark.parametrize("bits", [32, 8])
def test_two_graphs_of_one_optimizer(bits):
    """Each holds a norm and a step of gradients of its own; replayed in turn, with eager calls between."""
    torch.manual_seed(0)
    sizes = [40000, 77, 3001]
    start = [torch.randn(n, device="cuda").to(torch.bfloat16) for n in sizes]
    grads = [[torch.randn(n, device="cuda").to(torch.bfloat16) for n in sizes] for _ in range(2)]
    p, q = [t.clone() for t in start], [t.clone() for t in start]
    a, b = _optim(p, state_bits=bits), _optim(q, state_bits=bits)

    def step(opt, g):
        _, scale = opt.grad_norm(0.3, grads=g)
        opt.step(grads=g, scale=scale)

    step(b, grads[0])
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, g in zip(graphs, grads):
        with torch.cuda.graph(graph):
            step(b, g)
    step(a, grads[0])
    for turn in (0, 1, 1, 0, 1):
        graphs[turn].replay()
        step(a, grads[turn])
        if turn:
            step(a, grads[0])
            step(b, grads[0])
    torch.cuda.synchronize()
    assert a.steps() == b.steps()
    for s, t in zip((*p, *a.state.values()), (*q, *b.state.values())):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_state_buffers_that_are_not_aligned_are_refused():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    p = [torch.randn(256, device="cuda")]
    good = _optim(p, state_bits=8).state_dict()
    for name in ("m", "v"):
        buf = torch.zeros(256 + 64, device="cuda", dtype=torch.uint8)[16:272].view(torch.float8_e4m3fn)
        with pytest.raises(DominoError):
            _optim(p, state_bits=8, state=dict(good, **{name: buf}))


def test_the_same_gradient_for_two_parameters():
    p = [torch.randn(500, device="cuda"), torch.randn(500, device="cuda")]
    q = [t.clone() for t in p]
    g = torch.randn(500, device="cuda")
    a, b = _optim(p), _optim(q)
    a.step(grads=[g, g])
    b.step(grads=[g, g.clone()])
    assert all(torch.equal(s, t) for s, t in zip(p, q))
    assert abs(a.grad_norm(grads=[g, g])[0].item() - 2 ** 0.5 * g.double().norm().item()) < 1e-4


def test_gradients_of_any_container():
    p = [torch.randn(50, device="cuda"), torch.randn(60, device="cuda")]
    opt = _optim(iter(p))
    g = [torch.randn_like(t) for t in p]
    opt.step(grads=tuple(g))
    opt.step(grads=[g[0], None])
    for bad in ([g[0], 3.0], [g[0], g[1], g[1]], [g[0]]):
        with pytest.raises(ValueError, match="grads"):
            opt.step(grads=bad)
    with pytest.raises(TypeError):
        opt.step(grads=5)
    assert opt.steps() == 2


def test_parameters_of_a_module():
    """Leaves with gradients, several shapes, a bias, through a loss; a frozen one has none."""
    torch.manual_seed(1)
    m = torch.nn.Sequential(torch.nn.Linear(20, 33), torch.nn.SiLU(), torch.nn.Linear(33, 5)).cuda()
    m[0].bias.requires_grad_(False)
    start = [t.detach().double().clone() for t in m.parameters()]
    opt = _optim(m.parameters(), lr=1e-2, weight_decay=0.0)
    m(torch.randn(8, 20, device="cuda")).square().sum().backward()
    opt.step()
    for s, t in zip(start, m.parameters()):
        if t.grad is None:
            assert torch.equal(s, t.detach().double())
        else:
            # the first step moves every element by lr towards its gradient's other side
            want = s - 1e-2 * t.grad.double() / (t.grad.double().abs() + 1e-8)
            assert (t.detach().double() - want).abs().max() < 1e-2 * 64 * 2.0 ** -24 + 2.0 ** -24 * s.abs().max() * 2


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_but_empty_tensors(bits):
    p = [torch.zeros(0, device="cuda"), torch.zeros(3, 0, device="cuda")]
    opt = _optim(p, state_bits=bits)
    norm, scale = opt.grad_norm(grads=[torch.zeros_like(t) for t in p])
    opt.step(grads=[torch.zeros_like(t) for t in p], scale=scale)
    assert norm.item() == 0 and scale.item() == 1 and opt.steps() == 1
