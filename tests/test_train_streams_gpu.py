"""Table gradients of one context on several streams: they share its workspace,
so the library runs one after another."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

V, E, N = 60000, 256, 40000


def _inputs(count, n=N):
    g = np.random.default_rng(1)
    tok = [torch.as_tensor(np.minimum((g.random(n) ** 4 * V).astype(np.int32), V - 1)).cuda() for _ in range(count)]
    return tok, [torch.randn(n, E, device="cuda").to(torch.bfloat16) for _ in range(count)]


def _train(n=N):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    return DominoTrain(V, E=E, max_tokens=n, dtype="bf16")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [300, N, 140000])
def test_calls_on_two_streams(accumulate, n):
    tr = _train(n)
    tok, d = _inputs(2, n)
    want = [tr.embed_grad(d[k], tok[k], 2.0) for k in range(2)]
    got = [[torch.zeros(V, E, device="cuda") for _ in range(2)] for _ in range(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(6):
        for k in range(2):
            tr.embed_grad(d[k], tok[k], 2.0, out=got[turn][k], accumulate=accumulate, stream=streams[k])
    torch.cuda.synchronize()
    for turn in range(6):
        for k in range(2):
            assert torch.equal(got[turn][k], want[k])


def test_autograd_on_two_streams():
    """Autograd runs each backward on the stream of its forward."""
    from speculative_decoding_draft_lm_gb300.train import embedding
    tr = _train()
    tok, d = _inputs(2)
    W = torch.randn(V, E, device="cuda").to(torch.bfloat16).requires_grad_()
    want = [tr.embed_grad(d[k], tok[k], 1.0, grad_dtype=torch.bfloat16).float() for k in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        W.grad = None
        torch.cuda.synchronize()
        parts = []
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                parts.append((embedding(tr, W, tok[k]) * d[k]).sum(dtype=torch.float32))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        (parts[0] + parts[1]).backward()
        torch.cuda.synchronize()
        assert torch.equal(W.grad, (want[0] + want[1]).to(torch.bfloat16))


def test_two_streams_of_one_graph():
    tr = _train()
    tok, d = _inputs(2)
    want = [tr.embed_grad(d[k], tok[k], 2.0) for k in range(2)]
    out = [torch.empty(V, E, device="cuda") for _ in range(2)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        tr.embed_grad(d[0], tok[0], 2.0, out=out[0])
        tr.embed_grad(d[1], tok[1], 2.0, out=out[1], stream=side)
        main.wait_stream(side)
    for _ in range(3):
        for o in out:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    # ordinary calls after the capture, on another stream, and a second capture
    tr.embed_grad(d[1], tok[1], 2.0, out=out[0], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[1])
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again):
        tr.embed_grad(d[1], tok[1], 2.0, out=out[1])
    out[1].fill_(7.0)
    again.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1], want[1])


def test_a_stream_that_is_gone():
    """Contexts outlive streams: a call after its last one's stream was destroyed."""
    tr = _train()
    tok, d = _inputs(1)
    want = tr.embed_grad(d[0], tok[0])
    for _ in range(40):
        s = torch.cuda.Stream()
        out = torch.zeros(V, E, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        tr.embed_grad(d[0], tok[0], out=out, stream=s)
        s.synchronize()
        del s
        assert torch.equal(out, want)
