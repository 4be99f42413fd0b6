"""The device error word: read and cleared in the order of the caller's stream."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _tok(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def test_status_waits_for_its_own_stream_only():
    """Work on the default stream (a spin of about half a second) neither delays status() nor is waited for."""
    from speculative_decoding_draft_lm_gb300 import rollout as R
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    tr = DominoTrain(20, E=8, dtype="fp32")
    W, bad, side = torch.ones(20, 8, device="cuda"), _tok([3, 20]), torch.cuda.Stream()
    with torch.cuda.stream(side):  # a kernel's first launch loads it, which may wait for the device
        tr.embed(W, bad)
        assert tr.status() == R.DOMINO_ERR_BAD_TOKEN
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    busy = torch.cuda.Event()
    busy.record()
    with torch.cuda.stream(side):
        tr.embed(W, bad)
        assert tr.status() == R.DOMINO_ERR_BAD_TOKEN
        assert tr.status() == 0
    assert not busy.query()
    torch.cuda.synchronize()


def test_an_error_right_after_a_cleared_one_is_kept():
    from speculative_decoding_draft_lm_gb300 import rollout as R
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    tr = DominoTrain(20, E=8, dtype="fp32")
    W, bad, good, side = torch.ones(20, 8, device="cuda"), _tok([3, 20]), _tok([3, -1]), torch.cuda.Stream()
    out = torch.empty(2, 8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            tr.embed(W, bad, out=out)
            assert tr.status() == R.DOMINO_ERR_BAD_TOKEN
        tr.embed(W, good, out=out)
        assert tr.status() == 0


def test_launch_count_is_the_last_successful_calls():
    from speculative_decoding_draft_lm_gb300.rollout import DominoError
    from speculative_decoding_draft_lm_gb300.train import DominoTrain
    V, E = 50, 8
    tr = DominoTrain(V, E=E, max_tokens=4, dtype="fp32")
    x, W, tok = torch.randn(3, V, device="cuda"), torch.ones(V, E, device="cuda"), _tok([1, 2, 1])
    w, d = torch.ones(3, device="cuda"), torch.ones(3, E, device="cuda")
    ids, top, rest = tr.top_logits(x, 2)
    loss, stats = tr.distill_forward(x, ids, top, rest)
    out, table = torch.empty(3, E, device="cuda"), torch.zeros(V, E, device="cuda")
    calls = [lambda: tr.top_logits(x, 2), lambda: tr.distill_forward(x, ids, top, rest),
             lambda: tr.distill_backward(x, ids, top, rest, stats, w), lambda: tr.distill_step(x, ids, top, rest, w),
             lambda: tr.embed(W, tok), lambda: tr.embed_grad(d, tok)]
    refused = [lambda: tr.top_logits(x, 2, 0.0), lambda: tr.distill_forward(x, ids, top, rest, 0.0),
               lambda: tr.distill_backward(x, ids, top, rest, stats, w, 0.0),
               lambda: tr.distill_step(x, ids, top, rest, w, out=(loss, x)), lambda: tr.embed(W, tok, out=W[:3]),
               lambda: tr.embed_grad(torch.ones(9, E, device="cuda"), _tok([1] * 9))]
    for call in calls:
        call()
        count = tr.last_launch_count()
        assert count >= 1
        for bad in refused:
            with pytest.raises((DominoError, ValueError)):
                bad()
            assert tr.last_launch_count() == count
    tr.embed(W, tok[:0])
    assert tr.last_launch_count() == 0
    tr.embed(W, tok)
    tr.embed_grad(d[:0], tok[:0], out=table, accumulate=True)
    assert tr.last_launch_count() == 0
