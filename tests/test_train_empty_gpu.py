"""Calls without rows, whatever strides the empty tensors came with (numpy's are 0)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("strides", [(0, 0), (1, 1), (1, 40), (40, 1)])
def test_no_rows(strides):
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, distill_loss, embedding
    V, E, K = 40, 8, 3
    tr = DominoTrain(V, E=E, max_tokens=4, dtype="fp32")

    def none(cols):
        return torch.empty(0, device="cuda").as_strided((0, cols), strides)

    def flat(dtype=torch.float32):
        return torch.empty(0, dtype=dtype, device="cuda")

    ids, top, rest = tr.top_logits(none(V), K)
    assert ids.shape == top.shape == (0, K) and rest.shape == (0,)
    loss, grad = tr.distill_step(none(V), ids, top, rest, flat())
    assert loss.shape == (0,) and grad.shape == (0, V)
    loss, stats = tr.distill_forward(none(V), ids, top, rest)
    assert tr.distill_backward(none(V), ids, top, rest, stats, flat(), out=none(V)).shape == (0, V)
    W, tok = torch.ones(V, E, device="cuda", requires_grad=True), flat(torch.int32)
    assert tr.embed(W, tok, out=none(E)).shape == (0, E)
    assert not tr.embed_grad(none(E), tok).any()
    embedding(tr, W, tok).backward(none(E))
    assert W.grad.shape == (V, E) and not W.grad.any()
    x = none(V).requires_grad_()
    distill_loss(tr, x, ids, top).sum().backward()
    assert x.grad.shape == (0, V)
    assert tr.status() == 0
