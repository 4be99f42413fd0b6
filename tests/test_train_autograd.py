"""CPU checks of the autograd forms, with a stand-in for the context that does
the operators' arithmetic in torch."""
import pytest

torch = pytest.importorskip("torch")


class StandIn:
    """What the autograd functions call of DominoTrain."""
    max_tokens, torch_dtype = 64, torch.float32

    def distill_forward(self, logits, ids, top, rest, temperature):
        return self._loss(logits.detach(), ids, top, temperature), torch.zeros(logits.shape[0], 8)

    def distill_backward(self, logits, ids, top, rest, stats, dloss, temperature):
        x = logits.detach().requires_grad_()
        with torch.enable_grad():
            return torch.autograd.grad(self._loss(x, ids, top, temperature), x, dloss.detach())[0]

    def _loss(self, x, ids, top, T):
        p = torch.softmax(top / T, 1)
        return (p * (p.log() - torch.log_softmax(x / T, 1).gather(1, ids.long()))).sum(1)

    def embed(self, table, tokens, scale):
        return scale * table.detach()[tokens.long()]

    def embed_grad(self, dout, tokens, scale, grad_dtype=None):
        return torch.zeros(5, dout.shape[1]).index_add_(0, tokens.long(), scale * dout.detach())


def _distill():
    from speculative_decoding_draft_lm_gb300.train import distill_loss
    x = torch.randn(3, 7, requires_grad=True)
    ids = torch.tensor([[0, 2], [1, 6], [5, 3]], dtype=torch.int32)
    return x, distill_loss(StandIn(), x, ids, torch.randn(3, 2))


def _embedding():
    from speculative_decoding_draft_lm_gb300.train import embedding
    W = torch.randn(5, 4, requires_grad=True)
    return W, embedding(StandIn(), W, torch.tensor([0, 3, 3], dtype=torch.int32), 2.0)


@pytest.mark.parametrize("make", [_distill, _embedding])
def test_first_derivatives(make):
    x, y = make()
    (g,) = torch.autograd.grad((y ** 2).sum(), x)
    assert g.shape == x.shape and (g != 0).any()


@pytest.mark.parametrize("make", [_distill, _embedding])
def test_second_derivatives_are_refused(make):
    """Not silently dropped: a penalty on the gradient raises."""
    x, y = make()
    (g,) = torch.autograd.grad((y ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g ** 2).sum() + (x ** 2).sum()).backward()
