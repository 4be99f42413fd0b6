"""CPU checks of the scoring calls: argument checks that answer without a GPU, the
autograd form with a stand-in for the context, and the oracle."""
import ctypes
import os

import numpy as np
import pytest

from oracle import train_oracle as O

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_lm_gb300 import build, rollout, train
    if not os.path.exists(rollout.LIB_PATH):
        build.build()
    return train.load_library()


def test_null_context(lib):
    from speculative_decoding_draft_lm_gb300 import rollout as R
    bad = R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_train_logprobs_forward(None, None, 1, 8, 1, None, 1.0, None, None, 0, None, None, None, None) == bad
    assert lib.domino_train_logprobs_backward(None, None, 8, 1, None, 1.0, None, None, None, None, 8, None) == bad
    assert lib.domino_train_logprobs_step(None, None, 8, 1, None, 1.0, None, None, None, None, None, 8, None) == bad


def test_header_constants_match_the_binding():
    import re
    from speculative_decoding_draft_lm_gb300 import train
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "domino_train.h")).read()
    for name in ("DOMINO_TRAIN_MAX_ALTERNATIVES", "DOMINO_TRAIN_LOGPROB_STATS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(train, name)


class StandIn:
    """What the autograd function calls of DominoTrain, in torch."""
    torch_dtype = torch.float32

    def _values(self, x, tokens, T):
        lq = torch.log_softmax(x / T, 1)
        return lq.gather(1, tokens.long()[:, None])[:, 0], -(lq.exp() * lq).sum(1), lq

    def logprobs_forward(self, logits, tokens, temperature, alternatives, stats):
        lp, H, lq = self._values(logits.detach(), tokens, temperature)
        top = lq.topk(alternatives, 1)
        more = (top.indices.int(), top.values) if alternatives else ()
        return (lp, H, *more, torch.zeros(logits.shape[0], 4))

    def logprobs_backward(self, logits, tokens, stats, dlogprob, dentropy, temperature):
        x = logits.detach().requires_grad_()
        with torch.enable_grad():
            lp, H, _ = self._values(x, tokens, temperature)
            y = sum((d * v).sum() for d, v in ((dlogprob, lp), (dentropy, H)) if d is not None)
            return torch.autograd.grad(y, x)[0]


def test_autograd_form():
    from speculative_decoding_draft_lm_gb300.train import token_logprobs
    x = torch.randn(3, 7, requires_grad=True)
    tok = torch.tensor([1, 0, 6], dtype=torch.int32)
    lp, H, ids, alt = token_logprobs(StandIn(), x, tok, 2.0, alternatives=3)
    assert not ids.requires_grad and not alt.requires_grad
    (g,) = torch.autograd.grad((lp - H).sum(), x)
    y = x.detach().requires_grad_()
    lq = torch.log_softmax(y / 2.0, 1)
    (lq.gather(1, tok.long()[:, None]).sum() + (lq.exp() * lq).sum()).backward()
    assert torch.allclose(g, y.grad, atol=1e-6)
    lp, H = token_logprobs(StandIn(), x, tok)
    (g,) = torch.autograd.grad(lp.sum(), x, retain_graph=True, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        ((g ** 2).sum() + (x ** 2).sum()).backward()
    with pytest.raises(ValueError, match="logits"):
        token_logprobs(StandIn(), x.bfloat16(), tok)


def test_oracle_against_torch():
    g = np.random.default_rng(0)
    x = g.normal(0, 2, (4, 50))
    x[1, :20] = -np.inf
    x[2] = 1.0
    tok = np.asarray([3, 30, 7, -1], np.int32)
    lp, H, ids, alt, _ = O.logprobs(x, tok, 1.5, 6)
    lq = torch.log_softmax(torch.as_tensor(x) / 1.5, 1)
    for n in range(3):
        assert abs(lp[n] - lq[n, tok[n]].item()) < 1e-12
        assert abs(H[n] - torch.special.entr(lq[n].exp()).sum().item()) < 1e-12
    assert (ids[2] == np.arange(6)).all() and (ids[3] == -1).all() and lp[3] == 0
    assert (ids[0] == np.argsort(-x[0])[:6]).all() and np.allclose(alt[0], np.sort(lq[0].numpy())[::-1][:6])
    t = torch.as_tensor(x[:3]).requires_grad_()
    lq = torch.log_softmax(t / 1.5, 1)
    a, b = np.asarray([1.0, -2.0, 0.5, 1.0]), np.asarray([0.3, 0.2, -1.0, 1.0])
    y = (torch.as_tensor(a[:3]) * lq.gather(1, torch.as_tensor(tok[:3]).long()[:, None])[:, 0]).sum()
    q = lq.exp()
    y = y - (torch.as_tensor(b[:3])[:, None] * torch.where(q > 0, q * lq.clamp(min=-1e9), 0.0)).sum()
    y.backward()
    grad, _, _ = O.logprobs_grad(x, tok, 1.5, a, b)
    assert np.allclose(grad[:3], t.grad.numpy(), atol=1e-12) and (grad[3] == 0).all()
