"""The training example runs the operators together: its loss falls, its
gradients agree with a plain torch head's, and the rollout takes its weights."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("train_draft_head", os.path.join(ROOT, "examples", "train_draft_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss_and_the_rollout_drafts():
    losses, out = _example().main(steps=25, B=16, say=lambda *a: None)
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5]), losses
    assert out.shape == (4, 15) and (out >= 0).all() and (out < 4096).all()


def test_gradients_match_a_plain_torch_head():
    from speculative_decoding_draft_lm_gb300.train import DominoTrain, distill_loss
    m = _example()
    torch.manual_seed(3)
    V, E, G, F, B, K, T = 300, 16, 24, 20, 3, 12, 1.3
    mk = lambda *s: torch.randn(*s, device="cuda") * 0.3
    p = {"emb": mk(V, E), "w_ih": mk(3 * G, E), "w_hh": mk(3 * G, G), "fc1": mk(F, G), "fc2": mk(V, F), "b": mk(V)}
    tokens = torch.randint(0, V, (B, 15), device="cuda", dtype=torch.int32)
    s, base, target = mk(B, 15, F), mk(B, 16, V), mk(B * 14, V) * 10
    train = DominoTrain(V, E=E, max_tokens=B * 15, dtype="fp32")
    ids, top, rest = train.top_logits(target, K, T)

    a = {n: t.clone().requires_grad_() for n, t in p.items()}
    distill_loss(train, m.head_logits(train, a, tokens, s, base), ids, top, rest, T).mean().backward()

    # the same in double precision: buckets of the record and one of all others
    d = {n: t.double().requires_grad_() for n, t in p.items()}
    m.embedding = lambda train, table, tok: table[tok.long()]
    h0 = torch.zeros
    try:
        m.torch.zeros = lambda *sz, device=None: h0(*sz, device=device, dtype=torch.float64)
        logits = m.head_logits(None, d, tokens, s.double(), base.double())
    finally:
        m.torch.zeros = h0
    logq = torch.log_softmax(logits / T, 1)
    member = torch.zeros_like(logq, dtype=torch.bool).scatter_(1, ids.long(), True)
    q = torch.cat([logq.gather(1, ids.long()), torch.logsumexp(logq.masked_fill(member, float("-inf")), 1)[:, None]], 1)
    t = torch.cat([top.double() / T, rest.double()[:, None]], 1)
    torch.nn.functional.kl_div(q, torch.softmax(t, 1), reduction="sum").div(B * 14).backward()
    for n in p:
        ref = d[n].grad
        err = (a[n].grad.double() - ref).norm() / ref.norm()
        assert err < 1e-4, (n, err)
