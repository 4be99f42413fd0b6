"""Train a small Domino draft head on a target's logits, then draft with it.

    python examples/train_draft_head.py [--steps 60]

The pieces in the order of a training step: the target's logits become records
(``top_logits``), the teacher-forced tokens become GRU inputs (``embedding``),
the head runs as the rollout runs it (bias-free GRU, SiLU projector, base
logits added), ``distill_loss`` gives each position's loss and gradient, and
``DominoAdamW`` clips the gradients together and updates the weights.  What the
target thinks of the head's first choices (``logprobs_forward``) is said beside
the loss.  The trained weights then go to ``DominoRollout``.  Everything is synthetic: the
"target" is a fixed random function of the previous token.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from speculative_decoding_draft_lm_gb300 import inputs  # noqa: E402
from speculative_decoding_draft_lm_gb300.optim import DominoAdamW  # noqa: E402
from speculative_decoding_draft_lm_gb300.rollout import DominoRollout  # noqa: E402
from speculative_decoding_draft_lm_gb300.train import DominoTrain, distill_loss, embedding  # noqa: E402

STEPS = inputs.N_PROPOSALS - 1  # corrected steps of a block


def gru(x, h, w_hh):
    """One bias-free GRU update; x holds the input side of the gates r|z|n."""
    gi, gh = x.chunk(3, 1), (h @ w_hh.t()).chunk(3, 1)
    r, z = torch.sigmoid(gi[0] + gh[0]), torch.sigmoid(gi[1] + gh[1])
    return (1 - z) * torch.tanh(gi[2] + r * gh[2]) + z * h


def head_logits(train, p, tokens, s, base):
    """Corrected logits [B * 14, V]: tokens [B, 15] = verified, p_1 .. p_14; s and
    base are the steps' projector terms and base logits."""
    B = tokens.shape[0]
    x = embedding(train, p["emb"], tokens.reshape(-1).contiguous()).view(B, 15, -1)
    x = x @ p["w_ih"].t()
    h = torch.zeros(B, p["w_hh"].shape[1], device=x.device)
    out = []
    for u in range(15):
        h = gru(x[:, u], h, p["w_hh"])
        if u >= 1:
            a = torch.nn.functional.silu(h @ p["fc1"].t() + s[:, u])
            out.append(a @ p["fc2"].t() + p["b"] + base[:, u + 1])
    return torch.stack(out, 1).view(B * STEPS, -1)


def main(steps: int = 60, B: int = 32, K: int = 64, temperature: float = 1.5, seed: int = 0, say=print):
    torch.manual_seed(seed)
    dev, sh = "cuda", inputs.TINY
    shapes = inputs.weight_shapes(sh)
    scale = {"lm_head": 0.02, "emb": 1.0, "w_ih": sh.E ** -0.5, "w_hh": sh.G ** -0.5, "fc1": sh.G ** -0.5,
             "fc2": 0.1 * sh.F ** -0.5, "b": 0.0}
    p = {n: (torch.randn(shapes[n], device=dev) * scale[n]).requires_grad_(n != "lm_head") for n in shapes}
    # the target: what it says next depends on the token before, through a table of 8 classes
    likes = torch.randn(8, sh.V, device=dev) * 3.0
    train = DominoTrain(sh.V, E=sh.E, max_tokens=B * 15, dtype="fp32")
    opt = DominoAdamW([t for t in p.values() if t.requires_grad], lr=3e-3, weight_decay=0.0)
    losses = []
    for step in range(steps):
        hidden = torch.randn(B, 16, sh.H, device=dev)
        s = torch.randn(B, 15, sh.F, device=dev) * 0.1
        base = hidden @ p["lm_head"].t()
        tokens = torch.randint(0, sh.V, (B, 15), device=dev, dtype=torch.int32)
        target = likes[(tokens[:, 1:] % 8).long()] + base[:, 2:16]
        ids, top, rest = train.top_logits(target.reshape(B * STEPS, sh.V), K, temperature)
        logits = head_logits(train, p, tokens, s, base)
        loss = distill_loss(train, logits, ids, top, rest, temperature).mean()
        opt.zero_grad()
        loss.backward()
        _, clip = opt.grad_norm(max_norm=1.0)
        opt.step(scale=clip)
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            choice = logits.detach().argmax(1).to(torch.int32)
            logprob, _ = train.logprobs_forward(target.reshape(B * STEPS, sh.V), choice, temperature)
            say(f"step {step:3d}  loss {losses[-1]:.4f}  target's log probability of the head's choice "
                f"{logprob.mean().item():.3f}")
    if train.status() != 0:
        raise RuntimeError("a token or id was out of range")
    # draft one block per request with the trained head
    eng = DominoRollout(sh.V, sh.H, sh.E, sh.G, sh.F, max_B=4, dtype="fp32")
    eng.load_weights({n: t.detach().contiguous() for n, t in p.items()})
    verified = torch.arange(4, device=dev, dtype=torch.int32)
    out = eng.run(torch.randn(4, 16, sh.H, device=dev), torch.randn(4, 15, sh.F, device=dev) * 0.1, verified)
    torch.cuda.synchronize()
    say("proposals of request 0:", out[0].tolist())
    eng.close()
    opt.close()
    train.close()
    return losses, out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)
