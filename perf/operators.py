"""Workloads of the draft-head training operators, with their plain forms.

Three operators, in the order in which a training step uses them:

* ``top``: the record of a teacher's logits: the K largest per row (ids
  ascending, ties to the lower id) and the log-sum-exp of all the others;
* ``distill``: the divergence of a student's distribution from that record,
  with its gradient by the student's logits, either in one call (``step``) or
  as a forward call and a backward call (``pair``);
* ``embed`` / ``embed_grad``: the scaled embedding lookup and the dense
  gradient of its table.

``run`` computes the plain form with elementary torch operations in fp32, or,
where ``own`` is set, makes the calls a user makes of the package.  ``exact``
restates each definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

V_FULL = 151936   # vocabulary of the Qwen3-8B-shaped workloads
V_CUT = 80000     # the cut vocabulary of the profiling workloads


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "pad": 0, "temperature": 1.0}
    c.update(kw)
    return c


def listed():
    return [
        # teacher rows of one request's block: latency
        _case("top_block_k64", "top", N=15, V=V_FULL, K=64),
        # a training batch of 64 blocks, softened teacher
        _case("top_64_blocks_k256", "top", N=960, V=V_FULL, K=256, temperature=2.0),
        # fp32 logits of an odd vocabulary, as many candidates as the largest pool
        _case("top_odd_fp32_k2048", "top", N=333, V=V_CUT - 1, K=2048, dtype="fp32"),
        # loss and gradient of one request's block: latency
        _case("step_block_k64", "step", N=15, V=V_FULL, K=64),
        # the largest training batch: 256 blocks
        _case("step_256_blocks_k64", "step", N=3840, V=V_FULL, K=64),
        # a small fp32 model with an odd vocabulary
        _case("step_small_odd_fp32", "step", N=1021, V=4097, K=17, dtype="fp32", temperature=1.5),
        # forward and backward as autograd calls them, 64 blocks
        _case("pair_64_blocks_k256", "pair", N=960, V=V_FULL, K=256, temperature=2.0),
        # the same in fp32, odd vocabulary, rows inside a wider buffer
        _case("pair_odd_fp32_k512", "pair", N=240, V=V_CUT - 1, K=512, dtype="fp32", pad=33),
        # the embeddings of one block's tokens: latency
        _case("embed_block", "embed", N=16, V=V_FULL, E=1024),
        # the embeddings of a large batch at the larger target's width
        _case("embed_4096_blocks", "embed", N=61440, V=V_FULL, E=1536),
        # the table's gradient from 64 blocks: mostly untouched rows
        _case("embed_grad_64_blocks", "embed_grad", N=1024, V=V_FULL, E=1024),
        # the table's gradient from a large batch with frequent tokens
        _case("embed_grad_4096_blocks", "embed_grad", N=65536, V=V_FULL, E=1536),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "step", "pair", "embed", "embed_grad"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "pad": 0,
         "temperature": rng.choice([1.0, 0.7, 1.5, 2.0])}
    if op in ("embed", "embed_grad"):
        c["E"] = _log_int(rng, 40, 1536)
        if rng.random() < 0.5:
            c["E"] = max(8, c["E"] // 8 * 8)
        c["V"] = _log_int(rng, 1000, V_FULL)
        c["N"] = _log_int(rng, 1, 65536)
        c["pad"] = rng.choice([0, 0, 8, 3])
        return c
    c["V"] = _log_int(rng, 1000, V_FULL)
    if rng.random() < 0.5:
        c["V"] = c["V"] // 8 * 8
    most = 1.4e8 if op == "top" else 2.8e8  # elements
    c["N"] = _log_int(rng, 1, max(1, min(3840, int(most / c["V"]))))
    c["K"] = _log_int(rng, 1, min(2048, c["V"] // 2))
    c["pad"] = rng.choice([0, 0, 8, 33])
    return c


# ---- inputs ------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _dtype(case)
    N, V, op = case["N"], case["V"], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    if op in ("embed", "embed_grad"):
        E = case["E"]
        # ranks u^6 V (about a seventh of the tokens are the commonest one) spread
        # over the vocabulary by a fixed stride, and a few padding positions
        rank = (uniform(N).double().pow(6.0) * V).to(torch.int64).clamp_(0, V - 1)
        tok = ((rank * 7919 + 13) % V).to(torch.int32)
        tok[uniform(N) < 0.02] = -1
        s = {"tokens": tok, "scale": math.sqrt(E)}
        if op == "embed":
            s["table"] = torch.empty(V, E, device=dev, dtype=dt).normal_(0.0, 0.02, generator=g)
            s["out"] = torch.empty(N, E + case["pad"], device=dev, dtype=dt)[:, :E]
        else:
            s["dout"] = normal(N, E + case["pad"]).mul_(1e-2).to(dt)[:, :E]
            s["dtable"] = torch.empty(V, E, device=dev, dtype=torch.float32)
        return s

    K = case["K"]
    # logits: N(0, 2^2) with a grammar's mask (-inf) over part of every eighth row
    x = torch.empty(N, V + case["pad"], device=dev, dtype=dt).normal_(0.0, 2.0, generator=g)[:, :V]
    x[::8, : V // 3] = float("-inf")
    s = {"logits": x, "K": K, "temperature": case["temperature"]}
    if op == "top":
        s["ids"] = torch.empty(N, K, device=dev, dtype=torch.int32)
        s["top"] = torch.empty(N, K, device=dev, dtype=torch.float32)
        s["rest"] = torch.empty(N, device=dev, dtype=torch.float32)
        return s
    # the teacher's record: one id from each K-th of the vocabulary, their logits,
    # the mass of the others; short records (padded with -1) and empty ones
    edge = torch.arange(K + 1, device=dev) * V // K
    ids = edge[:-1] + (uniform(N, K) * (edge[1:] - edge[:-1])).to(torch.int64).clamp_(max=V // K - 1)
    top = normal(N, K).mul_(2.0).add_(4.0)
    x.scatter_(1, ids, (0.5 * top + 1.5 * normal(N, K)).to(dt))  # a student near its teacher; no mask on the record
    length = torch.where(uniform(N) < 0.1, (uniform(N) * K).to(torch.int64), torch.full((N,), K, device=dev))
    if N > 1:
        length[N // 2] = 0
    none = torch.arange(K, device=dev) >= length[:, None]
    ids[none] = -1
    rest = torch.where(length > 0, top.max(1).values / case["temperature"] + normal(N) - 1.0,
                       torch.full((N,), float("-inf"), device=dev))
    s.update(ids=ids.to(torch.int32), top=top, rest=rest,
             weight=torch.full((N,), 1.0 / N, device=dev) * (0.5 + uniform(N)),
             loss=torch.empty(N, device=dev, dtype=torch.float32),
             dlogits=torch.empty(N, V + case["pad"], device=dev, dtype=dt)[:, :V])
    if op == "pair":
        s["stats"] = torch.empty(N, 8, device=dev, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:
        from speculative_decoding_draft_lm_gb300.train import DominoTrain
        s["train"] = DominoTrain(case["V"], E=case.get("E", 0),
                                 max_tokens=case["N"] if case["op"] == "embed_grad" else 0, dtype=case["dtype"])
    return s


# ---- plain forms ---------------------------------------------------------------

def _log_sum_exp(a):
    m = a.max(dim=1, keepdim=True).values
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return (a - m).exp().sum(dim=1).log() + m[:, 0]


def _plain_top(s):
    x = s["logits"].float()
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : s["K"]].sort(dim=1).values
    top = x.gather(1, ids)
    rest = _log_sum_exp(x.scatter(1, ids, float("-inf")) / s["temperature"])
    return {"ids": ids.to(torch.int32), "top": top, "rest": rest}


def _max_and_sum(a):
    """(m, sum exp(a - m)) of each row, m its maximum (0 for a row of -inf)."""
    m = a.max(dim=1, keepdim=True).values
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return m[:, 0], (a - m).exp().sum(dim=1)


def _plain_distill(s):
    T = s["temperature"]
    ids, valid = s["ids"].long().clamp(min=0), s["ids"] >= 0
    t = torch.where(valid, s["top"] / T, float("-inf"))
    mt, st = _max_and_sum(torch.cat([t, s["rest"][:, None]], dim=1))
    has = st > 0
    st = torch.where(has, st, torch.ones_like(st))
    p = (t - mt[:, None]).exp() / st[:, None]
    p_rest = (s["rest"] - mt).exp() / st
    x = s["logits"].float() / T
    mx, sx = _max_and_sum(x)
    in_record = torch.zeros(x.shape, dtype=torch.int32, device=x.device).scatter_add_(1, ids, valid.int()) > 0
    outside = _log_sum_exp(x.masked_fill(in_record, float("-inf")))
    # sum p (log p - log q): the two normalisers as one difference, log(sx / st) + mx - mt
    loss = torch.where(p > 0, p * (t - x.gather(1, ids)), 0.0).sum(dim=1)
    loss = loss + torch.where(p_rest > 0, p_rest * (s["rest"] - outside), 0.0) + (mx - mt) + (sx / st).log()
    loss = torch.where(has, loss, 0.0)
    q = (x - mx[:, None]).exp() / sx[:, None]
    away = 1.0 - torch.where(p_rest > 0, p_rest * sx / (outside - mx).exp(), 0.0)
    grad = torch.where(in_record, q, q * away[:, None])
    grad.scatter_add_(1, ids, torch.where(valid, -p, 0.0))
    grad = grad * torch.where(has, s["weight"] / T, 0.0)[:, None]
    return {"loss": loss, "dlogits": grad.to(s["logits"].dtype)}


def _plain_embed(s):
    tok = s["tokens"].long()
    y = s["table"][tok.clamp(min=0)].float() * s["scale"]
    return {"out": torch.where((tok >= 0)[:, None], y, 0.0).to(s["table"].dtype)}


def _plain_embed_grad(s):
    tok = s["tokens"].long()
    y = torch.where((tok >= 0)[:, None], s["dout"].float(), 0.0)
    grad = torch.zeros_like(s["dtable"]).index_add_(0, tok.clamp(min=0), y)
    return {"dtable": grad * s["scale"]}


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"top": _plain_top, "step": _plain_distill, "pair": _plain_distill, "embed": _plain_embed,
                "embed_grad": _plain_embed_grad}[op](s)
    tr = s["train"]
    if op == "top":
        ids, top, rest = tr.top_logits(s["logits"], s["K"], s["temperature"], out=(s["ids"], s["top"], s["rest"]))
        return {"ids": ids, "top": top, "rest": rest}
    if op == "step":
        loss, grad = tr.distill_step(s["logits"], s["ids"], s["top"], s["rest"], s["weight"], s["temperature"],
                                     out=(s["loss"], s["dlogits"]))
        return {"loss": loss, "dlogits": grad}
    if op == "pair":
        loss, stats = tr.distill_forward(s["logits"], s["ids"], s["top"], s["rest"], s["temperature"],
                                         out=(s["loss"], s["stats"]))
        grad = tr.distill_backward(s["logits"], s["ids"], s["top"], s["rest"], stats, s["weight"], s["temperature"],
                                   out=s["dlogits"])
        return {"loss": loss, "dlogits": grad}
    if op == "embed":
        return {"out": tr.embed(s["table"], s["tokens"], s["scale"], out=s["out"])}
    return {"dtable": tr.embed_grad(s["dout"], s["tokens"], s["scale"], out=s["dtable"])}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    N, V, op = case["N"], case["V"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "embed":
        return {"bytes": 2.0 * N * case["E"] * e + 4.0 * N, "flops": float(N * case["E"])}
    if op == "embed_grad":
        return {"bytes": float(N * case["E"] * e + 4 * N + V * case["E"] * 4), "flops": float(N * case["E"])}
    K = case["K"]
    if op == "top":
        return {"bytes": float(N * V * e + N * (8 * K + 4)), "flops": 4.0 * N * V}
    record = N * (8 * K + 12)
    if op == "step":
        return {"bytes": float(2 * N * V * e + record), "flops": 8.0 * N * V}
    return {"bytes": float(3 * N * V * e + 2 * record + 32 * N), "flops": 8.0 * N * V}


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "embed":
        out = torch.zeros(case["N"], case["E"], dtype=torch.float64, device="cuda")
        at = (s["tokens"] >= 0).nonzero()[:, 0]
        out[at] = s["table"].index_select(0, s["tokens"][at].long()).double() * s["scale"]
        return {"out": out}
    if op == "embed_grad":
        # on the host: one row at a time in the order of the sorted tokens
        tok = s["tokens"].cpu().numpy().astype(np.int64)
        d = s["dout"].double().cpu().numpy()
        grad = np.zeros((case["V"], case["E"]))
        order = np.argsort(tok, kind="stable")
        order = order[tok[order] >= 0]
        if order.size:
            t = tok[order]
            first = np.flatnonzero(np.r_[True, t[1:] != t[:-1]])
            grad[t[first]] = np.add.reduceat(d[order], first, axis=0) * s["scale"]
        return {"dtable": torch.from_numpy(grad)}
    T, K = float(case["temperature"]), case["K"]
    N, V = case["N"], case["V"]
    if op == "top":
        ids, top, rest = [], [], []
        for n0 in range(0, N, 64):
            x = s["logits"][n0:n0 + 64].double()
            # the K-th largest value, then everything above it and the first ties
            kth = x.kthvalue(V - K + 1, dim=1).values[:, None]
            above, tie = x > kth, x == kth
            need = K - above.sum(1, keepdim=True)
            chosen = above | (tie & (tie.cumsum(1) <= need))
            i = chosen.nonzero()[:, 1].view(-1, K)
            ids.append(i.to(torch.int32))
            top.append(torch.gather(x, 1, i))
            rest.append(torch.logsumexp(torch.where(chosen, -math.inf, x / T), dim=1))
        return {"ids": torch.cat(ids), "top": torch.cat(top), "rest": torch.cat(rest)}
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    grad = torch.zeros(N, V, dtype=torch.float64 if N * V < 2 ** 30 else torch.float32, device="cuda")
    for n0 in range(0, N, 256):
        n1 = min(N, n0 + 256)
        x = s["logits"][n0:n1].double() / T
        ids = s["ids"][n0:n1].long()
        dest = torch.where(ids < 0, V, ids)  # padding goes to a column of its own
        dense = torch.full((n1 - n0, V + 1), -math.inf, dtype=torch.float64, device="cuda")
        dense.scatter_(1, dest, s["top"][n0:n1].double() / T)
        member = torch.zeros((n1 - n0, V + 1), dtype=torch.bool, device="cuda").scatter_(1, dest, True)[:, :V]
        dense = dense[:, :V]
        r = s["rest"][n0:n1].double()
        L = torch.logaddexp(torch.logsumexp(dense, 1), r)
        ok = L > -math.inf
        log_p = dense - L[:, None]
        log_q = torch.log_softmax(x, dim=1)
        terms = torch.where(log_p > -math.inf, log_p.exp() * (log_p - log_q), 0.0).sum(1)
        log_qr = torch.logsumexp(torch.where(member, -math.inf, log_q), 1)
        log_pr = r - L
        terms = terms + torch.where(log_pr > -math.inf, log_pr.exp() * (log_pr - log_qr), 0.0)
        loss[n0:n1] = torch.where(ok, terms, 0.0)
        q = log_q.exp()
        ratio = torch.where(log_pr > -math.inf, (log_pr - log_qr).exp(), 0.0)
        d = torch.where(member, q - log_p.exp(), q - q * ratio[:, None])
        w = (s["weight"][n0:n1].double() / T)[:, None]
        grad[n0:n1] = torch.where(ok[:, None], d * w, 0.0).to(grad.dtype)
    return {"loss": loss, "dlogits": grad}
