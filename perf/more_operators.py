"""Workloads of the operators that score a draft head and update its weights.

* ``score`` / ``pair`` / ``step``: the log probability of each row's token under
  softmax(logits / temperature), the row's entropy and its most likely
  alternatives; with the gradient of the first two by the logits, from a forward
  and a backward call (``pair``) or in one call (``step``);
* ``adamw``: one AdamW step over many tensors, with moments in 32 bits or in 8
  (e4m3 with a scale for every 128 elements, rounded stochastically), with or
  without an fp32 master copy, optionally clipped by the gradients' norm;
* ``norm``: that norm and the factor that clips it.

``run`` computes the plain form with elementary torch operations, or, where
``own`` is set, makes the calls a user makes of the package.  ``exact`` restates
each definition in 64 bits.
"""
import math
import random

import torch

own = False

V_FULL = 151936   # vocabulary of the Qwen3-8B-shaped workloads
V_CUT = 80000     # the cut vocabulary of the profiling workloads
BLOCK = 128       # elements that share a scale; tensors start at multiples of it in the flat buffers
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
MAX_NORM = 1.0
SEED = 20_26
COUNT = 100       # steps that the moments have seen


def _rows(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "pad": 0, "temperature": 1.0, "k": 0, "entropy": True}
    c.update(kw)
    return c


def _tensors(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "grad": "bf16", "bits": 32, "master": False, "clip": False,
         "V": 0, "E": 0, "many": 0, "most": 0, "pick": 0}
    c.update(kw)
    return c


def listed():
    return [
        # the sampled token of one request, with the alternatives a server returns: latency
        _rows("score_one_token_k20", "score", N=1, V=V_FULL, k=20),
        # a batch of 64 draft blocks scored
        _rows("score_64_blocks_k20", "score", N=960, V=V_FULL, k=20),
        # fp32 logits of an odd vocabulary inside a wider buffer, softened
        _rows("score_odd_fp32_k5", "score", N=333, V=V_CUT - 1, k=5, dtype="fp32", pad=33, temperature=0.7),
        # forward and backward as autograd calls them, with an entropy bonus, 64 blocks
        _rows("pair_64_blocks", "pair", N=960, V=V_FULL),
        # the largest training batch in one call: 256 blocks
        _rows("step_256_blocks", "step", N=3840, V=V_FULL),
        # a small fp32 model with an odd vocabulary, log probabilities alone
        _rows("step_small_odd_fp32", "step", N=1021, V=4097, dtype="fp32", temperature=1.5, entropy=False),
        # the tiny fp32 head, clipped: latency
        _tensors("adamw_tiny_head_fp32_clip", "adamw", V=4096, E=128, dtype="fp32", grad="fp32", clip=True),
        # many small tensors of odd sizes, 8-bit moments: launches and ragged ends
        _tensors("adamw_many_odd_8bit", "adamw", many=96, most=100_000, pick=7, bits=8),
        # the head at Qwen3-8B shapes: fp32 master weights and moments
        _tensors("adamw_head_master", "adamw", V=V_FULL, E=1024, master=True),
        # the same head with 8-bit moments, nothing held twice
        _tensors("adamw_head_8bit", "adamw", V=V_FULL, E=1024, bits=8),
        # the norm of the tiny head's gradients: latency
        _tensors("norm_tiny_head_fp32", "norm", V=4096, E=128, grad="fp32", bits=8),
        # the norm of the larger target's head
        _tensors("norm_large_head", "norm", V=V_FULL, E=1536, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "pair", "step", "adamw", "adamw", "adamw", "norm"])
    if op in ("adamw", "norm"):
        c = _tensors("", op, dtype=rng.choice(["bf16", "bf16", "fp32"]), grad=rng.choice(["bf16", "fp32"]))
        del c["name"]
        if op == "adamw":
            c["bits"] = rng.choice([8, 32])
            c["master"] = c["dtype"] == "bf16" and rng.random() < 0.4
            c["clip"] = rng.random() < 0.3
        if rng.random() < 0.5:
            c["V"], c["E"] = _log_int(rng, 1000, V_FULL), _log_int(rng, 40, 1024)
        else:
            c["many"], c["most"], c["pick"] = _log_int(rng, 1, 200), _log_int(rng, 10, 2_000_000), rng.randrange(1000)
        return c
    c = _rows("", op, dtype=rng.choice(["bf16", "bf16", "fp32"]), temperature=rng.choice([1.0, 0.7, 1.5, 2.0]),
              pad=rng.choice([0, 0, 8, 33]), entropy=rng.random() < 0.7)
    del c["name"]
    c["V"] = _log_int(rng, 1000, V_FULL)
    if rng.random() < 0.5:
        c["V"] = c["V"] // 8 * 8
    c["N"] = _log_int(rng, 1, max(1, min(3840, int((1.4e8 if op == "score" else 2.8e8) / c["V"]))))
    if op == "score":
        c["k"] = rng.choice([0, 1, 5, 20, 32])
    return c


# ---- inputs ------------------------------------------------------------------

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _sizes(case):
    """Elements of each tensor."""
    V, E = case["V"], case["E"]
    if V:  # embedding, the GRU's two, the projector's two, bias
        return [V * E, 3 * E * E, 3 * E * E, E * E, V * E, V]
    rng = random.Random(case["pick"])
    return [_log_int(rng, 1, case["most"]) for _ in range(case["many"])]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if case["op"] in ("adamw", "norm"):
        sizes = _sizes(case)
        at, total = [], 0
        for n in sizes:
            at.append(total)
            total += -(-n // BLOCK) * BLOCK
        held = torch.zeros(total, dtype=torch.bool, device="cuda")  # what is not between two tensors
        for i, n in zip(at, sizes):
            held[i:i + n] = True
        blocks = total // BLOCK
        # gradients whose size differs from block to block; none for the rows whose tokens did not occur
        size = (normal(blocks).mul_(1.5).exp_() * (uniform(blocks) < 0.7)).mul_(1e-3)
        grad = (normal(blocks, BLOCK) * size[:, None]).view(-1).mul_(held).to(TYPES[case["grad"]])
        s = {"grad": grad, "grads": [grad[i:i + n] for i, n in zip(at, sizes)], "max_norm": MAX_NORM,
             "norm": torch.empty((), device="cuda"), "scale": torch.full((), 0.75, device="cuda")}
        if case["op"] == "norm":
            return s
        p = (normal(total) * held).mul_(0.02)
        s["param"] = p.to(TYPES[case["dtype"]])
        s["params"] = [s["param"][i:i + n] for i, n in zip(at, sizes)]
        if case["master"]:
            s["master"] = p
        if case["bits"] == 32:
            s["m"] = normal(total).mul_(3e-4).mul_(held)
            s["v"] = normal(total).square_().add_(0.01).mul_(1e-6).mul_(held)
        else:
            m, v = normal(total).mul_(100.0), normal(total).square_().mul_(60.0)
            s["m"] = m.clamp_(-448, 448).mul_(held).to(torch.float8_e4m3fn)
            s["v"] = v.clamp_(2.0 ** -9, 448).mul_(held).to(torch.float8_e4m3fn)
            s["m_scale"] = uniform(blocks).add_(0.1).mul_(3e-6)
            s["v_scale"] = uniform(blocks).add_(0.1).mul_(1e-8)
        s["count"] = torch.full((1,), COUNT, dtype=torch.int64, device="cuda")
        return s

    N, V, dt = case["N"], case["V"], TYPES[case["dtype"]]
    # logits: N(0, 2^2) with a grammar's mask (-inf) over part of every eighth row, one row without a
    # logit left and every sixteenth one padding
    x = torch.empty(N, V + case["pad"], device="cuda", dtype=dt).normal_(0.0, 2.0, generator=g)[:, :V]
    x[::8, : V // 3] = float("-inf")
    if N > 4:
        x[N // 2] = float("-inf")
    tok = (uniform(N).double() * V).to(torch.int64).clamp_(max=V - 1)
    tok[5::16] = -1
    s = {"logits": x, "tokens": tok.to(torch.int32), "temperature": case["temperature"], "k": case["k"],
         "logprob": torch.empty(N, device="cuda"), "entropy": torch.empty(N, device="cuda")}
    if case["op"] == "score":
        s["ids"] = torch.empty(N, case["k"], dtype=torch.int32, device="cuda")
        s["alternatives"] = torch.empty(N, case["k"], device="cuda")
        return s
    # rows' gradients: an advantage of either sign, a small entropy bonus
    s["dlogprob"] = normal(N) / N
    s["dentropy"] = (uniform(N) * (0.1 / N)) if case["entropy"] else None
    s["stats"] = torch.empty(N, 4, device="cuda")
    s["dlogits"] = torch.empty(N, V + case["pad"], device="cuda", dtype=dt)[:, :V]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["clip"] = case["op"], case.get("clip", False)
    if own:
        if s["op"] == "adamw" or s["op"] == "norm":
            from speculative_decoding_draft_lm_gb300.optim import DominoAdamW
            keep = {n: s[n] for n in ("m", "v", "m_scale", "v_scale", "master", "count") if n in s}
            if s["op"] == "norm":  # of gradients alone: the optimizer's tensors are not touched
                keep, s["params"] = None, [torch.empty_like(t) for t in s["grads"]]
            s["opt"] = DominoAdamW(s["params"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                   state_bits=case["bits"], master=case["master"], seed=SEED, state=keep)
        else:
            from speculative_decoding_draft_lm_gb300.train import DominoTrain
            s["train"] = DominoTrain(case["V"], dtype=case["dtype"])
    return s


# ---- plain forms ---------------------------------------------------------------

def _plain_scores(s):
    T, tok = s["temperature"], s["tokens"].long()
    has = tok >= 0
    x = s["logits"].float()
    m = x.max(dim=1, keepdim=True).values
    some = has & (m[:, 0] > float("-inf"))
    d = torch.where(some[:, None], (x - m) / T, 0.0)
    e = d.exp()
    total = e.sum(dim=1)
    log_total = total.log()
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(dim=1) / total
    logprob = d.gather(1, tok.clamp(min=0)[:, None])[:, 0] - log_total
    logprob = torch.where(some, logprob, torch.where(has, float("-inf"), 0.0))
    out = {"logprob": logprob, "entropy": torch.where(some, entropy, 0.0)}
    return out, d, e / total[:, None], log_total, some


def _plain_score(s):
    out, d, _, log_total, some = _plain_scores(s)
    if s["k"]:
        ids = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, : s["k"]]
        lp = d.gather(1, ids) - log_total[:, None]
        real = some[:, None] & (lp > float("-inf"))
        out["ids"] = torch.where(real, ids, -1).to(torch.int32)
        out["alternatives"] = torch.where(real, lp, float("-inf"))
    return out


def _plain_gradient(s):
    out, d, q, log_total, some = _plain_scores(s)
    at = s["tokens"].long().clamp(min=0)[:, None]
    grad = -q * s["dlogprob"][:, None]
    grad.scatter_add_(1, at, s["dlogprob"][:, None])
    if s["dentropy"] is not None:
        log_q = (d - log_total[:, None]).clamp(min=-1e30)
        grad = grad - q * (log_q + out["entropy"][:, None]) * s["dentropy"][:, None]
    grad = torch.where(some[:, None], grad / s["temperature"], 0.0)
    out["dlogits"] = grad.to(s["logits"].dtype)
    return out


def _mix(h):
    """32 random bits from each 32-bit number (held in 64)."""
    h = (h ^ (h >> 15)) * 0x6A09E667 & 0xFFFFFFFF
    h = (h ^ (h >> 13)) * 0xBB67AE85 & 0xFFFFFFFF
    return h ^ (h >> 16)


def _words(total, t):
    """A random word for every position of the flat buffers, in step t."""
    key = _mix(_mix(t + 0x9E3779B9 & 0xFFFFFFFF) + SEED & 0xFFFFFFFF)
    at = torch.arange(total, device="cuda")
    high = at >> 32
    return _mix((at & 0xFFFFFFFF) * 0x9E3779B9 + key + high * 0x3C6EF373 & 0xFFFFFFFF)


def _round_e4m3(a, r, least):
    """(codes, scales) of the values `a`: r is 20 random bits for each, `least` the smallest code of what is not 0."""
    scale = (a.abs().view(-1, BLOCK).max(dim=1).values / 448.0).clamp(min=2.0 ** -120)
    y = (a.abs().view(-1, BLOCK) / scale[:, None]).view(-1).clamp(max=448.0)
    low = y < 2.0 ** -6
    word = torch.where(low, y + 2.0 ** -6, y).view(torch.int32).long()
    code = ((word + r) >> 20) - torch.where(low, 121 << 3, 120 << 3)
    code = torch.where(a != 0, code.clamp(min=least), 0) + torch.where(a < 0, 128, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale


def _plain_norm(s):
    norm = s["grad"].double().square().sum().sqrt()
    s["norm"].copy_(norm)
    s["scale"].copy_(torch.where(norm.isfinite(), (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0), float("nan")))
    return {"norm": s["norm"], "scale": s["scale"]}


def _plain_adamw(s):
    out = _plain_norm(s) if s["clip"] else {}
    s["count"].add_(1)
    t = s["count"].double()
    c1, c2 = 1.0 - BETA1 ** t, 1.0 - BETA2 ** t
    g = s["grad"].float() * s["scale"]
    m, v = s["m"].float(), s["v"].float()
    narrow = "m_scale" in s
    if narrow:
        m = (m.view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["v_scale"][:, None]).view(-1)
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    p = s["master"] if "master" in s else s["param"].float()
    p = p * (1.0 - LR * DECAY) - (LR / c1).float() * (m / (v.sqrt() / c2.sqrt().float() + EPS))
    lossy = s["param"].dtype == torch.bfloat16 and "master" not in s
    h = _words(p.numel(), s["count"]) if narrow or lossy else None
    if lossy:
        bits = p.view(torch.int32).long() + (h >> 4 & 0xFFFF)
        p = (bits & ~0xFFFF).to(torch.int32).view(torch.float32)
    if "master" in s:
        s["master"].copy_(p)
        out["master"] = s["master"]
    s["param"].copy_(p)
    if narrow:
        m, m_scale = _round_e4m3(m, h & 0xFFFFF, 0)
        v, v_scale = _round_e4m3(v, h >> 12, 1)
        s["m_scale"].copy_(m_scale)
        s["v_scale"].copy_(v_scale)
        out.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
    s["m"].copy_(m)
    s["v"].copy_(v)
    out.update(param=s["param"], m=s["m"], v=s["v"], count=s["count"])
    return out


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"score": _plain_score, "pair": _plain_gradient, "step": _plain_gradient, "adamw": _plain_adamw,
                "norm": _plain_norm}[op](s)
    if op == "norm":
        norm, scale = s["opt"].grad_norm(s["max_norm"], grads=s["grads"], out=(s["norm"], s["scale"]))
        return {"norm": norm, "scale": scale}
    if op == "adamw":
        out = {}
        if s["clip"]:
            out["norm"], out["scale"] = s["opt"].grad_norm(s["max_norm"], grads=s["grads"], out=(s["norm"], s["scale"]))
        s["opt"].step(grads=s["grads"], scale=s["scale"])
        out.update({n: s[n] for n in ("param", "m", "v", "m_scale", "v_scale", "master", "count") if n in s})
        return out
    tr = s["train"]
    if op == "score":
        names = ("logprob", "entropy", "ids", "alternatives")[: 4 if s["k"] else 2]
        r = tr.logprobs_forward(s["logits"], s["tokens"], s["temperature"], alternatives=s["k"],
                                out=tuple(s[n] for n in names))
        return dict(zip(names, r))
    if op == "step":
        logprob, entropy, grad = tr.logprobs_step(s["logits"], s["tokens"], s["dlogprob"], s["dentropy"],
                                                  s["temperature"], out=(s["logprob"], s["entropy"], s["dlogits"]))
        return {"logprob": logprob, "entropy": entropy, "dlogits": grad}
    logprob, entropy, stats = tr.logprobs_forward(s["logits"], s["tokens"], s["temperature"], stats=s["stats"],
                                                  out=(s["logprob"], s["entropy"]))
    grad = tr.logprobs_backward(s["logits"], s["tokens"], stats, s["dlogprob"], s["dentropy"], s["temperature"],
                                out=s["dlogits"])
    return {"logprob": logprob, "entropy": entropy, "dlogits": grad}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("adamw", "norm"):
        n = float(sum(_sizes(case)))
        g = 2 if case["grad"] == "bf16" else 4
        if op == "norm":
            return {"bytes": n * g, "flops": 2 * n}
        per = g + (2 if case["dtype"] == "bf16" else 4) * (1 if case["master"] else 2) + (8 if case["master"] else 0)
        per += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * per, "flops": 16 * n}
    N, V = case["N"], case["V"]
    e = 2 if case["dtype"] == "bf16" else 4
    passes = {"score": 1, "step": 2, "pair": 3}[op]
    return {"bytes": float(N * V * e * passes + N * (12 + 8 * case["k"])), "flops": (6.0 if op == "score" else 12.0) * N * V}


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_rows(case, s):
    T, N, V, k = float(case["temperature"]), case["N"], case["V"], case["k"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    logprob, entropy = torch.zeros(N, **f64), torch.zeros(N, **f64)
    ids = torch.full((N, k), -1, dtype=torch.int32, device="cuda")
    alternatives = torch.full((N, k), -math.inf, **f64)
    score = case["op"] == "score"
    grad = None if score else torch.zeros(N, V, device="cuda", dtype=torch.float64 if N * V < 2 ** 30 else torch.float32)
    for n in range(0, N, 256):
        rows = slice(n, min(N, n + 256))
        tok = s["tokens"][rows].long()
        x = s["logits"][rows].double()
        on = (tok >= 0) & (x > -math.inf).any(1)
        logprob[rows][tok >= 0] = -math.inf
        x, tok, where = x[on], tok[on], torch.arange(rows.start, rows.stop, device="cuda")[on]
        if not len(tok):
            continue
        log_q = torch.log_softmax(x / T, dim=1)
        q = log_q.exp()
        H = -torch.special.xlogy(q, q).sum(1)
        logprob[where] = log_q[torch.arange(len(tok), device="cuda"), tok]
        entropy[where] = H
        if k:
            # everything above the k-th largest value, then the first of its ties
            kth = x.kthvalue(V - k + 1, dim=1).values[:, None]
            tie = x == kth
            chosen = (x > kth) | (tie & (tie.cumsum(1) <= k - (x > kth).sum(1, keepdim=True)))
            i = chosen.nonzero()[:, 1].view(-1, k)
            i = i.gather(1, x.gather(1, i).sort(dim=1, descending=True, stable=True).indices)
            lp = log_q.gather(1, i)
            ids[where] = torch.where(lp > -math.inf, i, -1).to(torch.int32)
            alternatives[where] = lp
        if not score:
            a = s["dlogprob"][rows][on].double()[:, None]
            d = a * (torch.nn.functional.one_hot(tok, V).double() - q)
            if s["dentropy"] is not None:
                b = s["dentropy"][rows][on].double()[:, None]
                d = d - b * (torch.special.xlogy(q, q) + q * H[:, None])
            grad[where] = (d / T).to(grad.dtype)
    out = {"logprob": logprob, "entropy": entropy}
    if score:
        return dict(out, ids=ids, alternatives=alternatives) if k else out
    return dict(out, dlogits=grad)


def _exact_mix(x):
    for shift, by in ((15, 0x6A09E667), (13, 0xBB67AE85)):
        x = ((x ^ (x >> shift)) * by) % (1 << 32)
    return x ^ (x >> 16)


def _exact_e4m3(a, r, least):
    """The e4m3 values and the scales: |a| / scale to a multiple of its place's step, up with the probability of the
    rest; r is 20 random bits."""
    blocks = a.abs().reshape(-1, BLOCK)
    scale = torch.maximum(blocks.amax(1) / 448, torch.full((), 2.0 ** -120, dtype=a.dtype, device=a.device))
    y = (blocks / scale[:, None]).reshape(-1).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    q = torch.floor(y / step + r.double() / 2 ** 20) * step
    q = torch.where(a != 0, q.clamp(min=least * 2.0 ** -9), 0.0)
    return torch.where(a < 0, -q, q), scale


def _exact_norm(s):
    total = math.fsum(float(torch.dot(c, c)) for c in (g.double() for g in s["grad"].split(1 << 24)))
    norm = math.sqrt(total)
    return norm, min(1.0, s["max_norm"] / (norm + 1e-6))


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] not in ("adamw", "norm"):
        return _exact_rows(case, s)
    out = {}
    if case["op"] == "norm" or case["clip"]:
        norm, scale = _exact_norm(s)
        out = {"norm": torch.tensor(norm, dtype=torch.float64), "scale": torch.tensor(scale, dtype=torch.float64)}
        if case["op"] == "norm":
            return out
    else:
        scale = float(s["scale"])
    t = COUNT + 1
    key = _exact_mix((_exact_mix((t + 0x9E3779B9) % (1 << 32)) + SEED) % (1 << 32))
    total, part = s["grad"].numel(), 1 << 24
    names = ["param", "m", "v"] + (["master"] if case["master"] else []) + (["m_scale", "v_scale"] if case["bits"] == 8 else [])
    parts = {n: [] for n in names}
    for i in range(0, total, part):
        j = min(total, i + part)
        f64 = {n: s[n][i:j].double() for n in ("param", "m", "v", "grad")}
        g = f64["grad"] * scale
        m, v = f64["m"], f64["v"]
        if case["bits"] == 8:
            m = m * s["m_scale"][i // BLOCK:j // BLOCK].double().repeat_interleave(BLOCK)
            v = v * s["v_scale"][i // BLOCK:j // BLOCK].double().repeat_interleave(BLOCK)
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g.square(), v, BETA2)
        p = s["master"][i:j].double() if case["master"] else f64["param"]
        m_hat, v_hat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        p = p - LR * DECAY * p - LR * m_hat / (v_hat.sqrt() + EPS)
        at = torch.arange(i, j, device="cuda")
        h = _exact_mix((at * 0x9E3779B9 + key) % (1 << 32))
        parts["param"].append(p)
        if case["master"]:
            parts["master"].append(p)
        if case["bits"] == 8:
            m, m_scale = _exact_e4m3(m, h % (1 << 20), 0)
            v, v_scale = _exact_e4m3(v, h // (1 << 12), 1)
            parts["m_scale"].append(m_scale)
            parts["v_scale"].append(v_scale)
        parts["m"].append(m)
        parts["v"].append(v)
    out.update({n: torch.cat(c) for n, c in parts.items()})
    out["count"] = None
    return out
