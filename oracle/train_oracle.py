"""fp64 CPU restatement of the draft-head training operators (test
infrastructure only; it shares no code with the CUDA path).

Every function takes numpy arrays widened to float64 from the exact input
values and works row by row, in the plainest form of each definition.
"""
from __future__ import annotations

import numpy as np


def _lse(a: np.ndarray) -> float:
    """log sum exp of a vector; -inf for none or all -inf; NaN if any is."""
    if a.size == 0:
        return -np.inf
    if np.isnan(a).any():
        return np.nan
    m = a.max()
    if np.isinf(m):
        return m
    return float(m + np.log(np.exp(a - m).sum()))


def top_logits(x: np.ndarray, K: int, T: float):
    """(ids [N,K] ascending, top [N,K], rest [N]): NaN largest, ties to the lower id."""
    N, V = x.shape
    ids = np.empty((N, K), dtype=np.int32)
    top = np.empty((N, K))
    rest = np.empty(N)
    for n in range(N):
        key = np.where(np.isnan(x[n]), np.inf, x[n]) + 0.0
        # NaN before everything, then larger logits, then lower ids
        order = np.lexsort((np.arange(V), -key, ~np.isnan(x[n])))
        i = np.sort(order[:K])
        ids[n], top[n] = i, x[n, i]
        rest[n] = _lse(np.delete(x[n], i) / T)
    return ids, top, rest


def first_places(ids: np.ndarray, V: int) -> list:
    """The places of one row's record that take part: valid ids, first occurrences."""
    seen, out = set(), []
    for k, i in enumerate(ids.tolist()):
        if 0 <= i < V and i not in seen:
            seen.add(i)
            out.append(k)
    return out


def distill(x: np.ndarray, ids: np.ndarray, top: np.ndarray, rest, T: float):
    """(loss [N], grad [N,V] of each row's own loss, terms): terms holds, per row,
    the sum of the absolute parts of the loss, and per entry of grad the sum of
    its absolute parts, which the tolerances scale with."""
    N, V = x.shape
    loss, grad = np.zeros(N), np.zeros((N, V))
    loss_parts, grad_parts = np.zeros(N), np.zeros((N, V))
    with np.errstate(all="ignore"):
        for n in range(N):
            k = first_places(ids[n], V)
            S = ids[n][k]
            t = top[n][k] / T
            r = -np.inf if rest is None else rest[n]
            L = _lse(np.append(t, r))
            if L == -np.inf:
                continue
            p, pr = np.exp(t - L), np.exp(r - L)
            u = x[n] / T
            z = _lse(u)
            q = np.exp(u - z)
            outside = np.ones(V, dtype=bool)
            outside[S] = False
            log_qr = _lse(u[outside]) - z
            parts = [pk * (tk - L - (uk - z)) for pk, tk, uk in zip(p, t, u[S]) if pk != 0]
            if pr != 0:
                parts.append(pr * (r - L - log_qr))
            loss[n] = np.sum(parts)
            loss_parts[n] = (np.sum(np.abs(p[p != 0] * (t - u[S])[p != 0])) + abs(z - L)
                             + (abs(pr * (r - log_qr - z)) if pr != 0 else 0.0))
            ratio = 0.0 if pr == 0 or log_qr == -np.inf else np.exp(r - L - log_qr)
            g = q - q * ratio
            g[S] = q[S] - p
            a = q + q * ratio
            a[S] = q[S] + p
            if pr != 0 and log_qr == -np.inf:
                g[outside] = 0.0
            grad[n], grad_parts[n] = g / T, a / T
    return loss, grad, {"loss": loss_parts, "grad": grad_parts}


def logprobs(x: np.ndarray, tokens: np.ndarray, T: float, k: int = 0):
    """(logprob [N], entropy [N], ids [N,k], alternatives [N,k], terms): the k largest
    logits above -inf, largest first, NaN before all, ties to the lower id.  terms
    holds per row log s, sum q |d| and sum q d^2 for d = (x - max) / T, which the
    tolerances scale with."""
    N, V = x.shape
    logprob, entropy = np.zeros(N), np.zeros(N)
    ids, alt = np.full((N, k), -1, dtype=np.int32), np.full((N, k), -np.inf)
    terms = {"log_s": np.zeros(N), "a1": np.zeros(N), "a2": np.zeros(N)}
    with np.errstate(all="ignore"):
        for n in range(N):
            t = int(tokens[n])
            if not 0 <= t < V:
                continue
            if np.isnan(x[n]).any() or (x[n] == np.inf).any():
                lq, entropy[n] = np.full(V, np.nan), np.nan
            elif x[n].max() == -np.inf:
                logprob[n] = -np.inf
                continue
            else:
                d = (x[n] - x[n].max()) / T
                log_s = np.log(np.exp(d).sum())
                lq = d - log_s
                q = np.exp(lq)
                at = q > 0
                entropy[n] = -(q[at] * lq[at]).sum()
                terms["log_s"][n], terms["a1"][n] = log_s, (q[at] * -d[at]).sum()
                terms["a2"][n] = (q[at] * d[at] ** 2).sum()
            logprob[n] = lq[t]
            order = np.lexsort((np.arange(V), -(x[n] + 0.0), ~np.isnan(x[n])))
            order = [i for i in order[:k] if not x[n, i] == -np.inf]
            ids[n, :len(order)], alt[n, :len(order)] = order, lq[order]
    return logprob, entropy, ids, alt, terms


def logprobs_grad(x: np.ndarray, tokens: np.ndarray, T: float, g: np.ndarray, h: np.ndarray):
    """(gradient [N,V] of sum(g logprob + h entropy), q [N,V], log q + H [N,V]), zeros where a row takes no part."""
    N, V = x.shape
    grad, q, l = np.zeros((N, V)), np.zeros((N, V)), np.zeros((N, V))
    with np.errstate(all="ignore"):
        for n in range(N):
            t = int(tokens[n])
            if not 0 <= t < V or (g[n] == 0 and h[n] == 0) or x[n].max() == -np.inf:
                continue
            u = (x[n] - x[n].max()) / T  # far from zero the logarithm of the sum would be lost beside it
            lq = u - _lse(u)
            q[n] = np.exp(lq)
            H = -np.where(q[n] > 0, q[n] * lq, 0.0).sum()
            l[n] = np.where(q[n] > 0, lq + H, 0.0)
            hot = np.zeros(V)
            hot[t] = 1
            grad[n] = (g[n] * (hot - q[n]) - h[n] * q[n] * l[n]) / T
    return grad, q, l


def embed(table: np.ndarray, tokens: np.ndarray, scale: float) -> np.ndarray:
    V, E = table.shape
    out = np.zeros((tokens.size, E))
    for i, t in enumerate(tokens.tolist()):
        if 0 <= t < V:
            out[i] = scale * table[t]
    return out


def embed_grad(dout: np.ndarray, tokens: np.ndarray, V: int, scale: float):
    """(dtable [V,E], sum of absolute terms [V,E], occurrences [V])."""
    E = dout.shape[1]
    g, a, c = np.zeros((V, E)), np.zeros((V, E)), np.zeros(V, dtype=np.int64)
    for i, t in enumerate(tokens.tolist()):
        if 0 <= t < V:
            g[t] += scale * dout[i]
            a[t] += np.abs(scale * dout[i])
            c[t] += 1
    return g, a, c
