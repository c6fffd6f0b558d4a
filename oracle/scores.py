"""Oracle: scores of given tokens and their gradient (test infrastructure).

Row by row in float64, from the definitions:
  p = softmax(logits / T) over the unsuppressed ids (NaN as -inf; a row of -inf
  is uniform, a row with +inf uniform over its +inf ids),
  logprob = log p_t, entropy = -sum p log p, the largest logits in decreasing
  order (ties: the lower id) with their log p, ids of zero probability not
  listed,
  grad_v = (g (v == t) - p_v (g + h (log p_v + entropy))) / T.
log p comes from the maximum and log1p of the rest of the mass, so it stays
accurate on peaked rows.
"""
from collections import namedtuple

import numpy as np

Scores = namedtuple("Scores", ["logprob", "entropy", "top_ids", "top_logprobs", "logp"])


def log_softmax_row(row, T, suppress=()):
    """log p of every id of one float64 row, -inf at suppressed ids."""
    x = np.where(np.isnan(row), -np.inf, row)
    allowed = np.ones(x.shape[0], dtype=bool)
    allowed[list(suppress)] = False
    x = np.where(allowed, x, -np.inf)
    m = x[allowed].max()
    logp = np.full(x.shape[0], -np.inf)
    if np.isinf(m):
        support = allowed & (x == m)
        logp[support] = -np.log(support.sum())
        return logp
    d = (x - m) / T
    at = int(np.argmax(x))
    rest = np.exp(d[np.arange(x.shape[0]) != at]).sum()
    logp[allowed] = (d - np.log1p(rest))[allowed]
    return logp


def token_logprobs(logits, targets, T=1.0, suppress=(), top=0):
    """logits (B, L, V) float64, targets (B, L)."""
    B, L, V = logits.shape
    lp, ent = np.zeros((B, L)), np.zeros((B, L))
    ids = np.full((B, L, top), -1, dtype=np.int32)
    tops = np.full((B, L, top), -np.inf)
    logp = np.full((B, L, V), -np.inf)
    for b in range(B):
        for l in range(L):
            t = int(targets[b, l])
            if not 0 <= t < V:
                continue
            r = log_softmax_row(logits[b, l], T, suppress)
            logp[b, l] = r
            lp[b, l] = r[t]
            live = r > -np.inf
            ent[b, l] = -(np.exp(r[live]) * r[live]).sum()
            x = np.where(np.isnan(logits[b, l]), -np.inf, logits[b, l])
            order = sorted(np.flatnonzero(live), key=lambda v: (-x[v], v))[:top] if top else []
            ids[b, l, :len(order)] = order
            tops[b, l, :len(order)] = r[order]
    return Scores(lp, ent, ids, tops, logp)


def token_logprobs_grad(s, targets, g, h, T=1.0, suppress=()):
    """From Scores s; g, h (B, L)."""
    B, L, V = s.logp.shape
    out = np.zeros((B, L, V))
    for b in range(B):
        for l in range(L):
            t = int(targets[b, l])
            if not 0 <= t < V:
                continue
            p = np.exp(s.logp[b, l])
            lp = np.where(p > 0, s.logp[b, l], 0.0)
            d = -p * (g[b, l] + h[b, l] * (lp + s.entropy[b, l]))
            d[t] += g[b, l]
            d[list(suppress)] = 0.0
            out[b, l] = d / T
    return out
