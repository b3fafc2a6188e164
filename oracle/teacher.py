"""The most likely tokens of rows, and distillation from them, in double precision
(numpy), from their definitions in include/sampler.h. Plain loops over rows; nothing
is shared with the CUDA path."""
from __future__ import annotations

import numpy as np

from .losses import BAD_PARAM, OK, _row


def log_sum(x):
    """ln of the sum of e^x (-inf for none)."""
    m = x.max() if len(x) else -np.inf
    return m if m == -np.inf else m + np.log(np.exp(x - m).sum())


def top(logits, n, tokens=None, temperature=None, weight=None):
    """dict of ids and logprobs [N, n], rest, logprob, entropy, status [N]."""
    rows, V = logits.shape
    got = dict(ids=np.full((rows, n), -1, np.int32), logprobs=np.zeros((rows, n)), rest=np.zeros(rows),
               logprob=np.zeros(rows), entropy=np.zeros(rows), status=np.zeros(rows, np.int32))
    for r in range(rows):
        if weight is not None and weight[r] == 0:
            continue
        token = 0 if tokens is None else int(tokens[r])
        x = logits[r].astype(np.float64)
        st, logp = _row(x, 1.0 if temperature is None else temperature[r], token)
        got["status"][r] = st
        if st != OK:
            for k in ("logprobs", "rest", "logprob", "entropy"):
                got[k][r] = np.nan
            continue
        order = np.lexsort((np.arange(V), -x))[:n]
        order = order[x[order] > -np.inf]
        got["ids"][r, :len(order)] = order
        got["logprobs"][r] = -np.inf
        got["logprobs"][r, :len(order)] = logp[order]
        got["rest"][r] = log_sum(np.delete(logp, order))
        got["logprob"][r] = logp[token]
        p = np.exp(logp)
        with np.errstate(invalid="ignore"):
            got["entropy"][r] = -np.where(p > 0, p * logp, 0.0).sum()
    return got


def distill(logits, ids, logprobs, rest=None, tokens=None, token_coef=0.0, temperature=None, weight=None, grad_scale=1.0):
    """dict of loss, kl, logprob, status [N] and grad [N, V]."""
    rows, V = logits.shape
    kl, lp, status, grad = np.zeros(rows), np.zeros(rows), np.zeros(rows, np.int32), np.zeros((rows, V))
    loss = 0.0
    for r in range(rows):
        w = 1.0 if weight is None else float(weight[r])
        if w == 0:
            continue
        token = 0 if tokens is None else int(tokens[r])
        T = 1.0 if temperature is None else temperature[r]
        st, logp = _row(logits[r].astype(np.float64), T, token)
        there = ids[r] != -1
        at, l = ids[r][there].astype(int), logprobs[r][there].astype(np.float64)
        tail = -np.inf if rest is None else float(rest[r])
        if (len(set(at)) < len(at) or (at < 0).any() or (at >= V).any() or not (l < np.inf).all() or not tail < np.inf):
            st = BAD_PARAM
        status[r] = st
        if st != OK:
            kl[r] = lp[r] = np.nan
            grad[r] = np.nan
            loss = np.nan
            continue
        Te = 1.0 if np.float32(T) < np.float32(1e-5) else float(T)
        p = np.exp(logp)
        q, qr = np.exp(l), np.exp(tail)
        outside = np.ones(V, bool)
        outside[at] = False
        with np.errstate(invalid="ignore", divide="ignore"):
            k = np.where(q > 0, q * (l - logp[at]), 0.0).sum()
            ln_out = log_sum(logp[outside])
            if qr > 0:
                k += qr * (tail - ln_out)
        total = q.sum() + qr + token_coef
        g = total * p
        g[at] -= q
        if qr > 0 and ln_out > -np.inf:
            g[outside] -= qr * np.exp(logp[outside] - ln_out)
        each = k
        if token_coef:
            each = each - token_coef * logp[token]
            g[token] -= token_coef
        kl[r], lp[r] = k, logp[token]
        loss += w * each
        grad[r] = g * (w * grad_scale / Te)
    return dict(loss=loss, kl=kl, logprob=lp, status=status, grad=grad)
