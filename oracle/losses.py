"""Scoring, the losses and the 8-bit LM head in double precision (numpy), from
their definitions in include/sampler.h.

Plain loops over rows; nothing is shared with the CUDA path. Every function
takes float64 (or exactly widened) inputs and returns float64.
"""
from __future__ import annotations

import numpy as np

OK, NONFINITE, ALL_NEG_INF, BAD_PARAM = 0, 1, 2, 3
GREEDY_T = np.float32(1e-5)
E4M3_MAX = 448.0
LEAST = 2.0 ** -100


def _row(x, T, token):
    """(status, log-probabilities) of one row."""
    if not T >= 0 or np.isinf(T) or not 0 <= token < len(x):
        return BAD_PARAM, None
    if np.isnan(x).any() or (x == np.inf).any():
        return NONFINITE, None
    if (x == -np.inf).all():
        return ALL_NEG_INF, None
    y = x / (1.0 if np.float32(T) < GREEDY_T else float(T))
    y = y - y.max()  # first: next to a large maximum the logarithm would be lost
    return OK, y - np.log(np.exp(y).sum())


def score(logits, tokens, temperature=None, weight=None):
    """dict of logprob, entropy, status [N] and logp [N, V] (the rows' log-probabilities)."""
    n, V = logits.shape
    got = dict(logprob=np.zeros(n), entropy=np.zeros(n), status=np.zeros(n, np.int32), logp=np.zeros((n, V)))
    for r in range(n):
        if weight is not None and weight[r] == 0:
            continue
        st, logp = _row(logits[r].astype(np.float64), 1.0 if temperature is None else temperature[r], int(tokens[r]))
        got["status"][r] = st
        if st != OK:
            got["logprob"][r] = got["entropy"][r] = np.nan
            got["logp"][r] = np.nan
            continue
        p = np.exp(logp)
        got["logp"][r] = logp
        got["logprob"][r] = logp[tokens[r]]
        with np.errstate(invalid="ignore"):
            got["entropy"][r] = -np.where(p > 0, p * logp, 0.0).sum()
    return got


def logits_grad(got, tokens, by_logprob, by_entropy, temperature=None, weight=None):
    """The gradient of the logits [N, V] from those by each row's logprob and entropy."""
    n, V = got["logp"].shape
    grad = np.zeros((n, V))
    for r in range(n):
        if weight is not None and weight[r] == 0:
            continue
        if got["status"][r] != OK:
            grad[r] = np.nan
            continue
        T = 1.0 if temperature is None or np.float32(temperature[r]) < GREEDY_T else float(temperature[r])
        logp = got["logp"][r]
        p = np.exp(logp)
        one = np.zeros(V)
        one[tokens[r]] = 1.0
        a = 0.0 if by_logprob is None else by_logprob[r]
        b = 0.0 if by_entropy is None else by_entropy[r]
        with np.errstate(invalid="ignore"):
            h = np.where(p > 0, p * (logp + got["entropy"][r]), 0.0)
        grad[r] = (a * (one - p) - b * h) / T
    return grad


def policy(logits, tokens, old, advantage, ref=None, temperature=None, weight=None, clip_low=0.2, clip_high=0.2,
           kl_coef=0.0, entropy_coef=0.0, grad_scale=1.0):
    n = logits.shape[0]
    got = score(logits, tokens, temperature, weight)
    w = np.ones(n) if weight is None else weight.astype(np.float64)
    live = w != 0
    with np.errstate(over="ignore", invalid="ignore"):
        ratio = np.exp(got["logprob"] - old)
        cut = np.clip(ratio, 1.0 - clip_low, 1.0 + clip_high)
        term = -np.minimum(ratio * advantage, cut * advantage)
        decided = ((advantage > 0) & (ratio > 1.0 + clip_high)) | ((advantage < 0) & (ratio < 1.0 - clip_low))
        by_lp = np.where(decided, 0.0, -ratio * advantage)
        kl = np.zeros(n)
        if ref is not None:
            d = ref - got["logprob"]
            kl = np.where(np.isinf(d), np.inf, np.expm1(d) - d)
            if kl_coef != 0:
                term = term + kl_coef * kl
                by_lp = by_lp - kl_coef * np.expm1(d)
        if entropy_coef != 0:
            term = term - entropy_coef * got["entropy"]
    got["ratio"], got["kl"] = np.where(live, ratio, 0.0), np.where(live, kl, 0.0)
    got["loss"] = float((w * term)[live].sum())
    by_h = -entropy_coef * w * grad_scale if entropy_coef != 0 else None
    got["by_logprob"], got["by_entropy"] = np.where(live, w * by_lp * grad_scale, 0.0), by_h
    got["grad"] = logits_grad(got, tokens, got["by_logprob"], by_h, temperature, weight)
    return got


def preference(logits, tokens, offsets, ref=None, temperature=None, weight=None, beta=0.1, margin=0.0,
               label_smoothing=0.0, mean_over_tokens=False, grad_scale=1.0):
    n, pairs = logits.shape[0], (len(offsets) - 1) // 2
    got = score(logits, tokens, temperature, weight)
    w = np.ones(n) if weight is None else weight.astype(np.float64)
    reward, share = np.zeros(2 * pairs), np.ones(2 * pairs)
    spans = []
    for s in range(2 * pairs):
        b, e = int(offsets[s]), int(offsets[s + 1])
        if not 0 <= b <= e <= n:
            reward[s] = np.nan
            spans.append((0, 0))
            continue
        spans.append((b, e))
        rows = [r for r in range(b, e) if w[r] != 0]
        total = sum(w[r] * (got["logprob"][r] - (0.0 if ref is None else ref[r])) for r in rows)
        if mean_over_tokens:
            count = sum(w[r] for r in rows)
            share[s] = 1.0 / count if count != 0 else 0.0
        reward[s] = beta * share[s] * total
    by_lp = np.zeros(n)
    loss = 0.0
    for i in range(pairs):
        z = reward[2 * i] - reward[2 * i + 1] - margin
        if np.isnan(z):
            loss = np.nan
        else:
            loss += (1.0 - label_smoothing) * np.logaddexp(0.0, -z) + label_smoothing * np.logaddexp(0.0, z)
        with np.errstate(over="ignore"):
            by_z = 1.0 / (1.0 + np.exp(-z)) - (1.0 - label_smoothing)
        for k in range(2):
            b, e = spans[2 * i + k]
            by_lp[b:e] = (by_z if k == 0 else -by_z) * beta * share[2 * i + k] / pairs * w[b:e] * grad_scale
    inside = np.zeros(n, int)
    for b, e in spans:
        inside[b:e] += 1
    by_lp[inside > 1] = np.nan  # in more than one answer
    got["by_logprob"] = by_lp
    got["reward"], got["loss"] = reward, loss / pairs if pairs else 0.0
    got["grad"] = logits_grad(got, tokens, by_lp, None, temperature, weight)
    # a row whose pair has no finite margin takes a NaN gradient with it
    got["grad"][np.isnan(by_lp) & (w != 0)] = np.nan
    return got


def e4m3_table():
    """The 256 values of the e4m3 codes (NaN at 0x7f and 0xff)."""
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return t


def to_e4m3(x):
    """Codes of the nearest e4m3 values (ties to the even code), |x| up to 464."""
    positive = e4m3_table()[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(positive, a), 1, 126)
    lo = hi - 1
    below, above = a - positive[lo], positive[hi] - a
    code = np.where(below < above, lo, np.where(below > above, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= positive[126], 126, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize(src, block_rows):
    """(codes, scales) by the definition's own fp32 operations."""
    rows, cols = src.shape
    src = src.astype(np.float32)
    up, across = -(-rows // block_rows), -(-cols // 128)
    codes, scales = np.zeros((rows, cols), np.uint8), np.zeros((up, across), np.float32)
    for i in range(up):
        for j in range(across):
            at = np.s_[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128]
            b = src[at]
            if not np.isfinite(b).all():
                scales[i, j] = np.nan
                continue
            m = np.float32(max(np.abs(b).max(), np.float32(LEAST)))
            scales[i, j] = m / np.float32(E4M3_MAX)
            codes[at] = to_e4m3((b * (np.float32(E4M3_MAX) / m)).astype(np.float64))
    return codes, scales


def scaled_head(hidden, hidden_scale, weight, weight_scale):
    """(logits, sum of the products' magnitudes) from codes and scales; float64."""
    t = e4m3_table()
    rows, K = hidden.shape
    V = weight.shape[0]
    out, mag = np.zeros((rows, V)), np.zeros((rows, V))
    for b in range(-(-K // 128)):
        at = np.s_[:, 128 * b:128 * b + 128]
        h, w = t[hidden[at]], t[weight[at]]
        s = hidden_scale[:, b].astype(np.float64)[:, None] * np.repeat(weight_scale[:, b], 128)[:V].astype(np.float64)
        out += s * (h @ w.T)
        mag += np.abs(s) * (np.abs(h) @ np.abs(w).T)
    return out, mag
