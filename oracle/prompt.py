"""Prompts and single tokens of a hybrid model's layers -- TEST INFRASTRUCTURE ONLY.

Plain fp64 definitions, one sequence at a time: linear attention with a decay for each
head (token by token), causal attention over a whole prompt, attention of one token over
a cache, and the e4m3 cache row.  Beside each result the sum of the magnitudes of its
terms is returned where a test bounds the roundings of those terms by it.
"""
from __future__ import annotations

import math

import numpy as np


def oracle_linear(q, k, v, alpha, beta=None, skip=None, S0=None):
    """One sequence: q, k [T, Hk, dk], v [T, Hv, dv], alpha, beta [T, Hv], S0 [Hv, dv, dk]:
    S <- alpha S + beta v k^T, o = S q + skip v.  Returns (o, S, |o| terms, |S| terms)."""
    q, k, v, alpha = (np.asarray(t, np.float64) for t in (q, k, v, alpha))
    T, Hv, dv = v.shape
    group = np.arange(Hv) // (Hv // q.shape[1])
    beta = np.ones((T, Hv)) if beta is None else np.asarray(beta, np.float64)
    skip = np.zeros(Hv) if skip is None else np.asarray(skip, np.float64)
    S = np.zeros((Hv, dv, k.shape[2])) if S0 is None else np.array(S0, np.float64)
    Sa = np.abs(S)
    o, oa = np.zeros_like(v), np.zeros_like(v)
    for t in range(T):
        kt, qt = k[t][group], q[t][group]
        w = beta[t][:, None] * v[t]
        S = alpha[t][:, None, None] * S + w[:, :, None] * kt[:, None, :]
        Sa = alpha[t][:, None, None] * Sa + np.abs(w)[:, :, None] * np.abs(kt)[:, None, :]
        o[t] = np.einsum("hvk,hk->hv", S, qt) + skip[:, None] * v[t]
        oa[t] = np.einsum("hvk,hk->hv", Sa, np.abs(qt)) + np.abs(skip[:, None] * v[t])
    return o, S, oa, Sa


def _attend(q, k, v, scale):
    s = scale * (k @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v)


def oracle_prompt_attention(q, k, v, scale):
    """One sequence: q [T, Hq, d], k, v [T, Hkv, d]; token t sees tokens 0 .. t.  Returns
    (o, sum of p |v|)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    T, Hq, _ = q.shape
    rep = Hq // k.shape[1]
    o, oa = np.zeros_like(q), np.zeros_like(q)
    for h in range(Hq):
        kh, vh = k[:, h // rep], v[:, h // rep]
        for t in range(T):
            o[t, h], oa[t, h] = _attend(q[t, h], kh[:t + 1], vh[:t + 1], scale)
    return o, oa


def oracle_decode_attention(q, k, v, scale):
    """One token: q [Hq, d] over k, v [n, Hkv, d] (zeros for n = 0).  Returns (o, sum of p |v|)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    o, oa = np.zeros_like(q), np.zeros_like(q)
    if k.shape[0] == 0:
        return o, oa
    rep = q.shape[0] // k.shape[1]
    for h in range(q.shape[0]):
        o[h], oa[h] = _attend(q[h], k[:, h // rep], v[:, h // rep], scale)
    return o, oa


def oracle_pages(pages, table_row, n):
    """The first n positions of one sequence: pages [P, H, page, d] -> [n, H, d]."""
    page = pages.shape[2]
    out = np.zeros((n,) + pages.shape[1:2] + pages.shape[3:], pages.dtype)
    for j in range(n):
        out[j] = pages[table_row[j // page], :, j % page]
    return out


def _e4m3(y: float) -> float:
    """The e4m3 value nearest to y (ties to even; beyond 448 to 448; NaN stays)."""
    if math.isnan(y):
        return y
    a = abs(y)
    if a >= 448.0:
        return math.copysign(448.0, y)
    e = max(math.frexp(a)[1] - 1, -6) if a else -6
    step = math.ldexp(1.0, e - 3)
    return math.copysign(round(a / step) * step, y)          # Python's round: ties to even


def oracle_cache_row(x):
    """One row of the 8-bit cache: (scale byte, values that it stands for)."""
    x = np.asarray(x, np.float64)
    fine = np.abs(x[np.isfinite(x)])
    top = float(fine.max()) if fine.size else 0.0
    e = -118
    while e < 119 and top > math.ldexp(448.0, e):
        e += 1
    s = math.ldexp(1.0, e)
    return e + 127, np.array([_e4m3(float(v) / s) * s for v in x])
