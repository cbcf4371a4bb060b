"""Inputs and tolerances shared by the GPU tests of the prompt, single-token and cache calls.

Tolerances are element-wise and count roundings.  U is the relative size of a rounding to
bf16 (half a step, 2^-8); a result o = sum_i t_i whose terms are each rounded once to bf16
and which is itself rounded once is off by at most U |o| + U sum |t_i| (and U^2 terms,
below the slack).  fp32 work is counted at 2^-23 an operation (a matrix instruction may
truncate where an adder rounds) along the longest chain of operations."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -8
E = 2.0 ** -23


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).cuda()


def f32(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def within(got, ref, tol, what):
    got, ref, tol = np.asarray(got), np.asarray(ref), np.broadcast_to(tol, np.shape(ref))
    assert got.shape == ref.shape, what
    # A NaN of the definition (of a NaN among its terms) is a NaN of the result, and nothing else is.
    nan = np.isnan(ref)
    assert np.array_equal(nan, ~np.isfinite(got)), f"{what}: {np.count_nonzero(nan != ~np.isfinite(got))} values are not finite"
    off = np.where(nan, 0.0, np.abs(np.where(nan, 0.0, got) - np.where(nan, 0.0, ref)))
    over = off - np.where(nan, 0.0, tol)
    assert not over.size or over.max() <= 0, f"{what}: off by {off.flat[over.argmax()]:.3g}, allowed {tol.flat[over.argmax()]:.3g}"


def attention_tol(o, oa, score_abs):
    """bf16 output and probabilities; a score is a sum of 128 products and a probability's relative
    error is its score's error (twice: numerator and denominator)."""
    return U * np.abs(o) + (U + 2 * 130 * E * score_abs + 64 * E) * oa + 1e-30


def random_tables(rng, lens, page, spare=3):
    """Pages in random order; entries past a sequence's last page are out of range (never read)."""
    need = [-(-int(n) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(1, max(need, default=1)) + 1), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, max(1, sum(need) + spare)
