"""Plain float64 implementations of the operators around the head (the norm
with 8-bit output, the 8-bit head's codes and logits, the verification of
drafted tokens), written from their definitions in include/flashhead.h, and
the tolerances that the tests derive from the kernels' number formats."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128
FLOOR = 2.0 ** -126
U32 = 2.0 ** -24                                   # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def norm(x, residual, weight, eps, offset):
    """(t, y) in float64."""
    t = f64(x) + (f64(residual) if residual is not None else 0.0)
    w = f64(weight) if weight is not None else np.ones(t.shape[1])
    rms = np.sqrt((t * t).sum(1, keepdims=True) / t.shape[1] + eps)
    return t, t / rms * (w + offset)


# The row's sum of squares: at most 8 units of 8 values in a row per thread
# (64 fused adds), 6 steps across a wave and 4 across waves, all terms
# positive, each step off by half a step of fp32: 74, halved by the root.
# Then the mean, eps, the root, its reciprocal, two products, t's own sum and
# the weight's (with its offset): under 10 more.
NORM_STEPS = 74 / 2 + 10


def check_norm(y, y64):
    e = (NORM_STEPS * U32 + half_step(y.dtype)) * 1.001
    assert np.all(np.abs(f64(y) - y64) <= e * np.abs(y64) + 2.0 ** -133)


def blocks_max(a, by):
    """max |a| of each block of by x 128, cut at the ends."""
    v, d = a.shape
    out = np.zeros((-(-v // by), -(-d // BLOCK)))
    for i in range(out.shape[0]):
        rows = np.abs(a[i * by:(i + 1) * by])
        for j in range(out.shape[1]):
            out[i, j] = rows[:, j * BLOCK:(j + 1) * BLOCK].max()
    return out


def spread(scale, by, v, d):
    return np.repeat(np.repeat(scale, by, 0)[:v], BLOCK, 1)[:, :d]


def check_codes(codes, scale, a64, by, steps):
    """Codes and scales of a64, whose values the kernel has within `steps`
    half steps of fp32.  A code is the nearest e4m3 value: off by 2^-4 of
    itself at most, or by 2^-10 below the smallest normal code 2^-6."""
    v, d = a64.shape
    want = np.maximum(blocks_max(a64, by) / 448.0, FLOOR)
    got = f64(scale)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= (steps + 1) * U32 * 1.001 * want)
    s = spread(got, by, v, d)
    c = f64(codes)
    assert np.all(np.isfinite(c))
    q = a64 / s
    # the quotient's own rounding and the value's `steps`
    slack = (steps + 1) * U32 * 1.001 * np.abs(q)
    step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))), 2.0 ** -6) / 16
    assert np.all(np.abs(c - q) <= step + slack)


def dequant(codes, scale, by):
    return f64(codes) * spread(f64(scale), by, *codes.shape)


def logits(h8, hs, E8, es):
    """(z, sum of |products|) in float64."""
    h, E = dequant(h8, hs, 1), dequant(E8, es, BLOCK)
    return h @ E.T, np.abs(h) @ np.abs(E).T


def check_logits(out, z, mag, d):
    """Products of two e4m3 codes are exact in fp32.  A block's sum of 128 of
    them takes at most 128 additions, each off by at most one step of fp32 of
    the block's sum of magnitudes (the matrix instruction's own rounding is
    not stated, so a whole step each); then the scales' product, its product
    with the sum and one addition per block, half a step each.

    More than 16 rows with bf16 outputs may take the 8-bit matrix instruction,
    which drops the bits below 2^-13 of the largest product of each 8: the 7
    others lose less than 7 * 2^-13 of it, and the groups' largest products
    sum to no more than all magnitudes."""
    g = -(-d // BLOCK)
    e = (128 * 2 + 2 + g) * U32 * 1.001
    if out.dtype == torch.bfloat16 and out.shape[0] > 16:
        e += 7 * 2.0 ** -13
    assert np.all(np.abs(f64(out) - z) <= e * mag + half_step(out.dtype) * (1.001 * np.abs(z)
                  + e * mag) + 2.0 ** -133)


def verify(logits, row_start, draft_tokens, max_tokens, *, sample, tau=1.0, q=None,
           u_accept=None, u_sample=None):
    """(tokens, accepted, logp): the definition, one sequence after another.
    logits, q: float64 arrays; the others lists or arrays."""
    B, (rows, v) = len(row_start) - 1, logits.shape
    n_drafts = len(draft_tokens)
    k = 1.0 / tau if sample else 1.0
    tokens = np.full((B, max_tokens), -1, np.int64)
    logp = np.zeros((B, max_tokens))
    accepted = np.zeros(B, np.int64)

    def dist(r):
        z = logits[r]
        top = z.max()
        if not np.isfinite(top):                    # NaN, +inf, or all -inf
            return None, None, -1
        e = np.exp((z - top) * k)
        return e / e.sum(), (z - top) * k - math.log(e.sum()), int(z.argmax())

    for s in range(B):
        r0, r1 = int(row_start[s]), int(row_start[s + 1])
        n, d0 = r1 - r0 - 1, r0 - s
        if r0 < 0 or n < 0 or r1 > rows or n >= max_tokens or d0 < 0 or d0 + n > n_drafts or \
                any(not 0 <= int(draft_tokens[d0 + j]) < v for j in range(n)):
            accepted[s] = -1
            continue
        for j in range(n + 1):
            p, lp, best = dist(r0 + j)
            x = int(draft_tokens[d0 + j]) if j < n else -1
            if j < n and p is not None:
                if sample:
                    qx = q[d0 + j, x] if q is not None else 1.0
                    take = float(u_accept[d0 + j]) * qx < p[x]
                else:
                    take = x == best
                if take:
                    tokens[s, j], logp[s, j] = x, lp[x]
                    accepted[s] += 1
                    continue
            if p is None:
                break
            y = best
            if sample:
                w = p
                if j < n and q is not None:
                    w = np.fmax(p - q[d0 + j], 0.0)
                elif j < n:
                    w = p.copy()
                    w[x] = 0.0
                if not w.sum() > 0:
                    w = p
                c = np.cumsum(w)
                over = np.nonzero((c > float(u_sample[s]) * c[-1]) & (w > 0))[0]
                y = int(over[0]) if over.size else int(np.nonzero(w > 0)[0][-1])
            tokens[s, j], logp[s, j] = y, lp[y]
            break
    return tokens, accepted, logp
