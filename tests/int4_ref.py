"""Plain implementations of the 4-bit head's operators and of beam search's, in
64 bits, written from their definitions in include/flashhead.h."""
from __future__ import annotations

import numpy as np
import torch

TINY = 2.0 ** -126
# bits 4 n .. 4 n + 3 of the word of columns 8 i .. 8 i + 7 hold column 8 i + ORDER[n]
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def bf16(x) -> np.ndarray:
    """fp32 values rounded to bf16."""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def pack(q) -> torch.Tensor:
    """Codes in [-8, 7] (rows x d, d a multiple of 8) as bytes."""
    q = torch.as_tensor(q).to(torch.int64)
    w = q.view(q.shape[0], -1, 8)[:, :, ORDER] & 15
    return (w[:, :, 0::2] | (w[:, :, 1::2] << 4)).reshape(q.shape[0], -1).to(torch.uint8)


def unpack(E4) -> np.ndarray:
    b = E4.cpu().to(torch.int64)
    b = b.view(b.shape[0], -1, 4)
    q = np.zeros((b.shape[0], b.shape[1], 8), np.int64)
    for n, column in enumerate(ORDER):
        u = ((b[:, :, n // 2] >> (4 * (n % 2))) & 15).numpy()
        q[:, :, column] = np.where(u > 7, u - 16, u)
    return q.reshape(b.shape[0], -1)


def quantize(E, group, zero):
    """Codes, scales and zeros (groups x v) of E.  Quotients are fp32 numbers: one
    of two fp32 numbers rounded from 64 bits to 32 is that."""
    x = f64(E)
    v, d = x.shape
    G = -(-d // group)
    q = np.zeros((v, d), np.int64)
    scales, zeros = np.zeros((G, v)), np.zeros((G, v))

    def fp32(a):
        return a.astype(np.float32).astype(np.float64)

    for g in range(G):
        part = x[:, g * group:(g + 1) * group]
        if zero:
            lo, hi = np.minimum(part.min(1), 0), np.maximum(part.max(1), 0)
            s = fp32(fp32(hi / 15) - fp32(lo / 15))
        else:
            s = fp32(np.abs(part).max(1) / 7)
        s = bf16(np.maximum(s, TINY))
        if zero:
            zeros[g] = np.clip(-8 - np.rint(fp32(lo / s)), -8, 7)
        q[:, g * group:(g + 1) * group] = np.clip(
            np.rint(fp32(part / s[:, None])) + zeros[g][:, None], -8, 7)
        scales[g] = s
    return q, scales, zeros


def values(E4, scale, zero, group) -> np.ndarray:
    q = unpack(E4).astype(np.float64)
    d = q.shape[1]
    if zero is not None:
        q = q - np.repeat(f64(zero).T, group, 1)[:, :d]
    return q * np.repeat(f64(scale).T, group, 1)[:, :d]


def logits_bound(h, E4, scale, zero, group) -> np.ndarray:
    """A bound on the error of the kernel's fp32 logits.  Per group it adds at
    most 128 products of h with 24 and 128 with 24 + q <= 31 (three parts of each for an
    fp32 h), so no sum on the way is over 55 sum |h|, and each of the 2 * 128 *
    parts sums is off by a step of fp32 at most (2^-23: the matrix unit may cut
    instead of rounding).  Then zero times sum |h|, three roundings of that size,
    the product with the scale and the sum over groups with one rounding each.  A
    kernel may start a group's sums at 24 + zero times the sum of -h instead: those
    128 additions weigh 24 + z, and the 128 products are added to sums of 55 + z at
    most, 128 (79 + 2 z) in all, which is under 256 * 55 + 7 z for z up to 15."""
    a, parts = np.abs(f64(h)), 3 if h.dtype == torch.float32 else 1
    s = f64(scale)
    G = s.shape[0]
    out = np.zeros((a.shape[0], s.shape[1]))
    z = np.abs(f64(zero)) if zero is not None else np.zeros_like(s)
    for g in range(G):
        sums = a[:, g * group:(g + 1) * group].sum(1)
        n = 2 * min(group, 128) * parts
        out += np.outer(sums, s[g] * (55 * n + (55 + z[g]) * (3 + G + 4))) * 2.0 ** -23
    return out


def beam(logits, scores, finished, n, pad, eos):
    """(scores, parents, tokens, finished), each B x n."""
    z, at = f64(logits), f64(scores)
    B, K = at.shape
    v = z.shape[1]
    done = np.zeros((B, K), bool) if finished is None else finished.cpu().numpy().astype(bool)
    out = (np.full((B, n), -np.inf), np.full((B, n), -1, np.int64), np.full((B, n), -1, np.int64),
           np.zeros((B, n), bool))
    for b in range(B):
        keys, places = [], []
        for k in range(K):
            if not np.isfinite(at[b, k]):
                continue
            if done[b, k]:
                keys.append(np.array([at[b, k]]))
                places.append(np.array([k * v + pad]))
                continue
            row = z[b * K + k]
            top = row.max()
            if not np.isfinite(top):   # a NaN makes it one
                continue
            # (a logarithm added to a large top would leave nothing of it, or of `at`)
            key = at[b, k] + ((row - top) - np.log(np.exp(row - top).sum()))
            t = np.nonzero(row > -np.inf)[0]
            keys.append(key[t])
            places.append(k * v + t)
        if not keys:
            continue
        keys, places = np.concatenate(keys), np.concatenate(places)
        order = np.lexsort((places, -keys))[:n]
        m = len(order)
        out[0][b, :m], out[1][b, :m], out[2][b, :m] = keys[order], places[order] // v, \
            places[order] % v
        out[3][b, :m] = done[b, out[1][b, :m]] | (out[2][b, :m] == eos)
    return out
