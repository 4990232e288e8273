"""Attention over bounded and shared caches and eviction by weight (oracle side).

TEST INFRASTRUCTURE ONLY.  fp64 numpy, one query row at a time, from the definitions:

* a query at position t sees the rows j <= t with j < first or j > t - window;
* a decode row sees its request's entries j < n (those below the shared prefix read
  from request 0) and its window ring;
* one softmax with a sink logit: lse = ln(sum_j exp(z_j) + exp(sink)), weights
  exp(z_j - lse);
* an entry's weight is the sum of its weights over the heads;
* eviction keeps the protected slots, then the largest weights (ties: the lower slot),
  and moves the kept slots behind the budget into the given-up slots before it.

``attend`` also gives, per output, how far a computation may be from it that rounds the
rotated query to a sum of two bf16 values, the weights and the result to bf16, and
everything else to fp32.
"""

import numpy as np

from . import rope

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24     # half steps, relative


def visible(t, window, first):
    j = np.arange(t + 1)
    return j[(j < first) | (j > t - window)]


def attend(q, t, keys, sink, scale):
    """q [H, 512], keys [n, 512] (decoded), position t of the rotation.

    Returns (out [H, 512], lse [H], bound of out [H, 512], bound of lse [H]).
    """
    H = q.shape[0]
    ang = rope.angles(np.array([t]))[0]
    qr = rope.rotate_fp64(np.asarray(q, np.float64), ang[None, :])
    keys = np.asarray(keys, np.float64).reshape(-1, 512)
    n = keys.shape[0]
    zs = np.full(H, -np.inf) if sink is None else np.asarray(sink, np.float64)
    if n == 0:
        return np.zeros((H, 512)), zs.copy(), np.zeros((H, 512)), U_F32 * 2 * np.abs(np.where(np.isinf(zs), 0, zs))
    z = qr @ keys.T * scale
    M = np.maximum(z.max(1), zs)
    e = np.exp(z - M[:, None])
    den = e.sum(1) + np.exp(zs - M)
    p = e / den[:, None]
    lse = M + np.log(den)
    o = p @ keys
    out = rope.rotate_fp64(o, ang[None, :], inverse=True)
    # logits: the query's second half step (U_BF16 squared), fp32 products, sums, scaling and table
    dz = (U_BF16 ** 2 + (512 + 8) * U_F32) * (np.abs(qr) @ np.abs(keys).T) * scale + 8 * U_F32 * np.abs(z - M[:, None])
    # weights: the logits' error in numerator and denominator, sums of n terms, exp in fp32
    drel = 2 * dz.max(1) + (n + 16) * U_F32
    spread = p @ np.abs(keys)
    turned = spread.copy()
    c, s = np.abs(np.cos(ang)), np.abs(np.sin(ang))
    y0, y1 = spread[:, 448::2], spread[:, 449::2]
    turned[:, 448::2], turned[:, 449::2] = y0 * c + y1 * s, y0 * s + y1 * c
    b_out = (U_BF16 + drel[:, None] + (n + 16) * U_F32) * turned * 1.01 + U_BF16 * np.abs(out)
    b_lse = dz.max(1) + (n + 16) * U_F32 + 4 * U_F32 * np.abs(lse)
    return out, lse, b_out, b_lse


def weights(q, t, keys, lse, scale):
    """Sum over the heads of exp(z - lse) of every key, and its bound."""
    ang = rope.angles(np.array([t]))[0]
    qr = rope.rotate_fp64(np.asarray(q, np.float64), ang[None, :])
    keys = np.asarray(keys, np.float64).reshape(-1, 512)
    z = qr @ keys.T * scale
    lse = np.asarray(lse, np.float64)
    p = np.where(np.isneginf(lse)[:, None], 0.0, np.exp(z - lse[:, None]))
    dz = (U_BF16 ** 2 + (512 + 8) * U_F32) * (np.abs(qr) @ np.abs(keys).T) * scale
    dz += 8 * U_F32 * (np.abs(z) + np.where(np.isinf(lse), 0, np.abs(lse))[:, None])
    w = p.sum(0)
    return w, (p * dz).sum(0) * 1.01 + (q.shape[0] + 8) * U_F32 * w


def evict(acc, age, n, budget, fixed, recent):
    """(src [budget], m): slot i < m holds the entry of slot src[i]; -1 after m."""
    src = np.full(budget, -1, np.int64)
    m = min(n, budget)
    if n <= budget:
        src[:n] = np.arange(n)
        return src, m
    a = np.asarray(acc[:n], np.float64)
    safe = np.arange(n) < fixed
    if age is not None and recent > 0:
        g = np.asarray(age[:n], np.int64)
        safe |= g > g.max() - recent
    rank = [(0 if safe[i] else 1, 1 if np.isnan(a[i]) and not safe[i] else 0,
             0.0 if safe[i] or np.isnan(a[i]) else -a[i], i) for i in range(n)]
    keep = np.zeros(n, bool)
    keep[[r[3] for r in sorted(rank)[:m]]] = True
    src[:m] = np.arange(m)
    src[np.flatnonzero(~keep[:m])] = m + np.flatnonzero(keep[m:])
    return src, m
