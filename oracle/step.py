"""A step of new tokens: page tables and slot maps, positions of several axes, norms with the
rotation, and which keys a chunk's queries see (oracle side).

TEST INFRASTRUCTURE ONLY.  Python integers and numpy, from the definitions:

* a request of ctx tokens that gets n more has floor((ctx + n) / ratio) rows, 64 to a page; new
  pages come from the front of a ring of free ones, requests in order, and where none is left the
  table has -1; a request that ends gives the pages that it has back behind the ring's last one;
* pair k of the rotated dims turns by position * theta^(-2k/64) along its own axis;
* a norm and rotation is the compressor's contract for one token (its sums, roundings and codes);
* the query at position t sees the entries j < floor((t + 1) / ratio) and the rows
  max(0, t - window + 1) .. t.
"""

import numpy as np

from . import codecs, compress, rope

PAGE = 64
F32 = np.float32


def pages_of(rows):
    return (rows + PAGE - 1) // PAGE


def plan_step(ctx, new, T, ratio, ring_rows=0, table=None, free=None, state=None, shared=None):
    """Dict of cu, len, first_row, n_rows, req, pos1, slot, ring_slot, table, free, state (the last
    three copies with the step's changes; None without a table)."""
    table = None if table is None else np.array(table)
    free = None if free is None else np.array(free)
    head, count = (int(state[0]), int(state[1])) if table is not None else (0, 0)
    out = {k: [] for k in ("len", "first_row", "n_rows")}
    out["cu"] = [0]
    req, pos1, slot, ring = [-1] * T, [0] * T, [-1] * T, [-1] * T
    given, taken, short = [], 0, 0
    for b, (have, n) in enumerate(zip(ctx, new)):
        have, n, at = int(have), int(n), out["cu"][-1]
        ends = n < 0
        n = 0 if ends else min(n, T - at)
        after = 0 if ends else have + n
        first, rows = (0, 0) if ends else (have // ratio, after // ratio)
        if table is not None:
            if ends:
                own = 0 if shared is None else int(shared[b])
                given += [int(p) for p in table[b, min(own, pages_of(have // ratio)):pages_of(have // ratio)] if p >= 0]
            for lp in range(pages_of(first), pages_of(rows)):
                if taken < count:
                    table[b, lp] = free[(head + taken) % len(free)]
                    taken += 1
                else:
                    table[b, lp] = -1
                    short += 1
        for k in range(n):
            p = have + k
            req[at + k], pos1[at + k] = b, p + 1
            row = (p + 1) // ratio - 1
            if table is not None and (p + 1) % ratio == 0 and table[b, row // PAGE] >= 0:
                slot[at + k] = int(table[b, row // PAGE]) * PAGE + row % PAGE
            if ring_rows and p >= after - ring_rows:
                ring[at + k] = b * ring_rows + p % ring_rows
        out["cu"].append(at + n)
        out["len"].append(after)
        out["first_row"].append(first)
        out["n_rows"].append(rows)
    out.update(req=req, pos1=pos1, slot=slot, ring_slot=ring, table=table, free=free, state=None)
    if table is not None:
        for j, p in enumerate(given):
            free[(head + count + j) % len(free)] = p
        out["state"] = [(head + taken) % len(free), count - taken + len(given), short, 0]
    return out


def rope_cs(positions, axis_of, theta=rope.THETA_COMPRESSED, yarn=None):
    """[axes, T] integer positions -> float64 [T, 32, 2] of (cos, sin)."""
    f = rope.inv_freq(theta, yarn=yarn)
    a = np.asarray(positions, np.float64)[np.asarray(axis_of)].T * f
    return np.stack([np.cos(a), np.sin(a)], -1)


def norm_rope(x, norm, norm_w, eps, cs):
    """fp32 contract of x [n, D] (exact bf16 values): float32 [n, D] before any coding."""
    y = np.asarray(x, F32)
    if norm:
        ss = compress.pairwise_sum_f32((y * y).astype(F32))
        rr = (F32(1.0) / np.sqrt(((ss / F32(y.shape[-1])).astype(F32) + F32(eps)).astype(F32))).astype(F32)
        w = np.ones(y.shape[-1], F32) if norm_w is None else np.asarray(norm_w, F32)
        y = ((y * rr[..., None]).astype(F32) * w).astype(F32)
    if cs is not None:
        y = rope.rotate_table_fp32(y, cs)
    return y


def chunk_keys(t, ratio, n_entries, window):
    """(number of entries, first row, one past the last row) that a query at position t sees."""
    n = (t + 1) // ratio if ratio else n_entries
    if n_entries is not None:
        n = min(n, n_entries)
    return n, max(0, t - window + 1) if window else t + 1, t + 1
