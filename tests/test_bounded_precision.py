"""How exact window_attn, prefix_decode_attn and attn_weights are over many values, beside the
worst-case bounds of test_gpu_bounded_cache.py, which a computation with fewer terms of the query
would still meet.

include/cskvx.h states the errors of logits of N(0, 2): 2.2e-6 (rms) in the attention, whose
rotated query is the sum of two bf16 numbers, and 2.3e-7 in the weights, with three numbers and
four short sums (with the two longer ones of more than 64 heads still below the limit here).  A logit is measured by itself: as the log-sum-exp of a query that sees one row, and
as the weight of an entry for the one head whose log-sum-exp is not -inf.  Limits:

* rms: three times the stated error.  What the measurement adds is below that: a weight's
  argument of exp lies below 16 in base 2 (half steps up to 4.8e-7, 1.7e-7 rms after the product
  with ln 2), exp2 is off by 1.7e-7 at most and the sums of four parts by 6e-8 of 8; together
  3.4e-7 beside 6.9e-7.  A log-sum-exp is off by three half steps of 8, 7e-7 beside 6.6e-6.
* largest: five times the rms limit, which one of 5,000 normal values passes with 3e-3 odds if
  the rms itself stood at the limit, and practically never at the stated one.
* outputs: the norm of the error within a tenth of that of the documented roundings in fp64
  (weights to bf16 over the sum of the rounded ones, the result to bf16).  It is made of 10^5
  roundings and more, and of some hundred rows' few largest weights: a few percent of scatter.

The checks themselves are tested on the CPU: they pass the documented computation and refuse
the one with a term of the query left out."""

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import codecs, rope

SCALE = 512 ** -0.5
ATTENTION_LOGIT, WEIGHT_LOGIT = 2.2e-6, 2.3e-7


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def _turn(x, cs, back=False):
    """[rows, H, 512] with the last 64 dims turned by cs [rows, 32, 2], in fp64."""
    c, s = cs[:, None, :, 0].astype(np.float64), cs[:, None, :, 1].astype(np.float64) * (-1 if back else 1)
    y, y0, y1 = np.array(x, np.float64), x[..., 448::2], x[..., 449::2]
    y[..., 448::2], y[..., 449::2] = y0 * c - y1 * s, y0 * s + y1 * c
    return y


def _cut(x, terms):
    """The turned dims as a sum of `terms` bf16 numbers."""
    y = x.copy()
    rest, y[..., 448:] = x[..., 448:].copy(), 0.0
    for _ in range(terms):
        t = _bf16(rest)
        y[..., 448:] += t
        rest -= t
    return y


def _attend(q, keys, sink, cs, terms=None):
    """One softmax per row and head over keys [rows, n, 512]: exactly, or (terms) with the
    documented roundings."""
    r = _turn(q, cs)
    if terms is not None:
        r = _cut(r, terms)
    z = np.einsum("bhd,bnd->bhn", r, keys) * SCALE
    p = np.exp(z - z.max(-1, keepdims=True))
    total = p.sum(-1) + np.exp(sink - z.max(-1))
    w = p if terms is None else _bf16(p) * (p.sum(-1) / _bf16(p).sum(-1))[..., None]
    out = _turn(np.einsum("bhn,bnd->bhd", w, keys) / total[..., None], cs, back=True)
    return out if terms is None else _bf16(out)


def _logit_errors_are_within(err, stated):
    rms, largest = float(np.sqrt(np.mean(np.square(err)))), float(np.abs(err).max())
    return rms <= 3 * stated and largest <= 15 * stated


def _output_errors_are_within(out, q, keys, sink, cs):
    exact = _attend(q, keys, sink, cs)
    stated = np.linalg.norm(_attend(q, keys, sink, cs, terms=2) - exact)
    return np.linalg.norm(out - exact) <= 1.1 * stated


def _cs(pos):
    ang = rope.angles(np.asarray(pos, np.int64))
    return np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def _inputs(rows, H, n, seed, turned=False):
    """Queries with logits of N(0, 2); `turned`: all of it from the turned dims."""
    rs = np.random.default_rng(seed)
    q = _bf16(2.0 * rs.standard_normal((rows, H, 512)))
    if turned:
        q *= 8 ** 0.5 * (np.arange(512) >= 448)
        q = _bf16(q)
    keys = _bf16(rs.standard_normal((rows, n, 512)))
    return q, keys, rs.standard_normal(H), _cs(rs.integers(0, 100000, rows))


# --- the checks --------------------------------------------------------------------------------

@pytest.mark.parametrize("H", [1, 16])
def test_the_logit_checks_refuse_a_query_with_a_term_left_out(H):
    q, keys, _, cs = _inputs(80, H, 30, seed=H)
    r = _turn(q, cs)
    err = [(np.einsum("bhd,bnd->bhn", _cut(r, t) - r, keys) * SCALE).ravel() for t in range(4)]
    assert _logit_errors_are_within(err[2], ATTENTION_LOGIT)
    assert not _logit_errors_are_within(err[1], ATTENTION_LOGIT)
    assert _logit_errors_are_within(err[3], WEIGHT_LOGIT)
    assert not _logit_errors_are_within(err[2], WEIGHT_LOGIT)
    # sums in one run of roundings, as a product of all 512 dims in one accumulator has them
    rs = np.random.default_rng(1)
    assert not _logit_errors_are_within(ATTENTION_LOGIT * rs.standard_normal(5000), WEIGHT_LOGIT)
    assert _logit_errors_are_within(WEIGHT_LOGIT * rs.standard_normal(5000), WEIGHT_LOGIT)


def test_the_output_check_refuses_a_query_with_a_term_left_out():
    a = _inputs(24, 16, 300, seed=5, turned=True)
    assert _output_errors_are_within(_attend(*a, terms=2), *a)
    assert not _output_errors_are_within(_attend(*a, terms=1), *a)


# --- the kernels -------------------------------------------------------------------------------

def _paged(keys):
    """A cache whose request b has the rows keys[b] (BF16: exactly), in its own pages in order."""
    rows, n = keys.shape[:2]
    pages = (n + 63) // 64
    flat = np.zeros((rows, pages * 64, 512), np.float32)
    flat[:, :n] = keys
    pool = codecs.encode_rows(flat.reshape(-1, 512), codecs.FMT_BF16).reshape(rows * pages, 64 * 1024)
    table = np.arange(rows * pages, dtype=np.int32).reshape(rows, pages)
    return cskv.PagedCache(torch.from_numpy(pool).cuda(), torch.from_numpy(table).cuda(), cskv.FMT_BF16, 512)


def _dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 16, 64, 65, 128])
def test_logits_of_the_attention(H):
    """A query that sees one row: its log-sum-exp is the logit."""
    rows = 5000 // H + 1
    q, keys, _, cs = _inputs(rows, H, 1, seed=10 + H)
    z = np.einsum("bhd,bnd->bhn", _turn(q, cs), keys)[..., 0] * SCALE
    cache, one = _paged(keys), torch.ones(rows, dtype=torch.int32, device="cuda")
    bq, bcs = _dev(q, torch.bfloat16), _dev(cs)
    for lse in (cskv.window_attn(bq, cache, one, 1, 0, 1, None, SCALE, bcs, want_lse=True)[1],
                cskv.prefix_decode_attn(bq, cache, one, 0, 1, None, SCALE, bcs, want_lse=True)[1]):
        assert _logit_errors_are_within(lse.double().cpu().numpy() - z, ATTENTION_LOGIT)
    assert cskv.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 16, 64, 65, 128])
def test_logits_of_the_weights(H):
    """One head of each request has a log-sum-exp above -inf: an entry's weight is its exp(logit)."""
    rows, n = 10, 520
    q, keys, _, cs = _inputs(rows, H, n, seed=20 + H)
    head = np.random.default_rng(H).integers(0, H, rows)
    z = np.einsum("bhd,bnd->bhn", _turn(q, cs), keys)[np.arange(rows), head] * SCALE
    lse = np.full((rows, H), -np.inf, np.float32)
    lse[np.arange(rows), head] = 0.0
    acc = torch.zeros((rows, n), device="cuda")
    cskv.attn_weights(_dev(q, torch.bfloat16), _paged(keys), torch.full((rows,), n, dtype=torch.int32, device="cuda"), n,
                      SCALE, _dev(cs), _dev(lse), acc)
    assert cskv.device_status() == 0
    assert _logit_errors_are_within(acc.double().cpu().numpy() / np.exp(z) - 1.0, WEIGHT_LOGIT)


@pytest.mark.gpu
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("H,n", [(16, 237), (64, 300), (128, 1000)])
def test_errors_of_the_outputs(H, n, turned):
    rows = 320 // H + 4
    q, keys, sink, cs = _inputs(rows, H, n, seed=30 + H, turned=turned)
    sink = sink.astype(np.float32).astype(np.float64)
    cache, count = _paged(keys), torch.full((rows,), n, dtype=torch.int32, device="cuda")
    bq, bcs, bs = _dev(q, torch.bfloat16), _dev(cs), _dev(sink)
    for out in (cskv.window_attn(bq, cache, count, n, 0, n, bs, SCALE, bcs)[0],
                cskv.prefix_decode_attn(bq, cache, count, 0, n, bs, SCALE, bcs)[0]):
        assert _output_errors_are_within(out.double().cpu().numpy(), q, keys, sink, cs)
    assert cskv.device_status() == 0
