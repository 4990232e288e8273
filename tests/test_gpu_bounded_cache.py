"""GPU parity of window_attn, prefix_decode_attn, attn_weights and evict against the fp64
definitions on the same coded bytes, with bounds that count the roundings the calls document
(query as two bf16 numbers, weights and output bf16, the rest fp32)."""

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import bounded, codecs

from cases import HostPaged, bf16_values, cuda, swa_ring

pytestmark = pytest.mark.gpu

SCALE = 512 ** -0.5
BF16, FP8, FP4 = codecs.FMT_BF16, codecs.FMT_FP8, codecs.FMT_FP4
ERR_BOUNDS = 5


def _cache(fmt, rows, seed, scale=1.0):
    rs = np.random.default_rng(seed)
    c = HostPaged(fmt, 512, [max(1, n) for n in rows], seed=seed + 1)
    for b, n in enumerate(rows):
        c.fill(b, (scale * rs.standard_normal((max(1, n), 512))).astype(np.float32))
    return c


def _queries(T, H, seed, scale=2.0):
    return bf16_values(scale * np.random.default_rng(seed).standard_normal((T, H, 512)))


def _cs(pos1):
    return cuda(cskv.rope_table(np.maximum(np.asarray(pos1, np.int64) - 1, 0)))


def _i32(x):
    return cuda(np.asarray(x, np.int32))


def _check(out, lse, ref, where=""):
    o, l, bo, bl = ref
    out = out.float().cpu().numpy().astype(np.float64)
    d = np.abs(out - o)
    assert np.all(d <= bo + 1e-30), "%s out: %.3g over the bound" % (where, np.max(d / np.maximum(bo, 1e-30)))
    lse = lse.cpu().numpy().astype(np.float64)
    fin = np.isfinite(l)
    assert np.array_equal(lse[~fin], l[~fin]), where
    e = np.abs(lse[fin] - l[fin])
    assert np.all(e <= bl[fin] + 1e-30), "%s lse: %.3g over the bound" % (where, np.max(e / np.maximum(bl[fin], 1e-30)))


# --- window_attn ---------------------------------------------------------------------------

def _window(cache, q, pos1, window, first, req_of, sink, max_ctx=None, **kw):
    return cskv.window_attn(q[0].cuda(), cache.to_device(), _i32(pos1), window, first,
                            int(max(1, max(pos1))) if max_ctx is None else max_ctx,
                            None if sink is None else cuda(sink), SCALE, _cs(pos1),
                            req_of=None if req_of is None else _i32(req_of), want_lse=True, **kw)


def _window_ref(cache, q, i, pos1, window, first, req_of, sink):
    t = int(pos1[i]) - 1
    r = i if req_of is None else int(req_of[i])
    keys = cache.decoded[r][bounded.visible(t, window, first)] if t >= 0 else np.zeros((0, 512))
    return bounded.attend(q[1][i], max(t, 0), keys, sink, SCALE)


def _window_all(cache, q, pos1, window, first, req_of, sink, pick=None, **kw):
    out, lse = _window(cache, q, pos1, window, first, req_of, sink, **kw)
    assert cskv.device_status() == 0
    for i in (range(len(pos1)) if pick is None else pick):
        _check(out[i], lse[i], _window_ref(cache, q, i, pos1, window, first, req_of, sink), "query %d" % i)


@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
@pytest.mark.parametrize("H", [1, 5, 16, 20, 64, 96, 128])
def test_window_decode_heads_and_formats(fmt, H):
    pos1 = [700, 1, 129, 128, 64, 0, 257]
    cache = _cache(fmt, pos1, seed=H + 10 * fmt)
    sink = np.random.default_rng(3).standard_normal(H).astype(np.float32) if H % 2 == 0 else None
    _window_all(cache, _queries(len(pos1), H, H), pos1, 128, 4, None, sink)


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (2, 130), (63, 0), (127, 5), (128, 128), (129, 64),
                                          (300, 7), (5000, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_sizes(window, first):
    pos1 = [1, 2, 64, 65, 127, 128, 129, 130, 131, 256, 300, 513, 900]
    cache = _cache(FP8, pos1, seed=5)
    _window_all(cache, _queries(len(pos1), 8, 6), pos1, window, first, None, None)


@pytest.mark.parametrize("fmt,H,window,first", [(BF16, 20, 100, 7), (FP8, 64, 128, 4), (FP8, 3, 40, 0), (FP4, 16, 200, 64),
                                                (FP8, 128, 16, 1)])
def test_window_prompts(fmt, H, window, first):
    """Queries of three prompts in one call, in order; sampled against the definition."""
    L = [333, 64, 130]
    cache = _cache(fmt, L, seed=H)
    req = np.repeat(np.arange(3), L)
    pos1 = np.concatenate([np.arange(1, n + 1) for n in L])
    sink = np.random.default_rng(4).standard_normal(H).astype(np.float32)
    pick = sorted(set(np.random.default_rng(8).integers(0, len(req), 40).tolist()) | {0, 332, 333, 396, 397, 526})
    _window_all(cache, _queries(len(req), H, 7), pos1, window, first, req, sink, pick=pick)


def test_window_queries_in_any_order_with_padding():
    """Requests interleaved, positions far apart, descending and repeated, padding between."""
    L = [900, 40, 300]
    cache = _cache(FP8, L, seed=21)
    rs = np.random.default_rng(22)
    T, H = 61, 8
    req = rs.integers(0, 3, T)
    pos1 = np.array([rs.integers(0, L[r] + 1) for r in req])
    req[10:20], pos1[10:20] = 0, np.arange(900, 890, -1)
    req[20:24], pos1[20:24] = 0, 450
    pos1[30:33] = 0
    _window_all(cache, _queries(T, H, 23), pos1, 70, 3, req, rs.standard_normal(H).astype(np.float32))


def test_window_long_context_is_split_and_joined():
    """One request's long window: the keys are spread over the SMs and joined."""
    for pos1, window, first, H in (([20000], 15000, 64, 16), ([9001, 4000], 8000, 0, 64)):
        cache = _cache(FP8, pos1, seed=31)
        _window_all(cache, _queries(len(pos1), H, 32), pos1, window, first, None, None)


def test_window_pages_outside_the_window_are_never_read():
    """Table entries and rows behind the window hold rubbish: same bits, no error."""
    pos1 = [1000]
    cache = _cache(FP8, pos1, seed=41)
    q = _queries(1, 16, 42)
    a, la = _window(cache, q, pos1, 128, 4, None, None)
    assert cskv.device_status() == 0
    lo = (1000 - 128) // 64
    for p in range(1, lo):
        cache.block_table[0, p] = -77
    first_page = cache.block_table[0, 0]
    cache.pool[first_page, 4 * 528:] = 0x7F          # NaN codes behind the first four rows
    edge = cache.block_table[0, lo]
    cache.pool[edge, :(1000 - 128 - 64 * lo) * 528] = 0x7F
    b, lb = _window(cache, q, pos1, 128, 4, None, None)
    assert cskv.device_status() == 0
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_window_nan_rows_reach_only_their_queries(fmt):
    """A row that is not finite makes the queries that see it NaN and leaves the others exact."""
    L = 300
    cache = _cache(fmt, [L], seed=51)
    pos1 = np.arange(1, L + 1)
    req = np.zeros(L, np.int64)
    bad = 150
    rb = cache.page_bytes // 64
    page, slot = cache.block_table[0, bad // 64], bad % 64
    row = cache.pool[page, slot * rb:(slot + 1) * rb]
    if fmt == BF16:
        row.view(np.uint16)[300] = 0x7F80            # +inf in one dim
    else:
        row[300] = 0x7F                              # NaN code in one dim
    q = _queries(L, 16, 52)
    out, lse = _window(cache, q, pos1, 64, 2, req, None)
    assert cskv.device_status() == 0
    o = out.float().cpu().numpy()
    sees = (pos1 - 1 >= bad) & (bad > pos1 - 1 - 64)
    assert np.all(np.isnan(o[sees])) and np.all(np.isnan(lse.cpu().numpy()[sees]))
    for i in list(range(140, 150)) + list(range(214, 224)):
        assert not sees[i]
        _check(out[i], lse[i], _window_ref(cache, q, i, pos1, 64, 2, req, None), "query %d" % i)


def test_window_nan_query_stays_in_its_row():
    pos1 = [200, 300, 150]
    cache = _cache(FP8, pos1, seed=61)
    q = _queries(3, 16, 62)
    bad = q[0].clone()
    bad[1, 5, 17] = float("nan")
    a, la = _window(cache, q, pos1, 128, 4, None, None)
    b, lb = _window(cache, (bad, None), pos1, 128, 4, None, None)
    keep = torch.ones((3, 16), dtype=torch.bool)
    keep[1, 5] = False
    assert torch.equal(a.cpu()[keep], b.cpu()[keep]) and torch.equal(la.cpu()[keep], lb.cpu()[keep])
    assert torch.isnan(b[1, 5]).all() and torch.isnan(lb[1, 5])


def test_window_large_logits():
    """Logits of several hundred, growing along the keys: the running maximum moves often."""
    L = 700
    rs = np.random.default_rng(71)
    v = rs.standard_normal((L, 512)).astype(np.float32) * np.linspace(0.5, 8, L)[:, None].astype(np.float32)
    cache = HostPaged(BF16, 512, [L], seed=72)
    cache.fill(0, v)
    q = _queries(1, 16, 73, scale=12.0)
    sink = np.linspace(-300, 300, 16).astype(np.float32)
    _window_all(cache, q, [L], 650, 16, None, sink)


def test_window_sinks_of_minus_infinity_and_lowest():
    pos1 = [100, 0]
    cache = _cache(BF16, pos1, seed=75)
    sink = np.array([-np.inf, np.finfo(np.float32).min, 0.0, 5.0], np.float32)
    _window_all(cache, _queries(2, 4, 76), pos1, 64, 0, None, sink)


# --- prefix_decode_attn ----------------------------------------------------------------------

def _prefix_case(B, H, P, n, fmt, swa_fmt, seed, with_sink=True, ctx=None):
    cache = _cache(fmt, [max(1, max(n))] * B, seed)
    shared = P // 64
    for b in range(1, B):
        cache.block_table[b, :shared] = cache.block_table[0, :shared]
    ring = None
    if swa_fmt is not None:
        ring = swa_ring(np.random.default_rng(seed + 2).standard_normal((B, 128, 512)).astype(np.float32), swa_fmt)
    ctx = np.asarray([3 * x + 1 for x in n] if ctx is None else ctx)
    sink = np.random.default_rng(seed + 3).standard_normal(H).astype(np.float32) if with_sink else None
    return dict(cache=cache, ring=ring, swa_fmt=swa_fmt, ctx=ctx, n=np.asarray(n), P=P, H=H, B=B, sink=sink,
                q=_queries(B, H, seed + 4))


def _prefix_run(c, **kw):
    ring = {} if c["ring"] is None else dict(swa=cuda(c["ring"][0]), swa_fmt=c["swa_fmt"], ctx_len=_i32(c["ctx"]))
    return cskv.prefix_decode_attn(c["q"][0].cuda(), c["cache"].to_device(), _i32(c["n"]), c["P"],
                                   int(max(max(c["n"]), c["P"])), None if c["sink"] is None else cuda(c["sink"]), SCALE,
                                   _cs(c["ctx"]), want_lse=True, **dict(ring, **kw))


def _prefix_keys(c, b):
    n = int(c["n"][b])
    d = c["cache"].decoded
    keys = [d[0][:min(n, c["P"])], d[b][c["P"]:n]]
    if c["ring"] is not None:
        keys.append(c["ring"][1][b][:max(0, min(128, int(c["ctx"][b])))])
    return np.concatenate(keys)


def _prefix_all(c, out, lse):
    assert cskv.device_status() == 0
    for b in range(c["B"]):
        ref = bounded.attend(c["q"][1][b], max(0, int(c["ctx"][b]) - 1), _prefix_keys(c, b), c["sink"], SCALE)
        _check(out[b], lse[b], ref, "request %d" % b)


@pytest.mark.parametrize("fmt,swa_fmt", [(BF16, BF16), (FP8, FP8), (FP4, FP8), (FP4, None), (FP8, BF16)])
@pytest.mark.parametrize("H", [1, 7, 16, 64, 100, 128])
def test_prefix_formats_and_heads(fmt, swa_fmt, H):
    c = _prefix_case(5, H, 200, [331, 200, 201, 150, 264], fmt, swa_fmt, seed=100 + H, with_sink=H % 2 == 0)
    _prefix_all(c, *_prefix_run(c))


@pytest.mark.parametrize("P,n", [(0, [5, 0, 300]), (1, [1, 1, 1]), (64, [64, 65, 128]), (127, [128, 127, 3]),
                                 (128, [128, 0, 129]), (129, [500, 129, 130]), (1000, [1000, 1300, 0]),
                                 (0, [0, 0, 0])])
def test_prefix_lengths(P, n):
    """Requests with fewer entries than the prefix, without any, and with the prefix alone."""
    for swa_fmt, ctx in ((FP8, [1, 0, 500]), (None, [9, 9, 9])):
        c = _prefix_case(3, 16, P, n, FP8, swa_fmt, seed=200 + P, ctx=ctx)
        _prefix_all(c, *_prefix_run(c))


def test_prefix_batch_of_many_requests():
    n = [700 + 13 * b for b in range(33)]
    c = _prefix_case(33, 8, 640, n, FP8, FP8, seed=300)
    _prefix_all(c, *_prefix_run(c))


def test_prefix_long_and_split():
    """A long prefix for two requests: its keys are spread over the SMs and joined."""
    c = _prefix_case(2, 64, 9000, [9000, 9700], FP8, FP8, seed=310)
    _prefix_all(c, *_prefix_run(c))


def test_prefix_equals_sparse_decode_attn_without_a_prefix():
    """The same keys as the framework's HCA attention: both within their bounds of one another."""
    ratio, H = 128, 64
    ctx = np.array([128 * 300 + 5, 1000])
    n = ctx // ratio
    c = _prefix_case(2, H, 0, n.tolist(), FP8, FP8, seed=320, ctx=ctx)
    out, lse = _prefix_run(c)
    ref = cskv.sparse_decode_attn(c["q"][0].cuda(), c["cache"].to_device(), cuda(c["ring"][0]), FP8, _i32(ctx), None, 0,
                                  ratio, int(ctx.max()), cuda(c["sink"]), SCALE, _cs(ctx))
    assert cskv.device_status() == 0
    assert float((out.float() - ref.float()).norm() / ref.float().norm()) <= 1e-2


# --- attn_weights ----------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
@pytest.mark.parametrize("H", [1, 7, 16, 64, 65, 128])
def test_weights(fmt, H):
    n, first, cap, decay = [400, 0, 129, 64, 3], 3, 431, 0.75
    c = _prefix_case(5, H, 0, n, fmt, None, seed=400 + H)
    rs = np.random.default_rng(401)
    lse = (np.log(300.0) + 2 + rs.standard_normal((5, H))).astype(np.float32)
    lse[0, H // 2] = -np.inf
    acc = rs.uniform(0, 1, (5, cap)).astype(np.float32)
    got = cskv.attn_weights(c["q"][0].cuda(), c["cache"].to_device(), _i32(n), 400, SCALE, _cs(c["ctx"]), cuda(lse),
                            cuda(acc), decay=decay, first=first, acc_out=torch.full((5, cap), -9.0, device="cuda"))
    assert cskv.device_status() == 0
    got = got.cpu().numpy().astype(np.float64)
    for b in range(5):
        w, bound = bounded.weights(c["q"][1][b], int(c["ctx"][b]) - 1, c["cache"].decoded[b][:n[b]], lse[b], SCALE)
        ref = np.full(cap, -9.0)
        if n[b] > first:
            ref[first:n[b]] = decay * acc[b, first:n[b]].astype(np.float64) + w[first:]
            bound = bound[first:] + 3 * 2.0 ** -24 * np.abs(ref[first:n[b]])
            assert np.all(np.abs(got[b, first:n[b]] - ref[first:n[b]]) <= bound)
        rest = np.r_[0:min(first, cap), max(first, n[b]):cap]
        assert np.array_equal(got[b, rest], ref[rest])


def test_weights_in_place_and_sum_to_the_heads():
    """With the call's own lse the weights of a request sum to its heads (no sink, no ring)."""
    c = _prefix_case(3, 32, 100, [300, 257, 100], FP8, None, seed=420, with_sink=False)
    out, lse = _prefix_run(c)
    acc = torch.zeros((3, 300), device="cuda")
    for b in range(1, 3):      # the weights read each request's own rows: give it the prefix's
        for j in range(100):
            p, s = c["cache"].block_table[b, j // 64], j % 64
            p0 = c["cache"].block_table[0, j // 64]
            c["cache"].pool[p, s * 528:(s + 1) * 528] = c["cache"].pool[p0, s * 528:(s + 1) * 528]
    args = (c["q"][0].cuda(), c["cache"].to_device(), _i32(c["n"]), 300, SCALE, _cs(c["ctx"]), lse, acc)
    assert cskv.attn_weights(*args) is acc
    # each weight's relative error is the bound's logit term, far below 1e-4 at these values
    assert torch.allclose(acc.double().sum(1), torch.full((3,), 32.0, device="cuda", dtype=torch.float64), rtol=1e-4)
    once = acc.clone()
    cskv.attn_weights(*args)
    assert torch.allclose(acc, 2 * once, rtol=1e-6)
    assert cskv.device_status() == 0


def test_weights_nan_key_stays_in_its_entry():
    n = [200]
    c = _prefix_case(1, 16, 0, n, FP8, None, seed=430)
    lse = torch.full((1, 16), 6.0, device="cuda")
    args = lambda: (c["q"][0].cuda(), c["cache"].to_device(), _i32(n), 200, SCALE, _cs(c["ctx"]), lse,
                    torch.zeros((1, 200), device="cuda"))
    a = cskv.attn_weights(*args())
    p = c["cache"].block_table[0, 1]
    c["cache"].pool[p, 5 * 528 + 40] = 0x7F
    b = cskv.attn_weights(*args())
    keep = torch.arange(200) != 69
    assert torch.equal(a.cpu()[0, keep], b.cpu()[0, keep]) and torch.isnan(b[0, 69])


# --- evict -----------------------------------------------------------------------------------

def _evict_case(B, cap, n, fmts, seed, ties=False):
    rs = np.random.default_rng(seed)
    caches = []
    for f, (fmt, dim) in enumerate(fmts):
        c = HostPaged(fmt, dim, [cap] * B, seed=seed + f)
        for b in range(B):
            c.fill(b, rs.standard_normal((cap, dim)).astype(np.float32))
        caches.append(c)
    acc = np.exp(2 * rs.standard_normal((B, cap))).astype(np.float32)
    if ties:
        acc = np.round(acc).astype(np.float32)
        acc[:, ::7] = -0.0
        acc[:, 1::11] = np.nan
        acc[:, 2::13] = np.inf
        acc[:, 3::17] = -np.inf
    age = np.stack([rs.permutation(cap) for _ in range(B)]).astype(np.int32)
    return dict(caches=caches, acc=acc, age=age, n=np.asarray(n, np.int32), cap=cap, B=B)


def _slot_bytes(c, pool, b, s):
    """The bytes of slot s of request b (codes and, in page-split formats, the scale)."""
    pg, rb = pool[c.block_table[b, s // 64]], codecs.row_bytes(c.fmt, c.dim)
    s %= 64
    if c.fmt in (codecs.FMT_FP8_PAGESPLIT, codecs.FMT_FP4H_PAGESPLIT):
        d = rb - 4
        return np.concatenate([pg[s * d:(s + 1) * d], pg[64 * d + 4 * s:64 * d + 4 * s + 4]])
    return pg[s * rb:(s + 1) * rb]


def _evict_check(e, budget, fixed, recent, use_age, in_place):
    B, cap = e["B"], e["cap"]
    dev = [c.to_device() for c in e["caches"]]
    acc, age, n = cuda(e["acc"]), (cuda(e["age"]) if use_age else None), _i32(e["n"])
    kw = {}
    if not in_place:
        kw = dict(acc_out=torch.full((B, budget + 2), -5.0, device="cuda"), n_out=torch.full_like(n, -5),
                  age_out=torch.full((B, budget + 3), -5, dtype=torch.int32, device="cuda") if use_age else None)
    src, n_out, acc_out, age_out = cskv.evict(dev, acc, n, budget, fixed=fixed, recent=recent, age=age,
                                              max_entries=cap, **kw)
    assert cskv.device_status() == 0
    src, n_out, acc_out = src.cpu().numpy(), n_out.cpu().numpy(), acc_out.cpu().numpy()
    age_out = age_out.cpu().numpy() if use_age else None
    for b in range(B):
        ref, m = bounded.evict(e["acc"][b], e["age"][b] if use_age else None, int(e["n"][b]), budget, fixed, recent)
        assert n_out[b] == m
        assert np.array_equal(src[b], ref), b
        want = e["acc"][b].copy() if in_place else np.full(budget + 2, -5.0, np.float32)
        want[:m] = e["acc"][b][ref[:m]]
        assert np.array_equal(acc_out[b], want, equal_nan=True)
        if use_age:
            want = e["age"][b].copy() if in_place else np.full(budget + 3, -5, np.int32)
            want[:m] = e["age"][b][ref[:m]]
            assert np.array_equal(age_out[b], want)
    for c, d in zip(e["caches"], dev):
        want = c.pool.copy()
        for b in range(B):
            ref, m = bounded.evict(e["acc"][b], e["age"][b] if use_age else None, int(e["n"][b]), budget, fixed, recent)
            for i in np.flatnonzero(ref[:m] != np.arange(m)):
                _slot_bytes(c, want, b, i)   # address check
                pg, rb, s = want[c.block_table[b, i // 64]], codecs.row_bytes(c.fmt, c.dim), i % 64
                row = _slot_bytes(c, c.pool, b, ref[i])
                if c.fmt in (codecs.FMT_FP8_PAGESPLIT, codecs.FMT_FP4H_PAGESPLIT):
                    k = rb - 4
                    pg[s * k:(s + 1) * k], pg[64 * k + 4 * s:64 * k + 4 * s + 4] = row[:k], row[k:]
                else:
                    pg[s * rb:(s + 1) * rb] = row
        assert np.array_equal(d.pool.cpu().numpy(), want)


@pytest.mark.parametrize("fmts", [[(BF16, 512)], [(FP8, 512), (codecs.FMT_FP8_PAGESPLIT, 128)],
                                  [(FP4, 512), (codecs.FMT_FP4H_PAGESPLIT, 128), (BF16, 128), (FP8, 128)]])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_formats(fmts, in_place):
    e = _evict_case(3, 333, [333, 200, 331], fmts, seed=500, ties=True)
    _evict_check(e, 200, 5, 31, True, in_place)


@pytest.mark.parametrize("cap,n,budget,fixed,recent", [
    (1, [1, 0], 1, 0, 0), (2, [2, 1], 1, 0, 1), (2, [2, 2], 1, 1, 0), (70, [70, 69], 69, 0, 0), (70, [70, 3], 1, 0, 0),
    (129, [129, 129], 64, 64, 0), (129, [129, 100], 64, 0, 64), (129, [129, 65], 64, 30, 34),
    (1100, [1100, 1025], 1024, 7, 100), (1100, [1100, 900], 2000, 0, 0), (5000, [5000, 4999], 2500, 64, 500),
    (5000, [5000, 4097], 4096, 0, 0)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_sizes(cap, n, budget, fixed, recent, ties):
    e = _evict_case(2, cap, n, [(codecs.FMT_FP4H_PAGESPLIT, 128)], seed=510 + cap, ties=ties)
    _evict_check(e, budget, fixed, recent, True, cap % 2 == 0)


def test_evict_without_ages_and_equal_weights():
    e = _evict_case(2, 600, [600, 555], [(FP8, 128)], seed=530)
    e["acc"][:] = 1.0
    _evict_check(e, 300, 10, 0, False, True)
    e["acc"][:] = np.nan
    _evict_check(e, 300, 0, 0, False, False)


def test_evict_long_cache():
    e = _evict_case(1, 100000, [99999], [(codecs.FMT_FP4H_PAGESPLIT, 128)], seed=540)
    _evict_check(e, 60000, 64, 3000, True, True)


# --- together, streams, graphs, errors ---------------------------------------------------------

def test_decode_loop_with_a_bounded_cache():
    """Steps of a shared-prefix batch: attend, accumulate, evict, append; every step's outputs
    against the definition on the rows that the slots hold by then."""
    B, H, P, budget, cap = 3, 16, 70, 150, 192
    rs = np.random.default_rng(600)
    c = _prefix_case(B, H, P, [160, 150, 120], FP8, FP8, seed=601, ctx=[1000, 40, 7])
    cache = HostPaged(FP8, 512, [cap] * B, seed=602)
    vals = rs.standard_normal((B, cap, 512)).astype(np.float32)
    vals[:, :P] = vals[0, :P]
    for b in range(B):
        cache.fill(b, vals[b])
    held = [cache.decoded[b].copy() for b in range(B)]
    dev = cache.to_device()
    n = np.array([160, 150, 120])
    nd, acc = _i32(n), torch.zeros((B, cap), device="cuda")
    ages = np.tile(np.arange(cap, dtype=np.int32), (B, 1))
    age = cuda(ages)
    ring = cuda(c["ring"][0])
    for step in range(4):
        q_t, q_v = _queries(B, H, 610 + step)
        ctx = c["ctx"] + step
        out, lse = cskv.prefix_decode_attn(q_t.cuda(), dev, nd, P, cap, cuda(c["sink"]), SCALE, _cs(ctx), swa=ring,
                                           swa_fmt=FP8, ctx_len=_i32(ctx), want_lse=True)
        for b in range(B):
            keys = np.concatenate([held[b][:n[b]], c["ring"][1][b][:min(128, ctx[b])]])
            _check(out[b], lse[b], bounded.attend(q_v[b], int(ctx[b]) - 1, keys, c["sink"], SCALE), "step %d" % step)
        before = acc.cpu().numpy()
        cskv.attn_weights(q_t.cuda(), dev, nd, cap, SCALE, _cs(ctx), lse, acc, decay=0.9, first=P)
        a = acc.cpu().numpy()
        for b in range(B):
            w, bound = bounded.weights(q_v[b], int(ctx[b]) - 1, held[b][:n[b]], lse[b].cpu().numpy(), SCALE)
            ref = 0.9 * before[b, P:n[b]].astype(np.float64) + w[P:]
            assert np.all(np.abs(a[b, P:n[b]] - ref) <= bound[P:] + 1e-6 * np.abs(ref))
        src, nd, acc, age = cskv.evict([dev], acc, nd, budget, fixed=P, recent=20, age=age, max_entries=cap)
        src = src.cpu().numpy()
        for b in range(B):
            ref, m = bounded.evict(a[b], ages[b], int(n[b]), budget, P, 20)
            assert np.array_equal(src[b], ref)
            held[b][:m], ages[b][:m] = held[b][ref[:m]], ages[b][ref[:m]]
            n[b] = m
        assert np.array_equal(nd.cpu().numpy(), n)
        # the step's new entries, three for each request, go behind what is left
        new = rs.standard_normal((B, 3, 512)).astype(np.float32)
        cskv.encode_rows(cuda(new.reshape(-1, 512)), dev, req=_i32(np.repeat(np.arange(B), 3)),
                         row=_i32((n[:, None] + np.arange(3)).reshape(-1)))
        dec = codecs.decode_rows(codecs.encode_rows(new.reshape(-1, 512), FP8), FP8, 512).reshape(B, 3, 512)
        for b in range(B):
            held[b][n[b]:n[b] + 3] = dec[b]
            ages[b][n[b]:n[b] + 3] = 10000 + 3 * step + np.arange(3)
            acc[b, n[b]:n[b] + 3] = 0.0
        n = n + 3
        nd, age = _i32(n), cuda(ages)
    assert cskv.device_status() == 0


def test_captured_and_replayed_together_on_a_side_stream():
    """The three calls of a step captured into a graph, replayed on new inputs."""
    B, H, P = 2, 16, 300
    c = _prefix_case(B, H, P, [700, 650], FP8, FP8, seed=700)
    dev = c["cache"].to_device()
    q = c["q"][0].cuda()
    nd, ring, ctx, cs, sink = _i32(c["n"]), cuda(c["ring"][0]), _i32(c["ctx"]), _cs(c["ctx"]), cuda(c["sink"])
    acc = torch.zeros((B, 700), device="cuda")
    acc_out, n_out = torch.zeros((B, 700), device="cuda"), torch.zeros_like(nd)

    def step():
        o, l = cskv.prefix_decode_attn(q, dev, nd, P, 700, sink, SCALE, cs, swa=ring, swa_fmt=FP8, ctx_len=ctx,
                                       want_lse=True)
        w = cskv.attn_weights(q, dev, nd, 700, SCALE, cs, l, acc, acc_out=acc_out)
        s = cskv.evict([dev], w, nd, 640, fixed=P, n_out=n_out, acc_out=torch.zeros((B, 640), device="cuda"))
        return o, l, w, s[0], s[2]

    pool = dev.pool.clone()
    step()
    torch.cuda.synchronize()
    dev.pool.copy_(pool)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for seed in (1, 2):
        q.copy_(_queries(B, H, seed)[0])
        dev.pool.copy_(pool)
        g.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in got] + [dev.pool.clone()]
        dev.pool.copy_(pool)
        want = list(step()) + [dev.pool]
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
    assert cskv.device_status() == 0


def test_an_explicit_stream_and_the_same_call_twice():
    pos1 = [5000, 3000]
    cache = _cache(FP8, pos1, seed=710)
    q = _queries(2, 64, 711)
    a, la = _window(cache, q, pos1, 4096, 4, None, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, lb = _window(cache, q, pos1, 4096, 4, None, None, stream=side)
    d, ld = _window(cache, q, pos1, 4096, 4, None, None, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, d) and torch.equal(la, ld)


def test_bad_indices_are_skipped_and_reported():
    """Lengths beyond the host's bound, requests outside the table and pages outside the pool."""
    pos1 = [300, 200, 250]
    cache = _cache(FP8, pos1, seed=720)
    q = _queries(3, 16, 721)
    good, _ = _window(cache, q, pos1, 64, 2, None, None)
    assert cskv.device_status() == 0
    out, lse = _window(cache, q, pos1, 64, 2, [0, 7, 2], None)          # request 7 does not exist
    assert cskv.device_status() == ERR_BOUNDS
    assert torch.equal(out[[0, 2]], good[[0, 2]]) and not out[1].any() and torch.isneginf(lse[1]).all()
    out, _ = _window(cache, q, pos1, 64, 2, None, None, max_ctx=250)    # query 0 lies beyond the bound
    assert cskv.device_status() == ERR_BOUNDS
    assert torch.equal(out[1:], good[1:])
    keep = cache.block_table.copy()
    cache.block_table[1, 2] = cache.num_pages                            # rows 128 .. 191 of request 1
    out, lse = _window(cache, q, pos1, 64, 2, None, None)
    assert cskv.device_status() == ERR_BOUNDS
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    rows = [j for j in bounded.visible(199, 64, 2) if not 128 <= j < 192]
    _check(out[1], lse[1], bounded.attend(q[1][1], 199, cache.decoded[1][rows], None, SCALE))
    cache.block_table[:] = keep
    n = _i32([300, -3, 999])
    acc = torch.zeros((3, 300), device="cuda")
    cskv.attn_weights(q[0].cuda(), cache.to_device(), n, 250, SCALE, _cs(pos1), torch.zeros((3, 16), device="cuda"), acc)
    assert cskv.device_status() == ERR_BOUNDS
    assert not acc[1].any() and not acc[0, 250:].any() and (acc[0, :250] > 0).all()
    src, n_out, _, _ = cskv.evict([cache.to_device()], acc, n, 100, max_entries=250)
    assert cskv.device_status() == ERR_BOUNDS
    assert n_out.tolist() == [100, 0, 100] and (src[1] == -1).all()
    _window_all(cache, q, pos1, 64, 2, None, None)


def test_wrong_shapes_are_refused():
    cache = _cache(FP8, [100, 100], seed=730)
    dev = cache.to_device()
    q = _queries(2, 16, 731)[0].cuda()
    i, cs = _i32([100, 100]), _cs([100, 100])
    lse, acc = torch.zeros((2, 16), device="cuda"), torch.zeros((2, 100), device="cuda")
    with pytest.raises(ValueError, match="pos1"):
        cskv.window_attn(q, dev, i[:1].contiguous(), 8, 0, 100, None, SCALE, cs)
    with pytest.raises(ValueError, match="contiguous"):
        cskv.window_attn(q.transpose(0, 1), dev, i, 8, 0, 100, None, SCALE, cs)
    with pytest.raises(ValueError, match="q_rope_cs"):
        cskv.window_attn(q, dev, i, 8, 0, 100, None, SCALE, cs[:1].contiguous())
    with pytest.raises(ValueError, match="sink"):
        cskv.prefix_decode_attn(q, dev, i, 0, 100, torch.zeros(3, device="cuda"), SCALE, cs)
    with pytest.raises(ValueError, match="block table"):
        q3 = _queries(3, 16, 1)[0].cuda()
        cskv.prefix_decode_attn(q3, dev, _i32([1, 1, 1]), 0, 100, None, SCALE, _cs([1, 1, 1]))
    with pytest.raises(ValueError, match="swa"):
        cskv.prefix_decode_attn(q, dev, i, 0, 100, None, SCALE, cs, swa=torch.zeros((2, 128, 500), dtype=torch.uint8,
                                                                                   device="cuda"), swa_fmt=FP8, ctx_len=i)
    with pytest.raises(ValueError, match="acc"):
        cskv.attn_weights(q, dev, i, 101, SCALE, cs, lse, acc)
    with pytest.raises(ValueError, match="age"):
        cskv.evict([dev], acc, i, 50, age=torch.zeros((2, 40), dtype=torch.int32, device="cuda"))
    with pytest.raises(cskv.CskvError):
        cskv.evict([dev], acc, i, 50, fixed=30, recent=30, age=torch.zeros((2, 100), dtype=torch.int32, device="cuda"))
    with pytest.raises(cskv.CskvError):
        cskv.evict([], acc, i, 50)
    with pytest.raises(cskv.CskvError):
        cskv.window_attn(q, dev, i, 0, 0, 100, None, SCALE, cs)


@pytest.mark.parametrize("limit", [1, 2000, 20000])
def test_waits_that_run_out_end_their_kernels(limit):
    """With a limit far below a tile's time the kernels give up, report it and return; after it the
    same calls are exact."""
    pos1 = [3000, 2000, 1500]
    cache = _cache(FP8, pos1, seed=740)
    q = _queries(3, 16, 741)
    c = _prefix_case(3, 16, 500, [900, 800, 700], FP8, FP8, seed=742)
    prompt = _queries(600, 16, 743)
    long = _cache(FP8, [600], seed=744)
    lse = torch.zeros((3, 16), device="cuda")
    acc = torch.zeros((3, 900), device="cuda")
    good = [x.clone() for x in _window(cache, q, pos1, 2000, 4, None, None)]
    assert cskv.device_status() == 0
    cskv.set_spin_limit(limit)
    try:
        _window(cache, q, pos1, 2000, 4, None, None)
        _window(long, prompt, np.arange(1, 601), 128, 4, np.zeros(600, np.int64), None)
        _prefix_run(c)
        cskv.attn_weights(c["q"][0].cuda(), c["cache"].to_device(), _i32(c["n"]), 900, SCALE, _cs(c["ctx"]), lse, acc)
        assert cskv.device_status() in ((4,) if limit == 1 else (0, 4))
    finally:
        cskv.set_spin_limit(0)
    again = _window(cache, q, pos1, 2000, 4, None, None)
    assert cskv.device_status() == 0
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    _prefix_all(c, *_prefix_run(c))


def test_caches_beyond_four_gigabytes():
    """Pages at the end of a pool of more than 2^32 bytes."""
    page = 64 * 1024
    pages = (1 << 32) // page + 40
    pool = torch.zeros((pages, page), dtype=torch.uint8, device="cuda")
    L = 700
    small = _cache(BF16, [L], seed=750)
    per = small.max_pages
    bt = np.arange(pages - per, pages, dtype=np.int32)[None]
    for p in range(per):
        pool[int(bt[0, p])] = cuda(small.pool[small.block_table[0, p]])
    big = cskv.PagedCache(pool, cuda(bt), BF16, 512)
    q = _queries(1, 16, 751)
    args = (_i32([L]), 600, 4, L, None, SCALE, _cs([L]))
    a, la = cskv.window_attn(q[0].cuda(), big, *args, want_lse=True)
    b, lb = cskv.window_attn(q[0].cuda(), small.to_device(), *args, want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    acc = torch.rand((1, L), device="cuda")
    before = pool[int(bt[0, 0]):].clone()
    src, n, _, _ = cskv.evict([big], acc, _i32([L]), 300)
    src = src[0].long()
    rows = before.view(-1, 1024)
    assert torch.equal(pool[int(bt[0, 0]):].view(-1, 1024)[:300], rows[src])
    assert cskv.device_status() == 0


def test_calls_on_two_streams_at_once():
    """The same operators at the same time on two streams, each with its own workspace."""
    c = [_prefix_case(4, 32, 1000, [1500, 1400, 1300, 1200], FP8, FP8, seed=760 + k) for k in range(2)]
    want = [_prefix_run(x) for x in c]
    torch.cuda.synchronize()
    args = []
    for x in c:
        args.append(((x["q"][0].cuda(), x["cache"].to_device(), _i32(x["n"]), x["P"], 1500, cuda(x["sink"]), SCALE,
                      _cs(x["ctx"])), dict(swa=cuda(x["ring"][0]), swa_fmt=FP8, ctx_len=_i32(x["ctx"]), want_lse=True)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for k in range(2):
            got[k].append(cskv.prefix_decode_attn(*args[k][0], stream=streams[k], **args[k][1]))
    torch.cuda.synchronize()
    for k in range(2):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
    assert cskv.device_status() == 0


@pytest.mark.parametrize("fmt", [FP8, FP4])
def test_every_code_and_scale_is_read_exactly(fmt):
    """A query that sees one row gives that row back: every code under many scales, bit for bit
    (bf16 holds every such value except where the largest scales overflow it)."""
    rb = codecs.row_bytes(fmt, 512)
    if fmt == FP8:
        codes = np.concatenate([np.arange(256), np.arange(256)]).astype(np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x40
        scales = [0, 1, 7, 100, 119, 127, 134, 135, 140, 200, 245]
        rows = np.stack([np.concatenate([codes, np.full(16, s, np.uint8)]) for s in scales])
    else:
        packed = np.tile(np.arange(256).astype(np.uint8), 1)
        scales = [s for s in range(256) if (s & 0x7F) != 0x7F][::5]
        rows = np.stack([np.concatenate([packed, np.full(32, s, np.uint8)]) for s in scales])
    n = len(rows)
    cache = HostPaged(fmt, 512, [1] * n, seed=770)
    for b in range(n):
        cache.pool[cache.block_table[b, 0], :rb] = rows[b]
    want = codecs.decode_rows(rows, fmt, 512)
    cs = torch.zeros((n, 32, 2), device="cuda")
    cs[..., 0] = 1.0
    out, _ = cskv.window_attn(torch.zeros((n, 1, 512), dtype=torch.bfloat16, device="cuda"), cache.to_device(),
                              _i32([1] * n), 4, 0, 1, None, SCALE, cs)
    assert cskv.device_status() == 0
    assert np.array_equal(out[:, 0].float().cpu().numpy().astype(np.float64),
                          torch.from_numpy(want).to(torch.bfloat16).double().numpy())


def test_evict_with_one_table_in_place_and_one_apart():
    e = _evict_case(2, 500, [500, 300], [(FP8, 512)], seed=780)
    dev = [c.to_device() for c in e["caches"]]
    acc, age, n = cuda(e["acc"]), cuda(e["age"]), _i32(e["n"])
    age_out = torch.full((2, 400), -5, dtype=torch.int32, device="cuda")
    src, n_out, acc_out, _ = cskv.evict(dev, acc, n, 400, fixed=3, recent=40, age=age, age_out=age_out)
    assert acc_out is acc and n_out is n and cskv.device_status() == 0
    for b in range(2):
        ref, m = bounded.evict(e["acc"][b], e["age"][b], int(e["n"][b]), 400, 3, 40)
        assert np.array_equal(src[b].cpu().numpy(), ref) and int(n_out[b]) == m
        assert np.array_equal(acc_out[b, :m].cpu().numpy(), e["acc"][b][ref[:m]])
        assert np.array_equal(acc_out[b, m:].cpu().numpy(), e["acc"][b][m:])
        assert np.array_equal(age_out[b, :m].cpu().numpy(), e["age"][b][ref[:m]])
        assert (age_out[b, m:] == -5).all()
        assert np.array_equal(age[b].cpu().numpy(), e["age"][b])


def test_weights_of_many_requests():
    """More requests than share their tiles evenly (a block per request), some empty."""
    B, H = 70, 8
    n = [(37 * b) % 300 for b in range(B)]
    c = _prefix_case(B, H, 0, n, BF16, None, seed=790)
    lse = torch.full((B, H), 5.0, device="cuda")
    acc = torch.zeros((B, 300), device="cuda")
    cskv.attn_weights(c["q"][0].cuda(), c["cache"].to_device(), _i32(n), 300, SCALE, _cs(c["ctx"]), lse, acc)
    assert cskv.device_status() == 0
    got = acc.cpu().numpy()
    for b in range(B):
        w, bound = bounded.weights(c["q"][1][b], int(c["ctx"][b]) - 1, c["cache"].decoded[b][:n[b]], np.full(H, 5.0), SCALE)
        assert np.all(np.abs(got[b, :n[b]] - w) <= bound + 2.0 ** -24 * np.abs(w)) and not got[b, n[b]:].any()


def test_window_many_heads_of_one_query_group():
    """One head: 32 queries to a row block, several runs in it; and a prompt whose last block is short."""
    L = [97, 3, 200]
    cache = _cache(FP8, L, seed=800)
    req = np.repeat(np.arange(3), L)
    pos1 = np.concatenate([np.arange(1, n + 1) for n in L])
    for H in (1, 2, 63):
        _window_all(cache, _queries(len(req), H, 801), pos1, 33, 2, req, None,
                    pick=list(range(0, len(req), 7)) + [96, 97, 99, 100, len(req) - 1])


@pytest.mark.parametrize("H", [16, 64, 65, 96, 128])
@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
def test_weights_shares_that_span_requests(H, fmt):
    """More tiles than blocks: a block's share goes from one request to the next."""
    B = 24
    n = [1500 - 37 * b for b in range(B)]
    c = _prefix_case(B, H, 0, n, fmt, None, seed=810 + H)
    lse = torch.full((B, H), 5.0, device="cuda")
    acc = torch.zeros((B, 1500), device="cuda")
    cskv.attn_weights(c["q"][0].cuda(), c["cache"].to_device(), _i32(n), 1500, SCALE, _cs(c["ctx"]), lse, acc)
    assert cskv.device_status() == 0
    got = acc.cpu().numpy()
    for b in range(B):
        w, bound = bounded.weights(c["q"][1][b], int(c["ctx"][b]) - 1, c["cache"].decoded[b][:n[b]], np.full(H, 5.0), SCALE)
        assert np.all(np.abs(got[b, :n[b]] - w) <= bound + 2.0 ** -24 * np.abs(w)) and not got[b, n[b]:].any()


@pytest.mark.parametrize("H", [3, 64])
def test_window_of_many_parts(H):
    """A long window of one request: more parts than one thread per 8 dims joins, some rows of a
    second request without any key."""
    pos1 = [20000, 0, 17]
    cache = _cache(FP8, pos1, seed=820)
    _window_all(cache, _queries(3, H, 821), pos1, 20000, 3, None, np.linspace(-2, 3, H).astype(np.float32))


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_of_slices_beyond_shared_memory(in_place):
    """Longer slices than the shared memory has keys for: they are read again for every digit."""
    cap, n, budget, fixed, recent = 450001, 449999, 300000, 100, 20000
    pages = (cap + 63) // 64
    rs = np.random.default_rng(830)
    acc = np.exp(rs.standard_normal((1, cap))).astype(np.float32)
    acc[0, ::5] = 0.25
    age = rs.permutation(cap).astype(np.int32)[None]
    pool = torch.randint(0, 256, (pages, 64 * 256), dtype=torch.uint8, device="cuda",
                         generator=torch.Generator(device="cuda").manual_seed(831))
    bt = cuda(rs.permutation(pages).astype(np.int32)[None])
    rows = lambda: pool.view(pages, 64, 256)[bt[0].long()].view(-1, 256)
    before = rows().clone()
    a, g, nn = cuda(acc), cuda(age), _i32([n])
    kw = {} if in_place else dict(acc_out=torch.full((1, budget), -5.0, device="cuda"), n_out=_i32([0]),
                                  age_out=torch.full((1, budget), -5, dtype=torch.int32, device="cuda"))
    src, n_out, acc_out, age_out = cskv.evict([cskv.PagedCache(pool, bt, BF16, 128)], a, nn, budget, fixed=fixed,
                                              recent=recent, age=g, **kw)
    assert cskv.device_status() == 0
    ref, m = bounded.evict(acc[0], age[0], n, budget, fixed, recent)
    assert int(n_out[0]) == m and np.array_equal(src[0].cpu().numpy(), ref)
    assert np.array_equal(acc_out[0, :m].cpu().numpy(), acc[0][ref[:m]])
    assert np.array_equal(age_out[0, :m].cpu().numpy(), age[0][ref[:m]])
    after = rows()
    assert torch.equal(after[:m], before[torch.from_numpy(ref[:m]).long().cuda()])
    assert torch.equal(after[m:], before[m:])
