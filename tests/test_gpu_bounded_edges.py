"""window_attn, prefix_decode_attn, attn_weights and evict where a call is unusual: prompts of
many row blocks with padding, tables and pages of other shapes, extreme sinks and scales.  The
bounds are those of test_gpu_bounded_cache.py."""

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import bounded, codecs

from cases import cuda
from test_gpu_bounded_cache import (BF16, FP4, FP8, SCALE, _cache, _check, _cs, _i32, _prefix_all, _prefix_case,
                                    _prefix_run, _queries, _window, _window_all, _window_ref)

pytestmark = pytest.mark.gpu


# --- row blocks without any tile ---------------------------------------------------------------

@pytest.mark.parametrize("where", ["first", "last", "between", "stretches", "alternating", "all"])
@pytest.mark.parametrize("H", [64, 100])
def test_window_padding_in_prompts_of_many_row_blocks(where, H):
    """A prompt of 1,000 queries is several row blocks to each SM; those of padding have no tile."""
    T, L = 1000, 400
    cache = _cache(FP8, [L], seed=900 + H)
    pos1 = np.arange(T) % L + 1
    i = np.arange(T)
    empty = {"first": i < 500, "last": i >= 500, "between": (i > 150) & (i < 700),
             "stretches": (i // 152) % 2 == 0, "alternating": (i // 7) % 2 == 0, "all": i >= 0}[where]
    pos1 = np.where(empty, 0, pos1)
    q = _queries(T, H, 901)
    req = np.zeros(T, np.int64)
    sink = np.random.default_rng(902).standard_normal(H).astype(np.float32)
    for _ in range(3):
        out, lse = _window(cache, q, pos1, 128, 4, req, sink, max_ctx=L)
        assert cskv.device_status() == 0
        assert not out[cuda(empty)].any() and torch.equal(lse[cuda(empty)], cuda(sink).expand(int(empty.sum()), H))
    real = np.flatnonzero(~empty)
    for k in real[::max(1, len(real) // 12)]:
        _check(out[k], lse[k], _window_ref(cache, q, k, pos1, 128, 4, req, sink), "query %d" % k)


# --- sinks ---------------------------------------------------------------------------------------

def _check_with_sinks(out, lse, ref, sink):
    """A head whose sink is +inf: out 0, lse +inf; the others against the definition."""
    top = np.isposinf(sink)
    assert not out[cuda(top)].any() and torch.isposinf(lse[cuda(top)]).all()
    keep = cuda(~top)
    o, l, bo, bl = ref
    _check(out[keep], lse[keep], (o[~top], l[~top], bo[~top], bl[~top]))


SINKS = np.array([np.inf, np.finfo(np.float32).max, 3e38, 1e38, 200.0, -np.inf, 0.0], np.float32)


@pytest.mark.parametrize("pos1,window", [([200, 0, 60], 128), ([20000], 20000)])
def test_window_sinks_up_to_infinity(pos1, window):
    """Sinks above any logit, some beyond fp32 in base 2; one list and a split one."""
    cache = _cache(FP8, pos1, seed=920)
    q = _queries(len(pos1), len(SINKS), 921)
    out, lse = _window(cache, q, pos1, window, 4, None, SINKS)
    assert cskv.device_status() == 0
    finite = np.where(np.isposinf(SINKS), 0.0, SINKS)
    for i in range(len(pos1)):
        _check_with_sinks(out[i], lse[i], _window_ref(cache, q, i, pos1, window, 4, None, finite), SINKS)


@pytest.mark.parametrize("swa_fmt", [None, FP8, BF16])
def test_prefix_sinks_up_to_infinity(swa_fmt):
    c = _prefix_case(3, len(SINKS), 100, [300, 100, 0], FP8, swa_fmt, seed=922, ctx=[500, 20, 0])
    c["sink"] = SINKS
    out, lse = _prefix_run(c)
    assert cskv.device_status() == 0
    from test_gpu_bounded_cache import _prefix_keys
    finite = np.where(np.isposinf(SINKS), 0.0, SINKS)
    for b in range(3):
        ref = bounded.attend(c["q"][1][b], max(0, int(c["ctx"][b]) - 1), _prefix_keys(c, b), finite, SCALE)
        _check_with_sinks(out[b], lse[b], ref, SINKS)


# --- scales --------------------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-38, 2e-38, 1e-30, 1e-3])
def test_window_smallest_scales(scale):
    """Logits near 0, whatever the keys: the mean of the visible rows.  The first query's keys are all in
    the row block's first tile, the last one's all in its second."""
    L, H = 300, 16
    cache = _cache(FP8, [L], seed=930)
    pos1 = np.array([100, 160, 220, 280])
    q = _queries(4, H, 931)
    out, lse = cskv.window_attn(q[0].cuda(), cache.to_device(), _i32(pos1), 10, 0, L, None, scale, _cs(pos1),
                                req_of=_i32([0] * 4), want_lse=True)
    assert cskv.device_status() == 0
    for i in range(4):
        keys = cache.decoded[0][bounded.visible(pos1[i] - 1, 10, 0)]
        _check(out[i], lse[i], bounded.attend(q[1][i], pos1[i] - 1, keys, None, float(np.float32(scale))))


def test_largest_scale():
    """With zero queries every logit is 0 under the largest scale too."""
    cache = _cache(BF16, [200], seed=932)
    q = torch.zeros((1, 4, 512), dtype=torch.bfloat16, device="cuda")
    out, lse = cskv.window_attn(q, cache.to_device(), _i32([200]), 50, 2, 200, None, 1e38, _cs([200]), want_lse=True)
    assert cskv.device_status() == 0
    keys = cache.decoded[0][bounded.visible(199, 50, 2)]
    _check(out[0], lse[0], bounded.attend(np.zeros((4, 512)), 199, keys, None, 1e38))


# --- what a tensor, a cache and a workspace may be ------------------------------------------------

def test_a_parameter_as_queries_and_on_a_stream():
    pos1 = [300, 70]
    cache = _cache(FP8, pos1, seed=940)
    q = _queries(2, 16, 941)
    a, la = _window(cache, q, pos1, 128, 4, None, None)
    p = torch.nn.Parameter(q[0].cuda(), requires_grad=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (cache.to_device(), _i32(pos1), 128, 4, 300, None, SCALE, _cs(pos1))
    torch.cuda.synchronize()
    b, lb = cskv.window_attn(p, *args, want_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


# --- what is read ----------------------------------------------------------------------------------

def _rubbish(cache, b, keep):
    """Rows of request b that are not in `keep` become NaN codes and scales; entries of pages without
    a row to keep point nowhere."""
    rb = codecs.row_bytes(cache.fmt, cache.dim)
    keep = set(int(j) for j in keep)
    for p in range(cache.max_pages):
        rows = [s for s in range(64) if 64 * p + s in keep]
        page = cache.pool[cache.block_table[b, p]]
        for s in set(range(64)) - set(rows):
            page[s * rb:(s + 1) * rb] = 0xFF
        if not rows:
            cache.block_table[b, p] = -77 if p % 2 else cache.num_pages + 5


@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
@pytest.mark.parametrize("window,first,H", [(1, 0, 16), (1, 3, 16), (10, 0, 4), (20, 70, 32), (1, 0, 64)])
def test_window_rows_between_neighbouring_windows_never_count(fmt, window, first, H):
    """Queries of one request up to 64 positions apart, in either order and with jumps: the rows in
    the gaps hold NaN, and no page without a visible row is looked up."""
    L = 1500
    cache = _cache(fmt, [L], seed=950)
    pos1 = np.concatenate([100 + 64 * np.arange(5), 1500 - 64 * np.arange(4), [700, 640, 760, 701], [90]])
    see = set(j for p in pos1 for j in bounded.visible(p - 1, window, first).tolist())
    _rubbish(cache, 0, see)
    _window_all(cache, _queries(len(pos1), H, 951), pos1, window, first, np.zeros(len(pos1), np.int64), None)


@pytest.mark.parametrize("B,H,P,n", [(3, 16, 70, 200), (3, 64, 200, 330), (2, 128, 1, 140), (5, 8, 1000, 1064)])
def test_weights_behind_a_prefix_that_ends_inside_a_page(B, H, P, n):
    """The prefix lies in request 0's pages alone: the other requests' rows below it hold NaN, their table
    entries of whole prefix pages point nowhere.  The attention and the weights from n_prefix on are
    the same as with rows everywhere; the weights below it would be of each request's own rows."""
    c = _prefix_case(B, H, P, [n - 13 * b if n - 13 * b > P else P for b in range(B)], FP8, None, seed=960 + P)
    cache = c["cache"]
    for b in range(1, B):      # not the pages of request 0: rows below P of the page the prefix ends in
        edge = cache.block_table[b, P // 64]
        cache.pool[edge, :P % 64 * 528] = 0xFF
        cache.block_table[b, :P // 64] = -5
    out, lse = _prefix_run(c)
    _prefix_all(c, out, lse)
    acc = torch.full((B, n), 0.5, device="cuda")
    got = cskv.attn_weights(c["q"][0].cuda(), cache.to_device(), _i32(c["n"]), n, SCALE, _cs(c["ctx"]), lse, acc,
                            decay=0.5, first=P).cpu().numpy().astype(np.float64)
    assert cskv.device_status() == 0
    l = lse.cpu().numpy()
    for b in range(B):
        m = int(c["n"][b])
        w, bound = bounded.weights(c["q"][1][b], int(c["ctx"][b]) - 1, cache.decoded[b][P:m], l[b], SCALE)
        assert np.all(np.abs(got[b, P:m] - 0.25 - w) <= bound + 3 * 2.0 ** -24 * (0.25 + w))
        assert np.all(got[b, :P] == 0.5) and np.all(got[b, m:] == 0.5)


def _flat(cache):
    """Request 0's pages in order as a cache without a table."""
    pool = cache.pool[cache.block_table[0]]
    return cskv.PagedCache(cuda(pool), None, cache.fmt, cache.dim)


def _long_pages(cache, extra=48 + 16 * 1024):
    """The same cache with pages further apart, NaN codes between them."""
    pool = np.full((cache.num_pages, cache.page_bytes + extra), 0xFF, np.uint8)
    pool[:, :cache.page_bytes] = cache.pool
    return cskv.PagedCache(cuda(pool), cuda(cache.block_table), cache.fmt, cache.dim)


@pytest.mark.parametrize("other", [_flat, _long_pages])
@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
def test_caches_without_a_table_and_with_long_pages(other, fmt):
    """The same bits as with one table and 64-row pages, from all four calls (one request's rows)."""
    L, T, H = 700, 90, 16
    cache = _cache(fmt, [L], seed=970)
    a, b = cache.to_device(), other(cache)
    q = _queries(T, H, 971)[0].cuda()
    pos1 = np.random.default_rng(972).integers(1, L + 1, T)
    w = [cskv.window_attn(q, x, _i32(pos1), 100, 5, L, None, SCALE, _cs(pos1), req_of=_i32([0] * T), want_lse=True)
         for x in (a, b)]
    p = [cskv.prefix_decode_attn(q[:1], x, _i32([L]), 130, L, None, SCALE, _cs(pos1[:1]), want_lse=True) for x in (a, b)]
    acc = [cskv.attn_weights(q[:1], x, _i32([L]), L, SCALE, _cs(pos1[:1]), p[0][1], torch.zeros((1, L), device="cuda"))
           for x in (a, b)]
    for x in (w, p):
        assert torch.equal(x[0][0], x[1][0]) and torch.equal(x[0][1], x[1][1])
    assert torch.equal(acc[0], acc[1]) and (acc[0] > 0).all()
    for i in range(0, T, 9):
        _check(w[1][0][i], w[1][1][i], _window_ref(cache, (None, q.float().cpu().numpy().astype(np.float64)), i, pos1,
                                                   100, 5, [0] * T, None))
    before = b.pool.clone()
    src = [cskv.evict([x], acc[0].clone(), _i32([L]), 300, fixed=10)[0] for x in (a, b)]
    assert torch.equal(src[0], src[1]) and cskv.device_status() == 0
    rows = lambda c, pool: pool[:, :cache.page_bytes].reshape(pool.shape[0], 64, -1)[
        c.block_table[0].long() if c.block_table is not None else torch.arange(pool.shape[0], device="cuda")].flatten(0, 1)
    assert torch.equal(rows(a, a.pool), rows(b, b.pool))
    assert torch.equal(rows(b, b.pool)[:300], rows(b, before)[src[1][0].long()])
    assert torch.equal(b.pool[:, cache.page_bytes:], before[:, cache.page_bytes:])


def test_a_flat_cache_of_several_requests():
    """Without a table every request of a batch attends to the same rows."""
    cache = _cache(FP8, [500], seed=975)
    flat, n = _flat(cache), np.array([500, 3, 0, 257])
    q = _queries(4, 64, 976)
    out, lse = cskv.prefix_decode_attn(q[0].cuda(), flat, _i32(n), 100, 500, None, SCALE, _cs(n), want_lse=True)
    wo, wl = cskv.window_attn(q[0].cuda(), flat, _i32(n), 5000, 0, 500, None, SCALE, _cs(n), want_lse=True)
    acc = cskv.attn_weights(q[0].cuda(), flat, _i32(n), 500, SCALE, _cs(n), lse, torch.zeros((4, 500), device="cuda"))
    assert cskv.device_status() == 0
    for b in range(4):
        ref = bounded.attend(q[1][b], max(0, n[b] - 1), cache.decoded[0][:n[b]], None, SCALE)
        _check(out[b], lse[b], ref)
        _check(wo[b], wl[b], ref)
        if n[b]:
            w, bound = bounded.weights(q[1][b], int(n[b]) - 1, cache.decoded[0][:n[b]], lse[b].cpu().numpy(), SCALE)
            assert np.all(np.abs(acc[b, :n[b]].cpu().numpy() - w) <= bound + 2.0 ** -24 * w)
        assert not acc[b, n[b]:].any()


def test_workspaces_of_the_caller():
    """Of the stated size inside a larger buffer, full of NaN: the same results, nothing beyond it written."""
    c = _prefix_case(3, 16, 500, [3000, 2800, 600], FP8, BF16, seed=980)
    pos1 = [20000, 300]
    cache = _cache(FP8, pos1, seed=981)
    q = _queries(2, 16, 982)
    e_acc = torch.rand((2, 3000), device="cuda")
    e_cache = _cache(FP8, [3000, 3000], seed=983)

    def calls(ws):
        o = [_prefix_run(c, **ws(cskv.prefix_decode_attn_workspace_size(3, 16, 500, 3000, True))),
             _window(cache, q, pos1, 20000, 4, None, None, **ws(cskv.window_attn_workspace_size(2, 16, 20000, 20000, 4)))]
        d = e_cache.to_device()
        o.append(cskv.evict([d], e_acc.clone(), _i32([3000, 2500]), 1400, fixed=3,
                            **ws(cskv.evict_workspace_size(2, 3000, 1400)))[:3] + (d.pool,))
        return [t for x in o for t in x]

    guards = []

    def mine(nbytes):
        assert nbytes > 0
        buf = torch.full((nbytes + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        guards.append((buf, nbytes))
        return dict(workspace=buf[256:256 + nbytes])

    want, got = calls(lambda nbytes: {}), calls(mine)
    assert cskv.device_status() == 0 and len(guards) == 3
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for buf, nbytes in guards:
        assert (buf[:256] == 0xFF).all() and (buf[256 + nbytes:] == 0xFF).all()
    with pytest.raises(cskv.CskvError):
        _prefix_run(c, workspace=guards[0][0][256:256 + guards[0][1] - 256])
    with pytest.raises(cskv.CskvError):
        _prefix_run(c, workspace=guards[0][0][128:])


@pytest.mark.parametrize("B,H", [(3, 16), (3, 64), (33, 8)])
def test_prefix_longer_than_the_first_request(B, H):
    """Request 0's pages hold the prefix, though it sees a part of it (or nothing) itself."""
    c = _prefix_case(B, H, 200, [50] + [300 - b for b in range(1, B)], FP8, FP8, seed=985)
    _prefix_all(c, *_prefix_run(c))
    c["n"][0] = 0
    _prefix_all(c, *_prefix_run(c))


def test_weights_of_heads_whose_sink_takes_everything():
    """A log-sum-exp of +inf or far above the logits adds nothing, as the formula says."""
    c = _prefix_case(2, 4, 0, [300, 20], FP8, None, seed=990, with_sink=False)
    lse = np.array([[np.inf, 3e38, -np.inf, 2.0], [-np.inf, np.inf, 5.0, 6.0]], np.float32)
    acc = torch.zeros((2, 300), device="cuda")
    cskv.attn_weights(c["q"][0].cuda(), c["cache"].to_device(), _i32(c["n"]), 300, SCALE, _cs(c["ctx"]), cuda(lse), acc)
    assert cskv.device_status() == 0
    got = acc.cpu().numpy()
    for b, heads in ((0, [3]), (1, [2, 3])):
        m = int(c["n"][b])
        w, bound = bounded.weights(c["q"][1][b][heads], int(c["ctx"][b]) - 1, c["cache"].decoded[b][:m], lse[b, heads], SCALE)
        assert np.all(np.abs(got[b, :m] - w) <= bound + 2.0 ** -24 * w) and not got[b, m:].any()


def test_calls_whose_bounds_are_zero():
    """No position and no entry at all: outputs 0, log-sum-exps the sinks, nothing accumulated or moved."""
    cache = _cache(FP8, [64, 64], seed=991).to_device()
    q, z, sink = _queries(2, 16, 992)[0].cuda(), _i32([0, 0]), torch.arange(16, device="cuda", dtype=torch.float32)
    acc = torch.full((2, 8), 3.0, device="cuda")
    for out, lse in (cskv.window_attn(q, cache, z, 5, 0, 0, sink, SCALE, _cs([1, 1]), want_lse=True),
                     cskv.prefix_decode_attn(q, cache, z, 0, 0, sink, SCALE, _cs([1, 1]), want_lse=True)):
        assert not out.any() and torch.equal(lse, sink.expand(2, 16))
    cskv.attn_weights(q, cache, z, 0, SCALE, _cs([1, 1]), lse, acc)
    src, n, _, _ = cskv.evict([cache], acc, z, 4, max_entries=0)
    assert cskv.device_status() == 0
    assert (acc == 3.0).all() and (src == -1).all() and n.tolist() == [0, 0]
