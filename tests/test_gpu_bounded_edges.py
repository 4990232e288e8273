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
