"""GPU parity of chunk_attn against the fp64 definition on the same coded bytes, with bounds that
count the roundings the call documents, and a server's steps from lengths to attention."""

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import bounded, codecs, step

from cases import HostPaged, bf16_values, cuda
from test_gpu_bounded_cache import BF16, FP4, FP8, SCALE, _cache, _check, _i32, _queries

pytestmark = pytest.mark.gpu

ERR_BOUNDS, ERR_TIMEOUT = 5, 4


class Case:
    """R requests of `length` tokens, the last `new` of them in the call."""

    def __init__(self, new, length, H, ratio, fmt=FP8, window=0, rfmt=FP8, n=None, sink=False, seed=0, extra=0):
        rs = np.random.default_rng(seed)
        self.new, self.len = np.asarray(new), np.asarray(length)
        self.R, self.H, self.ratio, self.window = len(new), H, ratio, window
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.T = int(self.cu[-1]) + extra
        self.n = None if n is None else np.asarray(n)
        rows = None if ratio is None else [int(x) // ratio for x in length] if ratio else [int(x) for x in n]
        self.max_entries = 0 if rows is None else max(rows)
        self.entries = None if rows is None else _cache(fmt, rows, seed + 1)
        self.rows = _cache(rfmt, [int(x) for x in length], seed + 2) if window else None
        self.max_ctx = int(self.len.max())
        self.q = _queries(self.T, H, seed + 3)
        self.sink = rs.standard_normal(H).astype(np.float32) if sink else None
        self.req = np.repeat(np.arange(self.R), self.new)
        self.pos = np.concatenate([np.arange(l - n_, l) for l, n_ in zip(self.len, self.new)]) if self.cu[-1] else np.zeros(0, int)

    def args(self):
        pos = np.zeros(self.T, np.int64)
        pos[:len(self.pos)] = self.pos
        return dict(q=self.q[0].cuda(), cu_q=_i32(self.cu), ctx_len=_i32(self.len),
                    entries=None if self.entries is None else self.entries.to_device(), ratio=self.ratio or 0,
                    max_entries=self.max_entries, max_ctx_len=self.max_ctx, sink=None if self.sink is None else cuda(self.sink),
                    softmax_scale=SCALE, q_rope_cs=cuda(cskv.rope_table(pos)), n_entries=None if self.n is None else _i32(self.n),
                    rows=None if self.rows is None else self.rows.to_device(), window=self.window, want_lse=True)

    def run(self, **change):
        return cskv.chunk_attn(**dict(self.args(), **change))

    def keys(self, i):
        r, t = int(self.req[i]), int(self.pos[i])
        parts = [np.zeros((0, 512))]
        if self.entries is not None:
            m, _, _ = step.chunk_keys(t, self.ratio, None if self.n is None else int(self.n[r]), 0)
            parts.append(self.entries.decoded[r][:m])
        if self.window:
            _, lo, hi = step.chunk_keys(t, 1, None, self.window)
            parts.append(self.rows.decoded[r][lo:hi])
        return np.concatenate(parts)

    def want(self, i, scale=SCALE):
        return bounded.attend(self.q[1][i], int(self.pos[i]), self.keys(i), self.sink, scale)

    def check(self, out, lse, pick=None):
        assert cskv.device_status() == 0
        for i in (range(len(self.req)) if pick is None else pick):
            _check(out[i], lse[i], self.want(i), "query %d" % i)


def _some(T, n, seed=0):
    return sorted(set(np.random.default_rng(seed).integers(0, T, n).tolist()) | {0, T - 1})


@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
@pytest.mark.parametrize("H", [1, 5, 16, 20, 64, 65, 96, 128])
def test_single_tokens_of_several_requests(fmt, H):
    length = [700, 1, 129, 128, 64, 3, 257]
    c = Case([1] * 7, length, H, 4, fmt, window=128, rfmt=BF16 if fmt == FP4 else FP8, sink=H % 2 == 0, seed=H)
    c.check(*c.run())


@pytest.mark.parametrize("ratio", [1, 2, 4, 128])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 5000])
def test_ratios_and_windows(ratio, window):
    c = Case([70, 1, 33], [600, 300, 33], 8, ratio, FP8, window=window, rfmt=FP8, seed=ratio + window)
    c.check(*c.run(), pick=_some(104, 25))


@pytest.mark.parametrize("fmt,rfmt", [(BF16, FP8), (FP8, BF16), (FP4, FP8), (FP8, FP4), (FP4, FP4)])
@pytest.mark.parametrize("H", [3, 24, 64, 128])
def test_formats_of_entries_and_rows(fmt, rfmt, H):
    c = Case([40, 90], [1000, 777], H, 4, fmt, window=128, rfmt=rfmt, sink=True, seed=H + 7)
    c.check(*c.run(), pick=_some(130, 14))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500])
def test_chunk_and_cache_lengths(n):
    """Chunks of n tokens of a fresh request, and n entries behind."""
    c = Case([n], [n], 16, 1, BF16, seed=n)
    c.check(*c.run(), pick=_some(n, 12))
    c = Case([3], [n + 3], 20, 1, FP8, window=64, seed=n)
    c.check(*c.run())
    c = Case([2, 1], [2, 1], 64, 0, FP4, n=[n, max(0, n - 20)], seed=n)
    c.check(*c.run())


def test_attention_to_states_of_another_length():
    """Every query of a request sees all its states, whatever its position; some requests have none."""
    c = Case([37, 5, 1, 60], [900, 5, 40, 60], 32, 0, FP4, n=[1500, 0, 1, 333], sink=True, seed=3)
    c.check(*c.run(), pick=_some(103, 20))
    out, lse = c.run(ctx_len=None)
    c2, l2 = c.run()
    assert torch.equal(out, c2) and torch.equal(lse, l2)
    assert not out[37:42].any() and torch.equal(lse[37:42], cuda(c.sink).expand(5, 32))


def test_a_bound_of_entries_beside_the_positions():
    """n_entries below what the positions allow (a cache that was cut), with a window."""
    c = Case([30, 30], [800, 400], 16, 4, FP8, window=32, n=[77, 1000], seed=4)
    c.max_entries = 1000
    c.check(*c.run(), pick=_some(60, 16))


def test_windows_alone():
    c = Case([50, 20, 1], [300, 20, 129], 20, None, window=100, rfmt=FP8, sink=True, seed=5)
    c.check(*c.run(), pick=_some(71, 16))


def test_chunks_longer_than_their_requests_and_endless_windows():
    """Queries before position 0 see nothing; a window of any size reaches back to the first row."""
    c = Case([12, 3], [12, 3], 16, 1, FP8, window=2 ** 31 - 1, seed=30)
    c.check(*c.run())
    out, lse = c.run(ctx_len=_i32([5, 3]))
    assert cskv.device_status() == 0
    assert not out[:7].any() and torch.isneginf(lse[:7]).all()
    for i in range(7, 12):
        # the query at position i - 7, turned by the table's row of its own
        keys = np.concatenate([c.entries.decoded[0][:i - 6], c.rows.decoded[0][:i - 6]])
        _check(out[i], lse[i], bounded.attend(c.q[1][i], i, keys, None, SCALE))


def test_requests_without_queries_and_rows_behind_the_last_one():
    c = Case([0, 9, 0, 0, 4, 0], [100, 90, 0, 5, 40, 7], 16, 4, FP8, window=16, seed=6, extra=5)
    out = torch.full((c.T, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, 16), 7.0, device="cuda")
    c.run(out=out, lse=lse)
    c.check(out, lse)
    assert (out[13:] == 7.0).all() and (lse[13:] == 7.0).all()


def test_no_queries_at_all():
    c = Case([0, 0], [100, 90], 16, 4, FP8, seed=6, extra=3)
    out = torch.full((3, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert (out == 7.0).all() and cskv.device_status() == 0


def test_queries_without_keys():
    """Positions before the first entry: out 0, lse the sink, -inf without one."""
    for sink in (True, False):
        c = Case([10], [10], 16, 128, FP8, sink=sink, seed=8)
        c.max_entries = 5
        out, lse = c.run()
        assert cskv.device_status() == 0 and not out.any()
        want = cuda(c.sink).expand(10, 16) if sink else torch.full((10, 16), -float("inf"), device="cuda")
        assert torch.equal(lse, want)


def test_a_long_chunk_on_a_long_cache():
    c = Case([300, 41], [70000, 30000], 64, 128, FP8, window=128, sink=True, seed=9)
    a = c.run()
    c.check(*a, pick=_some(341, 6))
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("new,H", [([1], 16), ([1], 128), ([3, 2], 64), ([20], 5)])
def test_few_queries_on_a_long_cache_are_split(new, H):
    c = Case(new, [30000 + 17 * k for k in range(len(new))], H, 1, FP8, window=128, sink=True, seed=10)
    a = c.run()
    c.check(*a, pick=_some(sum(new), 2))
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_growing_logits_move_the_reference():
    """Keys whose logits grow along the list, and a first tile far below the rest."""
    H, n = 16, 1000
    rs = np.random.default_rng(12)
    c = Case([6], [n], H, 1, BF16, seed=12)
    d = rs.standard_normal(512)
    d /= np.linalg.norm(d)
    v = np.outer(np.linspace(-60, 120, n), d) + 0.1 * rs.standard_normal((n, 512))
    c.entries = HostPaged(BF16, 512, [n], seed=3)
    c.entries.fill(0, v.astype(np.float32))
    q = np.broadcast_to(8 * d, (6, H, 512)) + 0.1 * rs.standard_normal((6, H, 512))
    c.q = bf16_values(q)
    c.check(*c.run())


SINKS = np.array([np.inf, np.finfo(np.float32).max, 3e38, 1e38, 200.0, -np.inf, 0.0], np.float32)


@pytest.mark.parametrize("length", [60, 20000])
def test_sinks_up_to_infinity(length):
    c = Case([2], [length], len(SINKS), 1, FP8, seed=13)
    c.sink = SINKS
    out, lse = c.run()
    assert cskv.device_status() == 0
    top = np.isposinf(SINKS)
    assert not out[:, cuda(top)].any() and torch.isposinf(lse[:, cuda(top)]).all()
    c.sink = np.where(top, 0, SINKS).astype(np.float32)
    for i in range(2):
        o, l, bo, bl = c.want(i)
        _check(out[i][cuda(~top)], lse[i][cuda(~top)], (o[~top], l[~top], bo[~top], bl[~top]))


@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-30, 1e-3])
def test_smallest_scales(scale):
    c = Case([3], [300], 16, 1, FP8, window=10, seed=14)
    out, lse = c.run(softmax_scale=scale)
    assert cskv.device_status() == 0
    for i in range(3):
        _check(out[i], lse[i], c.want(i, float(np.float32(scale))))


def _poison(cache, r, rows, value=0xFF):
    rb = codecs.row_bytes(cache.fmt, 512)
    for j in rows:
        cache.pool[cache.block_table[r, j // 64], j % 64 * rb:(j % 64 + 1) * rb] = value


@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
def test_rows_that_nothing_sees_never_count(fmt):
    """NaN in the entries behind the visible ones, in the rows before the windows, in the pages'
    ends; tables that point nowhere there."""
    c = Case([9], [1000], 16, 4, fmt, window=50, rfmt=fmt, seed=15)
    c.check(*c.run())
    _poison(c.rows, 0, range(896, 1000 - 9 - 49))
    c.rows.block_table[0, :14] = [-77, 10 ** 6] * 7
    _poison(c.rows, 0, [])
    c.check(*c.run())
    c = Case([9], [1000], 16, 4, fmt, window=50, rfmt=fmt, n=[100], seed=15)
    c.max_entries = 250
    _poison(c.entries, 0, range(100, 250))
    c.entries.block_table[0, 2:] = -5
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [BF16, FP8, FP4])
@pytest.mark.parametrize("where", ["entry", "row"])
def test_a_row_that_is_not_finite_reaches_its_queries_alone(fmt, where):
    """A NaN row: the queries that see it are NaN, all others as without it."""
    c = Case([40, 30], [400, 30], 16, 1 if where == "entry" else 128, fmt, window=0 if where == "entry" else 20, rfmt=fmt, seed=16)
    base, blse = c.run()
    bad = 375                          # of request 0; queries sit at 360 .. 399
    cache = c.entries if where == "entry" else c.rows
    # one NaN: a code or a scale
    rb = codecs.row_bytes(fmt, 512)
    at = bad % 64 * rb
    page = cache.pool[cache.block_table[0, bad // 64]]
    if fmt == BF16:
        page[at + 10:at + 12] = [0xC0, 0x7F]
    elif fmt == FP8:
        page[at + 10] = 0x7F
    else:
        page[at + 256 + 3] = 0x7F
    out, lse = c.run()
    assert cskv.device_status() == 0
    t = np.arange(360, 400)
    sees = (t >= bad) if where == "entry" else (t >= bad) & (t < bad + 20)
    sees = np.concatenate([sees, np.zeros(30, bool)])
    nan = torch.isnan(out).flatten(1)
    assert nan[cuda(sees)].all() and torch.isnan(lse[cuda(sees)]).all()
    assert torch.equal(out[cuda(~sees)], base[cuda(~sees)]) and torch.equal(lse[cuda(~sees)], blse[cuda(~sees)])


def test_queries_that_are_not_finite_stay_alone():
    c = Case([20], [300], 4, 1, FP8, seed=17)
    base, blse = c.run()
    c.q[0][7, 2, 100] = float("nan")
    c.q[0][9, 0, 500] = float("inf")
    out, lse = c.run()
    keep = torch.ones((20, 4), dtype=torch.bool, device="cuda")
    keep[7, 2] = keep[9, 0] = False
    assert torch.equal(out[keep], base[keep]) and torch.equal(lse[keep], blse[keep])
    assert torch.isnan(out[7, 2]).all() and torch.isnan(out[9, 0]).any()


def test_pages_outside_the_pool_are_skipped_and_reported():
    c = Case([5, 4], [300, 200], 16, 1, FP8, seed=18)
    c.entries.block_table[0, 1] = c.entries.num_pages + 3
    c.entries.block_table[1, 2] = -1
    out, lse = c.run()
    assert cskv.device_status() == ERR_BOUNDS
    skip = {0: set(range(64, 128)), 1: set(range(128, 192))}
    for i in range(9):
        r, t = int(c.req[i]), int(c.pos[i])
        keep = [j for j in range(t + 1) if j not in skip[r]]
        _check(out[i], lse[i], bounded.attend(c.q[1][i], t, c.entries.decoded[r][keep], None, SCALE))
    c.check(*Case([5, 4], [300, 200], 16, 1, FP8, seed=18).run(), pick=[])


def test_lengths_beyond_their_bounds_are_cut_and_reported():
    c = Case([3], [500], 16, 1, FP8, seed=19)
    out, lse = c.run(max_entries=400)
    assert cskv.device_status() == ERR_BOUNDS
    for i in range(3):
        _check(out[i], lse[i], bounded.attend(c.q[1][i], int(c.pos[i]), c.entries.decoded[0][:400], None, SCALE))
    c.run(max_ctx_len=300)
    assert cskv.device_status() == ERR_BOUNDS
    c.run(ctx_len=_i32([-4]))
    assert cskv.device_status() == ERR_BOUNDS


def test_flat_caches_and_long_pages():
    """No block table, one request; pages further apart than their rows need."""
    c = Case([30], [500], 16, 1, FP8, window=0, seed=20)
    a = c.run()
    rb = codecs.row_bytes(FP8, 512)
    rows = np.concatenate([c.entries.pool[p][:64 * rb] for p in c.entries.block_table[0]]).reshape(-1, 64 * rb)
    b = c.run(entries=cskv.PagedCache(cuda(rows), None, FP8, 512))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pool = np.full((c.entries.num_pages, 64 * rb + 48), 0xFF, np.uint8)
    pool[:, :64 * rb] = c.entries.pool[:, :64 * rb]
    b = c.run(entries=cskv.PagedCache(cuda(pool), _i32(c.entries.block_table), FP8, 512))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_graph_and_a_stream_and_a_workspace_of_the_callers():
    c = Case([40, 1, 9], [900, 400, 9], 32, 4, FP8, window=128, sink=True, seed=21)
    a = c.args()
    want = cskv.chunk_attn(**a)
    R, T = 3, 50
    most = cskv.chunk_attn_max_keys(R, T, a["max_entries"], 128, a["max_ctx_len"])
    ws = torch.full((cskv.chunk_attn_workspace_size(R, T, 32, most) + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    a.update(out=out, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cskv.chunk_attn(**a, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cskv.chunk_attn(**a)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)          # nothing is kept there from one call to the next
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert cskv.device_status() == 0


def test_a_tighter_bound_of_keys_and_one_too_tight():
    c = Case([10, 10], [1000, 200], 16, 1, FP8, window=20, seed=22)
    up = lambda n: (n + 15) // 16 * 16
    need = [up(1000) + up(29), up(200) + up(29)]
    a = c.run(max_keys=sum(need))
    c.check(*a, pick=[0, 9, 10, 19])
    b = c.run(max_keys=sum(need) - 1)      # no room for the second request: no keys
    assert cskv.device_status() == ERR_BOUNDS
    c.check(*b, pick=[0, 9])               # (not the same bits: the row blocks' shares are others)
    assert not b[0][10:].any() and torch.isneginf(b[1][10:]).all()


def test_calls_that_are_refused():
    c = Case([3], [100], 16, 1, FP8, window=20, seed=23)
    a = c.args()
    for bad in (dict(q=a["q"].float()), dict(cu_q=a["cu_q"].long()), dict(ctx_len=_i32([1, 2])), dict(sink=torch.zeros(3, device="cuda")),
                dict(q_rope_cs=a["q_rope_cs"][:2]), dict(n_entries=_i32([1, 2])), dict(cu_q=_i32([0, 1, 3])),
                dict(out=a["q"][:2]), dict(lse=torch.zeros((3, 8), device="cuda"))):
        with pytest.raises(ValueError):
            cskv.chunk_attn(**dict(a, **bad))
    for bad in (dict(window=0), dict(rows=None), dict(entries=None, rows=None, window=0), dict(ratio=0), dict(ratio=-1),
                dict(softmax_scale=0.0), dict(max_entries=-1), dict(ctx_len=None)):
        with pytest.raises(cskv.CskvError):
            cskv.chunk_attn(**dict(a, **bad))


@pytest.mark.parametrize("new,length,H", [([300], [9000], 64), ([5], [300], 16), ([40, 1, 0, 7], [500, 60, 0, 9], 128)])
def test_waits_that_run_out_end_the_call_and_leave_the_next_one_exact(new, length, H):
    c = Case(new, length, H, 1, FP8, window=128, sink=True, seed=24)
    want = c.run()
    assert cskv.device_status() == 0
    cskv.set_spin_limit(64)
    try:
        for _ in range(3):
            c.run()
            assert cskv.device_status() == ERR_TIMEOUT
    finally:
        cskv.set_spin_limit(0)
    out, lse = c.run()
    assert cskv.device_status() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own; the same bits as one after the other."""
    cases = [Case([200, 30], [900, 400], 64, 1, FP8, window=64, sink=True, seed=25), Case([150], [4000], 20, 4, FP4, seed=26)]
    args = [c.args() for c in cases]
    want = [cskv.chunk_attn(**a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for k in (0, 1):
            got[k].append(cskv.chunk_attn(**args[k], stream=streams[k]))
    torch.cuda.synchronize()
    assert cskv.device_status() == 0
    for k in (0, 1):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_the_same_as_the_calls_for_windows_and_for_single_tokens():
    """window_attn with a window as long as the request, prefix_decode_attn without a prefix: the
    same definition, other kernels; each within its bound of it."""
    c = Case([40, 25], [300, 200], 16, 1, FP8, sink=True, seed=27)
    out, lse = c.run()
    pos1 = c.pos + 1
    w, wl = cskv.window_attn(c.q[0].cuda(), c.entries.to_device(), _i32(pos1), 300, 0, 300, cuda(c.sink), SCALE,
                             cuda(cskv.rope_table(c.pos)), req_of=_i32(c.req), want_lse=True)
    for i in range(0, 65, 7):
        ref = c.want(i)
        _check(out[i], lse[i], ref)
        _check(w[i], wl[i], ref)
    c = Case([1, 1, 1], [700, 129, 5], 64, 1, FP8, sink=True, seed=28)
    out, lse = c.run()
    p, pl = cskv.prefix_decode_attn(c.q[0].cuda(), c.entries.to_device(), _i32(c.len), 0, 700, cuda(c.sink), SCALE,
                                    cuda(cskv.rope_table(c.pos)), want_lse=True)
    for i in range(3):
        ref = c.want(i)
        _check(out[i], lse[i], ref)
        _check(p[i], pl[i], ref)


@pytest.mark.parametrize("H", [1, 2, 3, 7, 33, 50, 63, 127])
def test_heads_that_fill_a_row_block_unevenly(H):
    """Row blocks of 128 / H queries, in two halves that part between the heads of a query."""
    c = Case([9, 130, 2], [200, 130, 777], H, 1, FP8, window=20, rfmt=FP8, sink=True, seed=H)
    c.check(*c.run(), pick=_some(141, 16))


# --- a server's steps --------------------------------------------------------------------------

def test_a_servers_steps_from_lengths_to_attention():
    """Prompts in chunks, single tokens, a request that ends and another in its place: tables and
    slots from plan_step, angles from rope_cs, rows written by norm_rope, attention by chunk_attn;
    nothing but the tokens comes from the host.  The oracle keeps every request's rows in a list."""
    rs = np.random.default_rng(30)
    B, T, H, per, total, window = 3, 200, 8, 12, 20, 64
    pages = cskv.PageTable.allocate(B, per, total)
    maps = cskv.StepMaps(B, T, pages=True, ring=True)
    maps.new_len.zero_()
    plan = cskv.RopePlan()
    cache = cskv.PagedCache.allocate(total, cskv.FMT_FP8, 512, block_table=pages.block_table)
    ring = cskv.PagedCache.allocate(2 * B, cskv.FMT_BF16, 512)
    w = rs.uniform(0.5, 1.5, 512).astype(np.float32)
    rows = [np.zeros((0, 512)) for _ in range(B)]
    for new in ([100, 1, 0], [64, 1, 130], [1, 1, 1], [-1, 1, 1], [90, 0, 64], [1, 1, 1], [1, -1, 1]):
        n = np.maximum(new, 0)
        x, xv = bf16_values(1.5 * rs.standard_normal((T, 1, 512)))
        q, _ = bf16_values(2.0 * rs.standard_normal((T, H, 512)))
        cskv.plan_step(maps.new_len, _i32(new), T, pages, ring_rows=128, out=maps)
        cs = cskv.rope_cs(maps.pos1, plan, shift=-1)
        qn, _, _ = cskv.norm_rope([dict(x=q.cuda(), norm=True),
                                   dict(x=x.cuda(), norm=True, norm_w=cuda(w), rotate=True, cache=cache, slot=maps.slot),
                                   dict(x=x.cuda(), norm=True, norm_w=cuda(w), rotate=True, cache=ring, slot=maps.ring_slot)], cs)
        out, lse = cskv.chunk_attn(qn, maps.cu_new, maps.new_len, cache, 1, per * 64, per * 64, None, SCALE, cs, want_lse=True)
        # the last queries once more, over the window alone (the raw rows of the same pages)
        wout, wlse = cskv.chunk_attn(qn, maps.cu_new, maps.new_len, None, 0, 0, per * 64, None, SCALE, cs, rows=cache,
                                     window=window, want_lse=True)
        assert cskv.device_status() == 0 and int(pages.state[2]) == 0
        cs_h, qv = cs.cpu().numpy(), qn.float().cpu().numpy()
        i = 0
        for b in range(B):
            if new[b] < 0:
                rows[b] = np.zeros((0, 512))
                continue
            start = len(rows[b])
            y = step.norm_rope(xv[i:i + n[b], 0], True, w, 1e-6, cs_h[i:i + n[b]])
            rows[b] = np.concatenate([rows[b], codecs.decode_rows(codecs.encode_rows(y, codecs.FMT_FP8), codecs.FMT_FP8, 512)]) if n[b] else rows[b]
            for k in sorted({0, n[b] // 2, n[b] - 1} & set(range(n[b]))):
                t = start + k
                _check(out[i + k], lse[i + k], bounded.attend(qv[i + k], t, rows[b][:t + 1], None, SCALE), "request %d" % b)
                _check(wout[i + k], wlse[i + k], bounded.attend(qv[i + k], t, rows[b][max(0, t + 1 - window):t + 1], None, SCALE))
            i += n[b]
        assert maps.new_len.tolist() == [len(r) for r in rows]


@pytest.mark.parametrize("R", [255, 257, 1024, 1025, 2100])
def test_many_requests(R):
    """More requests than a block has threads, and than it sums up itself; some without new tokens, one
    with a row that is not finite."""
    rs = np.random.default_rng(R)
    length = rs.integers(1, 40, R)
    new = np.minimum(rs.choice([0, 1, 1, 2, 5], R), length)
    new[R - 2] = 1
    c = Case(new, length, 4, 1, FP8, window=8, seed=R)
    pick = sorted(set(_some(len(c.req), 30, R)) | {int(c.cu[R - 2])})
    out, lse = c.run()
    c.check(out, lse, pick)
    _poison(c.entries, R - 2, [0])
    bad, bad_lse = c.run()
    hit = np.flatnonzero(c.req == R - 2)
    assert np.isnan(bad[hit].float().cpu().numpy()).all() and np.isnan(bad_lse[hit].cpu().numpy()).all()
    rest = np.flatnonzero(c.req != R - 2)
    assert torch.equal(bad[rest], out[rest]) and torch.equal(bad_lse[rest], lse[rest])
    assert cskv.device_status() == 0


@pytest.mark.parametrize("R", [3, 300, 1025])
def test_queries_that_do_not_add_up_are_left_and_reported(R):
    """Borders that go back, again and again, below 0 or beyond T: each request alone would have all queries."""
    c = Case([1] * R, [40] * R, 8, 1, FP8, window=16, seed=R)
    back = np.tile([0, R], R)[:R + 1]
    low, high, one = c.cu.copy(), c.cu.copy(), c.cu.copy()
    low[1], high[R], one[R // 2] = -1, R + 1, one[R // 2 + 1] + 1
    for cu in (back, low, high, one):
        out = torch.full((R, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((R, 8), 5.0, device="cuda")
        c.run(cu_q=_i32(cu), out=out, lse=lse)
        assert cskv.device_status() == ERR_BOUNDS
        assert (out == 3.0).all() and (lse == 5.0).all()
    out, lse = c.run()
    c.check(out, lse, pick=_some(R, 9, R))


@pytest.mark.parametrize("new,length,H,ratio,window", [([77], [77], 128, 1, 0), ([76], [76], 128, 1, 0), ([75, 1], [75, 900], 128, 1, 0),
                                                       ([200, 33, 5], [200, 400, 700], 64, 1, 0), ([640], [1000], 32, 4, 128),
                                                       ([2100, 1, 40], [2100, 300, 40], 96, 128, 128), ([1, 700], [9000, 700], 64, 1, 0)])
def test_row_blocks_dealt_out_whole_and_cut(new, length, H, ratio, window):
    """As many row blocks as pairs, one more, some rounds, more than are dealt out, one long one among short ones."""
    c = Case(new, length, H, ratio, FP8, window=window, rfmt=BF16, sink=True, seed=len(new) + H)
    out, lse = c.run()
    c.check(out, lse, pick=sorted(set(_some(len(c.req), 14)) | {min(len(c.req) - 1, k) for k in (74, 75, 76, 77)}))
    again, lse2 = c.run()
    assert torch.equal(again, out) and torch.equal(lse2, lse)


def test_row_blocks_of_a_thousand_tiles_and_more_in_full_rounds():
    """Sizes beyond those that the plan tells apart: the same bits each time."""
    n = 132000
    c = Case([1], [n], 16, 1, FP4, seed=52)                 # its pages are every request's
    R = 2 * 76
    lens = n - 3 * np.arange(R)
    entries = c.entries.to_device()
    kw = dict(c.args(), q=c.q[0].repeat(R, 1, 1).cuda(), cu_q=_i32(np.arange(R + 1)), ctx_len=_i32(lens),
              q_rope_cs=cuda(cskv.rope_table(lens - 1)), max_keys=int(((lens + 15) // 16 * 16).sum()),
              entries=cskv.PagedCache(entries.pool, _i32(np.repeat(c.entries.block_table, R, 0)), FP4, 512))
    out, lse = cskv.chunk_attn(**kw)
    assert cskv.device_status() == 0
    for i in (0, 77, 151):
        _check(out[i], lse[i], bounded.attend(c.q[1][0], int(lens[i]) - 1, c.entries.decoded[0][:lens[i]], None, SCALE))
    for _ in range(3):
        again, lse2 = cskv.chunk_attn(**kw)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
