"""GPU parity of plan_step, rope_cs and norm_rope: whole numbers and coded rows equal to the
oracle's, tables of (cos, sin) within an ulp of the exact ones."""

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import codecs, rope, step

from cases import HostPaged, bf16_values, cuda

pytestmark = pytest.mark.gpu

ERR_BOUNDS = 5


def _i32(x):
    return cuda(np.asarray(x, np.int32))


# --- plan_step -----------------------------------------------------------------------------

def _pages_case(rs, ctx, ratio, per, spare, shared=None):
    """(table, free, state): each request's pages, the rest somewhere in a ring."""
    B = len(ctx)
    used = [step.pages_of(int(c) // ratio) for c in ctx]
    total = sum(used) + spare
    perm = rs.permutation(total + 7)[:total].astype(np.int32)
    table, at = np.full((B, per), -1, np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    cap = total + int(rs.integers(1, 9))
    head = int(rs.integers(0, cap))
    free = np.full(cap, -9, np.int32)
    for k in range(spare):
        free[(head + k) % cap] = perm[at + k]
    return table, free, np.array([head, spare, -5, -5], np.int32)


def _run_plan(ctx, new, T, ratio, ring, pages, shared=None, in_place=False, **kw):
    table, free, state = pages
    t = cskv.PageTable(_i32(table), _i32(free), _i32(state))
    so = None if in_place else torch.full((4,), -3, dtype=torch.int32, device="cuda")
    m = cskv.plan_step(_i32(ctx), _i32(new), T, t, ratio=ratio, ring_rows=ring,
                       shared_pages=None if shared is None else _i32(shared), state_out=so, **kw)
    return m, t, t.state if in_place else so


def _check_plan(m, t, state, ref, ring):
    got = {"cu": m.cu_new, "len": m.new_len, "first_row": m.first_row, "n_rows": m.n_rows, "req": m.req_of, "pos1": m.pos1,
           "slot": m.slot, "table": t.block_table, "free": t.free_pages, "state": state}
    if ring:
        got["ring_slot"] = m.ring_slot
    for k, v in got.items():
        assert np.array_equal(v.cpu().numpy(), np.asarray(ref[k])), k


@pytest.mark.parametrize("ratio", [1, 2, 4, 128])
@pytest.mark.parametrize("B,most,ring", [(1, 1, 0), (1, 700, 128), (3, 5, 7), (33, 300, 128), (70, 2, 16), (1500, 9, 128),
                                         (2049, 3, 0), (5, 20000, 128)])
def test_plans_of_random_steps(ratio, B, most, ring):
    rs = np.random.default_rng(B + 7 * ratio)
    ctx = rs.integers(0, 1000, B)
    new = rs.integers(0, most + 1, B)
    new[rs.random(B) < 0.2] = 0
    ends = rs.random(B) < 0.15
    new[ends] = -rs.integers(1, 5, int(ends.sum()))
    ctx[rs.random(B) < 0.1] = 0
    total = int(np.maximum(new, 0).sum())
    for T, spare in ((total + 13, 10 ** 4), (max(total, 1), 3)):       # enough pages; too few
        per = step.pages_of((1000 + most) // ratio) + 1
        need = sum(step.pages_of((int(c) + max(int(n), 0)) // ratio) for c, n in zip(ctx, new))
        pages = _pages_case(rs, ctx, ratio, per, min(spare, need + 5))
        ref = step.plan_step(ctx, new, T, ratio, ring, *pages)
        for in_place in (False, True):
            m, t, state = _run_plan(ctx, new, T, ratio, ring, pages, in_place=in_place)
            assert cskv.device_status() == 0
            _check_plan(m, t, state, ref, ring)


def test_plan_requests_without_tokens_and_no_tokens_at_all():
    rs = np.random.default_rng(2)
    for B, T in ((5, 0), (5, 9), (3000, 4), (40, 2049)):
        ctx, new = rs.integers(0, 300, B), np.zeros(B, np.int64)
        if B == 40:
            new[17] = 1           # the only one
        pages = _pages_case(rs, ctx, 1, 8, 4)
        m, t, state = _run_plan(ctx, new, T, 1, 32, pages)
        assert cskv.device_status() == 0
        _check_plan(m, t, state, step.plan_step(ctx, new, T, 1, 32, *pages), True)


def test_plan_shared_pages_stay_with_their_owner():
    rs = np.random.default_rng(3)
    ctx, new = np.array([640, 100, 0, 640, 63]), np.array([-1, -1, -1, 5, -2])
    shared = np.array([4, 9, 3, 2, 0])
    pages = _pages_case(rs, ctx, 1, 12, 6)
    m, t, state = _run_plan(ctx, new, 8, 1, 0, pages, shared)
    assert cskv.device_status() == 0
    ref = step.plan_step(ctx, new, 8, 1, 0, *pages, shared)
    _check_plan(m, t, state, ref, False)
    assert ref["state"][1] == 6 - 1 + (10 - 4) + 0 + 0 + 1


def test_plan_without_pages():
    ctx, new = np.array([5, 0, 90]), np.array([3, -1, 200])
    m = cskv.plan_step(_i32(ctx), _i32(new), 210, ring_rows=128)
    ref = step.plan_step(ctx, new, 210, 1, 128)
    assert m.slot is None
    for got, k in ((m.cu_new, "cu"), (m.req_of, "req"), (m.pos1, "pos1"), (m.ring_slot, "ring_slot"), (m.new_len, "len")):
        assert np.array_equal(got.cpu().numpy(), np.asarray(ref[k])), k


@pytest.mark.parametrize("T", [0, 1, 90, 300, 2500])
def test_plan_cuts_tokens_that_have_no_place(T):
    rs = np.random.default_rng(4)
    ctx, new = rs.integers(0, 200, 60), rs.integers(0, 100, 60)
    assert new.sum() > 2500
    pages = _pages_case(rs, ctx, 1, 6, 400)
    m, t, state = _run_plan(ctx, new, T, 1, 16, pages)
    assert cskv.device_status() == ERR_BOUNDS
    _check_plan(m, t, state, step.plan_step(ctx, new, T, 1, 16, *pages), True)


def test_plan_reports_what_it_cannot_place():
    """A request longer than its row of the table, a negative length, a ring that would overflow,
    a state that no ring has: nothing outside is touched, the status says so."""
    ctx, new = np.array([120, 60]), np.array([30, 1])
    table = np.array([[3, 5], [6, -1]], np.int32)
    m, t, state = _run_plan(ctx, new, 40, 1, 0, (table, np.arange(10, 20), np.array([0, 10, 0, 0])))
    assert cskv.device_status() == ERR_BOUNDS
    slot = m.slot.cpu().numpy()
    assert slot[:8].tolist() == list(range(5 * 64 + 56, 6 * 64)) and (slot[8:30] == -1).all() and slot[30] == 6 * 64 + 60
    assert np.array_equal(t.block_table.cpu().numpy(), table) and state.tolist() == [0, 10, 0, 0]

    m, t, state = _run_plan(np.array([-7, 3]), np.array([2, 1]), 4, 1, 0, (np.full((2, 2), -1), np.arange(4), np.array([0, 4, 0, 0])))
    assert cskv.device_status() == ERR_BOUNDS
    assert m.new_len.tolist() == [2, 4] and m.pos1.tolist() == [1, 2, 4, 0]

    m, t, state = _run_plan(np.array([640]), np.array([-1]), 1, 1, 0, (np.arange(10)[None], np.full(12, 77), np.array([3, 5, 0, 0])))
    assert cskv.device_status() == ERR_BOUNDS
    assert state.tolist() == [3, 12, 0, 0]
    assert t.free_pages.tolist() == [4, 5, 6] + [77] * 5 + [0, 1, 2, 3]

    for bad in ([9, 4, 0, 0], [-1, 4, 0, 0], [0, 9, 0, 0], [0, -2, 0, 0]):
        m, t, state = _run_plan(np.array([0]), np.array([64 * 3]), 200, 1, 0, (np.full((1, 4), -1), np.arange(4), np.array(bad)))
        assert cskv.device_status() == ERR_BOUNDS
        assert 0 <= state[0] < 4 and 0 <= state[1] <= 4


def test_plan_lengths_in_place_and_maps_used_again():
    """new_len written over ctx_len, the state over itself: a loop of steps on the device alone."""
    rs = np.random.default_rng(6)
    B, T, per, total = 7, 64, 20, 60
    t = cskv.PageTable.allocate(B, per, total)
    maps = cskv.StepMaps(B, T, pages=True, ring=True)
    maps.new_len.zero_()
    ctx, table = np.zeros(B, np.int64), np.full((B, per), -1, np.int32)
    free, state = np.arange(total, dtype=np.int32), [0, total, 0, 0]
    for k in range(40):
        new = rs.integers(0, 18, B)
        while new.sum() > T:
            new = new // 2
        if k % 9 == 8:
            new[k % B] = -1
        cskv.plan_step(maps.new_len, _i32(new), T, t, ring_rows=128, out=maps)
        ref = step.plan_step(ctx, new, T, 1, 128, table, free, state)
        assert cskv.device_status() == 0
        _check_plan(maps, t, t.state, ref, True)
        ctx, table, free, state = np.array(ref["len"]), ref["table"], ref["free"], ref["state"]


@pytest.mark.parametrize("T", [40, 5000])
def test_plan_in_a_graph_and_on_a_stream(T):
    rs = np.random.default_rng(8)
    B = 4
    ctx, new = _i32([0] * B), _i32([0] * B)
    pages = _pages_case(rs, [0] * B, 1, 60, 200)
    t = cskv.PageTable(_i32(pages[0]), _i32(pages[1]), _i32(pages[2]))
    so = torch.zeros(4, dtype=torch.int32, device="cuda")
    maps = cskv.StepMaps(B, T, ring=True)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cskv.plan_step(ctx, new, T, t, ring_rows=128, state_out=so, out=maps, workspace=ws, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cskv.plan_step(ctx, new, T, t, ring_rows=128, state_out=so, out=maps, workspace=ws)
    for _ in range(3):
        c, n = rs.integers(0, 60, B), rs.integers(0, T // B + 1, B)
        used = [step.pages_of(int(x)) for x in c]
        table = np.full((B, 60), -1, np.int32)
        for b in range(B):
            table[b, :used[b]] = 5000 + 60 * b + np.arange(used[b])
        ctx.copy_(_i32(c))
        new.copy_(_i32(n))
        t.block_table.copy_(_i32(table))
        g.replay()
        torch.cuda.synchronize()
        _check_plan(maps, t, so, step.plan_step(c, n, T, 1, 128, table, pages[1], pages[2]), True)


def test_plan_refuses_other_shapes():
    c = _i32([1, 2])
    t = cskv.PageTable.allocate(2, 3, 5)
    ok = dict(T=4, pages=t)
    cskv.plan_step(c, c, **ok)
    for bad in (dict(T=4, pages=cskv.PageTable.allocate(3, 3, 5)), dict(T=4, out=cskv.StepMaps(2, 4)),
                dict(T=5, pages=t, out=cskv.StepMaps(2, 4)), dict(T=4, pages=t, ring_rows=8, out=cskv.StepMaps(2, 4)),
                dict(T=4, shared_pages=c), dict(T=4, state_out=torch.zeros(4, dtype=torch.int32, device="cuda")),
                dict(T=4, pages=t, shared_pages=_i32([1])), dict(T=4, pages=t, state_out=c)):
        with pytest.raises(ValueError):
            cskv.plan_step(c, c, **bad)
    with pytest.raises(ValueError):
        cskv.plan_step(c, _i32([1, 2, 3]), **ok)
    with pytest.raises(cskv.CskvError):
        cskv.plan_step(c, c, T=4, pages=t, ratio=0)
    with pytest.raises(ValueError):
        cskv.PageTable(c, c, c)


# --- rope_cs ---------------------------------------------------------------------------------

def _cs_error(got, positions, axis_of, theta=rope.THETA_COMPRESSED, yarn=None):
    """Largest error in ulps of the exact value, less what double precision loses of the angle and what
    the fraction of a turn does not hold: its two products are cut at 2^-64 turns, and the speed's
    last bit, 2^-96 turns, counts up to 2^32 times: 3 * 2^-64 turns, 1.1e-18 in radians."""
    want = step.rope_cs(positions, axis_of, theta, yarn)
    f = rope.inv_freq(theta, yarn=yarn)
    a = np.abs(np.asarray(positions, np.float64)[np.asarray(axis_of)].T * f)
    slack = (a * 2.0 ** -52)[..., None] + 1.1e-18   # the product's rounding, and an ulp of f
    d = np.maximum(np.abs(got.cpu().numpy().astype(np.float64) - want) - slack, 0)
    return np.max(d / np.spacing(np.abs(want).astype(np.float32)).astype(np.float64))


@pytest.mark.parametrize("T", [1, 15, 16, 17, 1000, 40001])
@pytest.mark.parametrize("far", [50, 1 << 20, (1 << 31) - 1])
def test_rope_of_one_axis(T, far):
    rs = np.random.default_rng(T)
    p = rs.integers(0, far, T)
    p[0], p[-1] = 0, far
    plan = cskv.RopePlan()
    got = cskv.rope_cs(_i32(p), plan)
    # sums and products of the polynomials: below an ulp
    assert _cs_error(got, p[None], [0] * 32) < 1.0
    assert torch.equal(got[0, :, 0], torch.ones(32, device="cuda")) if T > 1 else True


def test_rope_negative_positions_shifts_and_the_ends_of_32_bits():
    p = np.array([-1, -5, -(1 << 31), (1 << 31) - 1, 7, -100000], np.int64)
    plan = cskv.RopePlan()
    assert _cs_error(cskv.rope_cs(_i32(p), plan), p[None], [0] * 32) < 1.0
    for shift in (-1, 12345, (1 << 31) - 1, -(1 << 31)):
        assert _cs_error(cskv.rope_cs(_i32(p), plan, shift=shift), p[None] + shift, [0] * 32) < 1.0


@pytest.mark.parametrize("sections", [(16, 16), (16, 8, 8), (8, 8, 8, 8), (32, 0), (0, 32)])
@pytest.mark.parametrize("T", [1, 333])
def test_rope_of_several_axes(sections, T):
    rs = np.random.default_rng(T)
    p = rs.integers(-50, 5000, (len(sections), T))
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    assert _cs_error(cskv.rope_cs(_i32(p), cskv.RopePlan(sections=sections)), p, axis) < 1.0
    turn = [k % len(sections) for k in range(32)]
    if max(turn) + 1 == len(sections):
        assert _cs_error(cskv.rope_cs(_i32(p), cskv.RopePlan(axis_of=turn)), p, turn) < 1.0


@pytest.mark.parametrize("theta,yarn", [(10000.0, None), (160000.0, rope.YARN_V4), (1.5, None), (1e30, None)])
def test_rope_speeds_and_the_host_table(theta, yarn):
    rs = np.random.default_rng(9)
    p = rs.integers(0, 1 << 20, 500)
    got = cskv.rope_cs(_i32(p), cskv.RopePlan(theta, yarn=yarn))
    assert _cs_error(got, p[None], [0] * 32, theta, yarn) < 1.0
    host = cskv.rope_table(p, theta, yarn=yarn)
    # both within an ulp of the exact values (beside the host's rounding of the angle)
    far = np.abs(p[:, None] * rope.inv_freq(theta, yarn=yarn))[..., None] * 2.0 ** -52 + 1.1e-18
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - host) <= 1.5 * np.spacing(np.abs(host)) + far)


def test_rope_into_a_given_tensor_and_without_positions():
    plan = cskv.RopePlan()
    out = torch.full((5, 32, 2), 7.0, device="cuda")
    assert cskv.rope_cs(_i32([1, 2, 3, 4, 5]), plan, out=out) is out and not (out == 7.0).any()
    assert cskv.rope_cs(_i32([]), plan).shape == (0, 32, 2)
    with pytest.raises(ValueError):
        cskv.rope_cs(_i32([1, 2]), plan, out=out)
    with pytest.raises(ValueError):
        cskv.rope_cs(_i32([[1, 2], [3, 4]]), plan)
    with pytest.raises(ValueError):
        cskv.rope_cs(_i32([1, 2]).long(), plan)
    with pytest.raises(ValueError):
        cskv.rope_cs(_i32([[1, 2], [3, 4]]).t(), cskv.RopePlan(sections=(16, 16)))


# --- norm_rope -------------------------------------------------------------------------------

def _cs(rs, T):
    return cskv.rope_table(rs.integers(0, 100000, T))


def _values(rs, shape, scale=1.5):
    return bf16_values(scale * rs.standard_normal(shape))


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def _want_heads(x, norm, w, eps, cs):
    y = step.norm_rope(x, norm, w, eps, None if cs is None else np.broadcast_to(cs[:, None], x.shape[:2] + (32, 2)))
    return _bits(torch.from_numpy(y).to(torch.bfloat16))


@pytest.mark.parametrize("dim", [128, 512])
@pytest.mark.parametrize("H", [1, 3, 4, 5, 20, 64])
@pytest.mark.parametrize("T,gap", [(1, 0), (7, 8), (33, 512)])
def test_norms_of_heads(dim, H, T, gap):
    rs = np.random.default_rng(H + T)
    t, v = _values(rs, (T, H * dim + gap))
    x, v = t.cuda()[:, gap // 2 // 8 * 8:][:, :H * dim].unflatten(1, (H, dim)), v[:, gap // 2 // 8 * 8:][:, :H * dim].reshape(T, H, dim)
    cs, w = _cs(rs, T), rs.uniform(0.5, 1.5, dim).astype(np.float32)
    for norm, weight, rotate in ((True, w, True), (True, None, False), (False, None, True), (False, None, False)):
        got, = cskv.norm_rope([dict(x=x, norm=norm, norm_w=None if weight is None else cuda(weight), rotate=rotate)], cuda(cs))
        assert np.array_equal(_bits(got), _want_heads(v, norm, weight, 1e-6, cs if rotate else None)), (norm, rotate)


def test_norms_in_place_and_into_slices():
    rs = np.random.default_rng(11)
    T, H = 9, 6
    t, v = _values(rs, (T, H, 512))
    cs = _cs(rs, T)
    buf = torch.full((T, H * 512 + 136), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 8:8 + H * 512].unflatten(1, (H, 512))
    cskv.norm_rope([dict(x=t.cuda(), norm=True, rotate=True, out=out, eps=1e-3)], cuda(cs))
    want = _want_heads(v, True, None, 1e-3, cs)
    assert np.array_equal(_bits(out), want)
    assert (buf[:, :8] == 3.0).all() and (buf[:, 8 + H * 512:] == 3.0).all()
    x = t.cuda()
    r, = cskv.norm_rope([dict(x=x, norm=True, rotate=True, out=x, eps=1e-3)], cuda(cs))
    assert r is x and np.array_equal(_bits(x), want)


def test_norms_of_extreme_values():
    """Zeros, the smallest and the largest numbers, NaN and infinities stay within their heads."""
    T, H, D = 1, 8, 512
    x = torch.ones((T, H, D), dtype=torch.bfloat16)
    x[0, 0] = 0
    x[0, 1] = 1e-38
    x[0, 2] = 1e18
    x[0, 3, 7] = float("nan")
    x[0, 4, 9] = float("inf")
    x[0, 5] = 3e38            # squares overflow: 1 / inf
    with np.errstate(all="ignore"):
        want = _want_heads(x.float().numpy(), True, None, 1e-6, None)
    got, = cskv.norm_rope([dict(x=x.cuda(), norm=True)])
    g, w = got[0].float().cpu().numpy(), torch.from_numpy(want).view(torch.bfloat16)[0].float().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(w))
    assert np.array_equal(g[~np.isnan(g)], w[~np.isnan(w)])
    assert np.isfinite(g[[0, 1, 2, 5, 6, 7]]).all() and np.isnan(g[3]).all()


def _rows_of(pool, fmt, dim, slots):
    """The stored bytes of physical rows, code part and scale part."""
    p = pool.cpu().numpy()
    out = []
    for s in slots:
        page, r = p[s // 64], int(s) % 64
        if fmt == codecs.FMT_FP8_PAGESPLIT:
            out.append(np.concatenate([page[r * dim:(r + 1) * dim], page[64 * dim + 4 * r:64 * dim + 4 * r + 4]]))
        elif fmt == codecs.FMT_FP4H_PAGESPLIT:
            out.append(np.concatenate([page[r * 64:(r + 1) * 64], page[64 * 64 + 4 * r:64 * 64 + 4 * r + 4]]))
        else:
            rb = codecs.row_bytes(fmt, dim)
            out.append(page[r * rb:(r + 1) * rb])
    return np.stack(out)


def _coded(y, fmt):
    n, dim = y.shape
    if fmt in (codecs.FMT_FP8_PAGESPLIT, codecs.FMT_FP4H_PAGESPLIT):
        pad = np.zeros(((n + 63) // 64 * 64, dim), np.float32)
        pad[:n] = y
        pages = (codecs.encode_pagesplit if fmt == codecs.FMT_FP8_PAGESPLIT else codecs.encode_fp4h_pagesplit)(pad)
        return _rows_of(torch.from_numpy(pages), fmt, dim, range(n))
    return codecs.encode_rows(y, fmt)


@pytest.mark.parametrize("fmt,dim", [(codecs.FMT_BF16, 512), (codecs.FMT_FP8, 512), (codecs.FMT_FP4, 512), (codecs.FMT_BF16, 128),
                                     (codecs.FMT_FP8, 128), (codecs.FMT_FP4, 128), (codecs.FMT_FP8_PAGESPLIT, 128),
                                     (codecs.FMT_FP4H_PAGESPLIT, 128)])
@pytest.mark.parametrize("T", [1, 50])
def test_rows_into_caches(fmt, dim, T):
    rs = np.random.default_rng(T + dim + fmt)
    t, v = _values(rs, (T, 1, dim))
    cs, w = _cs(rs, T), rs.uniform(0.5, 1.5, dim).astype(np.float32)
    cache = cskv.PagedCache.allocate(3, fmt, dim)
    cache.pool.fill_(0xA5)
    before = cache.pool.clone()
    slot = rs.permutation(192)[:T]
    if T > 1:
        slot[[3, 11]] = [-1, -7]
    got = cskv.norm_rope([dict(x=t.cuda(), norm=True, norm_w=cuda(w), rotate=True, cache=cache, slot=cuda(slot.astype(np.int64)))],
                         cuda(cs))
    assert got == [None] and cskv.device_status() == 0
    y = step.norm_rope(v[:, 0], True, w, 1e-6, cs)
    there = slot >= 0
    assert np.array_equal(_rows_of(cache.pool, fmt, dim, slot[there]), _coded(y[there], fmt))
    # everything else is as it was
    rest = [s for s in range(192) if s not in set(slot[there].tolist())]
    assert np.array_equal(_rows_of(cache.pool, fmt, dim, rest), _rows_of(before, fmt, dim, rest))


def test_several_jobs_and_the_rows_of_decode_append():
    """Queries, index queries, a window row and an index key in one launch; the row is what
    decode_append's ratio-1 job writes."""
    rs = np.random.default_rng(13)
    B = 5
    q, qv = _values(rs, (B, 20, 512))
    qi, qiv = _values(rs, (B, 8, 128))
    kv, _ = _values(rs, (B, 1, 512))
    ik, ikv = _values(rs, (B, 1, 128))
    pos = np.array([0, 127, 128, 300, 77])
    cs, w = cskv.rope_table(pos), rs.uniform(0.5, 1.5, 512).astype(np.float32)
    flat = cskv.PagedCache.allocate(2 * B, cskv.FMT_FP8, 512)
    keys = cskv.PagedCache.allocate(2, cskv.FMT_FP8_PAGESPLIT, 128)
    slot = np.arange(B) * 128 + pos % 128
    a, b, c, d = cskv.norm_rope([dict(x=q.cuda(), norm=True), dict(x=qi.cuda(), rotate=True),
                                 dict(x=kv.cuda(), norm=True, norm_w=cuda(w), rotate=True, cache=flat, slot=cuda(slot)),
                                 dict(x=ik.cuda(), rotate=True, cache=keys, slot=cuda(np.arange(B) + 60))], cuda(cs))
    assert c is None and d is None and cskv.device_status() == 0
    assert np.array_equal(_bits(a), _want_heads(qv, True, None, 1e-6, None))
    assert np.array_equal(_bits(b), _want_heads(qiv, False, None, 1e-6, cs))
    assert np.array_equal(_rows_of(keys.pool, 3, 128, np.arange(B) + 60), _coded(step.norm_rope(ikv[:, 0], False, None, 0, cs), 3))
    table = _i32(np.arange(2 * B).reshape(B, 2))
    ring = cskv.PagedCache.allocate(2 * B, cskv.FMT_FP8, 512, block_table=table)
    cskv.decode_append([dict(kv=kv.cuda(), ratio=1, norm_w=cuda(w), rope_cs=cuda(cs), ring_rows=128, out=ring)], _i32(pos))
    assert torch.equal(ring.pool, flat.pool)


def test_rows_outside_the_pool_are_skipped():
    rs = np.random.default_rng(14)
    t, v = _values(rs, (4, 1, 512))
    cache = cskv.PagedCache.allocate(2, cskv.FMT_BF16, 512)
    slot = np.array([128, 5, 1 << 40, 127])
    cskv.norm_rope([dict(x=t.cuda(), cache=cache, slot=cuda(slot))])
    assert cskv.device_status() == ERR_BOUNDS
    assert np.array_equal(_rows_of(cache.pool, 0, 512, [5, 127]), codecs.encode_rows(v[[1, 3], 0], 0))
    assert int((cache.pool != 0).any(1).sum()) == 2


def test_norm_calls_that_are_refused():
    x = torch.zeros((3, 2, 512), dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros((3, 32, 2), device="cuda")
    one = x[:, :1]
    cache, slot = cskv.PagedCache.allocate(1, 0, 512), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, :, :256]), dict(x=x.transpose(0, 1)), dict(x=x, out=x[:, :1]),
                dict(x=x, norm_w=cs), dict(x=one, cache=cache), dict(x=one, cache=cache, slot=slot.int()),
                dict(x=one, cache=cache, slot=slot, out=one), dict(x=x[0])):
        with pytest.raises(ValueError):
            cskv.norm_rope([bad], cs)
    for bad in (dict(x=x, rotate=True), dict(x=x, cache=cache, slot=slot), dict(x=x[:, :, :64].contiguous()),
                dict(x=x, eps=-1.0, norm=True), dict(x=one, cache=cskv.PagedCache.allocate(1, 0, 128), slot=slot)):
        with pytest.raises(cskv.CskvError):
            cskv.norm_rope([bad])
    with pytest.raises(ValueError):
        cskv.norm_rope([dict(x=x), dict(x=x[:2])], cs)
    with pytest.raises(ValueError):
        cskv.norm_rope([dict(x=x)], cs[:2])
    odd = torch.zeros((3, 1028), dtype=torch.bfloat16, device="cuda")[:, 4:].unflatten(1, (2, 512))
    with pytest.raises(cskv.CskvError):
        cskv.norm_rope([dict(x=odd)])
    assert cskv.norm_rope([dict(x=x[:0])], cs[:0])[0].shape == (0, 2, 512)


@pytest.mark.parametrize("B,T", [(64, 256), (65, 256), (64, 257), (1, 256), (63, 1)])
def test_plans_where_one_launch_ends(B, T):
    rs = np.random.default_rng(B + T)
    ctx, new = rs.integers(0, 700, B), np.zeros(B, np.int64)
    for b in rs.integers(0, B, T - T // 9):
        new[b] += 1
    new[new == 0] = rs.choice([0, -1], int((new == 0).sum()))
    pages = _pages_case(rs, ctx, 1, step.pages_of(int(ctx.max() + new.max())) + 1, 9)
    m, t, state = _run_plan(ctx, new, T, 1, 128, pages)
    assert cskv.device_status() == 0
    _check_plan(m, t, state, step.plan_step(ctx, new, T, 1, 128, *pages), True)


def test_norms_of_few_and_of_many_tokens_have_the_same_bits():
    rs = np.random.default_rng(31)
    T, H = 90, 61
    t, v = _values(rs, (T, H, 512))
    small, sv = _values(rs, (T, 7, 128))
    cs, w = _cs(rs, T), rs.uniform(0.5, 1.5, 512).astype(np.float32)
    x, y, c = t.cuda(), small.cuda(), cuda(cs)
    whole = None
    for n in (T, 80, 79, 78, 77, 5, 1):
        got = cskv.norm_rope([dict(x=x[:n], norm_w=cuda(w), rotate=True), dict(x=y[:n], norm=True, rotate=True)], c[:n])
        if whole is None:
            whole = got
            assert np.array_equal(_bits(got[0]), _want_heads(v, True, w, 1e-6, cs))
            assert np.array_equal(_bits(got[1]), _want_heads(sv, True, None, 1e-6, cs))
        assert all(torch.equal(a, b[:n]) for a, b in zip(got, whole)), n
