"""Pools that run out: plan_step keeps every page once, with a request or in the ring, and none in the
ring that is not there, however often requests with missing pages end (oracle on the CPU, kernels
on the GPU)."""

import numpy as np
import pytest

from oracle import step


def _oracle_step(new, s):
    r = step.plan_step(s["ctx"], new, int(np.maximum(new, 0).sum()), s["ratio"], 0, s["table"], s["free"], s["state"], s.get("shared"))
    return dict(s, ctx=np.array(r["len"]), table=r["table"], free=r["free"], state=r["state"]), r


def _start(B, per, total, capacity, ratio=1, head=0):
    free = np.full(capacity, -9)
    free[(head + np.arange(total)) % capacity] = np.arange(total)
    return dict(ctx=np.zeros(B, np.int64), table=np.full((B, per), -1), free=free, state=[head, total, 0, 0], ratio=ratio)


def _owned(s):
    pages = [step.pages_of(int(c) // s["ratio"]) for c in s["ctx"]]
    return [int(p) for b, n in enumerate(pages) for p in s["table"][b, :n] if p >= 0]


def _ring(s):
    return [int(s["free"][(s["state"][0] + k) % len(s["free"])]) for k in range(s["state"][1])]


def _random_new(rs, s, most):
    B, room = len(s["ctx"]), s["table"].shape[1] * 64 * s["ratio"] - s["ctx"]
    new = np.minimum(rs.integers(0, most, B), room)
    new[rs.random(B) < 0.3] = 0
    return np.where(rs.random(B) < 0.12, -1, new)


# a pool of 4 pages: (n_new, ring's count after it, pages that were missing)
OUT_OF_PAGES = [([192, 0], 1, 0), ([0, 256], 0, 3), ([0, -1], 1, 0), ([-1, 0], 4, 0), ([0, 320], 0, 1), ([0, -1], 4, 0)]


@pytest.mark.parametrize("capacity", [4, 8])
def test_the_oracle_gives_back_only_pages_that_are_there(capacity):
    s = _start(2, 6, 4, capacity)
    for new, count, short in OUT_OF_PAGES:
        s, r = _oracle_step(np.array(new), s)
        assert s["state"][1:3] == [count, short]
        assert sorted(_owned(s) + _ring(s)) == list(range(4))


@pytest.mark.parametrize("spare", [0, 11])
@pytest.mark.parametrize("B,per,total,most,ratio", [(5, 12, 20, 120, 1), (9, 4, 13, 900, 4), (40, 6, 70, 200, 1)])
def test_the_oracle_keeps_every_page_when_pages_run_out(B, per, total, most, ratio, spare):
    rs = np.random.default_rng(B + spare)
    s, short = _start(B, per, total, total + spare, ratio, head=3), 0
    for _ in range(200):
        s, r = _oracle_step(_random_new(rs, s, most), s)
        short += s["state"][2]
        assert sorted(_owned(s) + _ring(s)) == list(range(total))
    assert short > 20


def _device(s):
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    return cskv, i32, cskv.PageTable(i32(s["table"]), i32(s["free"]), i32(s["state"]))


def _kernel_step(cskv, i32, pages, s, new, T, **kw):
    """One step on the GPU against the oracle's, from the same state; returns the state after it."""
    m = cskv.plan_step(i32(s["ctx"]), i32(new), T, pages, ratio=s["ratio"], **kw)
    after, r = _oracle_step(new, s)
    assert cskv.device_status() == 0
    n = r["cu"][-1]
    for got, want in ((m.new_len, r["len"]), (m.cu_new, r["cu"]), (m.slot[:n], r["slot"]), (pages.block_table, r["table"]),
                      (pages.free_pages, r["free"]), (pages.state, r["state"])):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want))
    return after


@pytest.mark.gpu
@pytest.mark.parametrize("capacity", [4, 8])
@pytest.mark.parametrize("T", [256, 400])
def test_only_pages_that_are_there_come_back(capacity, T):
    s = _start(2, 6, 4, capacity)
    cskv, i32, pages = _device(s)
    for new, count, short in OUT_OF_PAGES[:4 if T == 256 else None]:   # (320 tokens need the places)
        s = _kernel_step(cskv, i32, pages, s, np.array(new), T)
        assert pages.state.tolist()[1:3] == [count, short]
        assert sorted(_owned(s) + _ring(s)) == list(range(4))


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [0, 11])
@pytest.mark.parametrize("B,per,total,most,ratio,steps", [(5, 12, 20, 50, 1, 150), (9, 4, 13, 900, 4, 60), (40, 6, 70, 200, 1, 60),
                                                          (1500, 3, 1600, 120, 1, 12)])
def test_every_page_is_kept_when_pages_run_out(B, per, total, most, ratio, steps, spare):
    """One launch and two, and more requests than a block has threads."""
    rs = np.random.default_rng(B + spare)
    s, short = _start(B, per, total, total + spare, ratio, head=3), 0
    cskv, i32, pages = _device(s)
    for _ in range(steps):
        new = _random_new(rs, s, most)
        s = _kernel_step(cskv, i32, pages, s, new, max(1, int(np.maximum(new, 0).sum())))
        short += s["state"][2]
        assert sorted(_owned(s) + _ring(s)) == list(range(total))
    assert short > 0   # (the case is of this kind)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 31, 32, 33, 255, 256, 257, 8191, 8193, 9000])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
def test_long_rows_with_holes_come_back_in_order(n, share):
    """Rows of up to more places than a block's warps read at once, some of whose pages are missing; one request
    gives back a part of its row, one goes on."""
    rs = np.random.default_rng(n)
    B, per = 3, n + 2
    table = rs.permutation(B * per).reshape(B, per)
    holes = rs.random((B, per)) < share
    holes[1] = False
    table[holes] = -1 - rs.integers(0, 5, int(holes.sum()))
    table[:, n:] = -1
    shared = np.array([0, 0, n // 3])
    s = dict(ctx=np.full(B, 64 * n - 1), table=table, free=np.full(B * per + 5, -9), state=[B * per, 0, 0, 0], ratio=1,
             shared=shared)
    cskv, i32, pages = _device(s)
    after = _kernel_step(cskv, i32, pages, s, np.array([-1, 1, -3]), 8, shared_pages=i32(shared))
    there = [int(p) for b, a in ((0, 0), (2, n // 3)) for p in table[b, a:n] if p >= 0]
    assert _ring(after) == there
