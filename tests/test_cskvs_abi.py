"""include/cskvs.h: binding, exports, refusals before any launch, and the host part of the
rotation plan (CPU only)."""

import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from oracle import rope

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_kv_gb300 import build, _lib
    build.build()
    return _lib.lib()


def test_header_binding_and_exports_agree(lib):
    from compressed_sparse_attention_kv_gb300 import _lib
    with open(os.path.join(ROOT, "include", "cskvs.h")) as f:
        declared = set(re.findall(r"CSKV_API\s+[\w\s\*]+?\b(cskvs_\w+)\s*\(", f.read()))
    assert set(_lib.STEP_SIGNATURES) == declared
    out = os.popen("nm -D --defined-only %s" % _lib.LIB_PATH).read()
    assert set(re.findall(r"\bT (cskvs_\w+)", out)) == declared


def _paged(fmt=1, dim=512, pool=FAKE, row=528, pages=4, table=FAKE, per=4):
    from compressed_sparse_attention_kv_gb300._lib import Paged
    return Paged(pool, table, 64 * row, pages, per, fmt, dim)


PLAN = dict(ctx=FAKE, new=FAKE, B=3, ratio=4, T=10, ring_rows=128, table=FAKE, max_pages=5, shared=None, free=FAKE,
            capacity=20, state=FAKE, state_out=FAKE, cu=FAKE, len=FAKE, first=FAKE, rows=FAKE, req=FAKE, pos1=FAKE,
            slot=FAKE, ring=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
CHUNK = dict(q=FAKE, cu=FAKE, ctx=FAKE, R=2, T=4, H=16, entries=_paged, ratio=4, n=None, max_entries=100, rows=_paged,
             window=128, max_ctx=400, sink=None, scale=0.04, cs=FAKE, out=FAKE, lse=None, max_keys=1000, ws=FAKE,
             ws_bytes=1 << 40, stream=None)

BAD_PLAN = [{"ctx": None}, {"new": None}, {"B": 0}, {"B": 65536}, {"ratio": 0}, {"ratio": (1 << 20) + 1}, {"T": -1},
            {"T": (1 << 27) + 1}, {"ring_rows": -1}, {"ring_rows": 0}, {"ring": None}, {"max_pages": 0}, {"free": None},
            {"capacity": 0}, {"state": None}, {"state_out": None}, {"cu": None}, {"len": None}, {"first": None},
            {"rows": None}, {"req": None}, {"pos1": None}, {"slot": None}, {"ws": None}, {"ws": FAKE + 16},
            {"ws_bytes": 100}, {"table": None}, {"ring_rows": (1 << 20) + 1}]
BAD_CHUNK = [{"q": None}, {"q": FAKE + 8}, {"cu": None}, {"ctx": None}, {"R": 0}, {"R": 65536}, {"T": 0},
             {"T": (1 << 23) + 1}, {"H": 0}, {"H": 129}, {"entries": None, "rows": None, "window": 0},
             {"entries": lambda: _paged(dim=128)}, {"entries": lambda: _paged(fmt=3, dim=128)},
             {"entries": lambda: _paged(fmt=4, dim=128)}, {"rows": lambda: _paged(pool=None)},
             {"rows": lambda: _paged(pages=0)}, {"rows": lambda: _paged(row=500)}, {"rows": lambda: _paged(per=0)},
             {"rows": None}, {"ratio": -1}, {"ratio": 0}, {"ratio": (1 << 20) + 1}, {"max_entries": -1},
             {"max_entries": (1 << 30) + 1}, {"window": 0}, {"window": -5}, {"max_ctx": -1}, {"max_ctx": (1 << 30) + 1},
             {"scale": 0.0}, {"scale": NAN}, {"scale": INF}, {"scale": 2e38}, {"cs": None}, {"cs": FAKE + 4},
             {"out": None}, {"out": FAKE + 2}, {"max_keys": -1}, {"max_keys": (1 << 40) + 1}]
BAD_PLAN += [{k: FAKE + 2} for k in ("ctx", "new", "table", "shared", "free", "state", "state_out", "cu", "len", "first", "rows",
                                     "req", "pos1")] + [{"slot": FAKE + 4}, {"ring": FAKE + 4}]
BAD_CHUNK += [{k: FAKE + 2} for k in ("cu", "ctx", "n", "sink", "lse")]


@pytest.mark.parametrize("change", BAD_PLAN)
def test_bad_plans_are_refused_before_any_launch(lib, change):
    assert lib.cskvs_plan_step(*dict(PLAN, **change).values()) == 1


@pytest.mark.parametrize("change", BAD_CHUNK)
def test_bad_chunks_are_refused_before_any_launch(lib, change):
    a = dict(CHUNK, **change)
    for k in ("entries", "rows"):
        if a[k] is not None:
            a[k] = ctypes.byref(a[k]())
    assert lib.cskvs_chunk_attn(*a.values()) == 1


def test_small_workspaces_are_refused(lib):
    assert lib.cskvs_plan_step_workspace_size(0) == 0
    w = lib.cskvs_plan_step_workspace_size(3)
    assert lib.cskvs_plan_step(*dict(PLAN, ws_bytes=w - 1).values()) == 1
    assert lib.cskvs_chunk_attn_workspace_size(2, 4, 0, 100) == 0
    assert lib.cskvs_chunk_attn_workspace_size(2, 4, 16, -1) == 0
    w = lib.cskvs_chunk_attn_workspace_size(2, 4, 16, 1000)
    if w:
        a = dict(CHUNK, ws_bytes=w - 1)
        a["entries"], a["rows"] = ctypes.byref(_paged()), ctypes.byref(_paged())
        assert lib.cskvs_chunk_attn(*a.values()) == 1


def test_the_bound_of_a_chunks_keys_holds(lib):
    rs = np.random.default_rng(0)
    for _ in range(300):
        R, window, ratio = int(rs.integers(1, 9)), int(rs.integers(0, 300)), int(rs.choice([1, 4, 128]))
        new = rs.integers(0, 60, R)
        ctx = new + rs.integers(0, 500, R)
        T = max(1, int(new.sum()) + int(rs.integers(0, 5)))
        up = lambda n: (n + 15) // 16 * 16
        keys = sum(up(c // ratio) + (up(min(c, n + window - 1)) if window else 0) for c, n in zip(ctx, new) if n)
        bound = lib.cskvs_chunk_attn_max_keys(R, T, int(max(ctx)) // ratio, window, int(max(ctx)))
        assert keys <= bound <= 16 * R + R * (up(int(max(ctx)) // ratio)) + (T + R * (window + 16) if window else 0)
    assert lib.cskvs_chunk_attn_max_keys(0, 1, 1, 1, 1) == lib.cskvs_chunk_attn_max_keys(1, 1, -1, 1, 1) == 0


def _norm_job(**change):
    from compressed_sparse_attention_kv_gb300._lib import NormJob
    j = NormJob(FAKE, 1024, 2, 512, 1, FAKE, 1e-6, 1, FAKE, 1024, _paged(), None)
    for k, v in change.items():
        setattr(j, k, v)
    return j


BAD_NORM = [dict(x=None), dict(x=FAKE + 8), dict(x_stride=1016), dict(x_stride=1028), dict(H=0), dict(H=1025), dict(dim=256),
            dict(dim=64), dict(norm_w=FAKE + 4), dict(norm=0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(out=None),
            dict(out=FAKE + 2), dict(out_stride=1016), dict(out_stride=1028), dict(out_stride=2048),
            dict(slot=FAKE), dict(slot=FAKE, H=1), dict(slot=FAKE + 4, H=1, out=None),
            dict(slot=FAKE, H=1, out=None, dim=128), dict(slot=FAKE, H=1, out=None, cache=lambda: _paged(pages=0)),
            dict(slot=FAKE, H=1, out=None, cache=lambda: _paged(fmt=3, row=516)),
            dict(slot=FAKE, H=1, out=None, cache=lambda: _paged(row=512))]


@pytest.mark.parametrize("change", BAD_NORM)
def test_bad_norm_jobs_are_refused_before_any_launch(lib, change):
    from compressed_sparse_attention_kv_gb300._lib import NormJob
    change = {k: v() if callable(v) else v for k, v in change.items()}
    jobs = (NormJob * 2)(_norm_job(), _norm_job(**change))
    assert lib.cskvs_norm_rope(jobs, 2, FAKE, 7, None) == 1


def test_bad_norm_calls_are_refused(lib):
    from compressed_sparse_attention_kv_gb300._lib import NormJob
    five = (NormJob * 5)(*[_norm_job() for _ in range(5)])
    assert lib.cskvs_norm_rope(five, 5, FAKE, 7, None) == 1
    assert lib.cskvs_norm_rope(five, 0, FAKE, 7, None) == 1
    assert lib.cskvs_norm_rope(None, 1, FAKE, 7, None) == 1
    assert lib.cskvs_norm_rope(five, 1, None, 7, None) == 1          # rotation without a table
    assert lib.cskvs_norm_rope(five, 1, FAKE + 4, 7, None) == 1
    assert lib.cskvs_norm_rope(five, 1, FAKE, -1, None) == 1
    assert lib.cskvs_norm_rope(five, 1, FAKE, (1 << 27) + 1, None) == 1
    assert lib.cskvs_norm_rope(five, 1, FAKE, 0, None) == 0          # no tokens: nothing to do


def _inv_two_pi(bits):
    """floor(2^bits / 2 pi), pi by Machin's formula in integers."""
    one = 1 << (bits + 64)

    def arctan(x):
        t = total = one // x
        n, sign = 3, -1
        while t:
            t //= x * x
            total += sign * (t // n)
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan(5) - arctan(239))
    return (one * one // (2 * pi)) >> 64


@pytest.mark.parametrize("theta,yarn", [(160000.0, None), (10000.0, None), (1.0001, None), (1e30, None), (1e300, None),
                                        (160000.0, rope.YARN_V4)])
def test_speeds_of_a_rotation_plan(theta, yarn):
    """Each speed is the double f_k over 2 pi, to 96 bits below the point."""
    import compressed_sparse_attention_kv_gb300 as cskv
    plan = cskv.RopePlan(theta, yarn=yarn)
    inv = Fraction(_inv_two_pi(300), 1 << 300)
    for k, f in enumerate(rope.inv_freq(theta, yarn=yarn)):
        w = plan.struct.speed[k]
        got = Fraction((w[0] << 64) | (w[1] << 32) | w[2], 1 << 96)
        want = Fraction(float(f)) * inv
        # the constant is cut at 2^-128, the product at 2^-96; pow of numpy and of C: an ulp of f each
        assert abs(got - want) <= Fraction(2, 1 << 96) + want * Fraction(8, 1 << 53)


def test_rotation_plans_of_several_axes(lib):
    import compressed_sparse_attention_kv_gb300 as cskv
    p = cskv.RopePlan(sections=(16, 8, 8))
    assert p.axes == 3 and list(p.struct.axis) == [0] * 16 + [1] * 8 + [2] * 8
    p = cskv.RopePlan(axis_of=[k % 4 for k in range(32)])
    assert p.axes == 4 and list(p.struct.axis) == [k % 4 for k in range(32)]
    assert cskv.RopePlan().axes == 1
    for bad in (dict(sections=(16, 8)), dict(sections=(40, -8)), dict(sections=(8, 8, 8, 4, 4)), dict(axis_of=[0] * 31),
                dict(axis_of=[4] * 32), dict(axis_of=[-1] * 32), dict(sections=(32,), axis_of=[0] * 32)):
        with pytest.raises(ValueError):
            cskv.RopePlan(**bad)
    for bad in (dict(theta=1.0), dict(theta=NAN), dict(theta=0.5), dict(yarn=dict(factor=2.0, original=0.0, beta_fast=32.0, beta_slow=1.0))):
        with pytest.raises(cskv.CskvError):
            cskv.RopePlan(**bad)
    plan = p.struct
    assert lib.cskvs_rope_cs(None, FAKE, 8, 0, 8, FAKE, None) == 1
    assert lib.cskvs_rope_cs(ctypes.byref(plan), None, 8, 0, 8, FAKE, None) == 1
    assert lib.cskvs_rope_cs(ctypes.byref(plan), FAKE + 2, 8, 0, 8, FAKE, None) == 1
    assert lib.cskvs_rope_cs(ctypes.byref(plan), FAKE, 7, 0, 8, FAKE, None) == 1       # axes overlap
    assert lib.cskvs_rope_cs(ctypes.byref(plan), FAKE, 8, 0, 8, FAKE + 8, None) == 1
    assert lib.cskvs_rope_cs(ctypes.byref(plan), FAKE, 8, 0, -1, FAKE, None) == 1
    plan.axis[5] = 7
    assert lib.cskvs_rope_cs(ctypes.byref(plan), FAKE, 8, 0, 8, FAKE, None) == 1
    assert lib.cskvs_rope_init(None, 1e4, 1.0, 1.0, 1.0, 1.0, 1, None) == 1
    assert lib.cskvs_rope_init(ctypes.byref(plan), 1e4, 1.0, 1.0, 1.0, 1.0, 5, None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    i = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cskv.plan_step(i, i, 4)
    with pytest.raises(ValueError, match="CUDA"):
        cskv.rope_cs(i, cskv.RopePlan())
    with pytest.raises(ValueError, match="shape"):
        cskv.rope_cs(i, cskv.RopePlan(sections=(16, 16)))
    with pytest.raises(ValueError, match="CUDA"):
        cskv.norm_rope([dict(x=torch.zeros((2, 1, 512), dtype=torch.bfloat16))])
    with pytest.raises(ValueError, match="1 to 4"):
        cskv.norm_rope([])
    with pytest.raises(ValueError, match="CUDA"):
        cskv.chunk_attn(torch.zeros((2, 4, 512), dtype=torch.bfloat16), i, i, None, 1, 1, 1, None, 1.0, i)


def test_the_oracle_of_a_step_gives_pages_once():
    """Random steps: no page is with two requests, free or owned twice, and none is lost."""
    from oracle import step
    rs = np.random.default_rng(1)
    B, per, total = 5, 12, 30
    table = np.full((B, per), -1)
    free, state = np.arange(total)[rs.permutation(total)], [7, total, 0, 0]
    ctx = np.zeros(B, np.int64)
    for _ in range(200):
        new = np.where(rs.random(B) < 0.1, -1, np.minimum(rs.integers(0, 90, B), per * 64 - ctx))
        r = step.plan_step(ctx, new, 10 ** 6, 1, 0, table, free, state)
        table, free, state, ctx = r["table"], r["free"], r["state"], np.array(r["len"])
        owned = [int(p) for b in range(B) for p in table[b, :step.pages_of(int(ctx[b]))]]
        ring = [int(free[(state[0] + k) % total]) for k in range(state[1])]
        if state[2]:        # a page was missing: start again
            table[:], ctx[:] = -1, 0
            free, state = np.arange(total), [0, total, 0, 0]
            continue
        assert sorted(owned + ring) == list(range(total))
