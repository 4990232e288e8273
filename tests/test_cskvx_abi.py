"""include/cskvx.h: binding, exports, refusals before any launch, and the oracle of eviction
against its definition (CPU only)."""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import bounded

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_kv_gb300 import build, _lib
    build.build()
    return _lib.lib()


def _declared():
    with open(os.path.join(ROOT, "include", "cskvx.h")) as f:
        return sorted(set(re.findall(r"CSKV_API\s+[\w\s\*]+?\b(cskvx_\w+)\s*\(", f.read())))


def test_header_binding_and_exports_agree(lib):
    from compressed_sparse_attention_kv_gb300 import _lib
    assert sorted(_lib.EXT_SIGNATURES) == _declared()
    out = os.popen("nm -D --defined-only %s" % _lib.LIB_PATH).read()
    assert set(re.findall(r"\bT (cskvx_\w+)", out)) == set(_declared())


def _paged(fmt=1, dim=512, pool=FAKE, row=528, pages=4, table=FAKE, per=4):
    from compressed_sparse_attention_kv_gb300._lib import Paged
    return Paged(pool, table, 64 * row, pages, per, fmt, dim)


WINDOW = dict(q=FAKE, rows=_paged, num_reqs=2, req_of=FAKE, pos1=FAKE, window=8, first=2, max_ctx=256, sink=None,
              scale=0.04, cs=FAKE, T=2, H=16, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, stream=None)
PREFIX = dict(q=FAKE, main=_paged, n=FAKE, n_prefix=10, max_entries=200, swa=FAKE, swa_fmt=1, ctx=FAKE, sink=None,
              scale=0.04, cs=FAKE, B=2, H=16, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, stream=None)
WEIGHTS = dict(q=FAKE, main=_paged, n=FAKE, first=0, max_entries=200, scale=0.04, cs=FAKE, lse=FAKE, B=2, H=16,
               decay=1.0, acc=FAKE, acc_stride=200, acc_out=FAKE, acc_out_stride=200, stream=None)
EVICT = dict(caches=None, ncaches=1, acc=FAKE, acc_stride=200, age=FAKE, age_stride=200, n=FAKE, B=2, max_entries=200,
             budget=100, fixed=4, recent=8, src=FAKE, acc_out=FAKE, acc_out_stride=200, age_out=FAKE,
             age_out_stride=200, n_out=FAKE, ws=FAKE, ws_bytes=1 << 40, stream=None)

INF, NAN = float("inf"), float("nan")
BAD = [
    ("window", {"q": None}), ("window", {"q": FAKE + 8}), ("window", {"pos1": None}), ("window", {"out": None}),
    ("window", {"out": FAKE + 2}), ("window", {"cs": None}), ("window", {"cs": FAKE + 4}), ("window", {"T": 0}),
    ("window", {"H": 0}), ("window", {"H": 129}), ("window", {"window": 0}), ("window", {"first": -1}),
    ("window", {"max_ctx": -1}), ("window", {"max_ctx": (1 << 30) + 1}), ("window", {"num_reqs": 0}),
    ("window", {"req_of": None, "num_reqs": 1}), ("window", {"scale": 0.0}), ("window", {"scale": -1.0}),
    ("window", {"scale": NAN}), ("window", {"scale": INF}), ("window", {"rows": lambda: _paged(fmt=3, dim=128)}),
    ("window", {"rows": lambda: _paged(dim=128)}), ("window", {"rows": lambda: _paged(pool=None)}),
    ("window", {"rows": lambda: _paged(pool=FAKE + 8)}), ("window", {"rows": lambda: _paged(pages=0)}),
    ("window", {"rows": lambda: _paged(row=512)}), ("window", {"rows": lambda: _paged(per=0)}),
    ("window", {"rows": lambda: _paged(fmt=5)}),
    ("prefix", {"q": None}), ("prefix", {"n": None}), ("prefix", {"out": None}), ("prefix", {"n_prefix": -1}),
    ("prefix", {"n_prefix": 201}), ("prefix", {"max_entries": (1 << 30) + 1}), ("prefix", {"swa": FAKE + 8}),
    ("prefix", {"swa_fmt": 2}), ("prefix", {"ctx": None}), ("prefix", {"B": 0}), ("prefix", {"H": 200}),
    ("prefix", {"scale": NAN}), ("prefix", {"main": lambda: _paged(fmt=4, dim=128)}),
    ("weights", {"q": None}), ("weights", {"n": None}), ("weights", {"lse": None}), ("weights", {"acc": None}),
    ("weights", {"acc_out": None}), ("weights", {"decay": NAN}), ("weights", {"decay": INF}),
    ("weights", {"first": -1}), ("weights", {"max_entries": -1}), ("weights", {"acc_stride": 199}),
    ("weights", {"acc_out_stride": 199}), ("weights", {"acc_out_stride": 201}), ("weights", {"B": 65536}),
    ("evict", {"ncaches": 0}), ("evict", {"ncaches": 5}), ("evict", {"acc": None}), ("evict", {"n": None}),
    ("evict", {"src": None}), ("evict", {"acc_out": None}), ("evict", {"n_out": None}), ("evict", {"budget": 0}),
    ("evict", {"fixed": -1}), ("evict", {"recent": -1}), ("evict", {"fixed": 60, "recent": 41}),
    ("evict", {"age": None}), ("evict", {"age_out": None}), ("evict", {"age": None, "age_out": None}),
    ("evict", {"acc_stride": 199}), ("evict", {"age_stride": 199}),
    ("evict", {"acc_out": 2 * FAKE, "acc_out_stride": 99}), ("evict", {"age_out": 2 * FAKE, "age_out_stride": 99}),
    ("evict", {"acc_out_stride": 300}), ("evict", {"age_out_stride": 300}), ("evict", {"B": 0}),
    ("evict", {"max_entries": -1}), ("evict", {"ws": None}), ("evict", {"ws": FAKE + 16}), ("evict", {"ws_bytes": 16}),
]


@pytest.mark.parametrize("what,change", BAD)
def test_bad_arguments_are_refused_before_any_launch(lib, what, change):
    from compressed_sparse_attention_kv_gb300._lib import Paged
    base, fn = {"window": (WINDOW, lib.cskvx_window_attn), "prefix": (PREFIX, lib.cskvx_prefix_decode_attn),
                "weights": (WEIGHTS, lib.cskvx_attn_weights), "evict": (EVICT, lib.cskvx_evict)}[what]
    a = dict(base, **change)
    if what == "evict":
        a["caches"] = (Paged * 5)(*[_paged() for _ in range(5)])
    assert fn(*[v() if callable(v) else v for v in a.values()]) == 1


def test_bad_caches_of_an_eviction_are_refused(lib):
    from compressed_sparse_attention_kv_gb300._lib import Paged
    for bad in (_paged(pool=None), _paged(fmt=7), _paged(fmt=3, dim=512, row=516), _paged(row=400)):
        arr = (Paged * 2)(_paged(), bad)
        assert lib.cskvx_evict(*list(dict(EVICT, caches=arr, ncaches=2).values())) == 1
    assert lib.cskvx_evict(*list(dict(EVICT, caches=None).values())) == 1


def test_small_workspaces_are_refused(lib):
    w = lib.cskvx_window_attn_workspace_size(1, 16, 100000, 50000, 4)
    if w:
        a = dict(WINDOW, T=1, max_ctx=100000, window=50000, first=4, ws_bytes=w - 1)
        assert lib.cskvx_window_attn(*[v() if callable(v) else v for v in a.values()]) == 1
    w = lib.cskvx_prefix_decode_attn_workspace_size(2, 16, 10, 200, 1)
    if w:
        a = dict(PREFIX, ws_bytes=w - 1)
        assert lib.cskvx_prefix_decode_attn(*[v() if callable(v) else v for v in a.values()]) == 1
    assert lib.cskvx_window_attn_workspace_size(0, 16, 100, 10, 4) == 0
    assert lib.cskvx_prefix_decode_attn_workspace_size(2, 16, 300, 200, 1) == 0
    assert lib.cskvx_evict_workspace_size(0, 100, 10) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    q = torch.zeros((2, 4, 512), dtype=torch.bfloat16)
    i = torch.ones(2, dtype=torch.int32)
    cs = torch.zeros((2, 32, 2))
    acc = torch.zeros((2, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.window_attn(q, None, i, 8, 0, 16, None, 0.04, cs)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.prefix_decode_attn(q, None, i, 0, 8, None, 0.04, cs)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.attn_weights(q, None, i, 8, 0.04, cs, acc, acc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.evict([], acc, i, 4)


# --- the oracle of eviction against the definition, entry by entry -----------------------

@pytest.mark.parametrize("seed", range(40))
def test_oracle_evict_follows_the_definition(seed):
    r = np.random.default_rng(seed)
    n = int(r.integers(1, 60))
    budget = int(r.integers(1, 60))
    fixed = int(r.integers(0, budget + 1))
    recent = int(r.integers(0, budget - fixed + 1))
    acc = r.choice([0.0, -0.0, 0.5, 1.0, np.nan, np.inf, -1.0, 2.0], size=n)
    age = r.permutation(n)
    src, m = bounded.evict(acc, age, n, budget, fixed, recent)
    assert m == min(n, budget) and np.all(src[m:] == -1)
    kept = src[:m]
    assert len(set(kept.tolist())) == m and (m == 0 or (kept.min() >= 0 and kept.max() < n))
    moved = kept != np.arange(m)
    assert np.all(kept[moved] >= m) and np.all(np.diff(kept[moved]) > 0)
    if n <= budget:
        return
    gone = sorted(set(range(n)) - set(kept.tolist()))
    safe = {i for i in range(n) if i < fixed or age[i] > age.max() - recent}
    assert safe <= set(kept.tolist())
    value = lambda i: -np.inf if np.isnan(acc[i]) else acc[i]
    for g in gone:
        for k in kept:
            if k in safe:
                continue
            assert np.isnan(acc[g]) and not np.isnan(acc[k]) or value(k) > value(g) or (
                value(k) == value(g) and np.isnan(acc[k]) == np.isnan(acc[g]) and k < g)


@pytest.mark.parametrize("what, change", [
    ("window", {"T": (1 << 23) + 1, "num_reqs": 1 << 24}), ("prefix", {"B": (1 << 23) + 1}),
    ("weights", {"B": 65536}), ("evict", {"B": 65536}), ("evict", {"max_entries": (1 << 30) + 1}),
    ("evict", {"budget": (1 << 30) + 1}), ("weights", {"max_entries": (1 << 30) + 1}),
])
def test_sizes_beyond_the_limits_are_refused(lib, what, change):
    test_bad_arguments_are_refused_before_any_launch(lib, what, change)


@pytest.mark.parametrize("seed", range(6))
def test_workspaces_of_any_size_are_finite(lib, seed):
    """A list is cut into 4 x 152 shares at most, a row sees a prefix, its own list and a ring: up to
    2 x 608 + 1 parts of 2 KB and 8 bytes a row."""
    rng = np.random.default_rng(900 + seed)
    for _ in range(500):
        T, H = int(2 ** rng.uniform(0, 14)), int(rng.integers(1, 129))
        ctx, window, first = (int(2 ** rng.uniform(0, 30)) for _ in range(3))
        w = lib.cskvx_window_attn_workspace_size(T, H, ctx, window, first)
        p = lib.cskvx_prefix_decode_attn_workspace_size(T, H, min(window, ctx), ctx, int(rng.integers(0, 2)))
        for need in (w, p):
            assert need % 256 == 0 and need <= T * H * (2 * 608 + 1) * (2048 + 8) + 512
