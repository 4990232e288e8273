"""include/cskvx.h through the binding and the C ABI without a GPU: what the calls take and refuse."""

import pytest

from test_cskvx_abi import EVICT, PREFIX, WEIGHTS, WINDOW, _paged, lib  # noqa: F401 (lib is a fixture)


def _values(a):
    return [v() if callable(v) else v for v in a.values()]


@pytest.mark.parametrize("scale", [1.0001e38, 3e38])
def test_scales_beyond_fp32_in_base_2_are_refused(lib, scale):  # noqa: F811
    assert lib.cskvx_window_attn(*_values(dict(WINDOW, scale=scale))) == 1
    assert lib.cskvx_prefix_decode_attn(*_values(dict(PREFIX, scale=scale))) == 1
    assert lib.cskvx_attn_weights(*_values(dict(WEIGHTS, scale=scale))) == 1


def test_one_flat_cache_of_several_requests_is_not_cut(lib):  # noqa: F811
    """Without a table all requests have the same rows: what one moves the others would overwrite."""
    from compressed_sparse_attention_kv_gb300._lib import Paged
    flat = _paged(table=None, per=0)
    for arr in ((Paged * 1)(flat), (Paged * 2)(_paged(), flat)):
        assert lib.cskvx_evict(*_values(dict(EVICT, caches=arr, ncaches=len(arr)))) == 1
