"""include/cskvx.h through the binding and the C ABI without a GPU: what the calls take and refuse."""

import pytest

from test_cskvx_abi import PREFIX, WEIGHTS, WINDOW, lib  # noqa: F401 (lib is a fixture)


def _values(a):
    return [v() if callable(v) else v for v in a.values()]


@pytest.mark.parametrize("scale", [1.0001e38, 3e38])
def test_scales_beyond_fp32_in_base_2_are_refused(lib, scale):  # noqa: F811
    assert lib.cskvx_window_attn(*_values(dict(WINDOW, scale=scale))) == 1
    assert lib.cskvx_prefix_decode_attn(*_values(dict(PREFIX, scale=scale))) == 1
    assert lib.cskvx_attn_weights(*_values(dict(WEIGHTS, scale=scale))) == 1
