"""include/cskvx.h through the binding and the C ABI without a GPU: what the calls take and refuse."""

import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
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


class _Subclass(torch.Tensor):
    pass


@pytest.mark.parametrize("wrap", [lambda t: torch.nn.Parameter(t, requires_grad=False),
                                  lambda t: t.as_subclass(_Subclass)])
def test_parameters_and_tensor_subclasses_are_tensors(lib, wrap):  # noqa: F811
    """They reach the argument checks (host tensors here), as they do in the other calls."""
    q = wrap(torch.zeros((2, 4, 512), dtype=torch.bfloat16))
    i, cs, acc = torch.ones(2, dtype=torch.int32), torch.zeros((2, 32, 2)), wrap(torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.window_attn(q, None, i, 8, 0, 16, None, 0.04, cs)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.prefix_decode_attn(q=q, main_kv=None, n_entries=i, n_prefix=0, max_entries=8, sink=None,
                                softmax_scale=0.04, q_rope_cs=cs)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.attn_weights(q, None, i, 8, 0.04, cs, acc, acc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.evict([], acc, i, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cskv.evict(caches=[], acc=acc, n_entries=i, budget=4)


def test_missing_arguments_are_named(lib):  # noqa: F811
    with pytest.raises(TypeError, match="acc"):
        cskv.evict([])
    with pytest.raises(TypeError, match="main_kv"):
        cskv.attn_weights()
