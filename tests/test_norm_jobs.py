"""norm_rope's jobs run in no order: calls in which one writes what another one reads or writes are
refused, columns of one buffer are not."""

import numpy as np
import pytest

FAKE = 1 << 20
E = 2 * 512                  # bytes of a head


@pytest.fixture(scope="module")
def lib():
    from compressed_sparse_attention_kv_gb300 import build, _lib
    build.build()
    return _lib.lib()


def _job(x, out, H=1, x_stride=None, out_stride=None, slot=None):
    from compressed_sparse_attention_kv_gb300._lib import NormJob, Paged
    cache = Paged(1 << 30, None, 64 * 1024, 4, 0, 0, 512)
    return NormJob(x, x_stride or 512 * H, H, 512, 1, None, 1e-6, 0, None if slot else out, out_stride or 512 * H, cache, slot)


# jobs over 7 tokens, (x, out, ...) each
MEETING = {
    "two jobs, one output": [(FAKE, 2 * FAKE), (3 * FAKE, 2 * FAKE)],
    "an output that is another job's input": [(FAKE, 2 * FAKE), (2 * FAKE, 3 * FAKE)],
    "in place, and read by another job": [(FAKE, FAKE), (FAKE, 3 * FAKE)],
    "in place, and coded into a cache": [(FAKE, FAKE), (FAKE, None, 1, None, None, 4096)],
    "in place twice": [(FAKE, FAKE), (FAKE, FAKE)],
    "its own input a head further": [(FAKE, FAKE + E, 2)],
    "its own input a token further": [(FAKE, FAKE + 2 * E, 2)],
    "its own input, 16 bytes before": [(FAKE, FAKE - 16)],
    "the last token's last bytes": [(FAKE, 2 * FAKE), (FAKE - 7 * E + 16, 3 * FAKE), (2 * FAKE + 7 * E - 16, 4 * FAKE)],
    "neighbouring columns that share 16 bytes": [(FAKE, 4 * FAKE, 1, 2048, 512), (3 * FAKE, FAKE + E - 16, 1, 512, 2048)],
    "a column of another token": [(FAKE, 4 * FAKE, 1, 2048, 512), (3 * FAKE, FAKE + 4 * 4 * E, 1, 512, 2048)],
    "strides that divide": [(FAKE, 4 * FAKE, 1, 1024, 512), (3 * FAKE, FAKE + E // 2, 1, 512, 2048)],
    "strides without a common column": [(FAKE, 4 * FAKE, 1, 520, 512), (3 * FAKE, FAKE, 1, 512, 768)],
}


@pytest.mark.parametrize("name", sorted(MEETING))
def test_jobs_that_meet_are_refused(lib, name):
    from compressed_sparse_attention_kv_gb300._lib import NormJob
    jobs = [_job(*j) for j in MEETING[name]]
    assert lib.cskvs_norm_rope((NormJob * len(jobs))(*jobs), len(jobs), None, 7, None) == 1
    assert lib.cskvs_norm_rope((NormJob * len(jobs))(*jobs[::-1]), len(jobs), None, 7, None) == 1


@pytest.mark.gpu
def test_columns_of_one_buffer_do_not_meet():
    """In place on one column beside others that are read, and from and to columns of one buffer; strides that differ."""
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    T = 11
    buf = torch.randn((T, 7 * 512), generator=gen, device="cuda").to(torch.bfloat16)
    col = lambda b, c, n=1: b[:, 512 * c:512 * (c + n)].unflatten(1, (n, 512))
    want = [cskv.norm_rope([dict(x=col(buf, c).contiguous(), norm=True)])[0] for c in range(7)]
    before = buf.clone()
    b = buf.clone()
    cskv.norm_rope([dict(x=col(b, 0), norm=True, out=col(b, 0)), dict(x=col(b, 1), norm=True, out=col(b, 3)),
                    dict(x=col(b, 2), norm=True, out=col(b, 4))])
    for c, w in ((0, want[0]), (1, col(before, 1)), (2, col(before, 2)), (3, want[1]), (4, want[2]), (5, col(before, 5))):
        assert torch.equal(col(b, c), w), c
    # every other token of a buffer and all tokens of its neighbour: strides of 10 and of 5 heads
    b = torch.randn((4 * T, 5 * 512), generator=gen, device="cuda").to(torch.bfloat16)
    x, out = b[:2 * T:2, 512:1024].unflatten(1, (1, 512)), b[2 * T:3 * T, :512].unflatten(1, (1, 512))
    y = x.clone()
    cskv.norm_rope([dict(x=x, norm=True, out=out)])
    assert torch.equal(out, cskv.norm_rope([dict(x=y, norm=True)])[0])
    other = b[:T, 1024:1536].unflatten(1, (1, 512))      # between x's tokens, another column
    cskv.norm_rope([dict(x=x, norm=True, out=other)])
    assert torch.equal(other, cskv.norm_rope([dict(x=y, norm=True)])[0])
    with pytest.raises(cskv.CskvError):
        cskv.norm_rope([dict(x=x, out=b[:T, 512:1024].unflatten(1, (1, 512)))])


def test_the_rule_of_strided_pieces_against_all_pairs(lib):
    """Random jobs of few tokens: refused whenever bytes are shared; with one stride, or one token, never otherwise.
    (What is not refused would launch on addresses that are none: without a GPU alone.)"""
    import torch
    from compressed_sparse_attention_kv_gb300._lib import NormJob
    if torch.cuda.is_available():
        pytest.skip("the addresses are none")
    rs = np.random.default_rng(0)
    met = passed = 0
    for _ in range(6000):
        T, H = int(rs.integers(1, 6)), int(rs.integers(1, 3))
        xs, os_ = (512 * H + 8 * int(rs.choice([0, 1, 64, 128, 300])) for _ in range(2))
        if rs.random() < 0.5:
            os_ = xs
        x, out = FAKE, FAKE + 16 * int(rs.integers(-1200, 1200))
        if x == out:
            continue
        shared = any(abs((x + 2 * i * xs) - (out + 2 * k * os_)) < E * H for i in range(T) for k in range(T))
        refused = lib.cskvs_norm_rope((NormJob * 1)(_job(x, out, H, xs, os_)), 1, None, T, None) == 1
        if shared or xs == os_ or T == 1:
            assert refused == shared, (T, H, xs, os_, out - x)
            met, passed = met + refused, passed + (not refused)
    assert met > 500 and passed > 500


@pytest.mark.gpu
def test_a_slot_without_a_cache_is_refused():
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    x, slot = torch.ones((3, 1, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for job in (dict(x=x, slot=slot), dict(x=x, slot=slot, out=torch.empty_like(x)), dict(x=x, slot=slot, cache=None)):
        with pytest.raises(ValueError, match="slot needs cache"):
            cskv.norm_rope([job])


@pytest.mark.gpu
def test_norm_follows_norm_w_and_not_against_it():
    import torch
    import compressed_sparse_attention_kv_gb300 as cskv
    x = torch.randn((3, 2, 512), device="cuda").to(torch.bfloat16)
    w = torch.rand(512, device="cuda")
    assert torch.equal(cskv.norm_rope([dict(x=x, norm_w=w)])[0], cskv.norm_rope([dict(x=x, norm_w=w, norm=True)])[0])
    assert torch.equal(cskv.norm_rope([dict(x=x)])[0], x)
    with pytest.raises(ValueError, match="norm_w without norm"):
        cskv.norm_rope([dict(x=x, norm_w=w, norm=False)])
