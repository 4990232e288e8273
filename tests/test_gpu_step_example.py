"""The documented step from lengths to attention, run as its example stands."""

import os
import re

import numpy as np
import pytest
import torch

import compressed_sparse_attention_kv_gb300 as cskv
from oracle import bounded, codecs, step

from cases import bf16_values, cuda
from test_gpu_bounded_cache import SCALE, _check, _i32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    with open(os.path.join(ROOT, "README.md")) as f:
        block, = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "chunk_attn(" in b]
    return block


@pytest.mark.gpu
def test_the_documented_step():
    """Two steps; each query turned once, at its own position, over every row up to its own."""
    rs = np.random.default_rng(40)
    B, T, H, per, total = 2, 48, 4, 3, 6
    pages = cskv.PageTable.allocate(B, per, total)
    cache = cskv.PagedCache.allocate(total, cskv.FMT_FP8, 512, block_table=pages.block_table)
    w_host, sink_host = rs.uniform(0.5, 1.5, 512).astype(np.float32), rs.standard_normal(H).astype(np.float32)
    env = dict(cskv=cskv, T=T, pages=pages, cache=cache, plan=cskv.RopePlan(), w=cuda(w_host), sink=cuda(sink_host), scale=SCALE,
               max_len=per * 64, ctx_len=_i32([0, 0]))
    rows = [np.zeros((0, 512)) for _ in range(B)]
    for new in ([30, 7], [1, 40]):
        kv, kvv = bf16_values(1.5 * rs.standard_normal((T, 1, 512)))
        q, qv = bf16_values(2.0 * rs.standard_normal((T, H, 512)))
        env.update(q=q.cuda(), kv=kv.cuda(), n_new=_i32(new))
        exec(_example(), env)
        env["ctx_len"] = env["maps"].new_len.clone()
        assert cskv.device_status() == 0
        cs = env["cs"].cpu().numpy()
        normed = torch.from_numpy(step.norm_rope(qv, True, None, 1e-6, None)).to(torch.bfloat16).float().numpy()
        i = 0
        for b in range(B):
            y = step.norm_rope(kvv[i:i + new[b], 0], True, w_host, 1e-6, cs[i:i + new[b]])
            start = len(rows[b])
            rows[b] = np.concatenate([rows[b], codecs.decode_rows(codecs.encode_rows(y, codecs.FMT_FP8), codecs.FMT_FP8, 512)])
            for k in range(new[b]):
                want = bounded.attend(normed[i + k], start + k, rows[b][:start + k + 1], sink_host, SCALE)
                _check(env["out"][i + k], env["lse"][i + k], want, "token %d of request %d" % (k, b))
            i += new[b]


@pytest.mark.gpu
@pytest.mark.parametrize("length", [40, 9000])
@pytest.mark.parametrize("logit", [1e3, 1e6, 2.0 ** 30])
def test_logits_up_to_two_to_the_thirty(logit, length):
    """A query that is one of its keys, +-1 in 448 dims, the logits as large as is allowed: that key alone, whole and
    split, by both calls.  (The other products with it are sums of 448 signs, below 448 / 2: their weights are less
    than e^-500.)"""
    rs = np.random.default_rng(41)
    H, hot = 3, length // 3
    t, v = bf16_values(rs.choice([-1.0, 1.0], (length, 512)))
    t[:, 448:] = 0                                                   # (nothing to rotate)
    cache = cskv.PagedCache.allocate((length + 63) // 64, cskv.FMT_BF16, 512,
                                     block_table=torch.arange((length + 63) // 64, dtype=torch.int32, device="cuda")[None])
    cache.pool.view(torch.bfloat16).view(-1, 512)[:length] = t.cuda()
    q = t[hot].cuda().expand(1, H, 512).contiguous()
    cs, n = cskv.rope_cs(_i32([length - 1]), cskv.RopePlan()), _i32([length])
    scale = logit / 448 * (1 - 2.0 ** -20)
    for out, lse in (cskv.chunk_attn(q, _i32([0, 1]), n, cache, 1, length, length, None, scale, cs, want_lse=True),
                     cskv.window_attn(q, cache, n, length, 0, length, None, scale, cs, want_lse=True)):
        assert cskv.device_status() == 0
        assert torch.equal(out, q)
        # the logit, its product with log2(e), and back: a few roundings of fp32
        assert float((lse.double() - logit).abs().max()) <= logit * 2.0 ** -19
