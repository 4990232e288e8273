"""compressed_sparse_attention_kv_gb300: DeepSeek-V4-style compressed-KV decode attention on GB300.

Thin Python binding over libcskv.so (include/cskv.h).  Every function here only
marshals arguments: torch tensors provide device memory and the current CUDA
stream; all arithmetic of the decode path runs in the library's sm_103a
kernels.  There is no CPU fallback: calling into the library without it being
built raises.

Calls (same names as the C ABI, without the ``cskv_`` prefix):

    compress(...)            gated per-channel pooling compressor -> cache rows
    compress_many(...)       several compressor jobs in one launch
    decode_append(...)       one decode step's compressor state ring and window update
    index_topk(...)          lightning-indexer scores + top-k selection
    sparse_decode_attn(...)  shared-KV attention over window + compressed entries
    sparse_prefill_attn(...) the same attention for many prompt queries
    decode_layer(...)        one layer's decode step, host buffers in and out
    encode_rows(...)         code rows of values into a cache format

and, from include/cskvx.h (prefix ``cskvx_``), attention over bounded and shared caches:

    window_attn(...)         a sliding window and the first rows of each request
    prefix_decode_attn(...)  a decode batch whose requests share their first entries
    attn_weights(...)        each entry's accumulated attention weight
    evict(...)               cuts each request's entries to a budget by that weight

and, from include/cskvs.h (prefix ``cskvs_``), one step of a server, from lengths to attention:

    plan_step(...)           block tables, slots and positions of a step's tokens, from lengths
    rope_cs(...)             the (cos, sin) table of positions on the GPU, one axis or several
    norm_rope(...)           norms of queries and rows with the rotation, rows coded into a cache
    chunk_attn(...)          new tokens' attention over all visible entries and a window
"""

import ctypes
import functools
import math

import numpy as np

from . import _lib

FMT_BF16 = 0
FMT_FP8 = 1
FMT_FP4 = 2
FMT_FP8_PAGESPLIT = 3
FMT_FP4H_PAGESPLIT = 4
PAGE_ROWS = 64
WINDOW = 128

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "device timeout",
           5: "device bounds"}


class CskvError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, _STATUS.get(status, "?"), status))


def _check(status, what):
    if status != 0:
        raise CskvError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _need(t, dtype, name, device=True):
    import torch
    if t is None:
        return
    if device and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def row_bytes(fmt, dim):
    return int(_lib.lib().cskv_row_bytes(fmt, dim))


def version():
    return int(_lib.lib().cskv_version())


def device_status(stream=None):
    """Synchronise the stream and return (and clear) the library's sticky device status."""
    return int(_lib.lib().cskv_device_status(_stream(stream)))


def set_spin_limit(cycles):
    _lib.lib().cskv_set_spin_limit(int(cycles))


def set_timing_events(begin, end):
    """Record torch.cuda.Event `begin`/`end` around every later indexer score kernel (None, None: off)."""
    if begin is None or end is None:
        _lib.lib().cskv_set_timing_events(None, None)
    else:
        _lib.lib().cskv_set_timing_events(begin.cuda_event, end.cuda_event)


class PagedCache:
    """A paged cache: `pool` uint8 [num_pages, page_bytes] on the GPU and an int32
    block table [batch, max_pages] (or None for a flat array of rows)."""

    def __init__(self, pool, block_table, fmt, dim):
        import torch
        _need(pool, torch.uint8, "pool")
        _need(block_table, torch.int32, "block_table")
        self.pool = pool
        self.block_table = block_table
        self.fmt = int(fmt)
        self.dim = int(dim)

    @classmethod
    def allocate(cls, num_pages, fmt, dim, block_table=None, device="cuda"):
        import torch
        rb = row_bytes(fmt, dim)
        page = PAGE_ROWS * rb
        page = (page + 15) // 16 * 16
        pool = torch.zeros((num_pages, page), dtype=torch.uint8, device=device)
        return cls(pool, block_table, fmt, dim)

    def desc(self):
        return _lib.Paged(self.pool.data_ptr(),
                          None if self.block_table is None else self.block_table.data_ptr(),
                          self.pool.shape[1], self.pool.shape[0],
                          0 if self.block_table is None else self.block_table.shape[1],
                          self.fmt, self.dim)


# YaRN of the compressed layers: 65,536 original positions stretched 16-fold, betas 32 / 1
YARN_V4 = dict(factor=16.0, original=65536, beta_fast=32.0, beta_slow=1.0)


def rope_table(positions, theta=160000.0, rope_dim=64, yarn=None):
    """float32 [..., 32, 2] (cos, sin) of every position, from cskv_rope_table (host code in
    the library): plain frequencies theta^(-2k/64), or with yarn (a dict like YARN_V4) the
    YaRN blend over the pair index."""
    if rope_dim != 64:
        raise ValueError("the kernels rotate 64 dims")
    pos = np.ascontiguousarray(np.asarray(positions), dtype=np.int64)
    out = np.empty(pos.shape + (32, 2), dtype=np.float32)
    y = yarn or {}
    st = _lib.lib().cskv_rope_table(pos.ctypes.data, int(pos.size), float(theta), float(y.get("factor", 1.0)),
                                    float(y.get("original", 1.0)), float(y.get("beta_fast", 1.0)),
                                    float(y.get("beta_slow", 1.0)), out.ctypes.data)
    _check(st, "cskv_rope_table")
    return out


def encode_rows(src, dst, req=None, row=None, stream=None):
    """Code rows of src (fp32 or bf16 [n, dim]) into the cache dst (rows row[i] of request req[i])."""
    import torch
    if src.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("src must be float32 or bfloat16")
    _need(src, None, "src")
    _need(req, torch.int32, "req")
    _need(row, torch.int32, "row")
    n, dim = src.shape
    st = _lib.lib().cskv_encode_rows(src.data_ptr(), int(src.dtype == torch.bfloat16), n, dim,
                                     _ptr(req), _ptr(row), dst.desc(), _stream(stream))
    _check(st, "cskv_encode_rows")


def compress(kv, gate, ape, ratio, overlap, out, req, first_entry, prev_kv=None, prev_gate=None,
             norm_w=None, eps=1e-6, rope_cs=None, stream=None):
    """Gated per-channel pooling of S sequences of T tokens (kv, gate: bf16 [S, T, coff, dim]);
    ape None = no slot bias (the V4.1 compressor)."""
    import torch
    for t, n in ((kv, "kv"), (gate, "gate"), (prev_kv, "prev_kv"), (prev_gate, "prev_gate")):
        _need(t, torch.bfloat16, n)
    for t, n in ((ape, "ape"), (norm_w, "norm_w"), (rope_cs, "rope_cs")):
        _need(t, torch.float32, n)
    _need(req, torch.int32, "req")
    _need(first_entry, torch.int32, "first_entry")
    S, T, coff, dim = kv.shape
    st = _lib.lib().cskv_compress(kv.data_ptr(), gate.data_ptr(), _ptr(prev_kv), _ptr(prev_gate),
                                  _ptr(ape), _ptr(norm_w), float(eps), _ptr(rope_cs),
                                  S, T, int(ratio), int(bool(overlap)), dim, req.data_ptr(),
                                  first_entry.data_ptr(), out.desc(), _stream(stream))
    _check(st, "cskv_compress")


def compress_many(jobs, stream=None):
    """Several compressor jobs in one launch.  Each job is a dict of compress()'s
    arguments (kv, gate, ape, ratio, overlap, out, req, first_entry and, optionally,
    prev_kv, prev_gate, norm_w, eps, rope_cs); same results as separate calls."""
    arr = _compress_jobs(jobs)
    st = _lib.lib().cskv_compress_many(arr, len(jobs), _stream(stream))
    _check(st, "cskv_compress_many")


def _compress_jobs(jobs, host_inputs=False):
    """ctypes array of struct cskv_compress_job for compress()-style job dicts.  With
    host_inputs (decode_layer), kv, gate, prev_kv, prev_gate and rope_cs may be pinned
    host tensors (read in place by the compressor)."""
    import torch

    def need_in(t, dtype, name):
        _need(t, dtype, name, device=not host_inputs)
        if t is not None and not t.is_cuda and not t.is_pinned():
            raise ValueError("%s must be a CUDA tensor or a pinned host tensor" % name)

    arr = (_lib.CompressJob * max(1, len(jobs)))()
    for i, j in enumerate(jobs):
        kv, gate = j["kv"], j["gate"]
        for t, n in ((kv, "kv"), (gate, "gate"), (j.get("prev_kv"), "prev_kv"), (j.get("prev_gate"), "prev_gate")):
            need_in(t, torch.bfloat16, n)
        need_in(j.get("rope_cs"), torch.float32, "rope_cs")
        for t, n in ((j.get("ape"), "ape"), (j.get("norm_w"), "norm_w")):
            _need(t, torch.float32, n)
        _need(j["req"], torch.int32, "req")
        _need(j["first_entry"], torch.int32, "first_entry")
        S, T, coff, dim = kv.shape
        arr[i] = _lib.CompressJob(kv.data_ptr(), gate.data_ptr(), _ptr(j.get("prev_kv")), _ptr(j.get("prev_gate")),
                                  _ptr(j.get("ape")), _ptr(j.get("norm_w")), float(j.get("eps", 1e-6)),
                                  _ptr(j.get("rope_cs")), S, T, int(j["ratio"]), int(bool(j["overlap"])), dim,
                                  j["req"].data_ptr(), j["first_entry"].data_ptr(), j["out"].desc())
    return arr


def decode_state(B, ratio, overlap, dim, device="cuda"):
    """A fresh per-request compressor state ring for decode_append: (state_kv, state_gate),
    bf16 [B, nblk * ratio, coff, dim] (nblk = coff = 2 with overlap, else 1), kv 0 and gate -inf."""
    import torch
    nblk = 2 if overlap else 1
    coff = 2 if overlap else 1
    shape = (B, nblk * ratio, coff, dim)
    return (torch.zeros(shape, dtype=torch.bfloat16, device=device),
            torch.full(shape, float("-inf"), dtype=torch.bfloat16, device=device))


def decode_append(jobs, pos, stream=None):
    """One decode step's state update.  Each job is a dict: kv, gate (bf16 [B, coff, dim]; gate
    may be None at ratio 1), state (the (state_kv, state_gate) pair of decode_state; None at
    ratio 1), ratio, overlap, out (PagedCache), and optionally ape, norm_w, eps, rope_cs
    (fp32 [B, 32, 2] at the position each request writes), ring_rows.  pos: int32 [B]
    positions of the new tokens (< 0: no token)."""
    import torch
    _need(pos, torch.int32, "pos")
    arr = (_lib.DecodeJob * len(jobs))()
    for i, j in enumerate(jobs):
        kv = j["kv"]
        _need(kv, torch.bfloat16, "kv")
        _need(j.get("gate"), torch.bfloat16, "gate")
        st = j.get("state")
        sk, sg = (st if st is not None else (None, None))
        _need(sk, torch.bfloat16, "state_kv")
        _need(sg, torch.bfloat16, "state_gate")
        for t, n in ((j.get("ape"), "ape"), (j.get("norm_w"), "norm_w"), (j.get("rope_cs"), "rope_cs")):
            _need(t, torch.float32, n)
        arr[i] = _lib.DecodeJob(kv.data_ptr(), _ptr(j.get("gate")), _ptr(sk), _ptr(sg), _ptr(j.get("ape")),
                                _ptr(j.get("norm_w")), float(j.get("eps", 1e-6)), _ptr(j.get("rope_cs")),
                                int(j["ratio"]), int(bool(j.get("overlap", 0))), int(kv.shape[-1]),
                                int(j.get("ring_rows", 0)), j["out"].desc())
    st = _lib.lib().cskv_decode_append(arr, len(jobs), pos.data_ptr(), int(pos.shape[0]), _stream(stream))
    _check(st, "cskv_decode_append")


def index_topk_workspace_size(B, max_ctx_len, ratio, Hi, k):
    return int(_lib.lib().cskv_index_topk_workspace_size(B, max_ctx_len, ratio, Hi, k))


def index_topk(q_idx, w, keys, ctx_len, ratio, k, max_ctx_len, topk_idx=None, topk_score=None,
               workspace=None, want_scores=True, stream=None):
    """Lightning-indexer top-k; returns (topk_idx int32 [B, k], topk_score fp32 [B, k] or None)."""
    import torch
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(w, torch.float32, "w")
    _need(ctx_len, torch.int32, "ctx_len")
    B, Hi, _ = q_idx.shape
    dev = q_idx.device
    if topk_idx is None:
        topk_idx = torch.empty((B, k), dtype=torch.int32, device=dev)
    if topk_score is None and want_scores:
        topk_score = torch.empty((B, k), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(index_topk_workspace_size(B, max_ctx_len, ratio, Hi, k),
                                dtype=torch.uint8, device=dev)
    st = _lib.lib().cskv_index_topk(q_idx.data_ptr(), w.data_ptr(), keys.desc(), ctx_len.data_ptr(),
                                    B, Hi, int(ratio), int(k), int(max_ctx_len), topk_idx.data_ptr(),
                                    _ptr(topk_score), workspace.data_ptr(), workspace.numel(),
                                    _stream(stream))
    _check(st, "cskv_index_topk")
    return topk_idx, topk_score


def sparse_decode_attn_workspace_size(B, H, max_ctx_len, ratio, k):
    return int(_lib.lib().cskv_sparse_decode_attn_workspace_size(B, H, max_ctx_len, ratio, k))


def sparse_decode_attn(q, main_kv, swa, swa_fmt, ctx_len, topk_idx, k, ratio, max_ctx_len, sink,
                       softmax_scale, q_rope_cs, out=None, workspace=None, stream=None):
    """Shared-KV decode attention; returns out bf16 [B, H, 512]."""
    import torch
    _need(q, torch.bfloat16, "q")
    _need(swa, torch.uint8, "swa")
    _need(ctx_len, torch.int32, "ctx_len")
    _need(topk_idx, torch.int32, "topk_idx")
    _need(sink, torch.float32, "sink")
    _need(q_rope_cs, torch.float32, "q_rope_cs")
    B, H, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    kk = int(k) if topk_idx is not None else 0
    if workspace is None:
        workspace = torch.empty(sparse_decode_attn_workspace_size(B, H, max_ctx_len, ratio, kk),
                                dtype=torch.uint8, device=q.device)
    st = _lib.lib().cskv_sparse_decode_attn(q.data_ptr(), main_kv.desc(), swa.data_ptr(), int(swa_fmt),
                                            ctx_len.data_ptr(), _ptr(topk_idx), kk, int(ratio),
                                            int(max_ctx_len), _ptr(sink), float(softmax_scale),
                                            q_rope_cs.data_ptr(), B, H, out.data_ptr(),
                                            workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(st, "cskv_sparse_decode_attn")
    return out


def sparse_prefill_attn(q, main_kv, window, pos1, topk_idx, k, ratio, max_ctx_len, sink, softmax_scale,
                        q_rope_cs, req_of=None, out=None, workspace=None, stream=None):
    """The attention of many prompt queries; query i of request req_of[i] sits at position
    pos1[i] - 1 and reads its window from `window` (raw rows by position).  Returns out
    bf16 [T, H, 512]."""
    import torch
    _need(q, torch.bfloat16, "q")
    _need(pos1, torch.int32, "pos1")
    _need(req_of, torch.int32, "req_of")
    _need(topk_idx, torch.int32, "topk_idx")
    _need(sink, torch.float32, "sink")
    _need(q_rope_cs, torch.float32, "q_rope_cs")
    T, H, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    kk = int(k) if topk_idx is not None else 0
    if workspace is None:
        workspace = torch.empty(sparse_decode_attn_workspace_size(T, H, max_ctx_len, ratio, kk),
                                dtype=torch.uint8, device=q.device)
    st = _lib.lib().cskv_sparse_prefill_attn(q.data_ptr(), main_kv.desc(), window.desc(), _ptr(req_of),
                                             pos1.data_ptr(), _ptr(topk_idx), kk, int(ratio), int(max_ctx_len),
                                             _ptr(sink), float(softmax_scale), q_rope_cs.data_ptr(), T, H,
                                             out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                             _stream(stream))
    _check(st, "cskv_sparse_prefill_attn")
    return out


def decode_layer(jobs, q_idx, w, keys, q, main_kv, swa, swa_fmt, ctx_len, k, ratio, max_ctx_len, sink,
                 softmax_scale, q_rope_cs, topk_idx=None, out=None, index_workspace=None, attn_workspace=None,
                 h_in=None, d_in=None, h_out=None, stream=None):
    """One decode step of one layer in one call (cskv_decode_layer): h_in (host uint8) is
    copied into d_in (device uint8, which the other tensors may view), then compress_many(jobs)
    (jobs may be empty), index_topk (skipped when q_idx is None: HCA) and sparse_decode_attn
    run, and out is copied into h_out (host, out's dtype and size or less) last.  Host
    buffers should be pinned; q, and the jobs' kv, gate, prev_kv, prev_gate and
    rope_cs, may be pinned host tensors (read in place by the attention and the
    compressor).  Returns (out, topk_idx); h_out holds the output once the stream has
    synchronised."""
    import torch
    for t, dt, n in ((q_idx, torch.bfloat16, "q_idx"), (w, torch.float32, "w"),
                     (swa, torch.uint8, "swa"), (ctx_len, torch.int32, "ctx_len"), (sink, torch.float32, "sink"),
                     (q_rope_cs, torch.float32, "q_rope_cs"), (d_in, torch.uint8, "d_in")):
        _need(t, dt, n)
    _need(q, torch.bfloat16, "q", device=False)
    if not q.is_cuda and not q.is_pinned():
        raise ValueError("q must be a CUDA tensor or a pinned host tensor")
    _need(h_in, torch.uint8, "h_in", device=False)
    _need(h_out, None, "h_out", device=False)
    for t, n in ((h_in, "h_in"), (h_out, "h_out")):
        if t is not None and t.is_cuda:
            raise ValueError("%s must be a host tensor" % n)
    if h_in is not None and (d_in is None or d_in.numel() < h_in.numel()):
        raise ValueError("d_in must be a device buffer at least as large as h_in")
    B, H, _ = q.shape
    dev = ctx_len.device
    csa = q_idx is not None
    Hi = q_idx.shape[1] if csa else 0
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if csa and topk_idx is None:
        topk_idx = torch.empty((B, k), dtype=torch.int32, device=dev)
    if csa and index_workspace is None:
        index_workspace = torch.empty(index_topk_workspace_size(B, max_ctx_len, ratio, Hi, k), dtype=torch.uint8,
                                      device=dev)
    kk = int(k) if csa else 0
    if attn_workspace is None:
        attn_workspace = torch.empty(sparse_decode_attn_workspace_size(B, H, max_ctx_len, ratio, kk),
                                     dtype=torch.uint8, device=dev)
    arr = _compress_jobs(jobs, host_inputs=True)
    empty = _lib.Paged(None, None, 0, 0, 0, 0, 128)
    a = _lib.DecodeLayerArgs(
        ctypes.cast(arr, ctypes.POINTER(_lib.CompressJob)) if jobs else None, len(jobs), _ptr(q_idx), _ptr(w), keys.desc() if csa else empty, Hi, kk,
        _ptr(topk_idx) if csa else None, _ptr(index_workspace) if csa else None,
        index_workspace.numel() if csa else 0, q.data_ptr(), main_kv.desc(), swa.data_ptr(), int(swa_fmt),
        ctx_len.data_ptr(), int(ratio), int(max_ctx_len), _ptr(sink), float(softmax_scale), q_rope_cs.data_ptr(),
        B, H, out.data_ptr(), attn_workspace.data_ptr(), attn_workspace.numel(),
        _ptr(h_in), _ptr(d_in), h_in.numel() if h_in is not None else 0,
        _ptr(h_out), h_out.numel() * h_out.element_size() if h_out is not None else 0)
    st = _lib.lib().cskv_decode_layer(ctypes.byref(a), _stream(stream))
    _check(st, "cskv_decode_layer")
    return out, topk_idx


def _refuse(name, t, dtype, shape, device):
    """Says what is wrong with an argument that _take did not accept."""
    _need(t, dtype, name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _take(name, t, dtype, shape, device):
    """The address of a contiguous tensor of this type, shape and device (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(name, t, dtype, shape, device)
    return t.data_ptr()


def _cache_on(name, cache, rows, device):
    """A cache whose pool and table (of at least `rows` requests) are on the device."""
    bt = cache.block_table
    if cache.pool.device != device or (bt is not None and bt.device != device):
        raise ValueError("%s must be on %s" % (name, device))
    if bt is not None and bt.shape[0] < rows:
        raise ValueError("%s's block table has %d rows for a batch of %d" % (name, bt.shape[0], rows))
    return cache.desc()


def _on_stream(f):
    """Runs f with its `stream` argument (if one is given) current, so that what f allocates for
    the call belongs to the stream that uses it, and with the first tensor's device current."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        import torch
        first = args[0] if args else kw.get("q", kw.get("acc", kw.get("ctx_len", kw.get("positions", kw.get("jobs")))))
        if isinstance(first, (list, tuple)) and first and isinstance(first[0], dict):   # norm_rope: its jobs
            first = first[0].get("x")
        if not isinstance(first, torch.Tensor):   # evict: its caches
            first = args[1] if len(args) > 1 else kw.get("acc")
            if not isinstance(first, torch.Tensor):
                return f(*args, **kw)             # which says what is missing
        device = first.device
        if stream is not None:
            if device.type == "cuda" and stream.device != device:
                raise ValueError("the stream must be on %s, got %s" % (device, stream.device))
            with torch.cuda.stream(stream):
                return f(*args, **kw)
        if device.type == "cuda" and device.index != torch._C._cuda_getDevice():
            with torch.cuda.device(device):
                return f(*args, **kw)
        return f(*args, **kw)
    return g


def _raw_stream(device):
    """The current stream of the (current) device, as the library takes it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(workspace, nbytes, device):
    """(tensor, address, bytes) of the caller's workspace, or of one of nbytes."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        import torch
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    _need(workspace, None, "workspace")
    if workspace.device != device:
        raise ValueError("workspace must be on %s, got %s" % (device, workspace.device))
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _query(q):
    """(rows, heads, device, address) of the queries."""
    import torch
    if q.dtype is not torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
        _need(q, torch.bfloat16, "q")
    if q.dim() != 3 or q.shape[2] != 512:
        raise ValueError("q must have shape (rows, heads, 512), got %s" % (tuple(q.shape),))
    T, H, _ = q.shape
    return T, H, q.device, q.data_ptr()


def _outputs(q, T, H, device, out, lse, want_lse):
    """(out, lse, their addresses); allocates what is not given."""
    import torch
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=device)
        po = out.data_ptr()
    else:
        po = _take("out", out, torch.bfloat16, (T, H, 512), device)
    if lse is not None:
        pl = _take("lse", lse, torch.float32, (T, H), device)
    elif want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=device)
        pl = lse.data_ptr()
    else:
        pl = None
    return out, lse, po, pl


def window_attn_workspace_size(T, H, max_ctx_len, window, first):
    return int(_lib.lib().cskvx_window_attn_workspace_size(T, H, max_ctx_len, window, first))


@_on_stream
def window_attn(q, rows, pos1, window, first, max_ctx_len, sink, softmax_scale, q_rope_cs, req_of=None, out=None,
                lse=None, want_lse=False, workspace=None, stream=None):
    """Attention over a sliding window and the first rows: query i (bf16 q [T, H, 512]) of
    request req_of[i] (None: request i) at position t = pos1[i] - 1 sees the rows j <= t of
    `rows` (a PagedCache of raw rows by position) with j < first or j > t - window; pos1[i]
    <= 0: a padding query (out 0).  Returns (out bf16 [T, H, 512], lse fp32 [T, H] or None)."""
    import torch
    T, H, dev, pq = _query(q)
    i32, f32 = torch.int32, torch.float32
    pp = _take("pos1", pos1, i32, (T,), dev)
    pr = _take("req_of", req_of, i32, (T,), dev)
    ps = _take("sink", sink, f32, (H,), dev)
    pc = _take("q_rope_cs", q_rope_cs, f32, (T, 32, 2), dev)
    desc = _cache_on("rows", rows, T if req_of is None else 1, dev)
    reqs = rows.block_table.shape[0] if rows.block_table is not None else 1 << 30
    out, lse, po, pl = _outputs(q, T, H, dev, out, lse, want_lse)
    L = _lib.lib()
    need = 0 if workspace is not None else L.cskvx_window_attn_workspace_size(T, H, max_ctx_len, window, first)
    workspace, pw, nw = _workspace(workspace, need, dev)
    _check(L.cskvx_window_attn(pq, desc, reqs, pr, pp, window, first, max_ctx_len, ps, softmax_scale, pc, T, H, po, pl,
                               pw, nw, _raw_stream(dev)), "cskvx_window_attn")
    return out, lse


def prefix_decode_attn_workspace_size(B, H, n_prefix, max_entries, with_swa):
    return int(_lib.lib().cskvx_prefix_decode_attn_workspace_size(B, H, n_prefix, max_entries, int(bool(with_swa))))


@_on_stream
def prefix_decode_attn(q, main_kv, n_entries, n_prefix, max_entries, sink, softmax_scale, q_rope_cs, swa=None,
                       swa_fmt=FMT_BF16, ctx_len=None, out=None, lse=None, want_lse=False, workspace=None, stream=None):
    """Decode attention of a batch whose requests share entries [0, n_prefix) (read through
    request 0's block-table row): request b sees its entries j < n_entries[b] and, with swa
    (uint8 [B, 128, row bytes] and ctx_len int32 [B]), its window ring.  Returns (out bf16
    [B, H, 512], lse fp32 [B, H] or None)."""
    import torch
    B, H, dev, pq = _query(q)
    i32, f32 = torch.int32, torch.float32
    pn = _take("n_entries", n_entries, i32, (B,), dev)
    ps = _take("sink", sink, f32, (H,), dev)
    pc = _take("q_rope_cs", q_rope_cs, f32, (B, 32, 2), dev)
    pr = px = None
    if swa is not None:
        pr = _take("swa", swa, torch.uint8, (B, WINDOW, row_bytes(swa_fmt, 512)), dev)
        if ctx_len is None:
            raise ValueError("swa needs ctx_len")
        px = _take("ctx_len", ctx_len, i32, (B,), dev)
    desc = _cache_on("main_kv", main_kv, B, dev)
    out, lse, po, pl = _outputs(q, B, H, dev, out, lse, want_lse)
    L = _lib.lib()
    need = 0 if workspace is not None else L.cskvx_prefix_decode_attn_workspace_size(B, H, n_prefix, max_entries,
                                                                                     swa is not None)
    workspace, pw, nw = _workspace(workspace, need, dev)
    _check(L.cskvx_prefix_decode_attn(pq, desc, pn, n_prefix, max_entries, pr, swa_fmt, px, ps, softmax_scale, pc, B, H,
                                      po, pl, pw, nw, _raw_stream(dev)), "cskvx_prefix_decode_attn")
    return out, lse


@_on_stream
def attn_weights(q, main_kv, n_entries, max_entries, softmax_scale, q_rope_cs, lse, acc, decay=1.0, first=0,
                 acc_out=None, stream=None):
    """acc_out[b, j] = decay * acc[b, j] + sum over heads of exp(z - lse) for the entries
    first <= j < n_entries[b] (lse as prefix_decode_attn gave it), read through each request's
    own block-table row: first >= that call's n_prefix, unless every request's pages hold the
    prefix.  acc, acc_out fp32 [B, >= max_entries], acc_out None: in place.  Returns acc_out."""
    import torch
    B, H, dev, pq = _query(q)
    f32 = torch.float32
    pn = _take("n_entries", n_entries, torch.int32, (B,), dev)
    pc = _take("q_rope_cs", q_rope_cs, f32, (B, 32, 2), dev)
    pl = _take("lse", lse, f32, (B, H), dev)
    if acc_out is None:
        acc_out = acc
    pa, wa = _table("acc", acc, f32, B, max_entries, dev)
    pb, wb = _table("acc_out", acc_out, f32, B, max_entries, dev)
    desc = _cache_on("main_kv", main_kv, B, dev)
    _check(_lib.lib().cskvx_attn_weights(pq, desc, pn, first, max_entries, softmax_scale, pc, pl, B, H, decay, pa, wa,
                                         pb, wb, _raw_stream(dev)), "cskvx_attn_weights")
    return acc_out


def _table(name, t, dtype, rows, least, device):
    """(address, columns) of a [rows, at least `least`] table (None: (None, 0))."""
    if t is None:
        return None, 0
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < least:
        _need(t, dtype, name)
        raise ValueError("%s must have shape (%d, at least %d), got %s" % (name, rows, least, tuple(shape)))
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _refuse(name, t, dtype, shape, device)
    return t.data_ptr(), shape[1]


_PAGED_ARRAYS = [_lib.Paged * max(1, n) for n in range(5)]


def evict_workspace_size(B, max_entries, budget):
    return int(_lib.lib().cskvx_evict_workspace_size(B, max_entries, budget))


@_on_stream
def evict(caches, acc, n_entries, budget, fixed=0, recent=0, age=None, max_entries=None, acc_out=None, age_out=None,
          n_out=None, src=None, workspace=None, stream=None):
    """Cuts each request's entries to `budget` slots: the first `fixed` slots and the `recent`
    newest ages stay, then the largest accumulated weights acc (fp32 [B, capacity]); kept
    entries from slot `budget` on move into the given-up slots of every cache in `caches` (with
    a block table each, unless there is one request; pages that requests share hold slots below
    `fixed` alone).
    age: int32 [B, capacity] or None (then recent is 0).  acc_out, age_out, n_out None: in
    place.  max_entries None: acc's capacity.  Returns (src int32 [B, budget], n_out, acc_out,
    age_out): slot i now holds the entry of slot src[:, i] (-1: none)."""
    import torch
    i32, f32 = torch.int32, torch.float32
    if acc.dim() != 2 or not acc.is_cuda:
        _need(acc, f32, "acc")
        raise ValueError("acc must have shape (requests, capacity), got %s" % (tuple(acc.shape),))
    B, dev = acc.shape[0], acc.device
    most = acc.shape[1] if max_entries is None else max_entries
    kept = min(most, budget)
    acc_out = acc if acc_out is None else acc_out
    age_out = age if age_out is None else age_out
    n_out = n_entries if n_out is None else n_out
    pa, wa = _table("acc", acc, f32, B, most, dev)
    pg, wg = _table("age", age, i32, B, most, dev)
    pb, wb = _table("acc_out", acc_out, f32, B, kept, dev)
    ph, wh = _table("age_out", age_out, i32, B, kept, dev)
    pn = _take("n_entries", n_entries, i32, (B,), dev)
    pm = _take("n_out", n_out, i32, (B,), dev)
    arr = _PAGED_ARRAYS[len(caches)] if len(caches) < 5 else _lib.Paged * len(caches)
    arr = arr(*[_cache_on("a cache", c, B, dev) for c in caches])
    if src is None:
        src = torch.empty((B, max(budget, 0)), dtype=i32, device=dev)
    px = _take("src", src, i32, (B, max(budget, 0)), dev)
    L = _lib.lib()
    need = 0 if workspace is not None else L.cskvx_evict_workspace_size(B, most, budget)
    workspace, pw, nw = _workspace(workspace, need, dev)
    _check(L.cskvx_evict(arr, len(caches), pa, wa, pg, wg, pn, B, most, budget, fixed, recent, px, pb, wb, ph, wh, pm,
                         pw, nw, _raw_stream(dev)), "cskvx_evict")
    return src, n_out, acc_out, age_out


class PageTable:
    """The pages of a batch and the free ones: `block_table` int32 [B, max_pages]; `free_pages`
    int32 [capacity], a ring of free pages' ids; `state` int32 [4]: where the ring starts, how
    many ids it holds, and (written by plan_step) how many pages a step lacked, 0."""

    def __init__(self, block_table, free_pages, state):
        import torch
        for t, n in ((block_table, "block_table"), (free_pages, "free_pages"), (state, "state")):
            _need(t, torch.int32, n)
        if block_table.dim() != 2 or free_pages.dim() != 1 or tuple(state.shape) != (4,):
            raise ValueError("block_table, free_pages and state must have shapes (B, max_pages), (capacity,) and (4,)")
        if free_pages.device != block_table.device or state.device != block_table.device:
            raise ValueError("free_pages and state must be on %s" % block_table.device)
        self.block_table = block_table
        self.free_pages = free_pages
        self.state = state

    @classmethod
    def allocate(cls, B, max_pages, num_pages, device="cuda"):
        """No request has a page, all num_pages are free."""
        import torch
        i32 = torch.int32
        state = torch.zeros(4, dtype=i32, device=device)
        state[1] = num_pages
        return cls(torch.full((B, max_pages), -1, dtype=i32, device=device),
                   torch.arange(num_pages, dtype=i32, device=device), state)


class StepMaps:
    """What plan_step writes, for B requests and T places for tokens: cu_new int32 [B + 1],
    new_len, first_row, n_rows int32 [B], req_of, pos1 int32 [T], slot int64 [T] (None without
    pages), ring_slot int64 [T] (None without a ring), and the call's workspace beside them.
    Made once, it may serve every step, one at a time."""

    def __init__(self, B, T, pages=True, ring=False, device="cuda"):
        import torch
        # one allocation: the step's workspace, the 64-bit maps, the others
        self.workspace_bytes = _lib.lib().cskvs_plan_step_workspace_size(B)
        wide = (self.workspace_bytes // 8,) + ((T,) if pages else ()) + ((T,) if ring else ())
        buf = torch.empty(sum(wide) + (4 * B + 2 + 2 * T) // 2, dtype=torch.int64, device=device)
        _, *slots, rest = buf.split_with_sizes(wide + (buf.shape[0] - sum(wide),))
        self.slot = slots[0] if pages else None
        self.ring_slot = slots[-1] if ring else None
        self.cu_new, self.new_len, self.first_row, self.n_rows, self.req_of, self.pos1, _ = \
            rest.view(torch.int32).split_with_sizes((B + 1, B, B, B, T, T, 1))
        self.workspace = buf.data_ptr()
        self.B, self.T, self.device = B, T, buf.device


@_on_stream
def plan_step(ctx_len, n_new, T, pages=None, ratio=1, ring_rows=0, shared_pages=None, state_out=None, out=None,
              workspace=None, stream=None):
    """Block tables and slot maps of a step on the GPU: request b has ctx_len[b] tokens (int32 [B])
    and gets n_new[b] more (0: none, < 0: the request ends and gives its pages back).  T: places
    for tokens; those behind the last one are padding (pos1 0, req_of and slots -1).  pages (a
    PageTable) gets pages from its ring for the rows floor(length / ratio) that its requests come
    to have; state_out int32 [4]: its state after the step (None: in place).  ring_rows > 0: the
    rows of a window ring per request.  shared_pages int32 [B]: leading pages that a request
    does not give back.  Returns the StepMaps (`out`, or a new one)."""
    import torch
    i32 = torch.int32
    if ctx_len.dim() != 1 or not ctx_len.is_cuda:
        _need(ctx_len, i32, "ctx_len")
        raise ValueError("ctx_len must have shape (requests,), got %s" % (tuple(ctx_len.shape),))
    B, dev = ctx_len.shape[0], ctx_len.device
    pc = _take("ctx_len", ctx_len, i32, (B,), dev)
    pn = _take("n_new", n_new, i32, (B,), dev)
    psh = _take("shared_pages", shared_pages, i32, (B,), dev)
    pt = pf = ps = po = None
    per = cap = 0
    if pages is not None:
        bt = pages.block_table
        per, cap = bt.shape[1], pages.free_pages.shape[0]
        pt = _take("block_table", bt, i32, (B, per), dev)
        pf, ps = pages.free_pages.data_ptr(), pages.state.data_ptr()
        po = ps if state_out is None else _take("state_out", state_out, i32, (4,), dev)
    elif shared_pages is not None or state_out is not None:
        raise ValueError("shared_pages and state_out need pages")
    if out is None:
        out = StepMaps(B, T, pages is not None, ring_rows > 0, dev)
    elif out.B != B or out.T != T or out.device != dev or (out.slot is None) != (pages is None) or \
            (out.ring_slot is None) != (ring_rows <= 0):
        raise ValueError("out must be a StepMaps of %d requests and %d tokens on %s, with slots as pages and ring_rows "
                         "say" % (B, T, dev))
    if workspace is None:
        pw, nw = out.workspace, out.workspace_bytes
    else:
        workspace, pw, nw = _workspace(workspace, 0, dev)
    _check(_lib.lib().cskvs_plan_step(pc, pn, B, ratio, T, ring_rows, pt, per, psh, pf, cap, ps, po,
                                      out.cu_new.data_ptr(), out.new_len.data_ptr(), out.first_row.data_ptr(),
                                      out.n_rows.data_ptr(), out.req_of.data_ptr(), out.pos1.data_ptr(), _ptr(out.slot),
                                      _ptr(out.ring_slot), pw, nw, _raw_stream(dev)), "cskvs_plan_step")
    return out


class RopePlan:
    """Speeds of the 32 rotated pairs (theta, yarn as in rope_table) and the axis of positions
    that each follows: sections (n_0, n_1, ...), pairs of axis 0 first, then of axis 1, ...
    (32 in all), or axis_of, 32 axes, pair by pair; neither: one axis.  Made once and kept."""

    def __init__(self, theta=160000.0, yarn=None, sections=None, axis_of=None):
        if sections is not None:
            if axis_of is not None:
                raise ValueError("sections and axis_of say the same")
            if any(n < 0 for n in sections) or sum(sections) != 32:
                raise ValueError("sections must add up to 32 pairs, got %s" % (tuple(sections),))
            axis_of = [a for a, n in enumerate(sections) for _ in range(n)]
        self.axes = 1 if axis_of is None else len(sections) if sections is not None else max(axis_of) + 1
        if axis_of is not None and (len(axis_of) != 32 or min(axis_of) < 0 or self.axes > 4):
            raise ValueError("axis_of must be 32 axes of at most four, got %s" % (axis_of,))
        y = yarn or {}
        self.struct = _lib.RopePlan()
        axis = None if axis_of is None else (ctypes.c_uint8 * 32)(*axis_of)
        st = _lib.lib().cskvs_rope_init(ctypes.byref(self.struct), float(theta), float(y.get("factor", 1.0)),
                                        float(y.get("original", 1.0)), float(y.get("beta_fast", 1.0)),
                                        float(y.get("beta_slow", 1.0)), self.axes,
                                        None if axis is None else ctypes.addressof(axis))
        _check(st, "cskvs_rope_init")
        self.ref = ctypes.byref(self.struct)


@_on_stream
def rope_cs(positions, plan, shift=0, out=None, stream=None):
    """fp32 [T, 32, 2] (cos, sin) of positions + shift on the GPU (int32 [T], or [axes, T] for a
    RopePlan of several axes): the table that compress, norm_rope and the attention calls take."""
    import torch
    shape = positions.shape
    if len(shape) == 1 and plan.axes == 1:
        T = shape[0]
    elif len(shape) == 2 and shape[0] == plan.axes:
        T = shape[1]
    else:
        raise ValueError("positions must have shape (%d, T), got %s" % (plan.axes, tuple(shape)))
    if positions.dtype is not torch.int32 or not positions.is_cuda or not positions.is_contiguous():
        _need(positions, torch.int32, "positions")
    dev = positions.device
    if out is None:
        out = torch.empty((T, 32, 2), dtype=torch.float32, device=dev)
        po = out.data_ptr()
    else:
        po = _take("out", out, torch.float32, (T, 32, 2), dev)
    _check(_lib.lib().cskvs_rope_cs(plan.ref, positions.data_ptr(), T, shift, T, po, _raw_stream(dev)), "cskvs_rope_cs")
    return out


def _heads(name, t, T, device):
    """(address, stride between tokens) of a bf16 [T, H, dim] tensor whose heads are contiguous."""
    import torch
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise ValueError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if t.device != device or t.dim() != 3 or t.shape[0] != T:
        raise ValueError("%s must have shape (%d, heads, dim) on %s, got %s on %s"
                         % (name, T, device, tuple(t.shape), t.device))
    s = t.stride()
    H, dim = t.shape[1], t.shape[2]
    if (s[2] != 1 and dim > 1) or (s[1] != dim and H > 1):
        raise ValueError("%s's heads must be contiguous, got strides %s" % (name, s))
    return t.data_ptr(), s[0] if T > 1 else H * dim


_NORM_ARRAYS = [_lib.NormJob * max(1, n) for n in range(5)]


@_on_stream
def norm_rope(jobs, rope_cs=None, stream=None):
    """Norms, rotation and coding of a step's queries and rows in one launch.  jobs: up to four
    dicts of x (bf16 [T, H, dim], dim 128 or 512, tokens any stride apart), norm_w (fp32 [dim] or
    None), norm (True with norm_w, else False), eps (1e-6), rotate (False), and either out (bf16 [T, H, dim], None: a
    new tensor; may be x) or cache (a PagedCache of that dim, H = 1) with slot (int64 [T],
    physical rows, < 0: skipped).  rope_cs: fp32 [T, 32, 2] (needed where a job rotates).  What a
    job writes no other job of the call reads or writes.
    Returns the list of outs (None for jobs with a cache)."""
    import torch
    if not 1 <= len(jobs) <= 4:
        raise ValueError("1 to 4 jobs, got %d" % len(jobs))
    x = jobs[0]["x"]
    T, dev = x.shape[0], x.device
    pc = _take("rope_cs", rope_cs, torch.float32, (T, 32, 2), dev)
    arr, outs = _NORM_ARRAYS[len(jobs)](), []
    for a, j in zip(arr, jobs):
        x = j["x"]
        a.x, a.x_stride = _heads("x", x, T, dev)
        a.H, a.dim = x.shape[1], x.shape[2]
        w = j.get("norm_w")
        if w is not None and not j.get("norm", True):
            raise ValueError("norm_w without norm")
        a.norm, a.eps, a.rotate = bool(j.get("norm", w is not None)), j.get("eps", 1e-6), bool(j.get("rotate"))
        a.norm_w = _take("norm_w", w, torch.float32, (a.dim,), dev)
        cache, out = j.get("cache"), j.get("out")
        if cache is not None:
            if out is not None:
                raise ValueError("a job has out or cache")
            if j.get("slot") is None:
                raise ValueError("cache needs slot")
            a.slot = _take("slot", j["slot"], torch.int64, (T,), dev)
            a.cache = _cache_on("cache", cache, 0, dev)
        else:
            if j.get("slot") is not None:
                raise ValueError("slot needs cache")
            if out is None:
                out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
            elif out.shape != x.shape:
                raise ValueError("out must have shape %s, got %s" % (tuple(x.shape), tuple(out.shape)))
            a.out, a.out_stride = _heads("out", out, T, dev)
        outs.append(out)
    _check(_lib.lib().cskvs_norm_rope(arr, len(jobs), pc, T, _raw_stream(dev)), "cskvs_norm_rope")
    return outs


def chunk_attn_max_keys(R, T, max_entries, window, max_ctx_len):
    """A bound of the keys that chunk_attn decodes, whatever the lengths."""
    return int(_lib.lib().cskvs_chunk_attn_max_keys(R, T, max_entries, window, max_ctx_len))


def chunk_attn_workspace_size(R, T, H, max_keys):
    return int(_lib.lib().cskvs_chunk_attn_workspace_size(R, T, H, max_keys))


@_on_stream
def chunk_attn(q, cu_q, ctx_len, entries, ratio, max_entries, max_ctx_len, sink, softmax_scale, q_rope_cs,
               n_entries=None, rows=None, window=0, max_keys=None, out=None, lse=None, want_lse=False, workspace=None,
               stream=None):
    """Attention of chunks of new tokens: the queries cu_q[r] .. cu_q[r + 1] - 1 of q (bf16
    [T, H, 512]) are the last tokens of request r, whose length is ctx_len[r]; the one at position
    t sees the entries j < floor((t + 1) / ratio) of `entries` (a PagedCache; ratio 0: all
    n_entries[r]; never more than n_entries[r], if given) and, with rows (a PagedCache of raw
    rows by position), the last `window` rows up to its own.  q is normed but not rotated: the call
    turns it by q_rope_cs, and its output back.  max_keys: a tighter bound than chunk_attn_max_keys
    (the workspace holds 1 KB for each).  Returns (out bf16 [T, H, 512], lse fp32 [T, H] or None)."""
    import torch
    T, H, dev, pq = _query(q)
    i32, f32 = torch.int32, torch.float32
    R = cu_q.shape[0] - 1
    pu = _take("cu_q", cu_q, i32, (R + 1,), dev)
    px = _take("ctx_len", ctx_len, i32, (R,), dev)
    pn = _take("n_entries", n_entries, i32, (R,), dev)
    ps = _take("sink", sink, f32, (H,), dev)
    pc = _take("q_rope_cs", q_rope_cs, f32, (T, 32, 2), dev)
    de = None if entries is None else ctypes.byref(_cache_on("entries", entries, R, dev))
    dr = None if rows is None else ctypes.byref(_cache_on("rows", rows, R, dev))
    out, lse, po, pl = _outputs(q, T, H, dev, out, lse, want_lse)
    L = _lib.lib()
    if max_keys is None:
        max_keys = L.cskvs_chunk_attn_max_keys(R, T, max_entries if entries is not None else 0, window, max_ctx_len)
    need = 0 if workspace is not None else L.cskvs_chunk_attn_workspace_size(R, T, H, max_keys)
    workspace, pw, nw = _workspace(workspace, need, dev)
    _check(L.cskvs_chunk_attn(pq, pu, px, R, T, H, de, ratio, pn, max_entries, dr, window, max_ctx_len, ps,
                              softmax_scale, pc, po, pl, max_keys, pw, nw, _raw_stream(dev)), "cskvs_chunk_attn")
    return out, lse


DEFAULT_SCALE = 1.0 / math.sqrt(512.0)
