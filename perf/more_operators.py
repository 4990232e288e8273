"""One step of a server of compressed-KV layers, from request lengths to attention.

Four operators:

* ``plan``   block tables, slot maps and positions of a step's tokens, made on the GPU from the
             requests' lengths;
* ``rope``   the (cos, sin) table of positions that are on the GPU, with one or several axes;
* ``norm``   norms of queries and rows for each head with the rotation in the same pass, rows coded
             into their cache;
* ``chunk``  attention of a chunk of new tokens over all visible entries of a paged cache (causal, or
             to states of another length) and a window of raw rows.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits; angles in
64), with ``own`` true the framework's calls.  ``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

D = 512
PAGE = 64
RING = 128
EPS = 1e-6
SCALE = 1.0 / math.sqrt(512.0)
THETA = 160000.0
BF16, FP8, FP4 = 0, 1, 2
ROW_BYTES = {BF16: 1024, FP8: 528, FP4: 288}
FORMATS = {"bf16": BF16, "fp8": FP8, "fp4": FP4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# pairs of the 32 that follow each axis: one axis; time, height and width of a video
SECTIONS = {1: (32,), 2: (16, 16), 3: (16, 8, 8)}


# ---------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 requests, raw rows, a few idle: latency
        {"name": "plan decode step", "op": "plan", "B": 64, "T": 64, "ctx": 32768, "ratio": 1, "ring": True},
        # prompts of 23 requests in one step, entries of ratio 4
        {"name": "plan ragged prompts", "op": "plan", "B": 23, "T": 8191, "ctx": 20000, "ratio": 4, "ring": True},
        # a large step of a large server
        {"name": "plan large step", "op": "plan", "B": 512, "T": 262144, "ctx": 65536, "ratio": 1, "ring": False},
        # the positions of a decode step
        {"name": "rope decode step", "op": "rope", "T": 64, "axes": 1, "far": 1048576},
        # a long video: time, height and width of every patch
        {"name": "rope video", "op": "rope", "T": 131071, "axes": 3, "far": 4096},
        # a decode step's queries, index queries and window rows: latency
        {"name": "norm decode step", "op": "norm", "T": 8, "H": 64, "Hi": 64, "fmt": "fp8", "gap": 512},
        # an odd number of prompt tokens, few heads, rows kept as they are
        {"name": "norm ragged prompts", "op": "norm", "T": 1037, "H": 20, "Hi": 0, "fmt": "bf16", "gap": 8},
        # a prompt chunk of 8,192 tokens
        {"name": "norm prompt chunk", "op": "norm", "T": 8192, "H": 64, "Hi": 64, "fmt": "fp8", "gap": 512},
        # a few tokens of one request behind 20,000 tokens at ratio 128: latency
        {"name": "chunk few tokens", "op": "chunk", "R": 1, "T": 5, "H": 16, "ctx": 20000, "ratio": 128, "window": 128,
         "fmt": "fp8", "rows": "fp8", "sink": True},
        # three prompts, every token sees all before it, odd sizes throughout
        {"name": "chunk ragged prompts", "op": "chunk", "R": 3, "T": 1037, "H": 20, "ctx": 1500, "ratio": 1, "window": 0,
         "fmt": "bf16", "rows": "bf16", "sink": False},
        # sixteen requests' tokens on encoder states of another length
        {"name": "chunk on encoder states", "op": "chunk", "R": 16, "T": 640, "H": 32, "ctx": 2000, "ratio": 0, "window": 0,
         "fmt": "fp4", "rows": "bf16", "sink": True},
        # the last chunk of a prompt of 1,048,576 tokens at ratio 128, with the 128-token window
        {"name": "chunk of a million tokens", "op": "chunk", "R": 1, "T": 4096, "H": 64, "ctx": 1048576, "ratio": 128,
         "window": 128, "fmt": "fp8", "rows": "fp8", "sink": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "norm", "chunk", "chunk", "chunk"])
    if op == "plan":
        B = _log(rng, 1, 512)
        T = B if rng.random() < 0.4 else max(B, _log(rng, 100, 200000))
        return {"op": op, "B": B, "T": T, "ctx": _log(rng, 100, 65536), "ratio": rng.choice([1, 2, 4, 128]),
                "ring": rng.random() < 0.5}
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 131071), "axes": rng.randint(1, 3), "far": _log(rng, 100, 1048576)}
    if op == "norm":
        H, Hi = rng.choice([1, 5, 16, 20, 32, 64, 128]), rng.choice([0, 0, 1, 8, 64])
        T = min(_log(rng, 1, 8192), 8192 * 80 // (H + Hi // 4))
        return {"op": op, "T": T, "H": H, "Hi": Hi, "fmt": rng.choice(["bf16", "fp8", "fp4"]),
                "gap": rng.choice([0, 8, 136, 512])}
    H = rng.choice([1, 5, 8, 16, 20, 32, 48, 64, 96, 128])
    R = _log(rng, 1, 16)
    ratio = rng.choice([0, 1, 4, 128, 128])
    ctx = _log(rng, 300, {0: 4096, 1: 8192, 4: 32768, 128: 1048576}[ratio])
    keys = ctx // max(ratio, 1) + 130
    T = max(R, min(_log(rng, 1, 4096), ctx * R // 2 if ratio else 4096, 1000000000 // (H * keys)))
    return {"op": op, "R": R, "T": T, "H": H, "ctx": ctx, "ratio": ratio,
            "window": rng.choice([0, 1, 100, 128, 128, 1000]) if ratio else 0,
            "fmt": rng.choice(["bf16", "fp8", "fp4"]), "rows": rng.choice(["bf16", "fp8"]), "sink": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _code_rows(x, fmt):
    """Values [n, 512] -> the bytes of their cache rows, uint8 [n, row bytes]."""
    if fmt == BF16:
        return x.to(torch.bfloat16).view(torch.uint8)
    if fmt == FP8:
        xb = x.unflatten(-1, (16, 32))
        a = xb.abs().amax(-1)
        # the smallest 2^e with a <= 448 2^e
        m, e = torch.frexp(a)
        e = torch.where(a > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.zeros_like(e)).clamp(-127, 127)
        codes = torch.ldexp(xb, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return torch.cat([codes.flatten(-2), (e + 127).to(torch.uint8)], -1)
    xb = x.unflatten(-1, (32, 16))
    sc = (xb.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    s = sc.float()[..., None]
    y = torch.where(s > 0, xb / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(xb))
    # to the nearest of the eight values, halves to the even code
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.int32)
    for i, (edge, up) in enumerate(((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                                    (5.0, False))):
        code = code + ((a >= edge) if up else (a > edge)).int()
    nib = (code | (torch.signbit(y) & (s > 0)).int() << 3).flatten(-2).unflatten(-1, (D // 2, 2))
    return torch.cat([(nib[..., 0] | (nib[..., 1] << 4)).to(torch.uint8), sc.view(torch.uint8)], -1)


def _pool(gen, pages, fmt):
    """A pool of `pages` pages of coded N(0, 1) rows."""
    rb = ROW_BYTES[fmt]
    pool = torch.empty((pages, PAGE * rb), dtype=torch.uint8, device="cuda")
    for p in range(0, pages, 4096):
        m = min(4096, pages - p)
        x = torch.randn((m * PAGE, D), generator=gen, device="cuda")
        pool[p:p + m] = _code_rows(x, fmt).view(m, PAGE * rb)
    return pool


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _shares(gen, n, total):
    """int64 [n] of random sizes, 1 at least, with the sum `total`."""
    w = torch.rand((n,), generator=gen, device="cuda") + 0.1
    cut = torch.round(torch.cumsum(w, 0) / w.sum() * (total - n)).long()
    cut[-1] = total - n
    return torch.diff(cut, prepend=torch.zeros_like(cut[:1])) + 1


def _speeds():
    k = torch.arange(32, dtype=torch.float64, device="cuda")
    return THETA ** (-k / 32.0)


def _axis_of(axes):
    return torch.repeat_interleave(torch.arange(axes), torch.tensor(SECTIONS[axes])).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev, i32 = "cuda", torch.int32
    s = {"case": case, "op": case["op"]}
    if case["op"] == "plan":
        B, T, r, ctx = case["B"], case["T"], case["ratio"], case["ctx"]
        have = torch.randint(0, ctx + 1, (B,), generator=gen, device=dev)
        b = torch.arange(B, device=dev)
        if T == B:          # one token each; every ninth request waits
            new = torch.where(b % 9 == 5, torch.zeros_like(b), torch.ones_like(b))
        else:               # nine tenths of the places are used
            new = _shares(gen, B, max(B, T * 9 // 10))
        done = b % 8 == 3   # requests that end with this step
        s["ctx"] = have.to(i32)
        s["new"] = torch.where(done, torch.full_like(new, -1), new).to(i32)
        rows0 = have // r
        # two pages more than a request that takes every new token would need
        s["max_pages"] = _pages((ctx + T) // r) + 1 if B <= 32 else _pages(ctx // r) + _pages(12 * T // B // r) + 2
        used = (rows0 + PAGE - 1) // PAGE
        total = B * s["max_pages"]
        perm = torch.randperm(total, generator=gen, device=dev).to(i32)
        lp = torch.arange(s["max_pages"], device=dev)[None]
        start = (torch.cumsum(used, 0) - used)[:, None]
        s["table"] = torch.where(lp < used[:, None], perm[(start + lp).clamp(max=total - 1)], torch.full_like(perm[:1], -1))
        s["table"] = s["table"].contiguous()
        # the free pages, somewhere in their ring
        n_used = used.sum()
        head = torch.randint(0, total, (1,), generator=gen, device=dev)
        at = (head + torch.arange(total, device=dev)) % total
        src = n_used + torch.arange(total, device=dev)
        free = torch.full((total,), -1, dtype=i32, device=dev)
        free[at] = torch.where(src < total, perm[src.clamp(max=total - 1)], torch.full_like(perm, -1))
        s["free"] = free
        s["state"] = torch.stack([head[0], total - n_used, torch.zeros_like(n_used), torch.zeros_like(n_used)]).to(i32)
        s["state_out"] = torch.zeros((4,), dtype=i32, device=dev)
        return s
    if case["op"] == "rope":
        T, axes = case["T"], case["axes"]
        s["pos"] = torch.randint(0, case["far"], (axes, T), generator=gen, device=dev).to(i32)
        s["axis"], s["speeds"] = _axis_of(axes), _speeds()
        s["sections"] = SECTIONS[axes]
        return s
    if case["op"] == "norm":
        T, H, Hi, fmt = case["T"], case["H"], case["Hi"], FORMATS[case["fmt"]]
        s["fmt"] = fmt
        # slices of what one projection wrote: queries, index queries, the row, and something behind
        buf = (1.5 * torch.randn((T, H * D + Hi * 128 + D + case["gap"]), generator=gen, device=dev)).to(torch.bfloat16)
        s["q"] = buf[:, :H * D].unflatten(1, (H, D))
        s["qi"] = buf[:, H * D:H * D + Hi * 128].unflatten(1, (Hi, 128)) if Hi else None
        s["kv"] = buf[:, H * D + Hi * 128:H * D + Hi * 128 + D].unflatten(1, (1, D))
        s["w"] = torch.rand((D,), generator=gen, device=dev) + 0.5
        a = torch.randint(0, 1048576, (T,), generator=gen, device=dev).double()[:, None] * _speeds()
        s["cs"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
        pages = _pages(T) + 1
        s["pool"] = torch.zeros((pages, PAGE * ROW_BYTES[fmt]), dtype=torch.uint8, device=dev)
        slot = torch.randperm(pages * PAGE, generator=gen, device=dev)[:T]
        s["slot"] = torch.where(torch.arange(T, device=dev) % 16 == 7, torch.full_like(slot, -1), slot)   # padding
        s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        s["out_i"] = torch.empty((T, Hi, 128), dtype=torch.bfloat16, device=dev) if Hi else None
        return s
    R, T, H, ctx, r = case["R"], case["T"], case["H"], case["ctx"], case["ratio"]
    new = _shares(gen, R, T)
    s["most_new"] = int(new.max())
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    s["cu"] = cu.to(i32)
    # lengths behind the chunk: ragged, ctx the longest, none shorter than its chunk
    less = torch.randint(0, max(1, ctx // 3), (R,), generator=gen, device=dev)
    less[0] = 0
    if r:
        s["len"] = torch.maximum(ctx - less, new).to(i32)
        s["max_ctx"] = max(ctx, s["most_new"])
        s["n"], s["max_entries"] = None, s["max_ctx"] // r
    else:
        s["len"], s["max_ctx"] = new.to(i32), s["most_new"]
        s["n"], s["max_entries"] = (ctx - less).to(i32), ctx
    pages = max(1, _pages(s["max_entries"]))
    s["fmt"] = FORMATS[case["fmt"]]
    s["pool"] = _pool(gen, R * pages, s["fmt"])
    s["bt"] = torch.randperm(R * pages, generator=gen, device=dev).to(i32).view(R, pages).contiguous()
    if case["window"]:
        # raw rows: of the pages before the window nothing is left but the table's entries
        s["rfmt"] = FORMATS[case["rows"]]
        all_pages = _pages(s["max_ctx"])
        keep = min(all_pages, _pages(s["most_new"] + case["window"]) + 1)
        s["rpool"] = _pool(gen, R * keep, s["rfmt"])
        perm = torch.randperm(R * keep, generator=gen, device=dev).to(i32).view(R, keep)
        last = ((s["len"].long() + PAGE - 1) // PAGE)[:, None]
        lp = torch.arange(all_pages, device=dev)[None]
        s["rbt"] = perm.gather(1, (lp - last + keep).clamp(0, keep - 1)).contiguous()
    req = torch.repeat_interleave(torch.arange(R, device=dev), new, output_size=T)
    pos = (s["len"].long() - new)[req] + torch.arange(T, device=dev) - cu[req]
    s["pos1"] = (pos + 1).to(i32)
    a = pos.double()[:, None] * _speeds()
    s["cs"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
    s["q"] = (2.0 * torch.randn((T, H, D), generator=gen, device=dev)).to(torch.bfloat16)
    s["sink"] = torch.randn((H,), generator=gen, device=dev) if case["sink"] else None
    return s


# ---------------------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------------------

def _plain_plan(s):
    c = s["case"]
    B, T, r, P = c["B"], c["T"], c["ratio"], s["max_pages"]
    ctx, new = s["ctx"].long(), s["new"].long()
    done = new < 0
    n = new.clamp(min=0)
    end = torch.cumsum(n, 0)
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    after = torch.where(done, torch.zeros_like(ctx), ctx + n)
    rows0 = torch.where(done, torch.zeros_like(ctx), ctx // r)
    rows1 = after // r
    used = (ctx // r + PAGE - 1) // PAGE
    first, last = (rows0 + PAGE - 1) // PAGE, (rows1 + PAGE - 1) // PAGE
    need, give = last - first, torch.where(done, used, torch.zeros_like(used))
    cap = s["free"].shape[0]
    head, count = s["state"][0].long(), s["state"][1].long()
    lp = torch.arange(P, device="cuda")[None]
    k = (torch.cumsum(need, 0) - need - first)[:, None] + lp
    fresh = (lp >= first[:, None]) & (lp < last[:, None])
    page = torch.where(k < count, s["free"][(head + k) % cap], torch.full_like(k, -1).int())
    j = (torch.cumsum(give, 0) - give)[:, None] + lp
    back = torch.where(lp < give[:, None], (head + count + j) % cap, torch.full_like(j, cap))
    free = torch.cat([s["free"], s["free"][:1]]).scatter(0, back.flatten(), s["table"].flatten())[:cap]
    s["free"].copy_(free)
    s["table"].copy_(torch.where(fresh, page, s["table"]))
    taken = torch.minimum(need.sum(), count)
    state = torch.stack([(head + taken) % cap, count - taken + give.sum(), need.sum() - taken, torch.zeros_like(taken)])
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(end, i, right=True).clamp(max=B - 1)
    live = i < end[-1]
    pos = ctx[b] + i - cu[b]
    row = (pos + 1) // r - 1
    p = s["table"][b, (row // PAGE).clamp(0, P - 1)].long()
    slot = torch.where(live & ((pos + 1) % r == 0) & (p >= 0), p * PAGE + row % PAGE, torch.full_like(p, -1))
    none = torch.full_like(i, -1)
    out = {"cu": cu.int(), "len": after.int(), "first_row": rows0.int(), "n_rows": rows1.int(),
           "req": torch.where(live, b, none).int(), "pos1": torch.where(live, pos + 1, torch.zeros_like(i)).int(),
           "slot": slot, "table": s["table"], "free": s["free"], "state": state.int()}
    if c["ring"]:
        out["ring_slot"] = torch.where(live & (pos >= after[b] - RING), b * RING + pos % RING, none)
    return out


def _plain_rope(s):
    a = s["pos"].double()[s["axis"]].t() * s["speeds"]
    return torch.stack([a.cos(), a.sin()], -1).float()


def _halves(x):
    """Sum over the last axis, neighbours first: x[2i] + x[2i + 1], again until one is left."""
    n = x.shape[-1]
    return x[..., 0] if n == 1 else _halves(x[..., 0::2] + x[..., 1::2])


def _turn(x, cs, back=False):
    """The last 64 dims turned by the table (..., 32, 2), forth or back."""
    c, s = cs[..., 0], cs[..., 1] * (-1.0 if back else 1.0)
    n = x.shape[-1] - 64
    y = x[..., n:].unflatten(-1, (32, 2))
    y0, y1 = y[..., 0], y[..., 1]
    return torch.cat([x[..., :n], torch.stack([y0 * c - y1 * s, y0 * s + y1 * c], -1).flatten(-2)], -1)


def _normed(x, w):
    x = x.float()
    r = 1.0 / torch.sqrt(_halves(x * x) / x.shape[-1] + EPS)
    y = x * r[..., None]
    return y if w is None else y * w


def _shown(pool, fmt):
    """A pool's rows as the values they hold: bf16; codes and scales of the other formats."""
    rows = pool.view(-1, PAGE, ROW_BYTES[fmt])
    if fmt == BF16:
        return {"rows": rows.view(torch.bfloat16)}
    if fmt == FP8:
        return {"codes": rows[..., :D].view(torch.float8_e4m3fn), "scales": rows[..., D:]}
    return {"codes": rows[..., :D // 2], "scales": rows[..., D // 2:].view(torch.float8_e4m3fn)}


def _plain_norm(s):
    cs = s["cs"][:, None]
    out = {"q": _normed(s["q"], None).to(torch.bfloat16)}
    if s["qi"] is not None:
        out["qi"] = _turn(s["qi"].float(), cs).to(torch.bfloat16)
    row = _code_rows(_turn(_normed(s["kv"], s["w"]), cs)[:, 0], s["fmt"])
    pool = s["pool"].view(-1, ROW_BYTES[s["fmt"]])
    # padding rows go behind the pool
    more = torch.cat([pool, pool[:1]])
    more[torch.where(s["slot"] < 0, torch.full_like(s["slot"], pool.shape[0]), s["slot"])] = row
    pool.copy_(more[:-1])
    return {**out, **_shown(s["pool"], s["fmt"])}


def _values(raw, fmt):
    """Row bytes [..., row bytes] -> fp32 values [..., 512]."""
    if fmt == BF16:
        return raw.view(torch.bfloat16).float()
    if fmt == FP8:
        v = raw[..., :D].contiguous().view(torch.float8_e4m3fn).float()
        return (v.unflatten(-1, (16, 32)) * torch.exp2(raw[..., D:].float() - 127.0)[..., None]).flatten(-2)
    c = raw[..., :D // 2].int()
    nib = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    mag = torch.tensor(E2M1, device=raw.device)[nib & 7]
    v = torch.where(nib >= 8, -mag, mag).unflatten(-1, (32, 16))
    return (v * raw[..., D // 2:].contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _gather(pool, bt, req, row, fmt):
    """fp32 values of rows `row` of requests `req` (same shapes)."""
    page = bt[req, row // PAGE].long()
    return _values(pool.view(-1, ROW_BYTES[fmt])[page * PAGE + row % PAGE], fmt)


def _plain_chunk(s):
    c = s["case"]
    R, T, H, r, window, most = c["R"], c["T"], c["H"], c["ratio"], c["window"], s["most_new"]
    cu, length = s["cu"].long(), s["len"].long()
    req = torch.arange(R, device="cuda")[:, None]
    n = cu[1:] - cu[:-1]
    # queries by request, padded to the longest chunk
    i = torch.arange(most, device="cuda")[None]
    live = i < n[:, None]
    at = (cu[:-1, None] + i).clamp(max=T - 1)
    pos1 = (length - n)[:, None] + i + 1
    q = _turn(s["q"].float(), s["cs"][:, None])[at]
    E = s["max_entries"]
    e = torch.arange(E, device="cuda").expand(R, E)
    kv = _gather(s["pool"], s["bt"], req.expand(R, E), e, s["fmt"])
    visible = pos1 // r if r else s["n"].long()[:, None].expand_as(pos1)
    see = e[:, None] < visible[..., None]
    if window:
        W = min(s["max_ctx"], most + window - 1)
        row = (length[:, None] - W) + torch.arange(W, device="cuda")[None]
        rows = _gather(s["rpool"], s["rbt"], req.expand(R, W), row.clamp(min=0), s["rfmt"])
        kv = torch.cat([kv, rows], 1)
        row = row[:, None]
        see = torch.cat([see, (row >= 0) & (row < pos1[..., None]) & (row >= pos1[..., None] - window)], -1)
    z = torch.bmm(q.flatten(1, 2), kv.transpose(1, 2)).unflatten(1, (most, H)) * SCALE
    z = z.masked_fill(~see[:, :, None], -math.inf)
    sink = s["sink"]
    m = z.amax(-1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(z - m[..., None])
    total = p.sum(-1)
    if sink is not None:
        total = total + torch.exp(sink - m)
    o = torch.bmm(p.flatten(1, 2), kv).unflatten(1, (most, H))
    o = torch.where((total > 0)[..., None], o / total[..., None], torch.zeros_like(o))
    lse = m + torch.log(total)
    # back to the tokens' order
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    o, lse = o[b, t - cu[b]], lse[b, t - cu[b]]
    return _turn(o, s["cs"][:, None], back=True).to(torch.bfloat16), lse


def _own_run(s):
    import compressed_sparse_attention_kv_gb300 as cskv
    c = s["case"]
    if s["op"] == "plan":
        pages = cskv.PageTable(s["table"], s["free"], s["state"])
        m = cskv.plan_step(s["ctx"], s["new"], c["T"], pages, ratio=c["ratio"], ring_rows=RING if c["ring"] else 0,
                           state_out=s["state_out"])
        out = {"cu": m.cu_new, "len": m.new_len, "first_row": m.first_row, "n_rows": m.n_rows, "req": m.req_of,
               "pos1": m.pos1, "slot": m.slot, "table": s["table"], "free": s["free"], "state": s["state_out"]}
        if c["ring"]:
            out["ring_slot"] = m.ring_slot
        return out
    if s["op"] == "rope":
        if "plan" not in s:     # made once by a program
            s["plan"] = cskv.RopePlan(THETA, sections=s["sections"])
        return cskv.rope_cs(s["pos"], s["plan"])
    if s["op"] == "norm":
        cache = cskv.PagedCache(s["pool"], None, s["fmt"], D)
        jobs = [dict(x=s["q"], norm=True, eps=EPS, out=s["out"]),
                dict(x=s["kv"], norm=True, norm_w=s["w"], eps=EPS, rotate=True, cache=cache, slot=s["slot"])]
        if s["qi"] is not None:
            jobs.append(dict(x=s["qi"], rotate=True, out=s["out_i"]))
        cskv.norm_rope(jobs, s["cs"])
        out = {"q": s["out"], **_shown(s["pool"], s["fmt"])}
        if s["qi"] is not None:
            out["qi"] = s["out_i"]
        return out
    rows = cskv.PagedCache(s["rpool"], s["rbt"], s["rfmt"], D) if c["window"] else None
    return cskv.chunk_attn(s["q"], s["cu"], s["len"], cskv.PagedCache(s["pool"], s["bt"], s["fmt"], D), c["ratio"],
                           s["max_entries"], s["max_ctx"], s["sink"], SCALE, s["cs"], n_entries=s["n"], rows=rows,
                           window=c["window"], want_lse=True)


def run(state):
    if own:
        return _own_run(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "norm": _plain_norm, "chunk": _plain_chunk}[state["op"]](state)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "plan":
        pages = T / case["ratio"] / PAGE + case["B"] / 8 * case["ctx"] / 2 / case["ratio"] / PAGE
        return {"bytes": T * (4 + 4 + 8 + (8 if case["ring"] else 0)) + case["B"] * 24 + pages * 8, "flops": T * 4}
    if op == "rope":
        return {"bytes": T * (4 * case["axes"] + 256), "flops": T * 32 * 20}
    if op == "norm":
        values = T * (case["H"] * D + case["Hi"] * 128)
        return {"bytes": values * 4 + T * (2 * D + ROW_BYTES[FORMATS[case["fmt"]]] + 256 + 8), "flops": values * 4}
    R, H, r, window, ctx = case["R"], case["H"], case["ratio"], case["window"], case["ctx"]
    # lengths are ragged: a sixth less than ctx in the mean, for all requests but the longest
    mean = ctx if R == 1 else ctx * 5 / 6
    entries = max(0.0, mean - T / R / 2) / r if r else mean
    seen = entries + min(window, mean)
    rows = R * (mean / max(r, 1) * ROW_BYTES[FORMATS[case["fmt"]]]
                + (min(mean, window + T / R) * ROW_BYTES[FORMATS[case["rows"]]] if window else 0))
    return {"bytes": T * H * (2048 + 4) + T * 256 + rows, "flops": T * H * seen * 4 * D}


# ---------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------

def _exact_row_values(raw, fmt):
    """Row bytes [n, row bytes] -> float64 [n, 512], from the bits of the formats."""
    b = raw.long()
    n = b.shape[0]

    def small_float(code, ebits, mbits, bias):
        e, f = (code >> mbits) & ((1 << ebits) - 1), code & ((1 << mbits) - 1)
        mag = torch.where(e == 0, f.double() * 2.0 ** (1 - bias - mbits),
                          (f + (1 << mbits)).double() * torch.exp2((e - bias - mbits).double()))
        return torch.where((code >> (ebits + mbits)) & 1 == 1, -mag, mag)

    if fmt == BF16:
        return small_float(b[:, 0::2] | (b[:, 1::2] << 8), 8, 7, 127)
    if fmt == FP8:
        step = torch.exp2(b[:, D:].double() - 127.0)
        return small_float(b[:, :D], 4, 3, 7) * step.repeat_interleave(32, 1)
    codes = torch.empty((n, D), dtype=torch.long, device=raw.device)
    codes[:, 0::2] = b[:, :D // 2] & 15
    codes[:, 1::2] = b[:, :D // 2] >> 4
    return small_float(codes, 2, 1, 1) * small_float(b[:, D // 2:], 4, 3, 7).repeat_interleave(16, 1)


def _exact_rotation(x, cs, sign):
    w = torch.view_as_complex(cs.double().contiguous())
    if sign < 0:
        w = w.conj()
    y = x.clone()
    n = x.shape[-1] - 64
    tail = torch.view_as_complex(x[..., n:].reshape(x.shape[:-1] + (32, 2)).contiguous()) * w
    y[..., n:] = torch.view_as_real(tail).flatten(-2)
    return y


def _exact_plan(case, s):
    ctx, new, r = s["ctx"].tolist(), s["new"].tolist(), case["ratio"]
    table, free = s["table"].cpu(), s["free"].cpu()
    cap, (head, count) = free.shape[0], s["state"].tolist()[:2]
    T, back = case["T"], []
    cu, length, first, rows = [0], [], [], []
    req, pos1, slot, ring = [-1] * T, [0] * T, [-1] * T, [-1] * T
    taken = short = 0
    for b, (have, n) in enumerate(zip(ctx, new)):
        if n < 0:
            back += table[b, :_pages(have // r)].tolist()
            cu.append(cu[-1])
            length.append(0)
            first.append(0)
            rows.append(0)
            continue
        for lp in range(_pages(have // r), _pages((have + n) // r)):
            if taken < count:
                table[b, lp] = free[(head + taken) % cap]
                taken += 1
            else:
                table[b, lp] = -1
                short += 1
        line = table[b].tolist()
        for p in range(have, have + n):
            i = cu[-1] + p - have
            req[i], pos1[i] = b, p + 1
            if (p + 1) % r == 0 and line[(p + 1) // r - 1 >> 6] >= 0:
                slot[i] = line[(p + 1) // r - 1 >> 6] * PAGE + ((p + 1) // r - 1) % PAGE
            if p >= have + n - RING:
                ring[i] = b * RING + p % RING
        cu.append(cu[-1] + n)
        length.append(have + n)
        first.append(have // r)
        rows.append((have + n) // r)
    for j, p in enumerate(back):
        free[(head + count + j) % cap] = p
    state = [(head + taken) % cap, count - taken + len(back), short, 0]

    def of(x, t=torch.int32):
        return torch.tensor(x, dtype=t, device="cuda")

    out = {"cu": of(cu), "len": of(length), "first_row": of(first), "n_rows": of(rows), "req": of(req), "pos1": of(pos1),
           "slot": of(slot, torch.int64), "table": table.cuda(), "free": free.cuda(), "state": of(state)}
    if case["ring"]:
        out["ring_slot"] = of(ring, torch.int64)
    return out


def _exact_norm(case, s):
    def rms(x, w=None):
        y = x.double()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
        return y if w is None else y * w.double()

    out = {"q": rms(s["q"])}
    cs = s["cs"][:, None]
    if s["qi"] is not None:
        out["qi"] = _exact_rotation(s["qi"].double(), cs, +1)
    row = _exact_rotation(rms(s["kv"], s["w"]), cs, +1)[:, 0]
    there = s["slot"] >= 0
    at, fmt = s["slot"][there], s["fmt"]
    if fmt == BF16:
        rows = torch.zeros((s["pool"].shape[0] * PAGE, D), dtype=torch.float64, device="cuda")
        rows[at] = row[there]
        return {**out, "rows": rows.view(-1, PAGE, D)}
    pool = s["pool"].view(-1, ROW_BYTES[fmt]).clone()
    pool[at] = _code_rows(row[there].float(), fmt)
    shown = _shown(pool, fmt)
    return {**out, **{k: v.double() if v.dtype == torch.float8_e4m3fn else v for k, v in shown.items()}}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(case, s)
    if op == "rope":
        turns = torch.empty((case["T"], 32, 2), dtype=torch.float64, device="cuda")
        k = 0
        for axis, pairs in enumerate(SECTIONS[case["axes"]]):
            for _ in range(pairs):
                a = s["pos"][axis].double() * float(THETA) ** (-2.0 * k / 64.0)
                turns[:, k, 0], turns[:, k, 1] = torch.cos(a), torch.sin(a)
                k += 1
        return turns
    if op == "norm":
        return _exact_norm(case, s)
    R, T, H, r, window = case["R"], case["T"], case["H"], case["ratio"], case["window"]
    if T * H * (s["max_entries"] + window) > 3e9:
        return None
    out = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
    cu, length = s["cu"].tolist(), s["len"].tolist()

    def rows_of(pool, bt, fmt, b, lo, hi):
        j = torch.arange(lo, hi, device="cuda")
        return _exact_row_values(pool.view(-1, ROW_BYTES[fmt])[bt[b].long()[j // PAGE] * PAGE + j % PAGE], fmt)

    for b in range(R):
        n = cu[b + 1] - cu[b]
        start = length[b] - n
        visible = length[b] // r if r else int(s["n"][b])
        entries = rows_of(s["pool"], s["bt"], s["fmt"], b, 0, visible)
        low = max(0, start - window + 1)
        raw = rows_of(s["rpool"], s["rbt"], s["rfmt"], b, low, length[b]) if window else None
        step = max(1, 30000000 // (H * (visible + window + 1)))
        for i in range(0, n, step):
            k = min(n, i + step)
            t = torch.arange(start + i, start + k, device="cuda")
            x = slice(cu[b] + i, cu[b] + k)
            q = _exact_rotation(s["q"][x].double(), s["cs"][x][:, None], +1)
            keys = entries
            see = torch.arange(visible, device="cuda") < ((t + 1) // r)[:, None] if r else \
                torch.ones((k - i, visible), dtype=torch.bool, device="cuda")
            if window:
                lo = max(0, start + i - window + 1)
                j = torch.arange(lo, start + k, device="cuda")
                keys = torch.cat([entries, raw[lo - low:start + k - low]])
                see = torch.cat([see, (j <= t[:, None]) & (j > t[:, None] - window)], 1)
            z = torch.where(see[:, None], (q @ keys.t()) * SCALE, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            if s["sink"] is not None:
                z = torch.cat([z, s["sink"].double()[None, :, None].expand(k - i, -1, 1)], -1)
            lse[x] = torch.logsumexp(z, -1)
            p = torch.exp(z - lse[x][..., None])[..., :keys.shape[0]]
            p = torch.where(torch.isfinite(lse[x])[..., None], p, torch.zeros_like(p))
            out[x] = _exact_rotation(p @ keys, s["cs"][x][:, None], -1)
    return out, lse
