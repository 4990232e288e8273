"""Operators over bounded and shared caches, as a server of compressed-KV layers calls them.

Four operators, all on paged caches of 512-d rows that are key and value of every head:

* ``window``   attention over a sliding window and the first rows of a request (raw rows by
               position), for prompt chunks and for single tokens;
* ``prefix``   decode attention of a batch whose requests share their first entries, each
               with entries of its own and a 128-slot window ring;
* ``weights``  each entry's attention weight, summed over the heads and accumulated;
* ``evict``    the entries of least accumulated weight leave, the survivors close the holes.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits), with
``own`` true the framework's calls.  ``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

D = 512
PAGE = 64
RING = 128
SCALE = 1.0 / math.sqrt(512.0)
BF16, FP8, FP4 = 0, 1, 2
ROW_BYTES = {BF16: 1024, FP8: 528, FP4: 288}
FORMATS = {"bf16": BF16, "fp8": FP8, "fp4": FP4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one request's next token on a layer without compression: latency
        {"name": "window one token", "op": "window", "T": 1, "reqs": 1, "H": 16, "ctx": 4096, "window": 128,
         "first": 4, "fmt": "bf16", "sink": True},
        # a decode batch of long requests on a layer with a long window
        {"name": "window decode batch", "op": "window", "T": 32, "reqs": 32, "H": 64, "ctx": 131072, "window": 4096,
         "first": 64, "fmt": "fp8", "sink": True},
        # prompts of three requests in one call, odd sizes throughout
        {"name": "window ragged prompts", "op": "window", "T": 1037, "reqs": 3, "H": 20, "ctx": 1500, "window": 1000,
         "first": 7, "fmt": "bf16", "sink": False},
        # a prompt of 8,192 tokens with the model's 128-token window
        {"name": "window prompt chunk", "op": "window", "T": 8192, "reqs": 1, "H": 64, "ctx": 8192, "window": 128,
         "first": 4, "fmt": "fp8", "sink": True},
        # two requests with a short common prompt: latency
        {"name": "prefix two requests", "op": "prefix", "B": 2, "H": 16, "prefix": 200, "tail": 37, "ring": False,
         "fmt": "bf16", "swa": "bf16", "sink": False},
        # 131,072 tokens at ratio 128, 7/8 of them a shared prompt
        {"name": "prefix batch of 32", "op": "prefix", "B": 32, "H": 64, "prefix": 896, "tail": 128, "ring": True,
         "fmt": "fp8", "swa": "fp8", "sink": True},
        # a shared prompt of 1,048,576 tokens at ratio 128, FP4 entries, 64 requests
        {"name": "prefix of a million tokens", "op": "prefix", "B": 64, "H": 64, "prefix": 8192, "tail": 512,
         "ring": True, "fmt": "fp4", "swa": "fp8", "sink": True},
        # one request's weights after a step: latency
        {"name": "weights one request", "op": "weights", "B": 1, "H": 16, "n": 1000, "first": 4, "fmt": "bf16"},
        # a batch of requests with 8,192 entries each
        {"name": "weights batch", "op": "weights", "B": 32, "H": 64, "n": 8192, "first": 0, "fmt": "fp8"},
        # a small cache cut to an odd budget
        {"name": "evict one request", "op": "evict", "B": 1, "n": 333, "budget": 200, "fixed": 4, "recent": 32,
         "caches": 1},
        # a batch that drops the page it has grown by
        {"name": "evict one page", "op": "evict", "B": 32, "n": 4160, "budget": 4096, "fixed": 64, "recent": 128,
         "caches": 1},
        # long caches cut to half
        {"name": "evict half", "op": "evict", "B": 8, "n": 65536, "budget": 32768, "fixed": 128, "recent": 4096,
         "caches": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "prefix", "prefix", "weights", "evict"])
    H = rng.choice([1, 5, 8, 16, 20, 32, 48, 64, 96, 128])
    fmt = rng.choice(["bf16", "fp8", "fp4"])
    if op == "window":
        fmt = rng.choice(["bf16", "fp8"])
        if rng.random() < 0.5:          # one token of each request
            T = reqs = _log(rng, 1, 64)
            ctx, window = _log(rng, 300, 32768), _log(rng, 1, 4096)
        else:                           # prompt chunks
            reqs = rng.randint(1, 4)
            window = _log(rng, 1, 1024)
            T = max(reqs + 1, min(_log(rng, 20, 4096), 64000000 // (H * (window + 130))))
            ctx = T + rng.randint(0, 2000)
        return {"op": op, "T": T, "reqs": reqs, "H": H, "ctx": ctx, "window": window,
                "first": rng.choice([0, 1, 4, 7, 64, 130]), "fmt": fmt, "sink": rng.random() < 0.5}
    if op == "prefix":
        return {"op": op, "B": min(_log(rng, 1, 64), 4096 // H), "H": H, "prefix": _log(rng, 1, 8192),
                "tail": _log(rng, 1, 512), "ring": rng.random() < 0.7, "fmt": fmt, "swa": rng.choice(["bf16", "fp8"]),
                "sink": rng.random() < 0.5}
    if op == "weights":
        return {"op": op, "B": _log(rng, 1, 32), "H": H, "n": _log(rng, 1, 8192), "first": rng.choice([0, 1, 64, 100]),
                "fmt": fmt}
    n = _log(rng, 2, 16384)
    budget = rng.randint(1, n)
    fixed = rng.randint(0, min(budget, 128))
    return {"op": op, "B": _log(rng, 1, 16), "n": n, "budget": budget, "fixed": fixed,
            "recent": rng.randint(0, budget - fixed), "caches": rng.randint(1, 2)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _code_rows(x, fmt):
    """Values [n, 512] -> the bytes of their cache rows, uint8 [n, row bytes]."""
    if fmt == BF16:
        return x.to(torch.bfloat16).view(torch.uint8)
    if fmt == FP8:
        xb = x.view(-1, 16, 32)
        e = torch.ceil(torch.log2(xb.abs().amax(-1) / 448.0)).clamp(-127, 127)
        codes = (xb * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return torch.cat([codes.reshape(-1, D), (e + 127).to(torch.uint8)], 1)
    xb = x.view(-1, 32, 16)
    sc = (xb.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = xb / sc.float().clamp(min=2.0 ** -9)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    nib = (torch.bucketize(y.abs(), edges) | ((y < 0).long() << 3)).reshape(-1, D // 2, 2)
    return torch.cat([(nib[..., 0] | (nib[..., 1] << 4)).to(torch.uint8), sc.view(torch.uint8)], 1)


def _pool(gen, pages, fmt):
    """A pool of `pages` pages of coded N(0, 1) rows."""
    rb = ROW_BYTES[fmt]
    pool = torch.empty((pages, PAGE * rb), dtype=torch.uint8, device="cuda")
    for p in range(0, pages, 4096):
        m = min(4096, pages - p)
        x = torch.randn((m * PAGE, D), generator=gen, device="cuda")
        pool[p:p + m] = _code_rows(x, fmt).view(m, PAGE * rb)
    return pool


def _rope(pos):
    """fp32 [..., 32, 2] (cos, sin) of positions (theta 160,000, 64 rotated dims)."""
    f = 160000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32.0)
    a = pos.double()[..., None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _pages(n):
    return (n + PAGE - 1) // PAGE


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"
    s = {"case": case, "op": case["op"]}
    i32 = torch.int32
    if case["op"] == "evict":
        B, n = case["B"], case["n"]
        pages = _pages(n)
        s["caches"] = [_pool(gen, B * pages, BF16) for _ in range(case["caches"])]
        s["bt"] = torch.randperm(B * pages, generator=gen, device=dev).to(i32).view(B, pages).contiguous()
        # weights of long use: heavy-tailed, with the zeros of entries that nothing looked at
        acc = torch.exp(2.0 * torch.randn((B, n), generator=gen, device=dev)) * 1e-3
        s["acc"] = torch.where(torch.rand((B, n), generator=gen, device=dev) < 0.05, torch.zeros_like(acc), acc)
        # births: the slots of the budget in the disorder that earlier calls left, then new ones in order
        m = case["budget"]
        age = torch.arange(n, device=dev, dtype=i32).repeat(B, 1)
        order = torch.argsort(torch.rand((B, m), generator=gen, device=dev), dim=1).to(i32)
        order[:, :case["fixed"]] = torch.arange(case["fixed"], device=dev, dtype=i32)
        age[:, :m] = order
        s["age"] = age.contiguous()
        # most requests are full, some have room left
        less = torch.randint(0, n, (B,), generator=gen, device=dev)
        s["n"] = torch.where(torch.arange(B, device=dev) % 4 == 3, n - less // 4, torch.full_like(less, n)).to(i32)
        s["acc_out"] = torch.zeros((B, m), device=dev)
        s["age_out"] = torch.zeros((B, m), dtype=i32, device=dev)
        s["n_out"] = torch.zeros((B,), dtype=i32, device=dev)
        s["src"] = torch.zeros((B, m), dtype=i32, device=dev)
        return s
    H, fmt = case["H"], FORMATS[case["fmt"]]
    s["fmt"] = fmt
    if case["op"] == "window":
        T, R, ctx = case["T"], case["reqs"], case["ctx"]
        pages = _pages(ctx)
        s["pool"] = _pool(gen, R * pages, fmt)
        s["bt"] = torch.randperm(R * pages, generator=gen, device=dev).to(i32).view(R, pages).contiguous()
        if T == R:      # one token of each request, at ragged lengths up to ctx
            s["req"] = None
            pos1 = ctx - torch.randint(0, max(1, ctx // 4), (T,), generator=gen, device=dev)
            pos1[0] = ctx
        else:           # each request's last tokens, in order
            per = [T // R + (1 if r < T % R else 0) for r in range(R)]
            s["req"] = torch.cat([torch.full((p,), r, device=dev) for r, p in enumerate(per)]).to(i32)
            pos1 = torch.cat([torch.arange(ctx - p + 1, ctx + 1, device=dev) for p in per])
        s["pos1"] = pos1.to(i32)
        rows = T
    else:
        B = rows = case["B"]
        n = case["prefix"] + case["tail"] if case["op"] == "prefix" else case["n"]
        s["max"] = n
        P = case["prefix"] if case["op"] == "prefix" else 0
        shared, pages = P // PAGE, _pages(n)
        s["pool"] = _pool(gen, shared + B * (pages - shared), fmt)
        perm = torch.randperm(s["pool"].shape[0], generator=gen, device=dev).to(i32)
        s["bt"] = torch.cat([perm[:shared].repeat(B, 1), perm[shared:].view(B, pages - shared)], 1).contiguous()
        if P % PAGE:    # the page that the prefix ends in: every request has its rows
            k = P % PAGE * ROW_BYTES[fmt]
            s["pool"][s["bt"][:, shared].long(), :k] = s["pool"][s["bt"][0, shared].long(), :k].clone()
        less = torch.randint(0, max(1, (n - P) // 2), (B,), generator=gen, device=dev)
        less[0] = 0
        s["n"] = (n - less).to(i32)
        pos1 = (s["n"] * 128 + 5).to(i32)
        s["pos1"] = pos1
        if case["op"] == "prefix" and case["ring"]:
            s["swa_fmt"] = FORMATS[case["swa"]]
            x = torch.randn((B * RING, D), generator=gen, device=dev)
            s["swa"] = _code_rows(x, s["swa_fmt"]).view(B, RING, -1).contiguous()
    s["q"] = (2.0 * torch.randn((rows, H, D), generator=gen, device=dev)).to(torch.bfloat16)
    s["cs"] = _rope(s["pos1"] - 1)
    s["sink"] = torch.randn((H,), generator=gen, device=dev) if case.get("sink") else None
    if case["op"] == "weights":
        # what the step's attention gave: the log of its sums, here of the entries with a little beside them
        s["lse"] = math.log(case["n"]) + 2.0 + 0.1 * torch.randn((rows, H), generator=gen, device=dev)
        s["acc"] = torch.rand((rows, s["max"]), generator=gen, device=dev)
        s["acc_out"] = torch.zeros((rows, s["max"]), device=dev)
    return s


# ---------------------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------------------

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


def _turn(x, cs, back=False):
    """The last 64 dims turned by the table (..., 32, 2), forth or back."""
    c, s = cs[..., 0], cs[..., 1] * (-1.0 if back else 1.0)
    y = x[..., D - 64:].unflatten(-1, (32, 2))
    y0, y1 = y[..., 0], y[..., 1]
    return torch.cat([x[..., :D - 64], torch.stack([y0 * c - y1 * s, y0 * s + y1 * c], -1).flatten(-2)], -1)


def _softmax_parts(z, sink):
    """exp of logits [..., H, keys] less their maximum, the sum with the sink, and the log of the sum."""
    m = z.amax(-1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(z - m[..., None])
    total = e.sum(-1)
    if sink is not None:
        total = total + torch.exp(sink - m)
    return e, total, m + torch.log(total)


def _plain_window(s):
    c = s["case"]
    pos = s["pos1"].long() - 1
    T = pos.shape[0]
    req = torch.arange(T, device="cuda") if s["req"] is None else s["req"].long()
    first, window = c["first"], c["window"]
    # keys of each query: the first rows, then the window's; a first row inside the window counts once
    a = torch.arange(first, device="cuda").expand(T, first)
    w = pos[:, None] - torch.arange(window, device="cuda").flip(0)
    row = torch.cat([a, w], 1)
    see = torch.cat([a < (pos - window + 1)[:, None], w >= 0], 1)
    kv = _gather(s["pool"], s["bt"], req[:, None].expand_as(row), row.clamp(min=0, max=c["ctx"] - 1), s["fmt"])
    q = _turn(s["q"].float(), s["cs"][:, None])
    z = torch.bmm(q, kv.transpose(1, 2)) * SCALE
    z = z.masked_fill(~see[:, None], -math.inf)
    e, total, lse = _softmax_parts(z, s["sink"])
    o = torch.bmm(e, kv) / total[..., None]
    return _turn(o, s["cs"][:, None], back=True).to(torch.bfloat16), lse


def _plain_prefix(s):
    c = s["case"]
    P, n, B, H = c["prefix"], s["max"], c["B"], c["H"]
    fmt = s["fmt"]
    j = torch.arange(P, device="cuda")
    shared = _gather(s["pool"], s["bt"], torch.zeros_like(j), j, fmt)
    jo = torch.arange(P, n, device="cuda").expand(B, n - P)
    mine = _gather(s["pool"], s["bt"], torch.arange(B, device="cuda")[:, None].expand_as(jo), jo, fmt)
    see = jo < s["n"].long()[:, None]
    if "swa" in s:
        mine = torch.cat([mine, _values(s["swa"], s["swa_fmt"])], 1)
        see = torch.cat([see, torch.arange(RING, device="cuda") < s["pos1"].long()[:, None]], 1)
    q = _turn(s["q"].float(), s["cs"][:, None])
    zs = (q.view(B * H, D) @ shared.t()).view(B, H, P) * SCALE
    zm = (torch.bmm(q, mine.transpose(1, 2)) * SCALE).masked_fill(~see[:, None], -math.inf)
    e, total, lse = _softmax_parts(torch.cat([zs, zm], -1), s["sink"])
    o = (e[..., :P].reshape(B * H, P) @ shared).view(B, H, D) + torch.bmm(e[..., P:], mine)
    return _turn(o / total[..., None], s["cs"][:, None], back=True).to(torch.bfloat16), lse


def _plain_weights(s):
    c = s["case"]
    n, B = s["max"], c["B"]
    j = torch.arange(n, device="cuda").expand(B, n)
    kv = _gather(s["pool"], s["bt"], torch.arange(B, device="cuda")[:, None].expand_as(j), j, s["fmt"])
    q = _turn(s["q"].float(), s["cs"][:, None])
    z = torch.bmm(q, kv.transpose(1, 2)) * SCALE
    w = torch.exp(z - s["lse"][..., None]).sum(1)
    see = (j >= c["first"]) & (j < s["n"].long()[:, None])
    return torch.where(see, 0.99 * s["acc"] + w, s["acc_out"])


def _plain_evict(s):
    c = s["case"]
    B, n, m = c["B"], c["n"], c["budget"]
    slot = torch.arange(n, device="cuda").expand(B, n)
    have = s["n"].long()[:, None]
    live = slot < have
    age = torch.where(live, s["age"], torch.full_like(s["age"], -1))
    newest = age.amax(1, keepdim=True)
    kept_for_sure = (slot < c["fixed"]) | (age > newest - c["recent"])
    rank = torch.where(kept_for_sure, torch.full_like(s["acc"], math.inf), s["acc"])
    rank = torch.where(live, rank, torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :m]
    keep = torch.zeros((B, n), dtype=torch.bool, device="cuda").scatter_(1, order, True) & live
    count = keep.sum(1, keepdim=True)
    # holes in ascending order, and the kept slots behind the count in ascending order
    hole = (slot < count) & ~keep
    mover = (slot >= count) & keep
    src = torch.where(slot < count, slot, torch.full_like(slot, -1))
    src[hole] = slot[mover]      # both run request by request, in ascending order, as many of each
    req = torch.arange(B, device="cuda")[:, None].expand(B, n)
    bt = s["bt"].long()
    to = bt[req[hole], slot[hole] // PAGE] * PAGE + slot[hole] % PAGE
    frm = bt[req[mover], slot[mover] // PAGE] * PAGE + slot[mover] % PAGE
    pools = [p.view(-1, 1024).view(torch.bfloat16).index_copy_(0, to, p.view(-1, 1024).view(torch.bfloat16)[frm])
             for p in s["caches"]]
    src = src[:, :m]
    there = src >= 0
    at = src.clamp(min=0)
    return {"src": src.int(), "n": count[:, 0].int(),
            "acc": torch.where(there, s["acc"].gather(1, at), s["acc_out"]),
            "age": torch.where(there, s["age"].gather(1, at), s["age_out"]), "caches": pools}


def _own_run(s):
    import compressed_sparse_attention_kv_gb300 as cskv
    c = s["case"]
    if s["op"] == "evict":
        caches = [cskv.PagedCache(p, s["bt"], BF16, D) for p in s["caches"]]
        src, n, acc, age = cskv.evict(caches, s["acc"], s["n"], c["budget"], fixed=c["fixed"], recent=c["recent"],
                                      age=s["age"], acc_out=s["acc_out"], age_out=s["age_out"], n_out=s["n_out"],
                                      src=s["src"])
        return {"src": src, "n": n, "acc": acc, "age": age,
                "caches": [p.view(-1, 1024).view(torch.bfloat16) for p in s["caches"]]}
    cache = cskv.PagedCache(s["pool"], s["bt"], s["fmt"], D)
    if s["op"] == "window":
        return cskv.window_attn(s["q"], cache, s["pos1"], c["window"], c["first"], c["ctx"], s["sink"], SCALE, s["cs"],
                                req_of=s["req"], want_lse=True)
    if s["op"] == "prefix":
        return cskv.prefix_decode_attn(s["q"], cache, s["n"], c["prefix"], s["max"], s["sink"], SCALE, s["cs"],
                                       swa=s.get("swa"), swa_fmt=s.get("swa_fmt", BF16), ctx_len=s["pos1"],
                                       want_lse=True)
    return cskv.attn_weights(s["q"], cache, s["n"], s["max"], SCALE, s["cs"], s["lse"], s["acc"], decay=0.99,
                             first=c["first"], acc_out=s["acc_out"])


def run(state):
    if own:
        return _own_run(state)
    return {"window": _plain_window, "prefix": _plain_prefix, "weights": _plain_weights,
            "evict": _plain_evict}[state["op"]](state)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "evict":
        B, n, m = case["B"], case["n"], case["budget"]
        free = max(1, n - case["fixed"] - case["recent"])
        drop = n - m
        # holes among the first m slots: the dropped slots that lie there, the rest lie behind
        holes = drop * max(0.0, min(1.0, (m - case["fixed"] - case["recent"] * m / n) / free))
        holes = min(holes, drop)
        return {"bytes": B * (n * 8 + m * 12 + holes * 2 * 1024 * case["caches"]), "flops": B * n}
    H, rb = case["H"], ROW_BYTES[FORMATS[case["fmt"]]]
    if op == "window":
        T, R = case["T"], case["reqs"]
        seen = min(case["ctx"], case["window"] + case["first"])
        if T == R:
            rows = T * seen
        else:
            rows = R * min(case["ctx"], case["window"] + case["first"] + T // R)
        return {"bytes": T * H * (2048 + 4) + rows * rb, "flops": T * H * seen * 4 * D}
    B = case["B"]
    if op == "prefix":
        own_keys = case["tail"] * 3 // 4
        keys = case["prefix"] + own_keys + (RING if case["ring"] else 0)
        ring = RING * ROW_BYTES[FORMATS[case["swa"]]] if case["ring"] else 0
        return {"bytes": B * H * (2048 + 4) + case["prefix"] * rb + B * (own_keys * rb + ring),
                "flops": B * H * keys * 4 * D}
    n = case["n"] * 3 / 4
    return {"bytes": B * (H * (1024 + 4) + n * (rb + 8)), "flops": B * H * n * 2 * D}


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


def _exact_rows(s, b, idx):
    place = s["bt"][b].long()[idx // PAGE] * PAGE + idx % PAGE
    return _exact_row_values(s["pool"].view(-1, ROW_BYTES[s["fmt"]])[place], s["fmt"])


def _exact_rotation(x, cs, sign):
    w = torch.view_as_complex(cs.double().contiguous())
    if sign < 0:
        w = w.conj()
    y = x.clone()
    tail = torch.view_as_complex(x[..., D - 64:].reshape(x.shape[:-1] + (32, 2)).contiguous()) * w
    y[..., D - 64:] = torch.view_as_real(tail).flatten(-2)
    return y


def _exact_attend(q, kv, see, sink):
    """q [t, H, 512], kv [n, 512], see [t, n] or None -> o [t, H, 512], lse [t, H]; all float64."""
    z = (q @ kv.t()) * SCALE
    if see is not None:
        z = torch.where(see[:, None], z, torch.full_like(z, -math.inf))
    if sink is not None:
        z = torch.cat([z, sink.double()[None, :, None].expand(z.shape[0], -1, 1)], -1)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None])[..., :kv.shape[0]]
    return p @ kv, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        B, m = case["B"], case["budget"]
        src = torch.full((B, m), -1, dtype=torch.int32, device="cuda")
        acc_out, age_out = torch.zeros((B, m), dtype=torch.float64, device="cuda"), torch.zeros_like(src)
        counts = torch.zeros((B,), dtype=torch.int32, device="cuda")
        pools = [p.view(-1, 1024).view(torch.bfloat16).double() if p.numel() < 1 << 28 else None for p in s["caches"]]
        for b in range(B):
            n = int(s["n"][b])
            a, births = s["acc"][b, :n].double(), s["age"][b, :n].long()
            slots = torch.arange(n, device="cuda")
            if n > m:
                safe = (slots < case["fixed"]) | (births > births.max() - case["recent"])
                # by weight, largest first; equal weights by slot; the safe ones before all
                value = torch.where(safe, torch.full_like(a, 1e300), a)
                kept = torch.argsort(-value, stable=True)[:m].sort().values
            else:
                kept = slots
            k = kept.numel()
            stays = kept[kept < k]
            holes = torch.ones((k,), dtype=torch.bool, device="cuda")
            holes[stays] = False
            now = torch.arange(k, device="cuda")
            now[holes] = kept[kept >= k]
            src[b, :k], counts[b] = now.int(), k
            acc_out[b, :k], age_out[b, :k] = a[now], births[now].int()
            rows = s["bt"][b].long()[slots // PAGE] * PAGE + slots % PAGE
            for p in pools:
                if p is not None:
                    p[rows[:k]] = p[rows[now]]
        return {"src": src, "n": counts, "acc": acc_out, "age": age_out, "caches": pools}
    q = s["q"].double()
    q = _exact_rotation(q, s["cs"][:, None], +1)
    if op == "window":
        T, H = case["T"], case["H"]
        out = torch.empty((T, H, D), dtype=torch.float64, device="cuda")
        lse = torch.empty((T, H), dtype=torch.float64, device="cuda")
        pos = s["pos1"].long() - 1
        req = torch.arange(T, device="cuda") if s["req"] is None else s["req"].long()
        step = 1 if s["req"] is None else 256
        starts = [0] + (torch.nonzero(req[1:] != req[:-1]).flatten() + 1).tolist() + [T]
        blocks = [(i, min(i + step, hi)) for lo, hi in zip(starts, starts[1:]) for i in range(lo, hi, step)]
        for i, k in blocks:
            t = pos[i:k]
            lo, hi = max(0, int(t.min()) - case["window"] + 1), int(t.max())
            idx = torch.cat([torch.arange(min(case["first"], lo), device="cuda"),
                             torch.arange(lo, hi + 1, device="cuda")])
            see = (idx <= t[:, None]) & ((idx < case["first"]) | (idx > t[:, None] - case["window"]))
            out[i:k], lse[i:k] = _exact_attend(q[i:k], _exact_rows(s, int(req[i]), idx), see, s["sink"])
        return _exact_rotation(out, s["cs"][:, None], -1), lse
    outs, logs = [], []
    for b in range(case["B"]):
        n = int(s["n"][b])
        kv = _exact_rows(s, b, torch.arange(n, device="cuda"))
        if op == "weights":
            p = torch.exp((q[b] @ kv.t()) * SCALE - s["lse"][b].double()[:, None]).sum(0)
            row = torch.zeros((s["max"],), dtype=torch.float64, device="cuda")
            f = case["first"]
            row[f:n] = 0.99 * s["acc"][b, f:n].double() + p[f:]
            outs.append(row)
            continue
        if "swa" in s:
            ring = _exact_row_values(s["swa"][b], s["swa_fmt"])
            kv = torch.cat([kv, ring[:min(RING, int(s["pos1"][b]))]])
        o, lse = _exact_attend(q[b:b + 1], kv, None, s["sink"])
        outs.append(o[0])
        logs.append(lse[0])
    if op == "weights":
        return torch.stack(outs)
    return _exact_rotation(torch.stack(outs), s["cs"][:, None], -1), torch.stack(logs)
