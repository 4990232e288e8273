"""Host model of the barriers of chunk_attn_kernel (chunk_attn.cu): both blocks of a pair, each with
its planning warp, its loading thread, its softmax and output warps, the even block's issuing
thread and the odd block's thread that tells of its copies; over the row blocks of a share, some
without any tile.

Products complete in the order of their issue, copies and messages after random times.  The roles
run with random speeds; the model checks that each finishes (a wait for a parity returns once the
phase with it has completed, so that a waiter must never fall two phases behind) and that what a
product or a warp reads is what it is meant to read: keys, dims, queries and weights of its tile,
logits that are read before they are overwritten, outputs that are read before the next row
block's products.  The controls are a single barrier for the blocks' output factors of all row
blocks, weights that are stored without waiting for the product before, and products that do not
wait for the outputs in their place."""

import random

import pytest

from test_list_attn_protocol import _Bar, _Sync, _drive


class _Pipe:
    """Products of one issuing thread: completed in order; a commit arrives when all before it are."""

    def __init__(self, rnd, now, events):
        self.rnd, self.now, self.events, self.end = rnd, now, events, 0

    def add(self, fn):
        self.end = max(self.end, self.now[0]) + self.rnd.randint(1, 12)
        self.events.append((self.end, fn))

    def commit(self, *bars):
        self.events.append((max(self.end, self.now[0] + 1), lambda: [b.arrive() for b in bars]))


class _Tx(_Bar):
    """A barrier that also counts messages: `count` arrivals and `tx` of them in a phase."""

    def __init__(self, count, tx):
        super().__init__(count + tx)


def _run(tiles, seed, warps=2, slow=None, one_factor_bar=False, weights_wait=True, places=3,
         outputs_wait=True):
    rnd = random.Random(seed)
    items, now, events = len(tiles), [0], []
    pipe = _Pipe(rnd, now, events)

    def later(fn):
        events.append((now[0] + rnd.randint(1, 30), fn))

    class Block:
        pass

    B = []
    for rank in range(2):
        b = Block()
        both = 2 if rank == 0 else 1
        b.k_full, b.k_free = [_Bar(both + 1) for _ in range(4)], [_Bar() for _ in range(4)]
        b.v_full, b.v_free = [_Bar(both + 1) for _ in range(2)], [_Bar() for _ in range(2)]
        b.s_full, b.moved = [_Bar(), _Bar()], [_Tx(1, warps + 1), _Tx(1, warps + 1)]
        b.p_full, b.q_full, b.q_free = _Bar(2 * warps), _Bar(2 * warps), _Bar()
        b.o_free = [_Bar(2 * warps) for _ in range(places)]
        b.l_full = [_Bar(warps), _Bar(warps)]
        b.f_full = [_Tx(1, warps)] * 2 if one_factor_bar else [_Tx(1, warps), _Tx(1, warps)]
        b.item_full, b.item_free = [_Bar(), _Bar()], [_Bar(2 + 2 * warps), _Bar(2 + 2 * warps)]
        b.sees_full, b.sees = [_Bar(), _Bar()], [None, None]
        b.soft, b.outs = _Sync(warps), _Sync(warps)
        b.item, b.keys, b.dims, b.q = [None, None], [None] * 4, [None] * 2, [None] * warps
        b.logits, b.read, b.weights = [None, None], {}, [None] * warps
        b.sums, b.factors = [None, None], [[None] * 2, [None] * 2]
        B.append(b)
    o = [None] * places           # which row block's sums of which block of dims each place holds, in either block
    out_read = {}

    def planner(b):
        for e in range(items):
            if e >= 2:
                yield lambda e=e: b.item_free[e & 1].done(((e >> 1) - 1) & 1)
            b.item[e & 1] = e
            b.item_full[e & 1].arrive()
            yield None
            b.sees[e & 1] = e
            b.sees_full[e & 1].arrive()
            yield None

    def there(b, e):
        return lambda: b.item_full[e & 1].done((e >> 1) & 1)

    def walk(b, keys, dims):
        e, t, fresh, first, early = 0, -1, True, True, False
        while e < items:
            if fresh:
                yield there(b, e)
                assert b.item[e & 1] == e
                s, t = e, -1
            fresh, ahead = tiles[s] == 0, False
            if not fresh:
                of, kt = s, t + 1
                send = kt < tiles[s]
                if not send and e + 1 < items:
                    yield there(b, e + 1)
                    of, kt = b.item[(e + 1) & 1], 0
                    send = ahead = tiles[of] > 0
                if send:
                    yield from keys((of, kt))
                if first or (t >= 0 and not early):
                    yield from dims((s, max(t, 0)))
                early, first = first, False
                if t + 1 < tiles[s]:
                    t += 1
                    continue
                s, t, fresh = of, 0, not ahead
            b.item_free[e & 1].arrive()
            e += 1

    def loader(b):
        gk = gv = 0

        def put(place, i, tile, bar):
            place[i] = tile
            bar.arrive()

        def keys(tile):
            nonlocal gk
            for m in range(4):
                if gk > 0:
                    yield lambda m=m, g=gk: b.k_free[m].done((g - 1) & 1)
                b.k_full[m].arrive()
                later(lambda m=m: put(b.keys, m, tile, b.k_full[m]))
            gk += 1

        def dims(tile):
            nonlocal gv
            for j in range(2):
                if gv > 0:
                    yield lambda j=j, g=gv: b.v_free[j].done((g - 1) & 1)
                b.v_full[j].arrive()
                later(lambda j=j: put(b.dims, j, tile, b.v_full[j]))
            gv += 1
        yield from walk(b, keys, dims)

    def teller():
        b, gk, gv = B[1], 0, 0

        def keys(tile):
            nonlocal gk
            for m in range(4):
                yield lambda m=m, g=gk: b.k_full[m].done(g & 1)
                later(B[0].k_full[m].arrive)
            gk += 1

        def dims(tile):
            nonlocal gv
            for j in range(2):
                yield lambda j=j, g=gv: b.v_full[j].done(g & 1)
                later(B[0].v_full[j].arrive)
            gv += 1
        yield from walk(b, keys, dims)

    def issuer():
        b, g, ahead = B[0], 0, False
        for e in range(items):
            yield there(b, e)
            nt = tiles[b.item[e & 1]]
            if not ahead:
                yield lambda e=e: b.q_full.done(e & 1)

            def products_s(t, e, i):
                for m in range(4):
                    yield lambda m=m, i=i: b.k_full[m].done(i & 1)

                    def product(m=m, t=t, i=i, e=e):
                        for c in B:
                            assert c.keys[m] == (e, t) and c.q == [e] * warps
                            if m == 0 and c.logits[i & 1] is not None:
                                assert c.read[c.logits[i & 1]] == warps     # the logits two tiles before
                            c.logits[i & 1] = (e, t)
                    pipe.add(product)
                    pipe.commit(B[0].k_free[m], B[1].k_free[m])
                pipe.commit(B[0].s_full[i & 1], B[1].s_full[i & 1])
                if t == tiles[e] - 1:
                    pipe.commit(B[0].q_free, B[1].q_free)

            def outputs_read(j, e=e):
                n = 2 * e + j
                if n >= places and outputs_wait:
                    yield lambda: b.o_free[n % places].done((n // places - 1) & 1)
            if nt == 0:
                yield from outputs_read(0)
                yield from outputs_read(1)
                pipe.commit(B[0].q_free, B[1].q_free)
            first, ahead = 0 if ahead else -1, False
            for t in range(first, nt):
                i = g + t
                if t + 1 < nt:
                    yield from products_s(t + 1, e, i + 1)
                elif nt and e + 1 < items:
                    def queries(f=e + 1):
                        return b.item_full[f & 1].done((f >> 1) & 1) and (b.item[f & 1] is not None and tiles[b.item[f & 1]] > 0) \
                            and b.q_full.done(f & 1)
                    yield lambda i=i: queries() or b.p_full.done(i & 1)
                    ahead = queries()
                    if ahead:
                        yield from products_s(0, e + 1, i + 1)
                if t < 0:
                    continue
                yield lambda i=i: b.p_full.done(i & 1)
                for j in range(2):
                    if t == 0:
                        yield from outputs_read(j)
                    yield lambda j=j, i=i: b.v_full[j].done(i & 1)

                    def product(j=j, t=t, e=e):
                        for c in B:
                            assert c.dims[j] == (e, t) and c.weights == [(e, t)] * warps
                        at = (2 * e + j) % places
                        if t == 0 and o[at] is not None:
                            assert out_read.get(o[at], 0) == 2 * warps
                        assert t == 0 or o[at] == (e, j)
                        o[at] = (e, j)
                    pipe.add(product)
                    pipe.commit(B[0].v_free[j], B[1].v_free[j])
            g += nt
            b.item_free[e & 1].arrive()
            yield None

    def softmax(b, peer, w):
        g = 0
        for e in range(items):
            yield lambda e=e: b.sees_full[e & 1].done((e >> 1) & 1)
            yield b.soft.arrive()
            assert b.item[e & 1] == e and b.sees[e & 1] == e
            for t in range(tiles[e]):
                yield lambda g=g: b.s_full[g & 1].done((g >> 1) & 1)
                assert b.logits[g & 1] == (e, t)
                b.read[(e, t)] = b.read.get((e, t), 0) + 1
                yield b.soft.arrive()
                later(peer.moved[g & 1].arrive)                  # a factor
                if w == 0:
                    later(peer.moved[g & 1].arrive)              # the flag
                    b.moved[g & 1].arrive()                      # how much is expected
                if g > 0 and weights_wait:
                    yield lambda g=g: b.v_free[1].done((g - 1) & 1)
                b.weights[w] = (e, t)
                yield lambda g=g: b.moved[g & 1].done((g >> 1) & 1)
                later(B[0].p_full.arrive)
                g += 1
            b.sums[e & 1] = e
            b.l_full[e & 1].arrive()
            b.item_free[e & 1].arrive()

    def outputs(b, peer, w, rank):
        g = 0
        if items:
            yield there(b, 0)
            yield b.outs.arrive()
            b.q[w] = 0
            later(B[0].q_full.arrive)
        for e in range(items):
            g += tiles[e]
            if e + 1 < items:
                yield there(b, e + 1)
                yield b.outs.arrive()
                assert b.item[(e + 1) & 1] == e + 1              # its queries into registers
            yield lambda e=e: b.q_free.done(e & 1)
            if e + 1 < items:
                b.q[w] = e + 1
                later(B[0].q_full.arrive)
            yield lambda e=e: b.l_full[e & 1].done((e >> 1) & 1)
            assert b.sums[e & 1] == e and b.item[e & 1] == e

            def factor(e=e):
                peer.factors[e & 1][rank] = e
                peer.f_full[e & 1].arrive()
            b.factors[e & 1][rank] = e
            later(factor)
            if w == 0:
                b.f_full[e & 1].arrive()
            yield b.outs.arrive()
            if one_factor_bar:
                yield lambda e=e: b.f_full[0].done(e & 1)
            else:
                yield lambda e=e: b.f_full[e & 1].done((e >> 1) & 1)
            if tiles[e]:
                yield lambda g=g: b.v_free[1].done((g - 1) & 1)
            for j in range(2):
                if tiles[e]:
                    assert o[(2 * e + j) % places] == (e, j)
                assert b.factors[e & 1] == [e, e]
                out_read[(e, j)] = out_read.get((e, j), 0) + 1
                later(B[0].o_free[(2 * e + j) % places].arrive)
                yield None
            b.item_free[e & 1].arrive()

    roles = {"issuer": issuer(), "teller": teller()}
    for rank in range(2):
        b, peer = B[rank], B[1 - rank]
        roles["planner %d" % rank] = planner(b)
        roles["loader %d" % rank] = loader(b)
        for w in range(warps):
            roles["softmax %d.%d" % (rank, w)] = softmax(b, peer, w)
            roles["outputs %d.%d" % (rank, w)] = outputs(b, peer, w, rank)
    return _drive(roles, rnd, now, events, slow)


def _row_blocks(seed):
    rnd = random.Random(2000 + seed)
    kind = seed % 5
    n = rnd.randint(1, 12)
    if kind == 0:
        return [0] * n
    if kind == 1:
        return [rnd.choice([0, 0, 1, 2]) for _ in range(n)]
    if kind == 2:
        return [1] * n
    if kind == 3:
        return [0] * rnd.randint(1, 4) + [rnd.randint(1, 3)] + [0] * rnd.randint(1, 4)
    return [rnd.randint(1, 5) for _ in range(n)]


@pytest.mark.parametrize("slow", [None, "issuer", "teller", "planner 1", "loader 0", "softmax 0.1", "outputs 1.0"])
@pytest.mark.parametrize("seed", range(40))
def test_every_role_finishes_and_reads_what_it_should(seed, slow):
    assert _run(_row_blocks(seed), seed, slow=slow) == "ok"


def _fails(**change):
    for seed in range(300):
        for slow in (None, "outputs 0.1", "softmax 1.1"):
            try:
                if _run(_row_blocks(seed), seed, slow=slow, **change) != "ok":
                    return True
            except AssertionError:
                return True
    return False


def test_weights_stored_without_waiting_are_found():
    """The control: a tile's weights in place of those that the product before still reads."""
    assert _fails(weights_wait=False)


def test_one_barrier_for_all_factors_is_found():
    """The control: a message for the next row block's factors counted in this one's phase."""
    assert _fails(one_factor_bar=True)


def test_products_in_place_of_unread_outputs_are_found():
    """The control: a row block's first products where outputs of one before are still read."""
    assert _fails(outputs_wait=False)
