"""Host models of the barriers of list_attn_kernel and weights_kernel (list_attn.cu): the
planning warp, the issuing thread and the working warps, over the row blocks that one block
takes in turn, some of them without any tile (padding queries, empty shares), and over a
block's tiles of several requests.

The mbarrier rule is the hardware's: a wait for parity p returns once the barrier's phase
with parity p has completed, so a waiter must never fall two phases behind its barrier.  The
roles run with random speeds; the model checks that each finishes and that the issuing
thread sees the queries, rows and weights that it is meant to.  A variant with one barrier
for the queries of all row blocks is the control: beside a row block without tiles nothing
keeps the working warps from completing a second phase before the issuing thread has seen
the first.  The weights' model has a control too: a release barrier per pair of chunk slots,
which two blocks of dims complete in turn, in place of one per block of dims."""

import random

import pytest


class _Bar:
    """An mbarrier with an arrival count and a phase counter."""

    def __init__(self, count=1):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class _Sync:
    """The named barrier of the working warps."""

    def __init__(self, count):
        self.count, self.seen, self.round = count, 0, 0

    def arrive(self):
        mine = self.round
        self.seen += 1
        if self.seen == self.count:
            self.seen, self.round = 0, self.round + 1
        return lambda: self.round > mine


def _drive(roles, rnd, now, events, slow):
    """Runs the roles (generators of conditions) and the asynchronous completions with random speeds."""
    cond = {k: None for k in roles}
    ready = {k: 0 for k in roles}
    idle = 0
    while roles:
        now[0] += 1
        for ev in [x for x in events if x[0] <= now[0]]:
            events.remove(ev)
            ev[1]()
        moved = False
        for k in list(roles):
            if ready[k] > now[0] or (cond[k] is not None and not cond[k]()):
                continue
            moved = True
            try:
                cond[k] = next(roles[k])
                ready[k] = now[0] + rnd.randint(1, 40 if k == slow else 6)
            except StopIteration:
                del roles[k], cond[k], ready[k]
        idle = 0 if moved or events else idle + 1
        if idle > 100:
            return "waiting: " + ", ".join(sorted(roles))
    return "ok"


def _run(tiles, seed, query_bars=2, slow=None, per_block=2):
    """tiles[e]: the tiles of the block's row block e.  Returns "ok" or the roles left waiting."""
    rnd = random.Random(seed)
    warps = 4 * per_block
    full = [_Bar(per_block) for _ in range(4)]
    free = [_Bar() for _ in range(4)]
    bar_s, bar_p = _Bar(2), _Bar(warps)
    bar_q = [_Bar(warps) for _ in range(query_bars)]
    plan_full, plan_free = [_Bar(), _Bar()], [_Bar(warps + 1), _Bar(warps + 1)]
    rows_full, rows_free = [_Bar(), _Bar()], [_Bar(warps), _Bar(warps)]
    sync = _Sync(warps)
    items = len(tiles)
    plan, rows = [None, None], [None, None]           # what the slots hold: a row block, a tile
    rotated = [0] * items                             # warps that have rotated a row block's queries
    filled = {}                                       # of a tile's blocks of dims
    weighed = {}
    now, events = [0], []

    def later(fn):
        events.append((now[0] + rnd.randint(1, 30), fn))

    def query_bar(e):
        return (bar_q[0], e & 1) if query_bars == 1 else (bar_q[e & 1], (e >> 1) & 1)

    def planner():
        g = 0
        for e in range(items):
            if e >= 2:
                yield lambda e=e: plan_free[e & 1].done(((e >> 1) - 1) & 1)
            plan[e & 1] = e
            plan_full[e & 1].arrive()
            for _ in range(tiles[e]):
                if g >= 2:
                    yield lambda g=g: rows_free[g & 1].done(((g >> 1) - 1) & 1)
                rows[g & 1] = g
                rows_full[g & 1].arrive()
                g += 1
                yield None

    def issuer():
        g = 0
        for e in range(items):
            yield lambda e=e: plan_full[e & 1].done((e >> 1) & 1)
            assert plan[e & 1] == e
            bar, parity = query_bar(e)
            yield lambda bar=bar, parity=parity: bar.done(parity)
            assert rotated[e] == warps
            for _ in range(tiles[e]):
                for b in range(4):
                    yield lambda b=b, g=g: full[b].done(g & 1)
                    assert filled.get((g, b), 0) == per_block
                assert rows[g & 1] == g
                later(bar_s.arrive)
                bar_s.arrive()
                yield lambda g=g: bar_p.done(g & 1)
                assert weighed.get(g, 0) == warps
                for b in range(4):
                    later(free[b].arrive)
                g += 1
            plan_free[e & 1].arrive()
            yield None

    def worker(w):
        block = w // per_block
        g, requested = 0, False

        def planned(e):
            return lambda: plan_full[e & 1].done((e >> 1) & 1)

        def looked_up(g):
            return lambda: rows_full[g & 1].done((g >> 1) & 1)
        for e in range(items):
            yield planned(e)
            assert plan[e & 1] == e
            yield sync.arrive()
            yield sync.arrive()                       # the queries are there
            rotated[e] += 1
            query_bar(e)[0].arrive()
            nt = tiles[plan[e & 1]]
            if nt > 0 and not requested:
                yield looked_up(g)
                assert rows[g & 1] == g
            for i in range(nt):
                if g > 0:
                    yield lambda g=g: free[block].done((g - 1) & 1)
                filled[(g, block)] = filled.get((g, block), 0) + 1
                full[block].arrive()
                last = i + 1 == nt
                if last and e + 1 < items:
                    yield planned(e + 1)
                    assert plan[(e + 1) & 1] == e + 1
                requested = not last or (e + 1 < items and tiles[e + 1] > 0)
                if requested:
                    yield looked_up(g + 1)
                    assert rows[(g + 1) & 1] == g + 1
                yield lambda g=g: bar_s.done(g & 1)
                assert rows[g & 1] == g
                yield sync.arrive()
                weighed[g] = weighed.get(g, 0) + 1
                bar_p.arrive()
                rows_free[g & 1].arrive()
                g += 1
            yield sync.arrive()
            yield sync.arrive()
            if nt > 0:
                yield lambda g=g: free[3].done((g - 1) & 1)
            if nt == 0 and e + 1 < items:
                yield planned(e + 1)
                yield sync.arrive()
            plan_free[e & 1].arrive()

    roles = {"planner": planner(), "issuer": issuer()}
    roles.update({"worker %d" % w: worker(w) for w in range(warps)})
    return _drive(roles, rnd, now, events, slow)


def _row_blocks(seed):
    rnd = random.Random(1000 + seed)
    kind = seed % 4
    n = rnd.randint(2, 14)
    if kind == 0:
        return [0] * n
    if kind == 1:
        return [rnd.choice([0, 0, 1, 2]) for _ in range(n)]
    if kind == 2:
        return [0] * rnd.randint(1, 4) + [rnd.randint(1, 3)] + [0] * rnd.randint(1, 4)
    return [rnd.randint(1, 4) for _ in range(n)]


@pytest.mark.parametrize("slow", [None, "issuer", "planner", "worker 3"])
@pytest.mark.parametrize("seed", range(40))
def test_every_role_finishes(seed, slow):
    assert _run(_row_blocks(seed), seed, slow=slow) == "ok"


def test_one_barrier_for_all_queries_is_missed_beside_an_empty_row_block():
    """The control: the model finds the fault that two barriers avoid, with empty row blocks only."""
    stuck = [_run(_row_blocks(s), s, query_bars=1, slow="issuer") for s in range(40)]
    assert any(r != "ok" for r in stuck)
    assert all(r == "ok" for s, r in enumerate(stuck) if s % 4 == 3)


# --- the weights -------------------------------------------------------------------------------

def _run_weights(runs, seed, slots, slow=None, per_block=2, release="block"):
    """runs: the tiles of each request in the block's share (each at least one); `slots` chunk slots."""
    rnd = random.Random(seed)
    warps, at_once = 4 * per_block, slots // 2
    full = [_Bar(per_block) for _ in range(4)]
    free = [_Bar() for _ in range(4)]
    bar_s, bar_p = [_Bar(2), _Bar(2)], [_Bar(warps), _Bar(warps)]
    bar_q = _Bar(warps)
    rows_full, rows_free = [_Bar(), _Bar()], [_Bar(warps), _Bar(warps)]
    sync = _Sync(warps)
    nt = sum(runs)
    tile0 = [sum(runs[:r]) for r in range(len(runs))]
    rows, chunk, queries = [None, None], [None] * at_once, [None]
    filled, weighed, sums = {}, {}, [None, None]
    now, events, order = [0], [], [0]

    def later(fn):   # products complete in the order of their issue
        order[0] = max(order[0], now[0]) + rnd.randint(0, 12)
        events.append((order[0], fn))

    def planner():
        for g in range(nt):
            if g >= 2:
                yield lambda g=g: rows_free[g & 1].done(((g >> 1) - 1) & 1)
            rows[g & 1] = g
            rows_full[g & 1].arrive()
            yield None

    def issuer():
        run = -1
        for i in range(nt):
            buf = i & 1
            if run + 1 < len(runs) and i == tile0[run + 1]:
                run += 1
                yield lambda run=run: bar_q.done(run & 1)
            assert queries[0] == (run, warps)
            if i >= 2:
                yield lambda i=i: bar_p[i & 1].done(((i >> 1) - 1) & 1)
                assert weighed.get(i - 2, 0) == warps
            for m in range(4):
                slot, fill = m % at_once, i * (8 // slots) + 2 * m // slots
                yield lambda slot=slot, fill=fill: full[slot].done(fill & 1)
                assert chunk[slot] == (i, m) and filled[(i, m)] == per_block
                later(free[m if release == "block" else slot].arrive)

            def complete(i=i, buf=buf):
                sums[buf] = i
                bar_s[buf].arrive()
            later(complete)
            bar_s[buf].arrive()
            yield None

    def worker(w):
        block = w // per_block

        def load(run):
            yield sync.arrive()
            yield sync.arrive()
            queries[0] = (run, queries[0][1] + 1 if queries[0] and queries[0][0] == run else 1)
            bar_q.arrive()

        def released(g):
            if release == "slot":   # the fills of a slot in turn
                fills = g * (4 // at_once) + block // at_once
                return None if fills == 0 else lambda: free[block % at_once].done((fills - 1) & 1)
            last, tile = (block + 4 - at_once) & 3, g - 1 if block < at_once else g
            return None if tile < 0 else lambda: free[last].done(tile & 1)

        def looked_up(g):
            return lambda: rows_full[g & 1].done((g >> 1) & 1)

        yield from load(0)
        yield looked_up(0)
        next_run, i, t = 1, 0, 0
        while t < nt:
            turn = next_run < len(runs) and i == tile0[next_run]
            if i < nt and (i == t or not turn):
                if turn:
                    yield from load(next_run)
                    next_run += 1
                wait = released(i)
                if wait is not None:
                    yield wait
                at = chunk[block % at_once]
                assert at == (i, block) or at is None or at < (i, block)
                chunk[block % at_once] = (i, block)
                filled[(i, block)] = filled.get((i, block), 0) + 1
                full[block % at_once].arrive()
                rows_free[i & 1].arrive()
                i += 1
                if i < nt:
                    yield looked_up(i)
                    assert rows[i & 1] == i
                if i < nt and i - t < 2:
                    continue
            yield lambda t=t: bar_s[t & 1].done((t >> 1) & 1)
            assert sums[t & 1] == t
            yield sync.arrive()
            weighed[t] = weighed.get(t, 0) + 1
            bar_p[t & 1].arrive()
            t += 1

    roles = {"planner": planner(), "issuer": issuer()}
    roles.update({"worker %d" % w: worker(w) for w in range(warps)})
    try:
        return _drive(roles, rnd, now, events, slow)
    except AssertionError as e:
        if release == "block":
            raise
        return "wrong: %s" % e


def _requests(seed):
    rnd = random.Random(2000 + seed)
    return [rnd.choice([1, 1, 2, 3, 6]) for _ in range(rnd.randint(1, 8))]


@pytest.mark.parametrize("slots", [4, 2])
@pytest.mark.parametrize("slow", [None, "issuer", "planner", "worker 5"])
@pytest.mark.parametrize("seed", range(30))
def test_every_role_of_the_weights_finishes(seed, slow, slots):
    assert _run_weights(_requests(seed), seed, slots, slow=slow) == "ok"


@pytest.mark.parametrize("slots", [4, 2])
def test_a_release_shared_by_blocks_of_dims_is_mistaken(slots):
    """The control: a wait that skips phases passes early by its parity."""
    assert any(_run_weights(_requests(s), s, slots, slow="worker 5", release="slot") != "ok" for s in range(60))
