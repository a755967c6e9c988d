"""The barrier protocols of the paged attention's tensor-core kernels
(fa_paged_tile2.cu: two query tiles that share the key tiles; fa_paged_tile.cu:
one, at d = 256), checked on models under random interleavings (host only).

A CTA works through items, each with some key tiles; key tiles n = 0, 1, ...
run on across the items, through K and V ring stages n % NS.  What the models
check: every product reads the K, V, Q and P it is meant to; the softmax reads
its own scores; O is complete where it is rescaled, stored and joined, and not
overwritten before; and no order of events ends in a deadlock.  They fail, as
they should, when a hand-off is left out.
"""

import random

import pytest


class _Violation(Exception):
    pass


class _Machine:
    """Barriers with phases and counts, the tensor pipe in issue order, copies in any order."""

    def __init__(self, rng):
        self.rng, self.count, self.phase, self.need = rng, {}, {}, {}
        self.pipe, self.copies = [], []

    def init(self, name, need=1):
        self.need[name] = need

    def arrive(self, name):
        self.count[name] = self.count.get(name, 0) + 1
        if self.count[name] == self.need.get(name, 1):
            self.count[name] = 0
            self.phase[name] = self.phase.get(name, 0) + 1

    def passed(self, name, parity):
        return (self.phase.get(name, 0) & 1) != parity

    def run(self, roles):
        waiting = dict.fromkeys(roles)
        alive = set(roles)
        while alive:
            ready = sorted(r for r in alive if waiting[r] is None or self.passed(*waiting[r]))
            extra = (["pipe"] if self.pipe else []) + (["copy"] if self.copies else [])
            if not ready and not extra:
                return "deadlock"
            r = self.rng.choice(ready + extra)
            if r == "pipe":
                self.pipe.pop(0)()
            elif r == "copy":
                self.copies.pop(self.rng.randrange(len(self.copies)))()
            else:
                try:
                    waiting[r] = next(roles[r])
                except StopIteration:
                    alive.discard(r)
        while self.pipe:
            self.pipe.pop(0)()
        return "ok"


def _expect(cond, what):
    if not cond:
        raise _Violation(what)


def _loads(mc, tiles, ns, nr, k, v, raw):
    """Producer and helpers: K and V of every tile into the rings (straight, or through raw slots
    that the helpers convert); the helpers say when V is whole."""
    def producer():
        for n in range(tiles):
            if nr:
                for kv, i in ((0, 2 * n), (1, 2 * n + 1)):
                    if i >= nr:
                        yield ("REMPTY", i % nr), ((i // nr) - 1) & 1

                    def land(i=i, kv=kv, n=n):
                        raw[i % nr] = (kv, n)
                        mc.arrive(("RFULL", i % nr))
                    mc.copies.append(land)
                continue
            for kv, ring in (("K", k), ("V", v)):
                if n >= ns:
                    yield (kv + "EMPTY", n % ns), ((n // ns) - 1) & 1

                def land(kv=kv, ring=ring, n=n):
                    ring[n % ns] = n
                    mc.arrive((kv + "FULL", n % ns))
                mc.copies.append(land)

    def helper(n, tail):
        """Of one key tile (a generator)."""
        st, ph = n % ns, ((n // ns) - 1) & 1
        if nr:
            for kv, i in ((0, 2 * n), (1, 2 * n + 1)):
                if n >= ns:
                    yield (("VEMPTY" if kv else "KEMPTY"), st), ph
                yield ("RFULL", i % nr), (i // nr) & 1
                _expect(raw[i % nr] == (kv, n), "conversion")
                (v if kv else k)[st] = n
                mc.arrive(("REMPTY", i % nr))
                mc.arrive(("VFIX" if kv else "KFULL", st))
        else:
            if n >= ns:
                yield ("VEMPTY", st), ph
            if tail:
                yield ("VFULL", st), (n // ns) & 1
                _expect(v[st] == n, "V's tail")
            mc.arrive(("VFIX", st))
    return producer, helper


def _two_tiles(items, ns, nr, rng, wait_split=True, s_after_pv=True, in_order=True):
    """items: (key tiles, split).  A split item's even key tiles go to tile 0, its odd to 1.
    in_order: an item's products begin with tile 0 (A), whose warps store and join the item
    before."""
    mc = _Machine(rng)
    total = sum(n for n, _ in items)
    k, v, raw = [None] * ns, [None] * ns, [None] * max(nr, 1)
    q, s = [None, None], [None, None]
    o = [[], []]            # (item, key tile) products in each tile's O
    producer, helper = _loads(mc, total, ns, nr, k, v, raw)
    first = (0, 1) if in_order else (1, 0)
    jobs = []               # (tile, key tile, item, first of the item in the tile, K's last use)
    n = 0
    for it, (tiles, split) in enumerate(items):
        for t in range(tiles):
            xs = [t % 2] if split else list(first)
            for x in xs:
                jobs.append((x, n, it, t < 2 if split else t == 0, x == xs[-1]))
            n += 1

    def helpers():
        n = 0
        for tiles, _ in items:
            for t in range(tiles):
                yield from helper(n, t == tiles - 1)
                n += 1

    def issuer():
        q_phase, p_phase, waiting, k_ready, v_ready = [0, 0], [0, 0], [], -1, -1
        ahead = iter(jobs)
        nxt = next(ahead, None)
        while nxt or waiting:
            while nxt and (not waiting or (len(waiting) == 1 and waiting[0][0] != nxt[0]) or
                           (not s_after_pv and len(waiting) == 1)):
                x, n, it, first, last = nxt
                if first:
                    yield ("QFULL", x), q_phase[x]
                    q_phase[x] ^= 1
                if n != k_ready:
                    yield ("KFULL", n % ns), (n // ns) & 1
                    k_ready = n

                def scores(x=x, n=n, it=it):
                    _expect(k[n % ns] == n, "S read another K")
                    _expect(q[x] == it, "S read another Q")
                    s[x] = ("S", n)
                mc.pipe.append(scores)
                mc.pipe.append(lambda x=x: mc.arrive(("SFULL", x)))
                if last:
                    mc.pipe.append(lambda n=n: mc.arrive(("KEMPTY", n % ns)))
                waiting.append(nxt)
                nxt = next(ahead, None)
            x, n, it, first, last = waiting.pop(0)
            if n != v_ready:
                if not nr:
                    yield ("VFULL", n % ns), (n // ns) & 1
                yield ("VFIX", n % ns), (n // ns) & 1
                v_ready = n
            yield ("PFULL", x), p_phase[x]
            p_phase[x] ^= 1

            def product(x=x, n=n, it=it, first=first):
                _expect(v[n % ns] == n, "P V read another V")
                _expect(s[x] == ("P", n), "P V read no P of its own")
                o[x] = ([] if first else o[x]) + [(it, n)]
            mc.pipe.append(product)
            mc.pipe.append(lambda x=x: mc.arrive(("ODONE", x)))
            if last:
                mc.pipe.append(lambda n=n: mc.arrive(("VEMPTY", n % ns)))

    def softmax(x):
        mine = [[j for j in jobs if j[0] == x and j[2] == it] for it in range(len(items))]
        todo = [it for it in range(len(items)) if mine[it]]
        done = joins = 0

        def load(it):
            q[x] = it
            mc.arrive(("QFULL", x))
        if todo:
            load(todo[0])
        for at, it in enumerate(todo):
            for i, (_, n, *_rest) in enumerate(mine[it]):
                yield ("SFULL", x), done & 1
                _expect(s[x] == ("S", n), "softmax read other scores")
                if i and rng.random() < 0.5:
                    yield ("ODONE", x), (done - 1) & 1
                    _expect(o[x] == [(it, j[1]) for j in mine[it][:i]], "rescale")
                s[x] = ("P", n)
                mc.arrive(("PFULL", x))
                done += 1
            if at + 1 < len(todo):
                load(todo[at + 1])
            yield ("ODONE", x), (done - 1) & 1
            both = items[it][1] and items[it][0] > 1
            if both and x == 1:
                mc.arrive("SPLIT")
                joins += 1
                continue
            _expect(o[x] == [(it, j[1]) for j in mine[it]], "O stored")
            if both:
                if wait_split:
                    yield "SPLIT", joins & 1
                joins += 1
                yield "tick", 1  # (reading takes a while)
                _expect(o[1] == [(it, j[1]) for j in jobs if j[0] == 1 and j[2] == it], "O joined")
    return mc.run({"producer": producer(), "helpers": helpers(), "issuer": issuer(),
                   "A": softmax(0), "B": softmax(1)})


def _one_tile(items, ns, nr, rng, q_empty=True):
    """items: key tiles of each; S two tiles ahead in three buffers, one Q tile."""
    mc = _Machine(rng)
    total = sum(items)
    k, v, raw = [None] * ns, [None] * ns, [None] * max(nr, 1)
    q, s, o = [None], [None] * 3, [[]]
    producer, helper = _loads(mc, total, ns, nr, k, v, raw)
    mc.init("QEMPTY", 2)
    jobs = [(n, it, t == 0, t == tiles - 1) for n, (it, t, tiles) in enumerate(
        (it, t, tiles) for it, tiles in enumerate(items) for t in range(tiles))]

    def helpers():
        n = 0
        for it, tiles in enumerate(items):
            if it and q_empty:
                yield "QEMPTY", (it - 1) & 1
            q[0] = it
            mc.arrive("QFULL")
            for t in range(tiles):
                yield from helper(n, t == tiles - 1)
                n += 1

    def issuer():
        def scores(n, it, first, last):
            if first:
                yield "QFULL", it & 1
            yield ("KFULL", n % ns), (n // ns) & 1

            def run():
                _expect(k[n % ns] == n, "S read another K")
                _expect(q[0] == it, "S read another Q")
                _expect(s[n % 3] is None or s[n % 3] == ("read", n - 3), "S over a P in use")
                s[n % 3] = ("S", n)
            mc.pipe.append(run)
            mc.pipe.append(lambda: mc.arrive(("SFULL", n % 3)))
            mc.pipe.append(lambda: mc.arrive(("KEMPTY", n % ns)))
            if last:
                mc.pipe.append(lambda: mc.arrive("QEMPTY"))
        for j in jobs[:2]:
            yield from scores(*j)
        for n, it, first, last in jobs:
            if not nr:
                yield ("VFULL", n % ns), (n // ns) & 1
            yield ("VFIX", n % ns), (n // ns) & 1
            yield ("PFULL", n % 3), (n // 3) & 1

            def product(n=n, it=it, first=first):
                _expect(v[n % ns] == n, "P V read another V")
                _expect(s[n % 3] == ("P", n), "P V read no P of its own")
                s[n % 3] = ("read", n)
                o[0] = ([] if first else o[0]) + [(it, n)]
            mc.pipe.append(product)
            mc.pipe.append(lambda: mc.arrive("ODONE"))
            mc.pipe.append(lambda n=n: mc.arrive(("VEMPTY", n % ns)))
            if last:
                mc.pipe.append(lambda: mc.arrive("FINAL"))
            if n + 2 < len(jobs):
                yield from scores(*jobs[n + 2])

    def softmax():
        n = 0
        for it, tiles in enumerate(items):
            yield "QFULL", it & 1
            mc.arrive("QEMPTY")  # (the rows' scales are read)
            for t in range(tiles):
                yield ("SFULL", n % 3), (n // 3) & 1
                _expect(s[n % 3] == ("S", n), "softmax read other scores")
                if t and rng.random() < 0.5:
                    yield "ODONE", (n - 1) & 1
                    _expect(o[0] == [(it, n - t + i) for i in range(t)], "rescale")
                s[n % 3] = ("P", n)
                mc.arrive(("PFULL", n % 3))
                n += 1
            yield "FINAL", it & 1
            _expect(o[0] == [(it, n - tiles + i) for i in range(tiles)], "O stored")
    return mc.run({"producer": producer(), "helpers": helpers(), "issuer": issuer(),
                   "softmax": softmax()})


def _outcomes(run, draw, seed, tries, **kw):
    rng = random.Random(seed)
    seen = {}
    for _ in range(tries):
        try:
            r = run(draw(rng), rng=rng, **kw)
        except _Violation as e:
            r = str(e)
        seen[r] = seen.get(r, 0) + 1
    return seen


def _two_items(rng):
    return [(rng.choice((1, 1, 2, 3, 5)), rng.random() < 0.5) for _ in range(rng.randint(1, 6))]


def _one_items(rng):
    return [rng.choice((1, 1, 2, 3, 5)) for _ in range(rng.randint(1, 6))]


@pytest.mark.parametrize("ns,nr", [(2, 0), (4, 0), (2, 2), (4, 4)])
def test_two_tiles_are_safe_under_any_interleaving(ns, nr):
    assert _outcomes(_two_tiles, _two_items, ns + nr, 400, ns=ns, nr=nr) == {"ok": 400}


@pytest.mark.parametrize("nr", [0, 2])
def test_one_tile_is_safe_under_any_interleaving(nr):
    assert _outcomes(_one_tile, _one_items, nr, 400, ns=2, nr=nr) == {"ok": 400}


@pytest.mark.parametrize("left_out", ["wait_split", "s_after_pv", "in_order"])
def test_two_tiles_fail_without(left_out):
    seen = _outcomes(_two_tiles, _two_items, 7, 400, ns=2, nr=0, **{left_out: False})
    assert set(seen) != {"ok"}, seen


def test_one_tile_fails_without_the_wait_for_q():
    seen = _outcomes(_one_tile, _one_items, 8, 400, ns=2, nr=0, q_empty=False)
    assert set(seen) != {"ok"}, seen
