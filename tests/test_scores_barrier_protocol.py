"""The barrier protocols of the shaped-score kernels that differ from the unshaped ones, checked on
models under random interleavings (host only, no GPU):

  dQ      (fa_scores_dq.cuh) goes through its key tiles twice where D is summed first, reads S before
          it asks for dP, and its row warps join their parts of D over a barrier of two phases;
  dK/dV   (fa_scores_dkdv.cuh) has one S and one dP buffer, and hands P and dS over in shared memory;
  forward (fa_scores_fwd2.cuh) has two query tiles that see different key tiles of one ring.

The roles meet only on mbarriers waited for by phase parity.  The tensor pipe runs what is issued
in issue order, each product reading its operands when it runs; a commit arrives once everything
issued before it has run; copies land in any order.  Each model checks every read, and finds the
mistakes that its kernel must not make.
"""

import random

import pytest


class _Violation(Exception):
    """A role or a product saw data of another step."""


class _Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


class _Machine:
    """Barriers, copies in flight and the tensor pipe; `run` interleaves the roles."""

    def __init__(self, rng, counts=None):
        self.rng, self.counts, self.bars = rng, counts or {}, {}
        self.in_flight, self.pipe = [], []

    def bar(self, name):
        kind = name[0] if isinstance(name, tuple) else name
        return self.bars.setdefault(name, _Barrier(self.counts.get(kind, 1)))

    def expect(self, cond, what):
        if not cond:
            raise _Violation(what)

    def load(self, stages, st, value, full):
        self.in_flight.append((stages, st, value, full))

    def issue(self, product):
        self.pipe.append(product)

    def commit(self, name):
        self.pipe.append(name)

    def _copy(self):
        stages, st, value, full = self.in_flight.pop(self.rng.randrange(len(self.in_flight)))
        stages[st] = value
        self.bar(full).arrive()

    def _run_pipe(self):
        op = self.pipe.pop(0)
        if callable(op):
            op()
        else:
            self.bar(op).arrive()

    def run(self, roles):
        waiting = dict.fromkeys(roles)
        while roles:
            ready = [r for r in roles
                     if waiting[r] is None or self.bar(waiting[r][0]).passed(waiting[r][1])]
            helpers = (["copy"] if self.in_flight else []) + (["pipe"] if self.pipe else [])
            if not ready and not helpers:
                return "deadlock"
            r = self.rng.choice(sorted(ready) + helpers)
            if r == "copy":
                self._copy()
            elif r == "pipe":
                self._run_pipe()
            else:
                try:
                    waiting[r] = next(roles[r])
                except StopIteration:
                    del roles[r]
        return "ok"


def _dq(n_keys, n_sum, nsk, nsv, warps, rng, dp_free=True, join=2, sum_ready=True):
    """n_sum steps that only add to D, then n_keys that make dQ.  `join`: the phases in which the
    row warps join their parts.  sum_ready: steps that only add hand their S buffer back too."""
    m = _Machine(rng, {"DSREADY": warps, "DPFREE": warps, "DSUM": warps})
    n = n_sum + n_keys
    s_buf, dp_buf = [None, None], [None]
    k_st, v_st = [None] * nsk, [None] * nsv
    holds = {}           # (buffer, warp): what that warp left in its columns of S
    parts, taken = {}, {}

    def producer():
        for j in range(n):
            if j >= nsk:
                yield ("KEMPTY", j % nsk), ((j // nsk) - 1) & 1
            m.load(k_st, j % nsk, j, ("KFULL", j % nsk))
            if j >= nsv:
                yield ("VEMPTY", j % nsv), ((j // nsv) - 1) & 1
            m.load(v_st, j % nsv, j, ("VFULL", j % nsv))

    def issuer():
        def s_of(j):
            yield ("KFULL", j % nsk), (j // nsk) & 1

            def product():
                m.expect(k_st[j % nsk] == j, "S's K")
                s_buf[j % 2] = j
                for w in range(warps):
                    holds[j % 2, w] = "S"
            m.issue(product)
            m.commit(("SFULL", j % 2))

        def dp_of(j):
            yield ("VFULL", j % nsv), (j // nsv) & 1

            def product():
                m.expect(v_st[j % nsv] == j, "dP's V")
                dp_buf[0] = j
            m.issue(product)
            m.commit("DPFULL")
            m.commit(("VEMPTY", j % nsv))

        yield from s_of(0)
        yield from dp_of(0)
        if n > 1:
            yield from s_of(1)
        for j in range(n):
            if j + 1 < n:
                if dp_free:
                    yield "DPFREE", j & 1
                yield from dp_of(j + 1)
            yield ("DSREADY", j % 2), (j >> 1) & 1

            def product(j=j):
                m.expect(s_buf[j % 2] == j and k_st[j % nsk] == j, "dQ's operands")
                m.expect(all(holds[j % 2, w] == "dS" for w in range(warps)), "dQ's dS")
            if j >= n_sum:
                m.issue(product)
            m.commit(("KEMPTY", j % nsk))
            if j + 2 < n:
                yield from s_of(j + 2)
            if j == n - 1:
                m.commit("DONE")

    def rows(w):
        for j in range(n):
            yield ("SFULL", j % 2), (j >> 1) & 1
            m.expect(s_buf[j % 2] == j and holds[j % 2, w] == "S", "the rows' S")
            yield "DPFULL", j & 1
            m.expect(dp_buf[0] == j, "the rows' dP")
            m.bar("DPFREE").arrive()
            if j < n_sum:
                if sum_ready:
                    m.bar(("DSREADY", j % 2)).arrive()
                if j == n_sum - 1:  # two rows of sums: the upper half of the warps first
                    half = warps // 2
                    if w >= half:
                        parts[w - half] = {w}
                    m.bar("DSUM").arrive()
                    if join == 2:
                        yield "DSUM", 0
                    if w < half:
                        parts[w] = parts.get(w, set()) | {w}
                    m.bar("DSUM").arrive()
                    yield "DSUM", 1 if join == 2 else 0
                    taken[w] = set().union(*parts.values())
                    m.expect(taken[w] == set(range(warps)), "the parts of D")
                continue
            holds[j % 2, w] = "dS"
            m.bar(("DSREADY", j % 2)).arrive()
        yield "DONE", 0

    roles = {"producer": producer(), "issuer": issuer()}
    roles.update({f"rows{w}": rows(w) for w in range(warps)})
    return m.run(roles)


def _dkdv(n, nq, ndo, warps, rng, s_after_p=True, dp_after_ds=True, final=True):
    m = _Machine(rng, {"P": warps, "DS": warps})
    q_st, do_st = [None] * nq, [None] * ndo
    s_buf, dp_buf = [None], [None]
    p_part, ds_part = [None] * warps, [None] * warps
    done = {"dV": 0, "dK": 0}

    def producer():
        for s in range(n):
            if s >= nq:
                yield ("QEMPTY", s % nq), ((s // nq) - 1) & 1
            m.load(q_st, s % nq, s, ("QFULL", s % nq))
            if s >= ndo:
                yield ("DOEMPTY", s % ndo), ((s // ndo) - 1) & 1
            m.load(do_st, s % ndo, s, ("DOFULL", s % ndo))

    def issuer():
        def s_of(s):
            yield ("QFULL", s % nq), (s // nq) & 1

            def product():
                m.expect(q_st[s % nq] == s, "S's Q")
                s_buf[0] = s
            m.issue(product)
            m.commit("S")

        def dp_of(s):
            yield ("DOFULL", s % ndo), (s // ndo) & 1

            def product():
                m.expect(do_st[s % ndo] == s, "dP's dO")
                dp_buf[0] = s
            m.issue(product)
            m.commit("DP")

        yield from s_of(0)
        yield from dp_of(0)
        for s in range(n):
            if not s_after_p and s + 1 < n:
                yield from s_of(s + 1)  # mistake: the rows may still read S
            yield "P", s & 1

            def dv(s=s):
                m.expect(p_part == [s] * warps and do_st[s % ndo] == s, "dV's operands")
                done["dV"] += 1
            m.issue(dv)
            m.commit(("DOEMPTY", s % ndo))
            if s_after_p and s + 1 < n:
                yield from s_of(s + 1)
            if not dp_after_ds and s + 1 < n:
                yield from dp_of(s + 1)  # mistake: the rows may still read dP
            yield "DS", s & 1

            def dk(s=s):
                m.expect(ds_part == [s] * warps and q_st[s % nq] == s, "dK's operands")
                done["dK"] += 1
            m.issue(dk)
            m.commit(("QEMPTY", s % nq))
            if s == n - 1 and final:
                m.commit("FINAL")
            if dp_after_ds and s + 1 < n:
                yield from dp_of(s + 1)

    def rows(w):
        for s in range(n):
            yield "S", s & 1
            m.expect(s_buf[0] == s, "the rows' S")
            yield None  # (the tanh's other way reads S once more)
            m.expect(s_buf[0] == s, "the rows' S, once more")
            p_part[w] = s
            m.bar("P").arrive()
            yield "DP", s & 1
            m.expect(dp_buf[0] == s, "the rows' dP")
            ds_part[w] = s
            m.bar("DS").arrive()
        if final:
            yield "FINAL", 0
        m.expect(done == {"dV": n, "dK": n}, "the sums at the end")

    roles = {"producer": producer(), "issuer": issuer()}
    roles.update({f"rows{w}": rows(w) for w in range(warps)})
    return m.run(roles)


def _forward(ranges, ns, warps, rng, s_after_pv=True, empty_for_unseen=True):
    """Query tile x sees the key tiles ranges[x] = (from, to) of those loaded, 0 .. n - 1."""
    m = _Machine(rng, {"P": warps})
    n = max(to for _, to in ranges)
    k_st, v_st = [None] * ns, [None] * ns
    s_buf = [[None] * warps, [None] * warps]  # ("S" or "P", tile), by softmax warp
    o = [[], []]

    def producer():
        for j in range(n):
            if j >= ns:
                yield ("KEMPTY", j % ns), ((j // ns) - 1) & 1
            m.load(k_st, j % ns, j, ("KFULL", j % ns))
            if j >= ns:
                yield ("VEMPTY", j % ns), ((j // ns) - 1) & 1
            m.load(v_st, j % ns, j, ("VFULL", j % ns))

    def issuer():
        phase = [0, 0]

        def s_of(x, j):
            def product():
                m.expect(k_st[j % ns] == j, "S's K")
                s_buf[x] = [("S", j)] * warps
            m.issue(product)
            m.commit(("SFULL", x))

        def sees(x, j):
            return ranges[x][0] <= j < ranges[x][1]

        yield ("KFULL", 0), 0
        for x in range(2):
            if sees(x, 0):
                s_of(x, 0)
        m.commit(("KEMPTY", 0))
        for j in range(n):
            yield ("VFULL", j % ns), (j // ns) & 1
            ready = False
            for x in range(2):
                if not s_after_pv and sees(x, j + 1) and sees(x, j):
                    if not ready:
                        yield ("KFULL", (j + 1) % ns), ((j + 1) // ns) & 1
                        ready = True
                    s_of(x, j + 1)  # mistake: before O += P V, over its P
                if sees(x, j):
                    yield ("P", x), phase[x]
                    phase[x] ^= 1

                    def product(x=x, j=j):
                        m.expect(s_buf[x] == [("P", j)] * warps and v_st[j % ns] == j,
                                 "O's operands")
                        o[x].append(j)
                    m.issue(product)
                    m.commit(("ODONE", x))
                if sees(x, j + 1) and (s_after_pv or not sees(x, j)):
                    if not ready:
                        yield ("KFULL", (j + 1) % ns), ((j + 1) // ns) & 1
                        ready = True
                    s_of(x, j + 1)
            m.commit(("VEMPTY", j % ns))
            if j + 1 < n:
                if not ready:  # (a tile that neither sees)
                    yield ("KFULL", (j + 1) % ns), ((j + 1) // ns) & 1
                    ready = True
                if empty_for_unseen or sees(0, j + 1) or sees(1, j + 1):
                    m.commit(("KEMPTY", (j + 1) % ns))

    def softmax(x, w):
        lo, hi = ranges[x]
        for j in range(lo, hi):
            yield ("SFULL", x), (j - lo) & 1
            m.expect(s_buf[x][w] == ("S", j), "the softmax's S")
            if j > lo and rng.random() < 0.5:  # a rescale of O
                yield ("ODONE", x), (j - lo - 1) & 1
                m.expect(o[x] == list(range(lo, j)), "O at a rescale")
            s_buf[x][w] = ("P", j)
            m.bar(("P", x)).arrive()
        if hi > lo:
            yield ("ODONE", x), (hi - lo - 1) & 1
            m.expect(o[x] == list(range(lo, hi)), "O at the end")

    roles = {"producer": producer(), "issuer": issuer()}
    roles.update({f"softmax{x}{w}": softmax(x, w) for x in range(2) for w in range(warps)})
    return m.run(roles)


def _outcomes(calls, seed, tries=20):
    rng = random.Random(seed)
    seen = {}
    for call in calls:
        for _ in range(tries):
            try:
                r = call(rng)
            except _Violation as e:
                r = str(e)
            seen[r] = seen.get(r, 0) + 1
    return seen


# Stages of K and V: d = 64, 96 and 128, 256.
DQ_STAGES = [(4, 4), (3, 2), (2, 1)]


def _dq_calls(stages, sums=(False, True), **kw):
    return [lambda rng, n=n, s=s: _dq(n, n if s else 0, *stages, 4, rng, **kw)
            for n in range(1, 7) for s in sums]


@pytest.mark.parametrize("stages", DQ_STAGES)
def test_dq_is_safe_under_any_interleaving(stages):
    assert set(_outcomes(_dq_calls(stages), 1)) == {"ok"}


@pytest.mark.parametrize("stages", DQ_STAGES)
def test_dq_with_dp_over_rows_that_read_it_fails_in_the_model(stages):
    assert set(_outcomes(_dq_calls(stages, dp_free=False), 2)) != {"ok"}


def test_dq_with_parts_of_d_joined_in_one_phase_fails_in_the_model():
    assert set(_outcomes(_dq_calls((3, 2), sums=(True,), join=1), 3)) != {"ok"}


def test_dq_whose_sums_keep_their_s_buffer_stops_in_the_model():
    assert "deadlock" in _outcomes(_dq_calls((3, 2), sums=(True,), sum_ready=False), 4)


# Stages of Q and dO: d = 64 and others.
DKDV_STAGES = [(2, 2), (2, 1)]


def _dkdv_calls(stages, **kw):
    return [lambda rng, n=n: _dkdv(n, *stages, 4, rng, **kw) for n in range(1, 8)]


@pytest.mark.parametrize("stages", DKDV_STAGES)
def test_dkdv_is_safe_under_any_interleaving(stages):
    assert set(_outcomes(_dkdv_calls(stages), 5)) == {"ok"}


@pytest.mark.parametrize("kw", [{"s_after_p": False}, {"dp_after_ds": False}, {"final": False}],
                         ids=["s_early", "dp_early", "no_final"])
def test_dkdv_mistakes_fail_in_the_model(kw):
    assert set(_outcomes(_dkdv_calls((2, 2), **kw), 6)) != {"ok"}


def test_dkdv_with_one_q_stage_stops_in_the_model():
    """S of the next step comes before dK of this one."""
    assert "deadlock" in _outcomes(_dkdv_calls((1, 1)), 10)


# Key tiles that the two query tiles see: alike, causal, windows, documents apart (with tiles that
# neither sees between them, and either one first), and one that sees nothing.
RANGES = [((0, 1), (0, 1)), ((0, 5), (0, 6)), ((0, 3), (1, 4)), ((0, 2), (4, 7)), ((5, 8), (0, 3)),
          ((0, 1), (9, 10)), ((0, 4), (0, 0)), ((0, 0), (0, 5)), ((2, 3), (0, 6))]


@pytest.mark.parametrize("ns", [4, 2])
def test_two_tile_forward_is_safe_under_any_interleaving(ns):
    calls = [lambda rng, r=r: _forward(r, ns, 4, rng) for r in RANGES]
    assert set(_outcomes(calls, 7)) == {"ok"}


def test_two_tile_forward_with_s_over_p_fails_in_the_model():
    calls = [lambda rng, r=r: _forward(r, 2, 4, rng, s_after_pv=False) for r in RANGES]
    assert set(_outcomes(calls, 8)) != {"ok"}


def test_two_tile_forward_that_keeps_unseen_tiles_stops_in_the_model():
    calls = [lambda rng, r=r: _forward(r, 2, 4, rng, empty_for_unseen=False) for r in RANGES]
    assert "deadlock" in _outcomes(calls, 9)
