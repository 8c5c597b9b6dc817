"""The hand-offs of the backward kernel's CTAs as models: every barrier is a count of completed
phases that a wait sees only through its parity, copies land and products finish in any order
their issuer allows, and the roles step in random order.  No order may leave a role waiting
for good, let a role use what is not there yet, or overwrite what is still read."""
import random

import pytest


class Bar:
    """A barrier of `need` arrivals a phase."""

    def __init__(self, need=1):
        self.need, self.phase, self.here = need, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.need:
            self.phase, self.here = self.phase + 1, 0

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


class Model:
    def __init__(self, rng):
        self.rng, self.pipes, self.copies = rng, {}, []

    def product(self, issuer, done):
        """Queued behind the issuer's others: `done` runs when it finishes."""
        self.pipes.setdefault(issuer, []).append(done)

    def run(self, roles):
        """roles: name -> generator that yields conditions to wait for."""
        waiting = {}
        for name, g in roles.items():
            waiting[name] = next(g, None)
        while True:
            ready = [n for n, c in waiting.items() if c is not None and c()]
            pipes = [n for n, q in self.pipes.items() if q]
            moves = [("role", n) for n in ready] + [("pipe", n) for n in pipes] + \
                    [("copy", i) for i in range(len(self.copies))]
            if not moves:
                return [n for n, c in waiting.items() if c is not None]
            kind, what = self.rng.choice(moves)
            if kind == "role":
                waiting[what] = next(roles[what], None)
            elif kind == "pipe":
                self.pipes[what].pop(0)()
            else:
                self.copies.pop(what)()


def dq_cta(E, ragged, rng, warps=3, KS=3, VS=2):
    m = Model(rng)
    kf, ke = [Bar() for _ in range(KS)], [Bar() for _ in range(KS)]
    vf, ve = [Bar() for _ in range(VS)], [Bar() for _ in range(VS)]
    s_full, s_free, dp_full, dp_free = Bar(), Bar(warps), Bar(), Bar(warps)
    ds_ready, dq_done, zero = Bar(warps), Bar(), Bar()
    k_in, v_in = [None] * KS, [None] * VS          # the step whose tile a stage holds
    s_tile = dp_tile = ds_tile = None              # the step a TMEM tile holds
    at = {w: (-1, 1) for w in range(warps)}        # (step, 0: S read, 1: dS written)
    clean = set()

    def producer():
        for i in range(E):
            if i >= KS:
                yield lambda: ke[i % KS].passed(i // KS - 1)
            m.copies.append(lambda i=i: (k_in.__setitem__(i % KS, i), kf[i % KS].arrive()))
            if i >= VS:
                yield lambda: ve[i % VS].passed(i // VS - 1)
            m.copies.append(lambda i=i: (v_in.__setitem__(i % VS, i), vf[i % VS].arrive()))
        if ragged:
            yield lambda: kf[(E - 1) % KS].passed((E - 1) // KS)
            assert k_in[(E - 1) % KS] == E - 1
            clean.add(E - 1)
            zero.arrive()

    def issuer_s():
        for i in range(E):
            yield lambda: kf[i % KS].passed(i // KS)
            if ragged and i == E - 1:
                yield lambda: zero.passed(0)
                assert i in clean
            if i:
                yield lambda: s_free.passed(i - 1)
            assert k_in[i % KS] == i
            assert all(a >= (i - 1, 0) for a in at.values()), "S overwritten while read"

            def done(i=i):
                nonlocal s_tile
                s_tile = i
                s_full.arrive()
            m.product("s", done)

    def issuer_dq():
        for i in range(E):
            yield lambda: kf[i % KS].passed(i // KS)
            yield lambda: ds_ready.passed(i)
            assert k_in[i % KS] == i and ds_tile == i
            assert all(a >= (i, 1) for a in at.values()), "dS not complete"
            m.product("dq", lambda i=i: (dq_done.arrive(), ke[i % KS].arrive()))

    def issuer_dp():
        for i in range(E):
            yield lambda: vf[i % VS].passed(i // VS)
            if i:
                yield lambda: dp_free.passed(i - 1)
            assert v_in[i % VS] == i

            def done(i=i):
                nonlocal dp_tile
                dp_tile = i
                dp_full.arrive()
                ve[i % VS].arrive()
            m.product("dp", done)

    def softmax(w):
        nonlocal ds_tile
        for i in range(E):
            yield lambda: s_full.passed(i)
            assert s_tile == i
            at[w] = (i, 0)
            s_free.arrive()
            yield lambda: dp_full.passed(i)
            assert dp_tile == i
            dp_free.arrive()
            if i:
                yield lambda: dq_done.passed(i - 1)
                assert dq_done.phase >= i, "dS overwritten while read"
            ds_tile = i
            at[w] = (i, 1)
            ds_ready.arrive()

    return m.run({"producer": producer(), "S": issuer_s(), "dQ": issuer_dq(), "dP": issuer_dp(),
                  **{f"warp {w}": softmax(w) for w in range(warps)}})


def dkdv_cta(n_blk, group, first, steps, ragged, rng, warps=2, QS=3, OS=2):
    m = Model(rng)
    qf, qe = [Bar() for _ in range(QS)], [Bar() for _ in range(QS)]
    of, oe = [Bar() for _ in range(OS)], [Bar(2) for _ in range(OS)]
    tf, te = [Bar() for _ in range(OS)], [Bar() for _ in range(OS)]
    s_full, dp_full = [Bar(), Bar()], Bar()
    p_ready, ds_ready = [Bar(warps), Bar(warps)], [Bar(warps), Bar(warps)]
    req, done_z = [Bar(), Bar()], [Bar(), Bar()]
    q_in, o_in, t_in = [None] * QS, [None] * OS, [None] * OS
    s_tile, dp_tile = [None, None], [None, None]
    block = lambda i: (first + i) % n_blk  # noqa: E731
    dirty = lambda i: block(i) == ragged   # noqa: E731
    clean = [set(), set()]

    def producer():
        for i in range(steps):
            if i >= QS:
                yield lambda: qe[i % QS].passed(i // QS - 1)
            m.copies.append(lambda i=i: (q_in.__setitem__(i % QS, i), qf[i % QS].arrive()))
            if i >= OS:
                yield lambda: oe[i % OS].passed(i // OS - 1)
            m.copies.append(lambda i=i: (o_in.__setitem__(i % OS, i), of[i % OS].arrive()))
            if i >= OS:
                yield lambda: te[i % OS].passed(i // OS - 1)
            m.copies.append(lambda i=i: (t_in.__setitem__(i % OS, i), tf[i % OS].arrive()))

    def take(i, w, ask, cleaned):
        yield (lambda: of[i % OS].passed(i // OS)) if w else (lambda: qf[i % QS].passed(i // QS))
        assert (o_in[i % OS] if w else q_in[i % QS]) == i
        if dirty(i):
            if ask:
                req[w].arrive()
            n = cleaned[w]
            cleaned[w] += 1
            yield lambda: done_z[w].passed(n)
            assert i in clean[w]

    def zeroes():
        time = 0
        for i in range(steps):
            if dirty(i):
                for w in (0, 1):
                    yield lambda: req[w].passed(time)
                    assert (o_in[i % OS] if w else q_in[i % QS]) == i
                    clean[w].add(i)
                    done_z[w].arrive()
                time += 1

    def issue_s(i, g):
        def done():
            s_tile[g] = ("S", i)
            s_full[g].arrive()
        m.product("x", done)

    def issue_dp(i):
        def done():
            assert o_in[i % OS] == i
            dp_tile[:] = [("dP", i)] * 2
            dp_full.arrive()
            oe[i % OS].arrive()
        m.product("y", done)

    def issuer_x():
        cleaned = [0, 0]
        yield from take(0, 0, True, cleaned)
        issue_s(0, 0)
        issue_s(0, 1)
        for i in range(steps):
            yield from take(i, 1, False, cleaned)
            if i + 1 < steps:
                yield from take(i + 1, 0, True, cleaned)
            for g in (0, 1):
                yield lambda: p_ready[g].passed(i)

                def dv(i=i, g=g):
                    assert s_tile[g] == ("P", i) and o_in[i % OS] == i
                    if g:
                        oe[i % OS].arrive()
                m.product("x", dv)
                if i + 1 < steps:
                    issue_s(i + 1, g)

    def issuer_y():
        cleaned = [0, 0]
        yield from take(0, 1, True, cleaned)
        issue_dp(0)
        for i in range(steps):
            yield lambda: qf[i % QS].passed(i // QS)
            assert q_in[i % QS] == i
            if i + 1 < steps:
                yield from take(i + 1, 1, True, cleaned)
            for g in (0, 1):
                yield lambda: ds_ready[g].passed(i)

                def dk(i=i, g=g):
                    assert dp_tile[g] == ("dS", i) and q_in[i % QS] == i
                    if g:
                        qe[i % QS].arrive()
                        te[i % OS].arrive()
                m.product("y", dk)
            if i + 1 < steps:
                issue_dp(i + 1)

    left = {}

    def softmax(g, w):
        for i in range(steps):
            yield lambda: s_full[g].passed(i)
            yield lambda: tf[i % OS].passed(i // OS)
            assert s_tile[g][1] == i and t_in[i % OS] == i
            left[g, i, "p"] = left.get((g, i, "p"), 0) + 1
            if left[g, i, "p"] == warps:
                s_tile[g] = ("P", i)
            p_ready[g].arrive()
            yield lambda: dp_full.passed(i)
            assert dp_tile[g][1] == i and t_in[i % OS] == i
            left[g, i, "d"] = left.get((g, i, "d"), 0) + 1
            if left[g, i, "d"] == warps:
                dp_tile[g] = ("dS", i)
            ds_ready[g].arrive()

    return m.run({"producer": producer(), "X": issuer_x(), "Y": issuer_y(), "zeroes": zeroes(),
                  **{f"group {g} warp {w}": softmax(g, w) for g in (0, 1) for w in range(warps)}})


@pytest.mark.parametrize("seed", range(4))
def test_dq(seed):
    rng = random.Random(seed)
    for _ in range(600):
        E = rng.randint(1, 12)
        assert dq_cta(E, rng.random() < 0.5, rng) == []


@pytest.mark.parametrize("seed", range(4))
def test_dkdv(seed):
    rng = random.Random(seed)
    for _ in range(400):
        n_blk, group = rng.randint(1, 5), rng.randint(1, 4)
        first = rng.randint(0, n_blk * group - 1)
        steps = rng.randint(1, n_blk * group - first)
        ragged = n_blk - 1 if rng.random() < 0.6 else -1
        assert dkdv_cta(n_blk, group, first, steps, ragged, rng) == []
