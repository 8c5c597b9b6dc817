"""The hand-offs between the two MMA issuers and the two softmax groups of the attention
kernels, as a model: every barrier is a count of completed phases that a wait sees only
through its parity, and the roles step in random order.

In the block-sparse kernel the P V issuer waits for the S two visits ahead on one of a ring of
barriers; the ring read from the kernel's source must never leave a role waiting for good,
whatever the order (a ring of four does).  In the window kernel it does not wait for S."""
import os
import random
import re

import pytest

from block_sparse_spatio_attn_b200 import build


def completes(visits, ring, rng):
    """Steps the roles through `visits` (the group of each visit) until no role can move;
    True when every one is done.  ring: barriers of the P V issuer's wait for S, 0 for none."""
    n = len(visits)
    s_full, p_full, o_done = ([0, 0] for _ in range(3))
    s_free = 0
    issued = [0] * ring
    passed = lambda count, parity: (count & 1) != parity  # noqa: E731  a wait on a parity
    s_next, extra = 0, 0
    pv_next, pv_of = 0, [0, 0]
    mine = [sum(v == g for v in visits) for g in (0, 1)]
    seen, stage = [0, 0], [0, 0]
    pipe = []
    while True:
        moves = []
        if s_next < n:
            g = visits[s_next]
            if s_next == 0 or passed(s_free, (s_next - 1) & 1):
                moves.append(("S", g))
        elif ring and extra < 2:
            moves.append(("behind the last S", 0))
        if pv_next < n:
            g, ahead = visits[pv_next], pv_next + 2
            if passed(p_full[g], pv_of[g] & 1) and (
                    not ring or passed(issued[ahead % ring], ahead // ring & 1)):
                moves.append(("PV", g))
        for g in (0, 1):
            if seen[g] < mine[g] and (
                    stage[g] == 0 and passed(s_full[g], seen[g] & 1) or
                    stage[g] == 1 and (seen[g] == 0 or passed(o_done[g], (seen[g] - 1) & 1)) or
                    stage[g] == 2):
                moves.append(("softmax", g))
        if pipe:
            moves.append(("tensor", 0))
        if not moves:
            return s_next == n and pv_next == n and seen == mine
        what, g = rng.choice(moves)
        if what == "S":
            pipe.append((s_full, g))
            if ring:
                issued[s_next % ring] += 1
            s_next += 1
        elif what == "behind the last S":
            issued[(n + extra) % ring] += 1
            extra += 1
        elif what == "PV":
            pipe.append((o_done, g))
            pv_of[g] += 1
            pv_next += 1
        elif what == "tensor":
            done, g = pipe.pop(0)
            done[g] += 1
        elif stage[g] == 0:      # S read into registers
            s_free += 1
            stage[g] = 1
        elif stage[g] == 1:      # the previous P V is done
            stage[g] = 2
        else:                    # P written
            p_full[g] += 1
            stage[g], seen[g] = 0, seen[g] + 1


def lists(rng, count):
    for _ in range(count):
        yield [g for _ in range(rng.randint(1, 7)) for g in rng.choice([(0,), (1,), (0, 1), (0, 1)])]


def ring_of(source):
    text = open(os.path.join(build.CSRC, source)).read()
    found = re.search(r"uint64_t s_issued\[(\d+)\]", text)
    return int(found.group(1)) if found else 0


@pytest.mark.parametrize("source", ["attention.cu", "window_fwd.cu"])
def test_no_order_leaves_a_role_waiting(source):
    rng = random.Random(1)
    ring = ring_of(source)
    assert ring == (8 if source == "attention.cu" else 0)
    for visits in lists(rng, 30000):
        assert completes(visits, ring, rng), visits


def test_the_model_sees_a_ring_that_is_too_short():
    rng = random.Random(1)
    assert not all(completes(v, 4, rng) for v in lists(rng, 30000))
