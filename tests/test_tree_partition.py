"""The tree kernel's work split, restated on the CPU: the planes' shares of the
blocks, every granule of every unit in exactly one block's range, cut units'
pieces in consecutive blocks that agree on their number and on the first of
them, and at most one piece a block of either kind (one that goes on behind its
range, one that began before it); and the counting by which the blocks of a cut
unit find each other, under every kind of interleaving."""
import random
import sys

import numpy as np
import pytest

UNIT_COST, MIN_SLACK, GRAIN, ROWS = 2, 5, 64, 128


@pytest.fixture(params=[(2, 5), (6, 10)], autouse=True)
def costs(request, monkeypatch):
    """A unit's fixed cost in granules, and how near its border a cut moves: fp16 pools, FP8 pools."""
    monkeypatch.setattr(sys.modules[__name__], "UNIT_COST", request.param[0])
    monkeypatch.setattr(sys.modules[__name__], "MIN_SLACK", request.param[1])


def units_of(lens, nodes, group, hk, plane, planes):
    out, at = [], 0
    for L, C in zip(lens, nodes):
        if C == 0:
            continue
        n = -(-L // GRAIN) + UNIT_COST
        m = -(-C * group // ROWS)
        for _ in range(hk * max(0, -(-(m - plane) // planes))):
            out.append((at, n))
            at += n
    return out, at


def blocks_of(work, grid):
    """[(first, one past the last) block] of each plane."""
    if len(set(work)) == 1 and work[0]:  # equal work: as many blocks each, in step
        each = grid // len(work)
        return [(x * each, (x + 1) * each) for x in range(len(work))]
    f = np.float32
    total = f(0)
    for w in work:
        total = f(total + f(w))
    share, upto, nxt, out = f(f(grid) / total), f(0), 0, []
    later = sum(w > 0 for w in work)
    for w in work:
        upto = f(upto + f(w))
        later -= w > 0
        end = min(max(int(np.rint(f(upto * share))), nxt + (w > 0)), grid - later)
        out.append((nxt, end))
        nxt = end
    return out


def split(units, W, blocks):
    G = min(blocks, max(W, 1))
    slack = max(MIN_SLACK, W // G // 16)

    def moved(x):
        if x >= W:
            return W
        U, n = next(u for u in units if u[0] <= x < u[0] + u[1])
        d0, d1 = x - U, U + n - x
        if min(d0, d1) > slack:
            return x
        return U if d0 <= d1 else U + n

    quo, rem = divmod(W, G)
    cuts = [moved(quo * c + rem * c // G) for c in range(G + 1)]
    return G, slack, cuts


def pieces(U, n, W, G, slack):
    a, b = U + slack + 1, U + n - slack - 1
    lo, hi = (a * G + W - 1) // W, ((b + 1) * G + W - 1) // W - 1
    return (hi - lo + 2 if a <= b and hi >= lo else 1), lo - 1


def check(lens, nodes, group, hk, grid, planes=1):
    per_plane = [units_of(lens, nodes, group, hk, x, planes) for x in range(planes)]
    work = [W for _, W in per_plane]
    if not any(work):
        return
    last = 0
    for (units, W), (first, end) in zip(per_plane, blocks_of(work, grid)):
        assert first == last and end >= first and (end > first or W == 0)
        last = end
        if W:
            check_plane(units, W, end - first)
    assert last <= grid


def check_plane(units, W, blocks):
    G, slack, cuts = split(units, W, blocks)
    assert cuts[0] == 0 and cuts[-1] == W and all(a <= b for a, b in zip(cuts, cuts[1:]))
    held = {}
    for c in range(G):
        goes_on = began = 0
        for U, n in units:
            a, b = max(cuts[c], U), min(cuts[c + 1], U + n)
            if a >= b:
                continue
            assert max(a - U - UNIT_COST, 0) < min(b - U - UNIT_COST, n - UNIT_COST)   # granules g0 < g1
            held.setdefault(U, []).append((c, a, b))
            if (a, b) != (U, U + n):
                if b == U + n:
                    began += 1
                else:
                    goes_on += 1
        assert goes_on <= 1 and began <= 1
    for U, n in units:
        got = held[U]
        P, first = pieces(U, n, W, G, slack)
        assert len(got) == P
        assert got[0][1] == U and got[-1][2] == U + n
        assert all(x[2] == y[1] for x, y in zip(got, got[1:]))
        if P > 1:
            assert [c for c, _, _ in got] == list(range(first, first + P))
            assert all(b - a > slack for _, a, b in (got[0], got[-1]))


@pytest.mark.parametrize("lens,nodes,group,hk", [
    ([1], [1], 6, 2),
    ([4096 + 16], [16], 6, 2),
    ([32768 + 8] * 4, [8] * 4, 6, 2),
    ([1049] * 32, [25] * 32, 6, 2),
    ([4160] * 64, [64] * 64, 6, 2),
    ([20] * 1000, [3] * 1000, 6, 2),
    ([130000], [1], 24, 1),
    ([5000] * 40 + [60], [2] * 40 + [60], 6, 2),       # one small row with several M blocks
])
def test_split_of_known_batches(lens, nodes, group, hk):
    for grid in (4, 7, 132, 152, 192):
        for planes in (1, 2, 3, 4):
            check(lens, nodes, group, hk, grid, planes)


def test_split_of_random_batches():
    rng = random.Random(0)
    for _ in range(300):
        rows = rng.randint(1, 40)
        nodes = [rng.choice([0, 1, rng.randint(1, 200)]) for _ in range(rows)]
        lens = [n + rng.choice([0, rng.randint(0, 300), rng.randint(0, 20000)]) for n in nodes]
        check(lens, nodes, rng.choice([1, 4, 6, 7, 24]), rng.choice([1, 2, 8]), rng.choice([5, 148, 152, 160]),
              rng.choice([1, 2, 3, 4]))


def gather(head, P, piece, patience, shares):
    """A block's steps from its arrival on, one atomic access a step (the
    device code's order); appends the shares that it merges."""
    def inc():
        old = head["count"]
        head["count"] = 0 if old >= 2 * P - 1 else old + 1
        return old

    n = inc() + 1
    yield
    last = n == P
    while n < P:
        if patience == 0:
            head["gone"] |= 1 << piece
            yield
            n = head["count"]
            yield
            if n < P:
                return
            old = head["gone"]
            head["gone"] &= ~(1 << piece)
            yield
            if not old >> piece & 1:
                return
            break
        patience -= 1
        n = head["count"]
        yield
    inc()
    yield
    shares.append(piece)
    if last:
        bits, head["gone"] = head["gone"], 0
        yield
        for k in range(P):
            if bits >> k & 1:
                inc()
                yield
                shares.append(k)


def test_every_share_is_merged_once_and_the_words_return_to_zero():
    rng = random.Random(1)
    for _ in range(4000):
        P = rng.randint(2, 6)
        head, shares = {"count": 0, "gone": 0}, []
        blocks = [gather(head, P, k, rng.choice([0, 0, 1, 3, 50]), shares) for k in range(P)]
        late = rng.choice([None, rng.randrange(P)])   # a block that starts when all others are through
        while blocks:
            can = [b for k, b in enumerate(blocks) if len(blocks) == 1 or late is None or k != late] or blocks
            b = rng.choice(can)
            try:
                next(b)
            except StopIteration:
                if late is not None and blocks.index(b) < late:
                    late -= 1
                blocks.remove(b)
        assert sorted(shares) == list(range(P)) and head == {"count": 0, "gone": 0}
