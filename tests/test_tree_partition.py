"""The tree kernel's work split, restated on the CPU: every granule of every
unit in exactly one block's range, cut units' pieces in consecutive blocks that
agree on their number and on the first of them, and at most one piece a block
of either kind (one that goes on behind its range, one that began before it)."""
import random

import pytest

MIN_GRANULES, GRANULE, ROWS = 4, 64, 128


def units_of(lens, nodes, group, hk):
    out, at = [], 0
    for L, C in zip(lens, nodes):
        if C == 0:
            continue
        n = -(-L // GRANULE)
        for _ in range(hk * -(-C * group // ROWS)):
            out.append((at, n))
            at += n
    return out, at


def split(units, W, grid):
    G = min(grid, max(W // MIN_GRANULES, 1))
    slack = max(MIN_GRANULES, W // G // 16)

    def moved(x):
        if x >= W:
            return W
        U, n = next(u for u in units if u[0] <= x < u[0] + u[1])
        d0, d1 = x - U, U + n - x
        if min(d0, d1) > slack:
            return x
        return U if d0 <= d1 else U + n

    cuts = [moved(W * c // G) for c in range(G + 1)]
    return G, slack, cuts


def pieces(U, n, W, G, slack):
    a, b = U + slack + 1, U + n - slack - 1
    lo, hi = (a * G + W - 1) // W, ((b + 1) * G + W - 1) // W - 1
    return (hi - lo + 2 if a <= b and hi >= lo else 1), lo - 1


def check(lens, nodes, group, hk, grid):
    units, W = units_of(lens, nodes, group, hk)
    if W == 0:
        return
    G, slack, cuts = split(units, W, grid)
    assert cuts[0] == 0 and cuts[-1] == W and all(a <= b for a, b in zip(cuts, cuts[1:]))
    held = {}
    for c in range(G):
        goes_on = began = 0
        for U, n in units:
            a, b = max(cuts[c], U), min(cuts[c + 1], U + n)
            if a >= b:
                continue
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
])
def test_split_of_known_batches(lens, nodes, group, hk):
    for grid in (1, 7, 132, 152, 192):
        check(lens, nodes, group, hk, grid)


def test_split_of_random_batches():
    rng = random.Random(0)
    for _ in range(300):
        rows = rng.randint(1, 40)
        nodes = [rng.choice([0, 1, rng.randint(1, 200)]) for _ in range(rows)]
        lens = [n + rng.choice([0, rng.randint(0, 300), rng.randint(0, 20000)]) for n in nodes]
        check(lens, nodes, rng.choice([1, 4, 6, 7, 24]), rng.choice([1, 2, 8]), rng.choice([3, 148, 152, 160]))
