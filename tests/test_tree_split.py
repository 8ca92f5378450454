"""The tree kernel's work split, its own source compiled for the host
(csrc/tree_split.cuh): every granule of every unit in exactly one block, cut
units' pieces in consecutive blocks that agree on how many there are and on the
first of them, ranges of nearly equal length, and sums that do not wrap."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_cache_06_gb300", "csrc")
GRAIN, ROWS, COST, SLACK = 64, 128, {False: 2, True: 6}, {False: 5, True: 10}


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Wno-unknown-pragmas",
                    "-I", CSRC, os.path.join(HERE, "tree_split_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.split_walk.restype = ctypes.c_longlong
    lib.split_walk.argtypes = [ctypes.c_int] * 2 + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 2 + \
        [ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong]
    return lib


def walk(host, fp8, cached, nodes, group, hk, grid, most=None):
    C, P = np.array(nodes, dtype=np.int32), np.array(cached, dtype=np.int32)
    units = int(sum(-(-c * group // ROWS) for c in nodes)) * hk if most is None else 0
    cap = units + 2 * grid + 8
    out = np.zeros((cap, 13), dtype=np.int32)
    n = host.split_walk(int(fp8), len(nodes), C.ctypes.data, P.ctypes.data, group, hk,
                        max(nodes, default=0) if most is None else most, grid, out.ctypes.data, cap)
    return out[:n] if n >= 0 else n


def check(host, fp8, cached, nodes, group, hk, grid):
    got = walk(host, fp8, cached, nodes, group, hk, grid)
    assert not isinstance(got, int), got
    want = {(r, k, m): -(-(p + c) // GRAIN) for r, (p, c) in enumerate(zip(cached, nodes)) if c
            for k in range(hk) for m in range(-(-c * group // ROWS))}
    held, blocks = {}, {}
    for block, plane, r, k, m, g0, g1, n, whole, np_, first, s0, e in got.tolist():
        assert want[r, k, m] == n and 0 <= g0 < g1 <= n
        held.setdefault((r, k, m), []).append((block, g0, g1, whole, np_, first))
        blocks.setdefault(block, []).append((r, k, m, g0, g1, n, np_, s0, e, plane))
    assert held.keys() == want.keys()
    for key, pieces in held.items():
        assert pieces == sorted(pieces)
        assert pieces[0][1] == 0 and pieces[-1][2] == want[key]
        assert all(x[2] == y[1] and y[0] == x[0] + 1 for x, y in zip(pieces, pieces[1:]))
        for block, _, _, whole, np_, first in pieces:
            assert bool(whole) == (len(pieces) == 1) and np_ == len(pieces)
            assert np_ == 1 or first == pieces[0][0]
    work = {}
    for r, k, m in want:
        x = m % planes_of(nodes, group)
        work[x] = work.get(x, 0) + want[r, k, m] + COST[fp8]
    for segs in blocks.values():
        # walked from the last unit to the first; a piece that goes on behind the range comes
        # first, one that began before it last
        assert [s[:3] for s in segs] == sorted((s[:3] for s in segs), reverse=True)
        for i, (r, k, m, g0, g1, n, np_, s0, e, plane) in enumerate(segs):
            assert plane == m % planes_of(nodes, group)
            assert g1 == n or i == 0
            assert g0 == 0 or i == len(segs) - 1
    if len(work) == 1:  # one plane: the blocks' ranges differ by no more than their moved cuts
        W = sum(work.values())
        quo = W // min(grid, W)
        assert all(s[0][8] - s[0][7] <= quo + 1 + 2 * max(SLACK[fp8], quo // 16) for s in blocks.values())


def planes_of(nodes, group):
    return min(4, max(1, -(-max(nodes) * group // ROWS)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cached,nodes,group,hk", [
    ([0], [1], 6, 2),
    ([4096], [16], 6, 2),
    ([32768] * 4, [8] * 4, 6, 2),
    ([1024] * 32, [25] * 32, 6, 2),
    ([4096] * 64, [64] * 64, 6, 2),
    ([20] * 1000, [3] * 1000, 6, 2),
    ([17] * 1024, [1] * 1023 + [500], 6, 2),
    ([130000], [1], 24, 1),
    ([2000000], [3], 6, 8),
    ([0], [16384], 4, 8),
    ([5000] * 40 + [0], [2] * 40 + [60], 6, 2),
    ([300, 0, 17], [0, 1, 0], 1, 1),
])
def test_known_batches(host, fp8, cached, nodes, group, hk):
    for grid in (4, 7, 132, 148, 152, 192):
        check(host, fp8, cached, nodes, group, hk, grid)


@pytest.mark.parametrize("fp8", [False, True])
def test_random_batches(host, fp8):
    rng = random.Random(int(fp8))
    for _ in range(200):
        rows = rng.choice([1, 2, rng.randint(1, 40), rng.randint(200, 1024)])
        top = 20000 if rows < 50 else 900
        nodes = [rng.choice([0, 1, rng.randint(1, 200)]) for _ in range(rows)]
        if not any(nodes):
            nodes[rng.randrange(rows)] = 1
        cached = [rng.choice([0, rng.randint(0, 300), rng.randint(0, top)]) for _ in range(rows)]
        check(host, fp8, cached, nodes, rng.choice([1, 4, 6, 7, 24]), rng.choice([1, 2, 8]),
              rng.choice([5, 148, 152, 160, 192]))


def test_work_beyond_31_bits_is_refused(host):
    """512 rows that all name 16384 nodes of eight KV heads over 200,000 tokens."""
    rows, T, L = 1024, 16384, 200000
    nodes = [T if r % 2 == 0 else 0 for r in range(rows)]
    assert walk(host, False, [L - c for c in nodes], nodes, 8, 8, 152, most=T) == -1
    assert walk(host, True, [L - c for c in nodes], nodes, 8, 8, 152, most=T) == -1


def test_division(host):
    rng = random.Random(3)
    cases = [(0, 1), (2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 2, 2 ** 31 - 1), (2 ** 31 - 1, 2)]
    for _ in range(200000):
        a, b = rng.getrandbits(rng.randint(1, 31)), max(1, rng.getrandbits(rng.randint(1, 31)))
        cases.append((a, b))
        cases.append((min(2 ** 31 - 1, a // b * b), b))
    for a, b in cases:
        assert host.split_div(a, b) == a // b, (a, b)
