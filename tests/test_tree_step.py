"""A step of several new tokens per row, without a GPU: the host functions
(rotary frequencies and rates, tree masks, the block manager's truncation) and
the refusals that are made before anything is launched."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_kv_cache_06_gb300 import ops
from paged_kv_cache_06_gb300.block_manager import BlockManager

INVALID, UNSUPPORTED, WORKSPACE, NOT_FOUND = 1, 2, 3, 7
FAKE = 0x100000       # aligned, non-null; never dereferenced by these calls
OTHER = 0x900000
ODD = 0x100008        # not 16-byte aligned


def P(x):
    return ctypes.c_void_p(x) if x else None


# ---- rotary frequencies and rates ----

def test_plain_frequencies():
    f = ops.rope_frequencies(64, base=500000.0)
    for i, x in enumerate(f.tolist()):
        assert x == pytest.approx(500000.0 ** (-2 * i / 64), rel=1e-14)


def test_linear_scaling_divides_every_frequency():
    f, g = ops.rope_frequencies(96), ops.rope_frequencies(96, scaling="linear", factor=4.0)
    assert torch.allclose(g * 4.0, f, rtol=1e-15, atol=0)


def test_base_scaling_keeps_the_fastest_pair_and_interpolates_the_slowest():
    f, g = ops.rope_frequencies(128), ops.rope_frequencies(128, scaling="base", factor=8.0)
    assert g[0] == f[0] == 1.0
    assert float(g[-1] * 8.0) == pytest.approx(float(f[-1]), rel=1e-12)
    assert bool((g[1:] < f[1:]).all())


def test_scaling_by_parts_leaves_fast_pairs_and_interpolates_slow_ones():
    f = ops.rope_frequencies(128)
    g = ops.rope_frequencies(128, scaling="by_parts", factor=8.0, original_len=4096.0, low=1.0, high=32.0)
    turns = 4096.0 * f / (2 * math.pi)
    assert bool((g[turns >= 32] == f[turns >= 32]).all())
    assert torch.allclose(g[turns <= 1] * 8.0, f[turns <= 1], rtol=1e-15, atol=0)
    between = (turns > 1) & (turns < 32)
    assert int(between.sum()) > 0
    w = (turns[between] - 1) / 31
    assert torch.allclose(g[between], w * f[between] + (1 - w) * f[between] / 8.0, rtol=1e-14, atol=0)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=15), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
    dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="linear", factor=float("inf")),
    dict(rot_dim=2, scaling="base", factor=2.0),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, original_len=0.0),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, original_len=100.0, low=4.0, high=4.0),
])
def test_bad_frequency_arguments(kw):
    with pytest.raises(ops.PagedKVError):
        ops.rope_frequencies(**kw)


def test_unknown_scaling_name():
    with pytest.raises(ValueError):
        ops.rope_frequencies(64, scaling="cubic")


def test_rates_are_fractions_of_a_turn():
    """rate / 2^64 is freq / 2 pi modulo one, to a double's relative precision."""
    freqs = torch.tensor([1.0, 0.5, 1e-3, 7.25e-9, 2 * math.pi / 4, 9.5, -0.25, 0.0], dtype=torch.float64)
    rates = ops.rope_rates(freqs, device="cpu")
    for f, r in zip(freqs.tolist(), rates.tolist()):
        got = Fraction(r % (1 << 64), 1 << 64)
        want = Fraction(f / (2 * math.pi)) % 1
        # the quotient is one rounding of a double; a negative one rounds once more on its way to [0, 1)
        off = abs(got - want)
        assert min(off, 1 - off) <= Fraction(1, 1 << 53) + Fraction(1, 1 << 64)


def test_rates_refuse_what_is_no_frequency():
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ops.PagedKVError):
            ops.rope_rates(torch.tensor([1.0, bad], dtype=torch.float64), device="cpu")
    with pytest.raises(ValueError):
        ops.rope_rates(torch.zeros(2, 2, dtype=torch.float64), device="cpu")


# ---- tree masks ----

def test_tree_mask_holds_a_node_and_its_ancestors():
    rng = np.random.default_rng(0)
    qs, parents = [0], []
    for n in (1, 0, 40, 7, 33):
        parents += [int(rng.integers(-1, i)) for i in range(n)]
        qs.append(qs[-1] + n)
    m = ops.tree_mask(parents, qs)
    assert m.shape == (81, 2) and m.dtype == torch.int32
    for a, b in zip(qs, qs[1:]):
        for i in range(b - a):
            seen, j = set(), i
            while j >= 0:
                seen.add(j)
                j = parents[a + j]
            words = [int(x) & 0xffffffff for x in m[a + i].tolist()]
            assert {j for j in range(64) if words[j // 32] >> (j % 32) & 1} == seen
    assert ops.tree_mask([], [0, 0]).shape == (0, 1)


def test_tree_mask_refusals():
    with pytest.raises(ValueError):
        ops.tree_mask([-1, 1], [0, 2])          # its own parent
    with pytest.raises(ValueError):
        ops.tree_mask([-1, -2], [0, 2])
    with pytest.raises(ValueError):
        ops.tree_mask([-1, 0], [0, 1])          # q_start does not cover the nodes
    with pytest.raises(ValueError):
        ops.tree_mask([-1] * 33, [0, 33], words=1)


# ---- refusals of the C entry points ----

def rope(**kw):
    a = dict(q_out=OTHER, k=FAKE, v=FAKE, ks=0, vs=0, bt=FAKE, sl=FAKE, qs=FAKE, rp=0, rates=FAKE, q=FAKE,
             kn=FAKE, vn=FAKE, sq=1536, sk=256, sv=256, rows=4, total=9, hq=12, hk=2, d=128, rot=128,
             layout=0, m=1.0, bs=16, mbpr=16, nb=64, msl=200)
    a.update(kw)
    return ops.lib().paged_kv_rope_append(
        *[P(a[n]) for n in ("q_out", "k", "v", "ks", "vs", "bt", "sl", "qs", "rp", "rates", "q", "kn", "vn")],
        a["sq"], a["sk"], a["sv"], a["rows"], a["total"], a["hq"], a["hk"], a["d"], a["rot"], a["layout"],
        a["m"], a["bs"], a["mbpr"], a["nb"], a["msl"], None, None)


def test_rope_append_refusals():
    for n in ("k", "v", "bt", "sl", "qs", "rates", "q", "kn", "vn", "q_out"):
        assert rope(**{n: 0}) == INVALID, n
    for n in ("k", "v", "q", "kn", "vn", "q_out"):
        assert rope(**{n: ODD}) == INVALID, n
    assert rope(rates=0x100004) == INVALID
    assert rope(ks=FAKE) == INVALID and rope(vs=FAKE) == INVALID       # one scale without the other
    assert rope(rot=0) == INVALID and rope(rot=144) == INVALID
    assert rope(rot=24) == UNSUPPORTED and rope(d=132, rot=128) == UNSUPPORTED
    assert rope(d=1040, rot=1040, sq=1 << 20, sk=1 << 20, sv=1 << 20) == UNSUPPORTED
    assert rope(hq=1024, sq=1 << 20) == UNSUPPORTED
    assert rope(layout=2) == INVALID and rope(m=float("nan")) == INVALID
    assert rope(sq=1528) == INVALID and rope(sq=1540) == INVALID       # too short; not a multiple of 8
    assert rope(sk=128) == INVALID and rope(sv=260) == INVALID
    assert rope(q_out=FAKE, sq=1544) == INVALID                        # in place needs equal layouts
    size = 9 * 12 * 128 * 2
    for off in (256, size - 16, -256, 16 - size):                      # over part of an input
        assert rope(q=OTHER + off) == INVALID, off
    for n, s in (("kn", "sk"), ("vn", "sv")):
        assert rope(**{n: OTHER}) == INVALID and rope(**{n: OTHER - 8 * 512 - 256, s: 256}) == INVALID
    assert rope(msl=257) == INVALID and rope(bs=0) == INVALID and rope(hk=0) == INVALID
    assert rope(nb=1 << 27, bs=16) == UNSUPPORTED
    assert rope(rows=0, k=0) == 0 and rope(total=0, q=0) == 0          # nothing to do


def tree(**kw):
    a = dict(out=OTHER, q=FAKE, k=FAKE, v=FAKE, ks=0, vs=0, bt=FAKE, sl=FAKE, qs=FAKE, mask=FAKE, words=1,
             rows=4, total=9, hq=12, hk=2, d=128, bs=16, scale=0.1, mbpr=16, nb=64, msl=200, ws=FAKE, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = ops.tree_workspace_size(4, 9, 12, 2, 128, 16)
    return ops.lib().paged_attention_tree(
        *[P(a[n]) for n in ("out", "q", "k", "v", "ks", "vs", "bt", "sl", "qs", "mask")], a["words"], a["rows"],
        a["total"], a["hq"], a["hk"], a["d"], a["bs"], a["scale"], a["mbpr"], a["nb"], a["msl"], P(a["ws"]),
        a["wsb"], None, None)


def test_tree_attention_refusals():
    for n in ("out", "q", "k", "v", "bt", "sl", "qs"):
        assert tree(**{n: 0}) == INVALID, n
    for n in ("out", "q", "k", "v"):
        assert tree(**{n: ODD}) == INVALID, n
    assert tree(ks=FAKE) == INVALID and tree(vs=FAKE) == INVALID
    assert tree(words=0) == INVALID and tree(words=33) == UNSUPPORTED
    assert tree(d=64) == UNSUPPORTED and tree(bs=24) == UNSUPPORTED and tree(rows=1025) == UNSUPPORTED
    assert tree(hq=12, hk=5) == INVALID and tree(scale=float("inf")) == INVALID
    for off in (0, 256, 9 * 12 * 256 - 16, 16 - 9 * 12 * 256):              # the output over the queries
        assert tree(q=OTHER + off) == INVALID, off
    assert tree(msl=257) == INVALID and tree(nb=0) == INVALID
    assert tree(ws=0) == WORKSPACE and tree(wsb=8) == WORKSPACE and tree(ws=0x100010) == WORKSPACE
    assert tree(rows=0, out=0) == 0 and tree(total=0, q=0) == 0


def test_tree_workspace_size_host_arithmetic():
    n = ops.tree_workspace_size(32, 500, 12, 2, 128, 64)
    assert n > 0 and n % 256 == 0
    assert ops.tree_workspace_size(32, 500, 12, 5, 128, 64) == 0
    assert ops.tree_workspace_size(-1, 500, 12, 2, 128, 64) == 0


def commit(**kw):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, qs=FAKE, path=FAKE, pl=FAKE, new=OTHER, layers=2, rows=4, mp=8,
             hk=2, d=128, eb=2, bs=16, mbpr=16, nb=64, msl=200)
    a.update(kw)
    return ops.lib().paged_kv_tree_commit(
        *[P(a[n]) for n in ("k", "v", "bt", "sl", "qs", "path", "pl", "new")], a["layers"], a["rows"], a["mp"],
        a["hk"], a["d"], a["eb"], a["bs"], a["mbpr"], a["nb"], a["msl"], None, None)


def test_tree_commit_refusals():
    for n in ("k", "v", "bt", "sl", "qs", "path", "pl"):
        assert commit(**{n: 0}) == INVALID, n
    assert commit(k=ODD) == INVALID and commit(v=ODD) == INVALID
    assert commit(new=FAKE) == INVALID and commit(new=FAKE + 12) == INVALID   # overlaps seq_lens
    for n, size in (("sl", 16), ("qs", 20), ("path", 128), ("pl", 16)):       # what every layer reads
        assert commit(**{n: OTHER - size + 4}) == INVALID and commit(**{n: OTHER + 12}) == INVALID, n
    assert commit(eb=4) == INVALID and commit(d=12) == UNSUPPORTED and commit(d=8, eb=1) == UNSUPPORTED
    assert commit(rows=-1) == INVALID and commit(mp=-1) == INVALID and commit(msl=257) == INVALID
    assert commit(nb=1 << 27) == UNSUPPORTED
    assert commit(rows=0, k=0) == 0 and commit(layers=0, k=0) == 0


def test_ops_refuse_cpu_tensors():
    h, i, w = torch.zeros(4, 12, 128, dtype=torch.float16), torch.zeros(4, dtype=torch.int32), None
    pool = torch.zeros(4, 16, 2, 128, dtype=torch.float16)
    bt, qs = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.tree_attention(h, h, pool, pool, bt, i, qs, 0.1, 16, ws, mask=w)
    with pytest.raises(ValueError):
        ops.rope_append(pool, pool, bt, i, qs, h[:, :2], h[:, :2], torch.zeros(64, dtype=torch.int64), 16)
    with pytest.raises(ValueError):
        ops.tree_commit(pool, pool, bt, i, qs, bt, i, 16)
    with pytest.raises(ValueError):
        ops.rope_append(pool, pool, bt, i, qs, h, h, torch.zeros(64, dtype=torch.int64), 16, layout="whole")


# ---- the block manager's side of a commit ----

def test_truncate_takes_drafted_tokens_back():
    bm = BlockManager(num_blocks=8, block_size=4, max_blocks_per_row=6)
    bm.admit(1, prompt_len=6, max_new_tokens=12)
    first, _ = bm.table(1)
    for k in range(7):
        assert bm.append_slot(1)[0] == 6 + k
    drafted, n = bm.table(1)
    assert n == 13 and (drafted[:4] >= 0).all()
    bm.truncate(1, 8)
    kept, n = bm.table(1)
    assert n == 8 and (kept == drafted).all()            # its blocks stay with it
    for k in range(6):                                   # and are used again, in the same order
        assert bm.append_slot(1)[0] == 8 + k
    again, n = bm.table(1)
    assert n == 14 and (again[:4] == drafted[:4]).all()
    assert bm.stats()["live_tokens"] == 14
    used = bm.stats()["used_blocks"]
    bm.free(1)
    assert used > 0 and bm.stats()["used_blocks"] == 0


def test_truncate_refusals():
    bm = BlockManager(num_blocks=4, block_size=4, max_blocks_per_row=4)
    bm.admit(1, prompt_len=6, max_new_tokens=4)
    for bad in (-1, 7):
        with pytest.raises(ops.PagedKVError) as e:
            bm.truncate(1, bad)
        assert e.value.status == INVALID
    with pytest.raises(ops.PagedKVError) as e:
        bm.truncate(2, 0)
    assert e.value.status == NOT_FOUND
    bm.truncate(1, 6)
    bm.truncate(1, 0)
    assert bm.table(1)[1] == 0


def test_truncate_into_a_shared_prefix_copies_on_the_next_write():
    bm = BlockManager(num_blocks=8, block_size=4, max_blocks_per_row=4)
    pid, ids = bm.register_prefix(8)
    bm.admit(1, prompt_len=9, max_new_tokens=4, prefix_id=pid)
    bm.truncate(1, 6)
    pos, cow = bm.append_slot(1)
    assert pos == 6 and cow is not None and cow[0] == int(ids[1])
