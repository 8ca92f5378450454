"""GPU parity of a step of several new tokens per row: rotary append, tree
attention and path commit against plain 64-bit forms, and the three together.

Tolerances are worst-case sums of the roundings that the operators are allowed
(u = 2^-24 for 32-bit arithmetic, h = 2^-11 for a rounding to fp16):

* rotary: the angle is within pi u (the turn fraction as a float) + 2^-30 of
  exact, sincospif within 2 ulp (4 u at most), the scaling, the two products
  and the sum 4 u: in all below 12 u m (|a| + |b|), then h |ref| (2^-25 below
  the normal range), or half an E4M3 step of the stored quotient.
* attention: with A = sum_t p_t |v_t|, weights rounded to fp16 give h A; a
  score's dot product is off by at most 130 u scale sum_d |q_d k_d| =: e, which
  moves weights and their sum by 2 e A; exponent and normalisation 8 u A; sums
  over L tokens L u A at most; a weight below fp16's normal range is off by
  2^-25 of the row's reference weight, sum_t |v_t| 2^-25 in all; the output
  h |ref| + 2^-25.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_06_gb300 import ops
from paged_kv_cache_06_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -11
ERR_BLOCK, ERR_LEN, ERR_POS, ERR_TIMEOUT, ERR_MASK = 1, 2, 4, 8, 32
NAN8 = 0x7F


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Step:
    """Rows of `prefix` cached tokens and `nodes` new ones, with block tables
    over a pool whose unused slots hold NaN."""

    def __init__(self, prefix, nodes, bs, hk=2, d=128, fp8=False, seed=0, extra=2, layers=None, fill=True):
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.prefix, self.nodes, self.bs, self.hk, self.d, self.fp8 = list(prefix), list(nodes), bs, hk, d, fp8
        self.rows = len(prefix)
        self.lens = [p + n for p, n in zip(prefix, nodes)]
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
        self.total = int(self.starts[-1])
        need = [(n + bs - 1) // bs for n in self.lens]
        self.nb = sum(need) + extra
        perm = rng.permutation(self.nb)
        self.tables = np.full((self.rows, max(1, max(need))), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(need):
            self.tables[r, :n] = perm[at:at + n]
            at += n
        self.max_len = max(self.lens)
        shape = ((layers,) if layers else ()) + (self.nb, bs, hk, d)
        self.k_scale = self.v_scale = None
        if fp8:
            self.k_scale = (0.02 + 0.02 * torch.rand(hk, generator=self.gen))
            self.v_scale = (0.02 + 0.02 * torch.rand(hk, generator=self.gen))
            pools = [self.codes(shape) for _ in range(2)]
        else:
            pools = [torch.randn(shape, generator=self.gen).half() for _ in range(2)]
        self.k_pool, self.v_pool = pools
        if fill and not layers:  # slots that no row's tokens occupy
            free = torch.ones(self.nb * bs, dtype=torch.bool)
            for r in range(self.rows):
                free[self.slots(r)] = False
            for p in pools:
                p.view(-1, hk, d)[free] = NAN8 if fp8 else float("nan")

    def codes(self, shape):
        x = torch.randn(shape, generator=self.gen) / 0.03
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def slots(self, r, a=0, b=None):
        t = np.arange(a, self.lens[r] if b is None else b)
        return torch.from_numpy(self.tables[r, t // self.bs].astype(np.int64) * self.bs + t % self.bs)

    def values(self, pool, r, scale):
        """Row r's tokens as float64 [L][hk][d]."""
        x = pool.view(-1, self.hk, self.d)[self.slots(r)]
        x = x.view(torch.float8_e4m3fn).double() if self.fp8 else x.double()
        return x * scale.double()[:, None] if scale is not None else x

    def gpu(self, **kw):
        a = dict(k_pool=self.k_pool.cuda(), v_pool=self.v_pool.cuda(), block_tables=i32(self.tables),
                 seq_lens=i32(self.lens), q_start=i32(self.starts),
                 k_scale=None if self.k_scale is None else self.k_scale.cuda(),
                 v_scale=None if self.v_scale is None else self.v_scale.cuda())
        a.update(kw)
        return a


def random_parents(nodes, seed):
    rng = np.random.default_rng(seed)
    return [int(rng.integers(max(-1, i - 9), i)) for n in nodes for i in range(n)]


def seen_of(step, mask):
    """Per row [C][C] booleans from mask words (None: a chain)."""
    out = []
    for r, n in enumerate(step.nodes):
        if mask is None:
            out.append(torch.tril(torch.ones(n, n, dtype=torch.bool)))
        else:
            w = mask[step.starts[r]:step.starts[r] + n].long() & 0xffffffff
            j = torch.arange(n)
            out.append((w[:, j // 32] >> (j % 32) & 1).bool() if n else torch.ones(0, 0, dtype=torch.bool))
    return out


def tree_ref(step, q, seen, scale, skip=None):
    """(output, tolerance) in float64; skip: per row, tokens that nobody sees."""
    hq = q.shape[1]
    g = hq // step.hk
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    for r, n in enumerate(step.nodes):
        if n == 0:
            continue
        a = int(step.starts[r])
        k = step.values(step.k_pool, r, step.k_scale).permute(1, 0, 2).repeat_interleave(g, 0)
        v = step.values(step.v_pool, r, step.v_scale).permute(1, 0, 2).repeat_interleave(g, 0)
        x = q[a:a + n].double().permute(1, 0, 2)
        vis = torch.cat([torch.ones(n, step.prefix[r], dtype=torch.bool), seen[r]], 1)
        vis[:, (skip or {}).get(r, [])] = False
        kz, vz = torch.nan_to_num(k, posinf=0, neginf=0), torch.nan_to_num(v, posinf=0, neginf=0)
        s = (x @ kz.transpose(1, 2)) * scale
        s = torch.where(vis, s, torch.full_like(s, -np.inf))
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        p = torch.where(l > 0, p / torch.where(l > 0, l, torch.ones_like(l)), torch.zeros_like(p))
        o, big = p @ vz, p @ vz.abs()
        e = 130 * U * abs(scale) * (x.abs() @ kz.abs().transpose(1, 2)).where(vis, torch.zeros(())).amax(-1, keepdim=True)
        low = 2.0 ** -25 * (vis.double() @ vz.abs())
        out[a:a + n] = o.permute(1, 0, 2)
        tol[a:a + n] = (H * o.abs() + (H + 2 * e + (8 + step.lens[r]) * U) * big + low + 2.0 ** -25).permute(1, 0, 2)
    return out, tol


def check(got, ref, tol, what=""):
    got = got.double().cpu()
    assert bool(torch.isfinite(got).all()), what
    over = (got - ref).abs() - tol
    if bool((over > 0).any()):
        i = np.unravel_index(int(over.argmax()), over.shape)
        pytest.fail(f"{what}: {int((over > 0).sum())} of {over.numel()} outside tolerance; worst at {i}: "
                    f"{float(got[i])} for {float(ref[i])}, allowed {float(tol[i])}")


def tree_run(step, q, mask, scale, err=None, stream=None, workspace=None, total=None, **kw):
    hq = q.shape[1]
    gq = q.cuda()
    out = torch.full(gq.shape, float("nan"), dtype=torch.float16, device="cuda")
    ws = workspace if workspace is not None else ops.alloc_tree_workspace(
        step.rows, q.shape[0], hq, step.hk, step.d, step.bs)
    a = step.gpu(**kw)
    gm = None if mask is None else mask.cuda()
    torch.cuda.synchronize()
    ops.tree_attention(out, gq, a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], scale,
                       step.max_len, ws, mask=gm, k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err,
                       stream=stream)
    torch.cuda.synchronize()
    return out


TREES = [
    # prefix, nodes, block size, q heads, kv heads
    ([0], [1], 16, 12, 2),                              # one token, nothing cached
    ([1, 0, 17, 200], [1, 2, 3, 8], 16, 12, 2),
    ([63, 64, 65, 127, 128, 129], [1, 1, 1, 1, 1, 1], 64, 12, 2),
    ([63, 64, 65, 127, 128, 129], [7, 64, 33, 1, 130, 2], 64, 12, 2),   # nodes over tile borders
    ([1000, 5, 333], [0, 21, 22], 48, 12, 2),           # a row without nodes; one query tile and one more
    ([4096], [16], 64, 12, 2),
    ([9000, 3, 40, 700], [5, 5, 31, 32], 32, 12, 2),    # one long row among short ones
    ([50] * 60, [4] * 60, 16, 12, 2),                   # many short rows
    ([700, 130], [150, 200], 128, 12, 2),               # several query tiles a row
    ([300, 31], [9, 40], 16, 4, 4),                     # heads of their own
    ([300, 31], [9, 40], 16, 32, 8),
    ([300, 2000], [9, 40], 112, 28, 4),
    ([257, 90], [11, 3], 16, 24, 1),                    # a group wider than the decode kernels take
    ([90, 20], [3, 300], 16, 5, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree_matches_the_formula(cuda_device, case, fp8):
    prefix, nodes, bs, hq, hk = TREES[case]
    step = Step(prefix, nodes, bs, hk=hk, fp8=fp8, seed=100 + case)
    q = torch.randn(step.total, hq, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(nodes, case), step.starts)
    err = err_word()
    ref, tol = tree_ref(step, q, seen_of(step, mask), 0.0883)
    got = tree_run(step, q, mask, 0.0883, err)
    assert int(err.item()) == 0
    check(got, ref, tol, f"tree {case}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", [1, 3, 6, 8, 11])
def test_chain_matches_the_formula(cuda_device, case, fp8):
    prefix, nodes, bs, hq, hk = TREES[case]
    step = Step(prefix, nodes, bs, hk=hk, fp8=fp8, seed=200 + case)
    q = torch.randn(step.total, hq, 128, generator=step.gen).half()
    ref, tol = tree_ref(step, q, seen_of(step, None), 0.0883)
    check(tree_run(step, q, None, 0.0883), ref, tol, f"chain {case}")


@pytest.mark.parametrize("prefix,nodes,hq,hk", [
    ([300, 17, 2000, 64], [22] * 4, 12, 2),      # two M blocks a row, the second nearly empty
    ([300, 17, 2000, 64], [43, 64, 50, 60], 12, 2),              # three, of unequal nodes
    ([0] * 40, [86] * 40, 6, 1),                 # four and a part: not even
    ([900, 31, 700] * 6, [85] * 18, 12, 2),      # four
    ([20000], [64], 12, 2),                      # one row over all blocks
    ([1], [33], 4, 1),                           # less work than blocks
    ([100, 5000, 3], [64, 0, 64], 8, 2),         # and a row without nodes
])
def test_rows_of_equally_many_query_tiles(cuda_device, prefix, nodes, hq, hk):
    """Blocks that read the same tokens for different query tiles load them
    together: against 64 bits, with numbers that are none in unseen and seen
    values, a bad table entry, and the same bits every time."""
    step = Step(prefix, nodes, 16, hk=hk, seed=sum(nodes))
    q = torch.randn(step.total, hq, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(nodes, 5), step.starts)
    ref, tol = tree_ref(step, q, seen_of(step, mask), 0.0883)
    err = err_word()
    got = tree_run(step, q, mask, 0.0883, err)
    assert int(err.item()) == 0
    check(got, ref, tol)
    for _ in range(3):
        assert torch.equal(tree_run(step, q, mask, 0.0883), got)
    # a cached token's block out of range: nobody sees its sixteen tokens
    r = int(np.argmax([p if n else -1 for p, n in zip(step.prefix, step.nodes)]))
    if step.prefix[r] >= 32:
        t = step.tables.copy()
        t[r, 1] = step.nb
        ref, tol = tree_ref(step, q, seen_of(step, mask), 0.0883, skip={r: list(range(16, 32))})
        check(tree_run(step, q, mask, 0.0883, err, block_tables=i32(t)), ref, tol)
        assert ops.check_error(err) == ERR_BLOCK
    # the first row's last node holds an infinity in V: it reaches those who see it alone
    a, n = int(step.starts[0]), step.nodes[0]
    step.v_pool.view(-1, hk, 128)[step.slots(0, step.prefix[0] + n - 1)] = float("inf")
    got2 = tree_run(step, q, mask, 0.0883)
    sees = torch.zeros(step.total, dtype=torch.bool)
    sees[a:a + n] = seen_of(step, mask)[0][:, n - 1]
    assert torch.equal(got2[~sees.cuda()], got[~sees.cuda()])
    assert bool(torch.isinf(got2[sees.cuda()]).all())


def test_large_scores_and_scale(cuda_device):
    """Scores far apart: the running maximum moves late and often."""
    step = Step([1500, 700], [20, 9], 64, seed=7)
    q = (torch.randn(step.total, 12, 128, generator=step.gen) * 6).half()
    for r in range(2):  # keys grow along the row
        s = step.slots(r)
        f = torch.linspace(0.05, 4.0, len(s))[:, None, None]
        kp = step.k_pool.view(-1, 2, 128)
        kp[s] = (kp[s].float() * f).half()
    mask = ops.tree_mask(random_parents(step.nodes, 3), step.starts)
    for scale in (0.3, -0.2):
        ref, tol = tree_ref(step, q, seen_of(step, mask), scale)
        check(tree_run(step, q, mask, scale), ref, tol, f"scale {scale}")


def test_masks_that_leave_nothing_or_only_others(cuda_device):
    """Rows with no cached token whose nodes see nothing, only a later node, or
    all; and bits set past the row's nodes."""
    step = Step([0, 0, 40], [5, 70, 3], 16, seed=9)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = torch.zeros(step.total, 4, dtype=torch.int32)
    mask[1, 0] = 1 << 4                  # node 1 of row 0 sees node 4 alone
    mask[3, 0] = -1                      # node 3 sees all five (and bits past them)
    mask[3, 1:] = -1
    mask[5 + 10, 2] = 1 << 5             # node 10 of row 1 sees node 69
    mask[5 + 69, :] = -1
    mask[75, 1] = -1                     # row 2: bits of nodes that are not there
    ref, tol = tree_ref(step, q, seen_of(step, mask), 0.1)
    got = tree_run(step, q, mask, 0.1)
    check(got, ref, tol, "sparse masks")
    empty = [0, 2, 4] + [5 + i for i in range(69) if i != 10]
    assert bool((got[empty] == 0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_what_a_node_does_not_see_does_not_reach_it(cuda_device, fp8):
    """Infinities and NaN in nodes that others do not see."""
    step = Step([100, 0, 250], [12, 40, 9], 16, fp8=fp8, seed=11)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(step.nodes, 5), step.starts)
    # nodes 4 and 7 of row 0, 33 of row 1, 2 of row 2 hold what is no number
    bad = [(0, 4), (0, 7), (1, 33), (2, 2)]
    kp, vp = step.k_pool.view(-1, 2, 128), step.v_pool.view(-1, 2, 128)
    for i, (r, j) in enumerate(bad):
        s = step.slots(r)[step.prefix[r] + j]
        for p in (kp, vp):
            if fp8:
                p[s, :, 3:9] = NAN8 | (0x80 if i % 2 else 0)
            else:
                p[s, :, 3:9] = [float("inf"), float("nan"), float("-inf"), float("nan")][i]
    seen = seen_of(step, mask)
    touched = torch.zeros(step.total, dtype=torch.bool)
    for r, j in bad:
        a = int(step.starts[r])
        touched[a:a + step.nodes[r]] |= seen[r][:, j]
    assert 0 < int(touched.sum()) < step.total
    ref, tol = tree_ref(step, q, seen, 0.1)
    got = tree_run(step, q, mask, 0.1)
    ok = ~touched
    check(got[ok.cuda()], ref[ok], tol[ok], "unseen")
    # a node that sees a NaN key has no number for an answer
    for r, j in bad:
        if fp8 or not (r, j) in ((0, 4), (1, 33)):
            a = int(step.starts[r])
            rows = torch.nonzero(seen[r][:, j]).flatten() + a
            assert bool(torch.isnan(got[rows.cuda()]).all())


def test_values_that_are_no_numbers_reach_those_who_see_them(cuda_device):
    """Only V is not finite: exactly the dims concerned follow, for the nodes
    that see it."""
    step = Step([130, 20], [30, 6], 16, seed=12)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(step.nodes, 6), step.starts)
    vp = step.v_pool.view(-1, 2, 128)
    s0, s1 = step.slots(0)[130 + 3], step.slots(1)[20 + 1]
    vp[s0, 0, 10], vp[s0, 0, 90], vp[s1, 1, 64] = float("inf"), float("-inf"), float("nan")
    seen = seen_of(step, mask)
    ref, tol = tree_ref(step, q, seen, 0.1)
    got = tree_run(step, q, mask, 0.1).double().cpu()
    want = ref.clone()
    a = torch.nonzero(seen[0][:, 3]).flatten()
    b = torch.nonzero(seen[1][:, 1]).flatten() + 30
    want[a, 0:6, 10], want[a, 0:6, 90] = float("inf"), float("-inf")
    for n in b.tolist():
        want[n, 6:12, 64] = float("nan")
    plain = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    assert bool(((got - ref).abs()[plain] <= tol[plain]).all())


def test_one_node_equals_decode_and_a_chain_equals_prefill(cuda_device):
    """The same attention through the operators that were there (2e-3 + 2e-3
    |ref| is their tolerance; both sides take half of it at most)."""
    step = Step([300, 0, 64], [1, 1, 1], 64, seed=13)
    q = torch.randn(3, 12, 128, generator=step.gen).half()
    a = step.gpu()
    out = torch.empty(3, 12, 128, dtype=torch.float16, device="cuda")
    ws = ops.alloc_workspace(3, 12, 2, 128, step.max_len, 64)
    ops.decode(out, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, step.max_len, ws)
    got = tree_run(step, q, None, 0.0883)
    assert bool(((got - out).float().abs() <= 2e-3 + 2e-3 * out.float().abs()).all())
    step = Step([300, 0, 64], [40, 129, 5], 64, seed=14)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    a = step.gpu()
    out = torch.empty(step.total, 12, 128, dtype=torch.float16, device="cuda")
    ops.prefill(out, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.0883,
                step.max_len)
    got = tree_run(step, q, None, 0.0883)
    assert bool(((got - out).float().abs() <= 2e-3 + 2e-3 * out.float().abs()).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_every_time_and_under_another_block_order(cuda_device, fp8):
    step = Step([5000, 40, 900, 0], [9, 33, 17, 50], 16, fp8=fp8, seed=15)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(step.nodes, 7), step.starts)
    ws = ops.alloc_tree_workspace(4, step.total, 12, 2, 128, 16)
    first = tree_run(step, q, mask, 0.1, workspace=ws)
    for _ in range(3):
        assert torch.equal(tree_run(step, q, mask, 0.1, workspace=ws), first)
    perm = torch.randperm(step.nb, generator=step.gen)
    inv = torch.argsort(perm)
    kp, vp = step.k_pool[perm].cuda(), step.v_pool[perm].cuda()
    t = step.tables.copy()
    t[t >= 0] = inv.numpy()[t[t >= 0]]
    assert torch.equal(tree_run(step, q, mask, 0.1, workspace=ws, k_pool=kp, v_pool=vp, block_tables=i32(t)), first)


def test_rows_behind_the_last_sequence_are_left_as_they_were(cuda_device):
    step = Step([30, 70], [4, 9], 16, seed=16)
    q = torch.randn(step.total + 6, 12, 128, generator=step.gen).half()
    mask = torch.cat([ops.tree_mask(random_parents(step.nodes, 8), step.starts),
                      torch.full((6, 1), -1, dtype=torch.int32)])
    got = tree_run(step, q, mask, 0.1)
    assert bool(torch.isnan(got[step.total:]).all())
    ref, tol = tree_ref(step, q[:step.total], seen_of(step, mask), 0.1)
    check(got[:step.total], ref, tol)


def test_bad_rows_and_blocks_are_flagged_and_skipped(cuda_device):
    step = Step([30, 70, 200, 10], [4, 9, 3, 40], 16, seed=17)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask2 = torch.full((step.total, 2), -1, dtype=torch.int32)
    good = tree_run(step, q, mask2, 0.1)
    # a row of more nodes than the mask has bits
    err = err_word()
    got = tree_run(step, q, mask2[:, :1].contiguous(), 0.1, err)
    assert ops.check_error(err) == ERR_MASK and ops.check_error(err) == 0
    assert bool(torch.isnan(got[16:]).all()) and torch.equal(got[:16], good[:16])
    # a length above the bound, and one below the row's nodes
    for lens, gone in (([34, 10000, 203, 50], slice(4, 13)), ([34, 8, 203, 50], slice(4, 13)),
                       ([-1, 79, 203, 50], slice(0, 4))):
        err = err_word()
        got = tree_run(step, q, mask2, 0.1, err, seq_lens=i32(lens))
        assert ops.check_error(err) == ERR_LEN
        assert bool(torch.isnan(got[gone]).all())
        keep = torch.ones(step.total, dtype=torch.bool)
        keep[gone] = False
        assert torch.equal(got[keep.cuda()], good[keep.cuda()])
    # block ids out of range: their tokens are skipped
    t = step.tables.copy()
    t[2, 3], t[2, 12] = step.nb, -7     # tokens 48..63 and 192..202 of row 2 (its nodes among them)
    err = err_word()
    got = tree_run(step, q, mask2, 0.1, err, block_tables=i32(t))
    assert ops.check_error(err) == ERR_BLOCK
    want, tol = tree_ref(step, q, seen_of(step, mask2), 0.1, skip={2: [*range(48, 64), *range(192, 203)]})
    check(got[13:16], want[13:16], tol[13:16], "skipped blocks")
    keep = torch.ones(step.total, dtype=torch.bool)
    keep[13:16] = False
    assert torch.equal(got[keep.cuda()], good[keep.cuda()])


def test_two_streams_and_captured_graphs(cuda_device):
    """Two calls at once on workspaces of their own; two captured graphs that
    share a workspace, replayed in turn with changed inputs."""
    steps = [Step([3000, 20, 150], [9, 30, 1], 16, seed=18), Step([800] * 12, [5] * 12, 64, fp8=True, seed=19)]
    qs = [torch.randn(s.total, 12, 128, generator=s.gen).half() for s in steps]
    masks = [ops.tree_mask(random_parents(s.nodes, 9), s.starts) for s in steps]
    want = [tree_run(s, q, m, 0.1) for s, q, m in zip(steps, qs, masks)]
    args, outs = [], []
    for s, q, m in zip(steps, qs, masks):
        a = s.gpu()
        outs.append(torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda"))
        args.append((outs[-1], q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"],
                     0.1, s.max_len, m.cuda(), a["k_scale"], a["v_scale"]))

    def call(i, ws, stream=None):
        o, q, k, v, bt, sl, st, sc, ml, m, ks, vs = args[i]
        ops.tree_attention(o, q, k, v, bt, sl, st, sc, ml, ws, mask=m, k_scale=ks, v_scale=vs, stream=stream)

    ws = [ops.alloc_tree_workspace(s.rows, s.total, 12, 2, 128, s.bs) for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, ws[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    # graphs on one workspace, of the larger step's size
    shared = max(ws, key=lambda x: x.numel())
    graphs = []
    for i in range(2):
        outs[i].fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, shared)
        graphs.append(g)
    for k in range(4):
        graphs[k % 2].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    args[0][1].copy_(-args[0][1])     # new queries under the same graph
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], tree_run(steps[0], -qs[0], masks[0], 0.1))


# ---- rotary append ----

def rotate_ref(x, pos, freqs, layout, m):
    """float64 rotation of [T][heads][d]; (result, 12 u m (|a| + |b|))."""
    rot = 2 * len(freqs)
    x = x.double()
    ang = pos.double()[:, None] * freqs[None, :]
    c, s = (m * torch.cos(ang))[:, None], (m * torch.sin(ang))[:, None]
    y, e = x.clone(), torch.zeros_like(x)
    if layout == "half":
        ia, ib = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    else:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    e[..., ia] = e[..., ib] = 12 * U * abs(m) * (a.abs() + b.abs())
    return y, e


def fp16_tol(ref):
    return H * ref.abs() + 2.0 ** -25


def code_values(x):
    return x.view(torch.float8_e4m3fn).double()


def e4m3_tol(ref):
    """Half a step: 2^-4 of the value's binade, 2^-10 below the normal range."""
    return torch.clamp(torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -6)))) * 2.0 ** -4, min=2.0 ** -10)


ROPES = [
    # prefix, nodes, bs, q heads, kv heads, head dim, rotated, layout
    ([0], [1], 16, 12, 2, 128, 128, "half"),
    ([5, 0, 100, 31], [1, 3, 0, 9], 16, 12, 2, 128, 128, "half"),
    ([5, 0, 100, 31], [1, 3, 0, 9], 16, 12, 2, 128, 128, "interleaved"),
    ([5, 7, 100, 31], [17, 3, 64, 9], 5, 12, 2, 128, 64, "half"),
    ([5, 7, 100, 31], [17, 3, 64, 9], 48, 32, 8, 128, 96, "interleaved"),
    ([11] * 40, [1] * 40, 64, 4, 4, 64, 32, "half"),
    ([11, 900], [700, 301], 64, 12, 2, 128, 128, "half"),        # several tokens a block
    ([11, 900], [700, 301], 64, 7, 1, 80, 16, "interleaved"),
    ([3, 1], [400, 600], 16, 3, 1, 256, 256, "half"),
    ([3] * 1100, [1] * 1100, 16, 2, 1, 64, 64, "interleaved"),   # more rows than a block has threads
    ([7, 300, 0], [1500, 0, 907], 64, 12, 2, 128, 128, "half"),  # four tokens a block, the last one part full
    ([1], [25000], 128, 1, 1, 64, 32, "half"),                   # the most tokens a block
    ([9], [9200], 16, 1, 1, 1024, 1024, "interleaved"),          # a table of factors of the most pairs
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(ROPES)))
def test_rope_append_matches_the_formula(cuda_device, case, fp8):
    prefix, nodes, bs, hq, hk, d, rot, layout = ROPES[case]
    step = Step(prefix, nodes, bs, hk=hk, d=d, fp8=fp8, seed=300 + case, fill=False)
    T = step.total
    m = [1.0, 1.25][case % 2]
    # every second case takes views of one projection's output
    if case % 2:
        qkv = torch.randn(T, hq + 2 * hk, d, generator=step.gen).half().cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = (torch.randn(T, n, d, generator=step.gen).half().cuda() for n in (hq, hk, hk))
    freqs = ops.rope_frequencies(rot, base=10000.0, scaling="by_parts", factor=4.0, original_len=2048.0)
    rng = np.random.default_rng(case)
    pos = torch.from_numpy(rng.integers(-5000, 2_000_000, T)) if case != 1 else None
    own = torch.cat([torch.arange(p, p + n) for p, n in zip(prefix, nodes)])
    a = step.gpu()
    q_out = torch.full((T, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    err = err_word()
    ops.rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], k, v,
                    ops.rope_rates(freqs), step.max_len, layout=layout, q=q, q_out=q_out,
                    rope_positions=None if pos is None else pos.to(torch.int32).cuda(), mscale=m,
                    k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    at = own if pos is None else pos
    ref, e = rotate_ref(q.cpu(), at, freqs, layout, m)
    check(q_out, ref, e + fp16_tol(ref), "queries")
    slots = torch.cat([step.slots(r, step.prefix[r]) for r in range(step.rows)])
    kref, ke = rotate_ref(k.cpu(), at, freqs, layout, m)
    kp, vp = a["k_pool"].cpu(), a["v_pool"].cpu()
    got_k, got_v = kp.view(-1, hk, d)[slots], vp.view(-1, hk, d)[slots]
    if fp8:
        s = step.k_scale.double()[:, None]
        check(code_values(got_k), kref / s, (ke + U * kref.abs()) / s + e4m3_tol(kref / s), "keys")
        bits = v.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)
        at_block, at_slot = np.divmod(slots.numpy().astype(np.int32), bs)   # a row of one block per token
        _, want_v = oracle.paged_append_fp8(step.k_pool.numpy(), step.v_pool.numpy(), step.k_scale.numpy(),
                                            step.v_scale.numpy(), at_block[:, None], at_slot, bits, bits)
        assert np.array_equal(vp.numpy(), want_v)
    else:
        check(got_k, kref, ke + fp16_tol(kref), "keys")
        assert torch.equal(got_v.view(torch.int16), v.cpu().view(torch.int16))
    # nothing else was written
    rest = torch.ones(step.nb * bs, dtype=torch.bool)
    rest[slots] = False
    it = torch.uint8 if fp8 else torch.int16
    for got, was in ((kp, step.k_pool), (vp, step.v_pool)):
        assert torch.equal(got.view(-1, hk, d)[rest].view(it), was.view(-1, hk, d)[rest].view(it))


def test_rope_far_positions_keep_their_digits(cuda_device):
    """One pair a token, at positions up to 2^31 - 1: cos and sin as exact as
    near zero."""
    T = 64
    step = Step([0], [T], 16, hk=1, d=64, seed=1, fill=False)
    q = torch.zeros(T, 1, 64, dtype=torch.float16)
    q[..., :32] = 1.0
    pos = torch.tensor([0, 1, 2 ** 31 - 1, -2 ** 31, 1_000_003, 131072] + list(range(10 ** 9, 10 ** 9 + T - 6)))
    freqs = ops.rope_frequencies(64)
    a = step.gpu()
    out = torch.empty(T, 1, 64, dtype=torch.float16, device="cuda")
    kv = torch.zeros(T, 1, 64, dtype=torch.float16, device="cuda")
    ops.rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], kv, kv,
                    ops.rope_rates(freqs), step.max_len, q=q.cuda(), q_out=out,
                    rope_positions=pos.to(torch.int32).cuda())
    # the reference multiplies exactly, in integers: position * round(freq / 2 pi * 2^100)
    got = out.double().cpu()[:, 0]
    two_pi = 6283185307179586476925286766559005768394
    for i in range(32):
        rate = int(freqs[i].item() * 2 ** 60) * (10 ** 39 << 40) // two_pi   # of a turn, in 2^-100
        for t in range(T):
            turn = (int(pos[t]) * rate) % (1 << 100) / (1 << 100)
            c, s = math.cos(2 * math.pi * turn), math.sin(2 * math.pi * turn)
            # 2^31 positions times the relative 2^-53 of a rate below a sixth of a turn
            slack = 12 * U + 2 * math.pi * 2 ** 31 * 2.0 ** -53 / 6
            assert abs(got[t, i] - c) <= H * abs(c) + slack
            assert abs(got[t, 32 + i] - s) <= H * abs(s) + slack


def test_rope_in_place_without_queries_and_padded(cuda_device):
    step = Step([20, 9], [6, 3], 16, seed=21, fill=False)
    T, pad = step.total, 5
    q = torch.randn(T + pad, 12, 128, generator=step.gen).half().cuda()
    k, v = (torch.randn(T + pad, 2, 128, generator=step.gen).half().cuda() for _ in range(2))
    rates = ops.rope_rates(ops.rope_frequencies(128))
    a, b, c = step.gpu(), step.gpu(), step.gpu()
    rows = lambda x: (x["k_pool"], x["v_pool"], x["block_tables"], x["seq_lens"], x["q_start"])  # noqa: E731
    out = torch.full_like(q, float("nan"))
    ops.rope_append(*rows(a), k, v, rates, step.max_len, q=q, q_out=out)
    assert bool(torch.isnan(out[T:]).all()) and bool(torch.isfinite(out[:T]).all())
    same = q.clone()
    ops.rope_append(*rows(b), k, v, rates, step.max_len, q=same, q_out=same)
    assert torch.equal(same[:T], out[:T]) and torch.equal(same[T:], q[T:])
    ops.rope_append(*rows(c), k, v, rates, step.max_len)
    for x in (b, c):
        assert torch.equal(x["k_pool"], a["k_pool"]) and torch.equal(x["v_pool"], a["v_pool"])


def test_rope_append_flags_what_it_cannot_place(cuda_device):
    step = Step([20, 9, 40], [6, 3, 2], 16, seed=22, fill=False)
    q = torch.randn(11, 12, 128, generator=step.gen).half().cuda()
    k, v = (torch.randn(11, 2, 128, generator=step.gen).half().cuda() for _ in range(2))
    rates = ops.rope_rates(ops.rope_frequencies(128))

    def go(**kw):
        a = step.gpu(**kw)
        out, err = torch.full_like(q, float("nan")), err_word()
        ops.rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], k, v, rates,
                        step.max_len, q=q, q_out=out, dev_err=err)
        return a["k_pool"], out, ops.check_error(err)

    kp, out, e = go()
    assert e == 0
    for lens in ([26, 2, 42], [26, 1000, 42]):        # below its nodes; above the bound
        kq, o, e = go(seq_lens=i32(lens))
        assert e == ERR_LEN and bool(torch.isnan(o[6:9]).all())
        assert torch.equal(o[:6], out[:6]) and torch.equal(o[9:], out[9:])
        s = step.slots(1, 9)
        assert torch.equal(kq.view(-1, 2, 128)[s.cuda()], step.k_pool.view(-1, 2, 128)[s].cuda())
    t = step.tables.copy()
    t[1, 0] = step.nb
    kq, o, e = go(block_tables=i32(t))
    assert e == ERR_BLOCK and torch.equal(o, out)      # queries are turned all the same
    changed = (kq != kp).any(-1).any(-1).view(-1)
    assert set(torch.nonzero(changed).flatten().tolist()) == set(step.slots(1, 9).tolist())


def test_rope_append_captured_and_on_another_stream(cuda_device):
    step = Step([20, 9], [6, 3], 16, fp8=True, seed=23, fill=False)
    q = torch.randn(9, 12, 128, generator=step.gen).half().cuda()
    k, v = (torch.randn(9, 2, 128, generator=step.gen).half().cuda() for _ in range(2))
    rates = ops.rope_rates(ops.rope_frequencies(64))
    a, b = step.gpu(), step.gpu()
    pos = i32(range(9))

    def go(x, out, stream=None):
        ops.rope_append(x["k_pool"], x["v_pool"], x["block_tables"], x["seq_lens"], x["q_start"], k, v, rates,
                        step.max_len, layout="interleaved", q=q, q_out=out, rope_positions=pos,
                        k_scale=x["k_scale"], v_scale=x["v_scale"], stream=stream)

    one, two = torch.empty_like(q), torch.empty_like(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    go(a, one, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(b, two)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(a["k_pool"], b["k_pool"])
    pos.add_(1000)
    g.replay()
    go(a, one)
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(a["k_pool"], b["k_pool"])


# ---- commit ----

def commit_ref(step, pools, paths):
    out = [p.clone() for p in pools]
    for r, path in enumerate(paths):
        P = step.prefix[r]
        s = step.slots(r)
        for src, dst in zip(pools, out):
            a = src.view(-1, step.nb * step.bs, step.hk, step.d)
            b = dst.view(-1, step.nb * step.bs, step.hk, step.d)
            for j, n in enumerate(path):
                b[:, s[P + j]] = a[:, s[P + n]]
    return out


def commit_run(step, paths, err=None, new=True, **kw):
    width = max([len(p) for p in paths] + [1])
    path = np.full((step.rows, width), -1, dtype=np.int32)
    for r, p in enumerate(paths):
        path[r, :len(p)] = p
    a = step.gpu(**kw)
    nl = torch.full((step.rows,), -5, dtype=torch.int32, device="cuda") if new else None
    ops.tree_commit(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], i32(path),
                    i32([len(p) for p in paths]), step.max_len, new_seq_lens=nl, dev_err=err)
    torch.cuda.synchronize()
    return a["k_pool"].cpu(), a["v_pool"].cpu(), nl


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layers,hk,d,bs", [(None, 2, 128, 16), (1, 2, 128, 64), (5, 2, 128, 16), (3, 8, 128, 48),
                                            (2, 1, 64, 7), (2, 9, 128, 16)])
def test_commit_moves_the_path(cuda_device, layers, hk, d, bs, fp8):
    nodes = [1, 8, 0, 90, 40, 12, 64]
    step = Step([0, 13, 5, 31, 100, 16, 3], nodes, bs, hk=hk, d=d, fp8=fp8, seed=31, layers=layers)
    rng = np.random.default_rng(4)
    paths = [[0], [1, 2, 5], [], sorted(rng.choice(90, 70, replace=False).tolist()), [], list(range(12)),
             list(range(1, 64))]    # one step along: every source but the first is a destination too
    err = err_word()
    k, v, nl = commit_run(step, paths, err)
    assert int(err.item()) == 0
    wk, wv = commit_ref(step, (step.k_pool, step.v_pool), paths)
    it = torch.uint8 if fp8 else torch.int16
    assert torch.equal(k.view(it), wk.view(it)) and torch.equal(v.view(it), wv.view(it))
    assert nl.tolist() == [p + len(x) for p, x in zip(step.prefix, paths)]


def test_commit_flags_what_is_no_path(cuda_device):
    step = Step([10, 20, 30], [8, 50, 4], 16, seed=32)
    good = [[1, 3], [2, 40], [0]]
    for bad, at in (([3, 3], 0), ([5, 2], 0), ([8], 0), ([-1, 2], 0), (list(range(33)) + [50], 1),
                    ([0, 1, 2, 3, 3], 2)):
        paths = [list(p) for p in good]
        paths[at] = bad
        err = err_word()
        k, v, nl = commit_run(step, paths, err)
        assert ops.check_error(err) == ERR_POS
        paths[at] = []
        wk, wv = commit_ref(step, (step.k_pool, step.v_pool), paths)
        assert torch.equal(k.view(torch.int16), wk.view(torch.int16))
        assert torch.equal(v.view(torch.int16), wv.view(torch.int16))
        want = [p + len(x) for p, x in zip(step.prefix, paths)]
        want[at] = -5
        assert nl.tolist() == want
    err = err_word()
    k, v, nl = commit_run(step, good, err, seq_lens=i32([18, 70, 3]))
    assert ops.check_error(err) == ERR_LEN and nl.tolist() == [12, 22, -5]
    t = step.tables.copy()
    t[1, 3] = -1                      # node 40's block (position 60) of row 1
    err = err_word()
    k, v, nl = commit_run(step, good, err, new=False, block_tables=i32(t))
    assert ops.check_error(err) == ERR_BLOCK and nl is None
    wk, _ = commit_ref(step, (step.k_pool, step.v_pool), [[1, 3], [2], [0]])
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16))


# ---- the step as a whole ----

@pytest.mark.parametrize("fp8", [False, True])
def test_calls_back_to_back_keep_the_streams_order(cuda_device, fp8):
    """Every call reads what the one before wrote (queries and keys from the
    last output, committed slots, lengths): with a wait after each, without,
    and captured, the same bits.  A decode that starts early follows each tree
    (fp16 pools)."""
    hq, hk, d, rounds = 12, 2, 128, 8
    step = Step([300, 17, 2000, 60], [9, 4, 13, 1], 16, fp8=fp8, seed=77, fill=False)
    T = step.total
    x0 = torch.randn(T, hq, d, generator=step.gen).half().cuda()
    mask = ops.tree_mask(random_parents(step.nodes, 4), step.starts).cuda()
    rates = ops.rope_rates(ops.rope_frequencies(d))
    paths = [[0, 2, 3, 8], [1, 3], [4, 5, 6, 12], [0]]
    path = i32([p + [-1] * (4 - len(p)) for p in paths])
    lens = i32([len(p) for p in paths])
    at = i32([n - 1 for n in step.lens])
    new = x0[:step.rows, :hk].contiguous()

    def run(how):
        a = step.gpu()
        x, y, out = x0.clone(), torch.empty_like(x0), torch.empty_like(x0)
        nl = torch.zeros(step.rows, dtype=torch.int32, device="cuda")
        z = torch.zeros(step.rows, hq, d, dtype=torch.float16, device="cuda")
        ws = ops.alloc_tree_workspace(step.rows, T, hq, hk, d, 16)
        dws = ops.alloc_workspace(step.rows, hq, hk, d, step.max_len, 16)
        err = err_word()
        rows = (a["block_tables"], a["seq_lens"], a["q_start"])
        scales = dict(k_scale=a["k_scale"], v_scale=a["v_scale"])
        wait = torch.cuda.synchronize if how == "waits" else lambda: None

        def go():
            for _ in range(rounds):
                ops.rope_append(a["k_pool"], a["v_pool"], *rows, x[:, :hk], x[:, hk:2 * hk], rates, step.max_len,
                                q=x, q_out=y, dev_err=err, **scales)
                wait()
                ops.tree_attention(out, y, a["k_pool"], a["v_pool"], *rows, 0.09, step.max_len, ws, mask=mask,
                                   dev_err=err, **scales)
                wait()
                if not fp8:
                    ops.append_decode(z, out[:step.rows], a["k_pool"], a["v_pool"], *rows[:2], at, new, new, 0.09,
                                      step.max_len, dws, pdl=True, dev_err=err)
                    wait()
                    ops.tree_attention(x, out, a["k_pool"], a["v_pool"], *rows, 0.09, step.max_len, ws, mask=mask,
                                       dev_err=err)
                    wait()
                ops.tree_commit(a["k_pool"], a["v_pool"], *rows, path, lens, step.max_len, new_seq_lens=nl, dev_err=err)
                wait()
                ops.tree_attention(x, out, a["k_pool"], a["v_pool"], *rows, 0.09, step.max_len, ws, mask=mask,
                                   dev_err=err, **scales)
                wait()

        if how == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                go()
            g.replay()
        else:
            go()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return [t.cpu() for t in (x, y, out, z, nl, a["k_pool"].view(torch.uint8), a["v_pool"].view(torch.uint8))]

    want = run("waits")
    assert bool(torch.isfinite(want[0]).all()) and want[4].tolist() == [p + len(q) for p, q in zip(step.prefix, paths)]
    for how in ("stream", "stream", "graph"):
        for name, w, g in zip(("x", "y", "out", "z", "lens", "k", "v"), want, run(how)):
            assert torch.equal(w.view(torch.uint8) if w.dtype == torch.float16 else w,
                               g.view(torch.uint8) if g.dtype == torch.float16 else g), (how, name)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_drafted_step_end_to_end(cuda_device, fp8):
    """Block manager, rotary append of a tree, tree attention, commit of an
    accepted path, truncation, and a second step of one token over what was
    committed: equal to plain causal attention over the accepted tokens."""
    hq, hk, d, bs, scale = 12, 2, 128, 16, 0.0883
    gen = torch.Generator().manual_seed(5)
    prompts, n_nodes = [37, 5, 90], [11, 6, 17]
    bm = BlockManager(num_blocks=64, block_size=bs, max_blocks_per_row=12)
    for r, n in enumerate(prompts):
        bm.admit(r, n, 60)
    freqs = ops.rope_frequencies(d)
    rates = ops.rope_rates(freqs)
    dt = torch.uint8 if fp8 else torch.float16
    kp, vp = (torch.zeros(64, bs, hk, d, dtype=dt, device="cuda") for _ in range(2))
    ks = torch.full((hk,), 0.03, device="cuda") if fp8 else None
    vs = torch.full((hk,), 0.025, device="cuda") if fp8 else None
    err = err_word()
    raw = [[], [], []]  # each row's committed (k, v) rows, before rotation

    def feed(tokens, counts, depth_pos, mask):
        """One step of the packed tokens [(q, k, v)]: rope append, then attention."""
        q, k, v = tokens
        tables, lens = bm.tables([0, 1, 2])
        starts = np.concatenate([[0], np.cumsum(counts)])
        bt, sl, st = i32(tables), i32(lens), i32(starts)
        ml = int(lens.max())
        qo, out = torch.empty_like(q), torch.empty_like(q)
        ops.rope_append(kp, vp, bt, sl, st, k, v, rates, ml, q=q, q_out=qo,
                        rope_positions=None if depth_pos is None else i32(depth_pos), k_scale=ks, v_scale=vs,
                        dev_err=err)
        ws = ops.alloc_tree_workspace(3, q.shape[0], hq, hk, d, bs)
        ops.tree_attention(out, qo, kp, vp, bt, sl, st, scale, ml, ws,
                           mask=None if mask is None else mask.cuda(), k_scale=ks, v_scale=vs, dev_err=err)
        return out, bt, sl, st, ml

    def draw(n):
        return [torch.randn(n, h, d, generator=gen).half().cuda() for h in (hq, hk, hk)]

    # prompts: a chain a row
    t = draw(sum(prompts))
    feed(t, prompts, None, None)
    at = 0
    for r, n in enumerate(prompts):
        raw[r] += [(t[1][at + i], t[2][at + i]) for i in range(n)]
        at += n
    # a drafted tree a row
    for r, n in enumerate(n_nodes):
        for i in range(n):
            assert bm.append_slot(r)[0] == prompts[r] + i
    parents = random_parents(n_nodes, 3)
    starts = np.concatenate([[0], np.cumsum(n_nodes)])
    depth, paths = [], []
    for r, n in enumerate(n_nodes):
        dep = []
        for i in range(n):
            p = parents[starts[r] + i]
            dep.append(0 if p < 0 else dep[p] + 1)
        depth += [prompts[r] + x for x in dep]
        i, path = int(np.argmax(dep)), []   # the deepest node's ancestors are accepted
        while i >= 0:
            path.append(i)
            i = parents[starts[r] + i]
        paths.append(path[::-1])
    t = draw(sum(n_nodes))
    _, bt, sl, st, ml = feed(t, n_nodes, depth, ops.tree_mask(parents, starts))
    width = max(map(len, paths))
    path = np.array([p + [-1] * (width - len(p)) for p in paths], dtype=np.int32)
    nl = torch.empty(3, dtype=torch.int32, device="cuda")
    ops.tree_commit(kp, vp, bt, sl, st, i32(path), i32([len(p) for p in paths]), ml, new_seq_lens=nl, dev_err=err)
    for r, p in enumerate(paths):
        bm.truncate(r, prompts[r] + len(p))
        raw[r] += [(t[1][starts[r] + i], t[2][starts[r] + i]) for i in p]
    assert nl.tolist() == [len(x) for x in raw] == list(bm.tables([0, 1, 2])[1])
    # one token more a row
    for r in range(3):
        assert bm.append_slot(r)[0] == len(raw[r])
    t = draw(3)
    out, *_ = feed(t, [1, 1, 1], None, None)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for r in range(3):
        raw[r].append((t[1][r], t[2][r]))
        n = len(raw[r])
        k = torch.stack([x for x, _ in raw[r]]).cpu()
        v = torch.stack([x for _, x in raw[r]]).cpu().double()
        kr, ke = rotate_ref(k, torch.arange(n), freqs, "half", 1.0)
        qr, qe = rotate_ref(t[0][r:r + 1].cpu(), torch.tensor([n - 1]), freqs, "half", 1.0)
        g = hq // hk
        kr, ke, v = (x.permute(1, 0, 2).repeat_interleave(g, 0) for x in (kr, ke, v))
        qr, qe = qr.permute(1, 0, 2), qe.permute(1, 0, 2)
        s = (qr @ kr.transpose(1, 2)) * scale
        p = torch.softmax(s, -1)
        want, big = p @ v, p @ v.abs()
        # what storing costs: half a step of each key and value
        if fp8:
            kd = e4m3_tol(kr / 0.03) * 0.03 * 1.001 + ke
            vd = (e4m3_tol(v / 0.025) * 0.025 * 1.001)
        else:
            kd, vd = fp16_tol(kr) + ke, torch.zeros_like(v)
        qd = fp16_tol(qr) + qe
        e = scale * ((qr.abs() + qd) @ kd.transpose(1, 2) + qd @ kr.abs().transpose(1, 2)).amax(-1, keepdim=True)
        e = e + 130 * U * scale * (qr.abs() @ kr.abs().transpose(1, 2)).amax(-1, keepdim=True)
        grow = torch.expm1(2 * e)           # every weight over the sum: within e^(2 e)
        tol = H * want.abs() + grow * big + (1 + grow) * ((H + (8 + n) * U) * big + p @ vd) + 2.0 ** -25 * (1 + v.abs().sum(1, keepdim=True))
        check(out[r:r + 1], want.permute(1, 0, 2), tol.permute(1, 0, 2), f"row {r}")
