"""GPU parity of the calls that keep a cache within a budget: head norms with
the rotary append, and eviction, against plain 64-bit forms.

Tolerances of the norms (u = 2^-24, h = 2^-11): a head's squares add up within 16
u (at most 16 terms a lane and five additions across lanes), the mean's factor
and sum within 2 u, its root halves that and takes 4 u itself, the two products 2 u:
15 u of each normalised value, 16 u with the second order; the rotation 12 u m
(|a| + |b|) on top (derived at the rotary append's tests), in all 28 u m (|a| +
|b|), 30 u with the second order; then h |ref| (2^-25 below the normal range), or
half an E4M3 step of the stored quotient (2^-4 of it, 2^-10 below the normal range).
Eviction moves bits: equality.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from paged_kv_cache_06_gb300 import ops
from paged_kv_cache_06_gb300.block_manager import BlockManager
from test_gpu_tree_step import ERR_BLOCK, ERR_LEN, Step, check, err_word, i32

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -11


# ---- norms of queries and keys with the rotary append ----

def norm_ref(x, weight, eps):
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def turned(y, pos, freqs, layout, mscale):
    """(rotated, tolerance before the output's rounding), both float64."""
    rot = 2 * freqs.shape[0]
    ang = torch.as_tensor(pos, dtype=torch.float64)[:, None] * freqs[None, :]
    c, s = (mscale * f(ang)[:, None, :] for f in (torch.cos, torch.sin))
    out, tol = y.clone(), 16 * U * y.abs()
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = y[..., i], y[..., j]
    out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    tol[..., i] = tol[..., j] = 30 * U * abs(mscale) * (a.abs() + b.abs())
    return out, tol


def rounded(ref, tol):
    return tol + H * ref.abs() + 2.0 ** -25


NORMS = [
    # prefix, nodes, block, q heads, kv heads, dim, rotated
    ([5], [1], 16, 12, 2, 128, 128),
    ([0, 63, 64, 700], [1, 1, 1, 1], 64, 12, 2, 128, 64),
    ([3, 0, 90], [7, 0, 40], 48, 32, 8, 128, 32),
    ([10, 2], [33, 5], 16, 4, 4, 64, 64),
    ([10, 2], [9, 5], 16, 8, 1, 96, 96),            # a head of six lanes
    ([10, 2], [9, 5], 16, 8, 2, 80, 16),            # of five
    ([1, 2, 3], [300, 1, 77], 32, 28, 4, 256, 256),
    ([0], [3], 16, 2, 1, 512, 128),
    ([0], [3], 16, 2, 1, 16, 16),                   # a head of one lane
    ([11] * 50, [60] * 50, 64, 12, 2, 128, 128),    # several tokens a block
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", range(len(NORMS)))
def test_norm_rope_append_matches_the_formula(cuda_device, case, layout, fp8):
    prefix, nodes, bs, hq, hk, d, rot = NORMS[case]
    step = Step(prefix, nodes, bs, hk=hk, d=d, fp8=fp8, seed=300 + case)
    gen, eps, mscale = step.gen, (1e-6, 0.25)[case % 2], (1.0, 1.3)[case % 3 == 1]
    qkv = torch.randn(step.total, hq + 2 * hk, d, generator=gen).half()
    qkv[:, 0] *= 30                                  # a loud head, a faint one
    qkv[:, hq] *= 0.01
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=gen)).half() for _ in range(2))
    pos = np.concatenate([[(0, 123456)[case % 2] + p + i for i in range(n)] for p, n in zip(prefix, nodes)])
    freqs = ops.rope_frequencies(rot)
    a, err, x = step.gpu(), err_word(), qkv.cuda()
    q_out = torch.full((step.total, hq, d), float("nan"), dtype=torch.float16, device="cuda")
    ops.norm_rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"],
                         x[:, hq:hq + hk], x[:, hq + hk:], ops.rope_rates(freqs), kw.cuda(), step.max_len, eps=eps,
                         layout=layout, q=x[:, :hq], q_out=q_out, q_weight=qw.cuda(), rope_positions=i32(pos),
                         mscale=mscale, k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref, tol = turned(norm_ref(qkv[:, :hq], qw, eps), pos, freqs, layout, mscale)
    check(q_out, ref, rounded(ref, tol), "queries")
    ref, tol = turned(norm_ref(qkv[:, hq:hq + hk], kw, eps), pos, freqs, layout, mscale)
    slots = torch.cat([step.slots(r, prefix[r]) for r in range(step.rows)])
    rest = torch.ones(step.nb * bs, dtype=torch.bool)
    rest[slots] = False
    for name, pool, scale in (("k_pool", step.k_pool, step.k_scale), ("v_pool", step.v_pool, step.v_scale)):
        was, got = pool.view(-1, hk, d), a[name].cpu().view(-1, hk, d)
        as_bits = torch.uint8 if fp8 else torch.int16
        assert torch.equal(got.view(as_bits)[rest], was.view(as_bits)[rest]), name   # nothing else is written
        if name == "v_pool":
            want = qkv[:, hq + hk:]
            if fp8:
                want = (want.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(got[slots].view(as_bits), want.view(as_bits))
        elif fp8:
            want, off = ref / scale.double()[:, None], tol / scale.double()[:, None]
            want = want.clamp(-448, 448)
            check(got[slots].view(torch.float8_e4m3fn).float(), want,
                  off + torch.maximum((want.abs() + off) * 2.0 ** -4, torch.tensor(2.0 ** -10)), "keys")
        else:
            check(got[slots], ref, rounded(ref, tol), "keys")


def norm_call(step, qkv, hq, weights, **kw):
    hk, d = step.hk, step.d
    a, x = step.gpu(), qkv.cuda()
    args = dict(q=x[:, :hq], q_out=torch.zeros(qkv.shape[0], hq, d, dtype=torch.float16, device="cuda"),
                q_weight=weights[0].cuda())
    tables, lens = kw.pop("block_tables", a["block_tables"]), kw.pop("seq_lens", a["seq_lens"])
    starts = kw.pop("q_start", a["q_start"])
    args.update(kw)
    ops.norm_rope_append(a["k_pool"], a["v_pool"], tables, lens, starts, x[:, hq:hq + hk], x[:, hq + hk:],
                         ops.rope_rates(ops.rope_frequencies(d)), weights[1].cuda(), step.max_len, **args)
    torch.cuda.synchronize()
    return args["q_out"], a["k_pool"], a["v_pool"]


def norm_step(prefix, nodes, bs=16, seed=0):
    step = Step(prefix, nodes, bs, seed=seed, fill=False)
    qkv = torch.randn(step.total + 3, 16, 128, generator=step.gen).half()
    return step, qkv, [(1 + 0.1 * torch.randn(128, generator=step.gen)).half() for _ in range(2)]


def test_norm_rope_append_without_queries_in_place_and_behind_the_last_row(cuda_device):
    step, qkv, w = norm_step([30, 5, 0], [4, 1, 20], seed=1)
    out, k, v = norm_call(step, qkv, 12, w)
    assert bool((out[step.total:] == 0).all())                   # tokens behind the last row are left alone
    none = norm_call(step, qkv, 12, w, q=None, q_out=None, q_weight=None)
    assert torch.equal(none[1], k) and torch.equal(none[2], v)   # keys and values alone
    q = qkv[:, :12].contiguous().cuda()
    norm_call(step, qkv, 12, w, q=q, q_out=q)                    # over its own input
    assert torch.equal(q[:step.total], out[:step.total])
    assert torch.equal(q[step.total:].cpu(), qkv[step.total:, :12])


def test_norm_rope_append_skips_and_flags_bad_rows(cuda_device):
    step, qkv, w = norm_step([30, 5, 9], [4, 1, 20], seed=2)
    out, k, v = norm_call(step, qkv, 12, w)
    err, lens = err_word(), list(step.lens)
    lens[1] = step.max_len + 1
    got = norm_call(step, qkv, 12, w, seq_lens=i32(lens), dev_err=err)
    assert ops.check_error(err) == ERR_LEN
    assert bool((got[0][4] == 0).all()) and torch.equal(got[0][5:], out[5:]) and torch.equal(got[0][:4], out[:4])
    t = step.tables.copy()
    t[2, 0] = step.nb                                            # tokens 9 .. 15 of row 2
    got = norm_call(step, qkv, 12, w, block_tables=i32(t), dev_err=err)
    assert ops.check_error(err) == ERR_BLOCK
    assert torch.equal(got[0], out)                              # its queries are rotated all the same
    lost, kept = step.slots(2, 9, 16), step.slots(2, 16)
    for new, was, pool in ((got[1], k, step.k_pool), (got[2], v, step.v_pool)):
        new, was = new.cpu().view(-1, 2, 128), was.cpu().view(-1, 2, 128)
        assert torch.equal(new[lost], pool.view(-1, 2, 128)[lost]) and torch.equal(new[kept], was[kept])


def test_norms_of_heads_that_are_zero_huge_or_no_number(cuda_device):
    step, qkv, w = norm_step([0], [6], seed=3)
    qkv[0, 0] = 0
    qkv[1, 1] = 65504
    qkv[2, 2, 5] = float("inf")
    qkv[3, 3, 7] = float("nan")
    qkv[4, 4] = 2.0 ** -24
    out, _, _ = norm_call(step, qkv, 12, w, eps=1e-6)
    assert bool((out[0, 0] == 0).all()) and bool(torch.isfinite(out[1, 1]).all())
    assert bool(torch.isnan(out[3, 3]).all()) and bool(torch.isnan(out[2, 2, [5, 69]]).all())
    pos, freqs = np.arange(6), ops.rope_frequencies(128)
    clean = torch.ones(6, 12, dtype=torch.bool)
    clean[2, 2] = clean[3, 3] = False
    ref, tol = turned(norm_ref(qkv[:6, :12], w[0], 1e-6), pos, freqs, "half", 1.0)
    check(out[:6][clean.cuda()], ref[clean], rounded(ref, tol)[clean])


# ---- weights ----

def weights_ref(step, q, scale, queries, used, skip=(), extra=lambda n, mag: 0):
    """What the last used[r] of row r's queries[r] give: (sums [rows][hk] of tensors [L], their
    tolerance before they are added to anything), and the queries' outputs.  extra: further roundings
    of an exponent, in U."""
    hq = q.shape[1]
    g, out = hq // step.hk, []
    a = 0
    for r, n in enumerate(step.lens):
        a += queries[r]
        u = used[r]
        if not u or not n:
            out.append(None)
            continue
        k = step.values(step.k_pool, r, step.k_scale).permute(1, 0, 2).repeat_interleave(g, 0)
        v = step.values(step.v_pool, r, step.v_scale).permute(1, 0, 2).repeat_interleave(g, 0)
        x = q[a - u:a].double().permute(1, 0, 2)
        s = (x @ k.transpose(1, 2)) * scale
        hide = torch.arange(n)[None, :] > torch.arange(n - u, n)[:, None]
        hide[:, [t for rr, t in skip if rr == r]] = True
        s = s.masked_fill(hide, -np.inf)
        p = torch.softmax(s, -1)
        e = 130 * U * abs(scale) * (x.abs() @ k.abs().transpose(1, 2)).masked_fill(hide, 0).amax(-1, keepdim=True)
        mag = s.masked_fill(hide, 0).abs().amax(-1, keepdim=True)
        tol = p * (2 * e + (12 + n + 4 * mag + extra(n, mag)) * U)
        shape = (step.hk, g * u, n)
        out.append((p.reshape(shape).sum(1), (tol + g * u * U * p).reshape(shape).sum(1), (p @ v, p @ v.abs(), e)))
    return out


def check_weights(step, got, before, ref, own):
    """got, before: [rows][hk][stride]; row r's last own[r] tokens start from zero."""
    got, before = got.cpu().double(), before.cpu().double()
    for r, n in enumerate(step.lens):
        assert torch.equal(got[r, :, n:], before[r, :, n:])
        if ref[r] is None:
            assert torch.equal(got[r], before[r])
            continue
        w = before[r, :, :n].clone()
        w[:, n - own[r]:] = 0
        want = w + ref[r][0]
        check(got[r, :, :n], want, ref[r][1] + 2 * U * want.abs() + 2.0 ** -126, f"weights of row {r}")


DECODES = [
    ([1], 16, 12, 2),
    ([16, 1, 0, 33, 200], 16, 12, 2),
    ([63, 64, 65, 4100], 64, 12, 2),
    ([700, 3, 129], 48, 32, 8),
    ([513, 40], 112, 28, 4),
    ([300, 31, 2], 32, 4, 4),
    ([257, 90], 16, 8, 1),
    ([20000, 50], 64, 12, 2),
    ([300 + 7 * i for i in range(70)], 16, 6, 2),       # units cut between blocks, odd groups
    ([1024] * 40, 64, 10, 2),
    ([i * 37 % 500 for i in range(300)], 16, 12, 2),    # many short rows, some of nothing
    ([5000, 70, 0], 16, 8, 1),
    ([300 + 7 * i for i in range(70)] + [4200], 16, 6, 2),  # the same beside rows too long for clusters
    ([1024] * 40 + [4097], 64, 10, 2),
    ([i * 37 % 500 for i in range(300)] + [4300], 16, 12, 2),
    ([1 + i * 331 % 1024 for i in range(200)], 16, 12, 2),      # a block a unit, more than there is room for
    ([i * 7 % 70 for i in range(400)], 32, 14, 2),
    ([2048, 1, 0, 1025] + [i * 61 % 700 for i in range(110)], 64, 16, 2),  # clusters of two, their largest shares
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode_weights_match_the_formula(cuda_device, case, fp8):
    """Weights: a score is off by e (a dot product of 128 terms), m U (its scaling and the
    maximum taken from it, m the largest score) and so its weight by 2 e + 4 m U of
    itself, exponent, reciprocal and products 12 U, the sum over L weights L U, over the
    heads g U.  The output as the tree's."""
    lens, bs, hq, hk = DECODES[case]
    step = Step(lens, [0] * len(lens), bs, hk=hk, fp8=fp8, seed=500 + case)
    q = torch.randn(len(lens), hq, 128, generator=step.gen).half()
    before = torch.rand(len(lens), hk, step.max_len + 5, generator=step.gen)
    a, err = step.gpu(), err_word()
    ws = ops.alloc_decode_weights_workspace(len(lens), hq, hk, 128, step.max_len, bs)
    ref = weights_ref(step, q, 0.0883, [1] * len(lens), [1] * len(lens))
    outs = []
    for _ in range(2):
        out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        w = before.cuda()
        ops.decode_weights(out, w, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883,
                           step.max_len, ws, k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
        torch.cuda.synchronize()
        outs.append((out, w))
    assert int(err.item()) == 0
    assert all(torch.equal(x, y) for x, y in zip(*outs))              # the same bits every time
    check_weights(step, w, before, ref, [1] * len(lens))
    for r, n in enumerate(lens):
        if n == 0:
            assert bool((out[r] == 0).all())
            continue
        o, big, e = (x[:, 0] for x in ref[r][2])
        low = 2.0 ** -25 * step.values(step.v_pool, r, step.v_scale).abs().sum(0).repeat_interleave(hq // hk, 0)
        check(out[r], o, H * o.abs() + (H + 2 * e + (8 + n) * U) * big + low + 2.0 ** -25, f"output of row {r}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [48, 5000])
def test_decode_weights_of_values_that_cancel(cuda_device, cap, fp8):
    """Nearly equal weights of values of both signs.  A weight reaches the output within 2^-22 of itself and 2^-32 of the
    largest, so what is left of the sum is good to that share of A = sum p |v|, and to half a step of its own."""
    lens = [2, 4, 6, 10, 16, 40]
    step = Step(lens, [0] * 6, 16, fp8=fp8, seed=32)
    values = (90 + 20 * torch.rand(step.v_pool.shape, generator=step.gen)) * (1 - 2 * (torch.arange(16) % 2))[:, None, None]
    if fp8:
        step.k_scale, step.v_scale = torch.full((2,), 0.02), torch.ones(2)
        step.v_pool = values.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        step.v_pool = values.half()
    q = (0.05 * torch.randn(6, 12, 128, generator=step.gen)).half()
    ref = weights_ref(step, q, 0.0883, [1] * 6, [1] * 6)
    tables = np.concatenate([step.tables, np.full((6, (cap + 15) // 16 - step.tables.shape[1]), -1, dtype=np.int32)], 1)
    before = torch.zeros(6, 2, cap)
    a, err, w = step.gpu(block_tables=i32(tables)), err_word(), before.cuda()
    out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    ops.decode_weights(out, w, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, cap,
                       ops.alloc_decode_weights_workspace(6, 12, 2, 128, cap, 16), k_scale=a["k_scale"],
                       v_scale=a["v_scale"], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_weights(step, w, before, ref, [1] * 6)
    for r, n in enumerate(lens):
        o, big, e = (x[:, 0] for x in ref[r][2])
        low = 2.0 ** -32 * step.values(step.v_pool, r, step.v_scale).abs().sum(0).repeat_interleave(6, 0)
        check(out[r], o, H * o.abs() + (2.0 ** -22 + 2 * e + (12 + n) * U) * big + low + 2.0 ** -25, f"output of row {r}")


@pytest.mark.parametrize("cap", [80, 5000])
def test_decode_weights_of_infinite_values(cuda_device, cap):
    """An infinite value is its dim's output, two of both signs are no number, and other dims keep their bits."""
    step = Step([70, 30], [0, 0], 16, seed=33)
    q = torch.randn(2, 12, 128, generator=step.gen).half().cuda()
    tables = np.concatenate([step.tables, np.full((2, (cap + 15) // 16 - step.tables.shape[1]), -1, dtype=np.int32)], 1)
    ws = ops.alloc_decode_weights_workspace(2, 12, 2, 128, cap, 16)

    def run():
        a, w, out = step.gpu(block_tables=i32(tables)), torch.zeros(2, 2, cap, device="cuda"), torch.zeros_like(q)
        ops.decode_weights(out, w, q, a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, cap, ws)
        torch.cuda.synchronize()
        return out.cpu(), w.cpu()

    clean, weights = run()
    v, slots, inf = step.v_pool.view(-1, 2, 128), step.slots(0), float("inf")
    v[slots[3], 0, 5], v[slots[60], 0, 77], v[slots[20], 1, 8], v[slots[66], 1, 8] = inf, -inf, inf, -inf
    out, w = run()
    assert torch.equal(w, weights)
    assert bool((out[0, :6, 5] == inf).all()) and bool((out[0, :6, 77] == -inf).all()) and bool(torch.isnan(out[0, 6:, 8]).all())
    same = torch.ones(2, 12, 128, dtype=torch.bool)
    same[0, :6, [5, 77]] = same[0, 6:, 8] = False
    assert torch.equal(out[same], clean[same])


SPLITS = [
    ([1024 - 9 * i for i in range(32)], 12, 2),                    # clusters of four, as many as fit
    ([1024 - 7 * i for i in range(48)], 12, 2),                    # of two
    ([2048, 1, 0, 1025] + [i * 61 % 700 for i in range(60)], 16, 2),    # of two, their largest shares
    ([2048 - 100 * i for i in range(16)], 6, 2),                   # of eight
    ([1000 - 3 * i for i in range(96)], 12, 2),                    # a block a unit
    ([2000 - 9 * i for i in range(90)], 8, 2),                     # the even cut, with rows that clusters could take
    ([4096, 0, 3000] + [i * 31 % 300 for i in range(35)], 12, 2),  # eight blocks for rows taken for few
    ([4096, 0, 3000] + [i * 31 % 300 for i in range(36)], 12, 2),  # and one row more
    ([4200] + [i * 17 % 90 for i in range(429)], 8, 1),            # two blocks an SM
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(SPLITS)))
def test_decode_weights_at_the_borders_of_the_work_split(cuda_device, case, fp8):
    """Tolerances as where the weights are compared with the formula."""
    lens, hq, hk = SPLITS[case]
    step = Step(lens, [0] * len(lens), 32, hk=hk, fp8=fp8, seed=560 + case)
    q = torch.randn(len(lens), hq, 128, generator=step.gen).half()
    before = torch.rand(len(lens), hk, step.max_len + 1, generator=step.gen)
    a, err, w = step.gpu(), err_word(), before.cuda()
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    ops.decode_weights(out, w, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, step.max_len,
                       ops.alloc_decode_weights_workspace(len(lens), hq, hk, 128, step.max_len, 32),
                       k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref = weights_ref(step, q, 0.0883, [1] * len(lens), [1] * len(lens))
    check_weights(step, w, before, ref, [1] * len(lens))
    for r, n in enumerate(lens):
        if n == 0:
            assert bool((out[r] == 0).all())
            continue
        o, big, e = (x[:, 0] for x in ref[r][2])
        low = 2.0 ** -32 * step.values(step.v_pool, r, step.v_scale).abs().sum(0).repeat_interleave(hq // hk, 0)
        check(out[r], o, H * o.abs() + (H + 2 * e + (8 + n) * U) * big + low + 2.0 ** -25, f"output of row {r}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("more,hq,hk", [(24, 12, 2), (66, 8, 1), (55, 6, 1)])
def test_decode_weights_whatever_the_order_of_the_rows(cuda_device, more, hq, hk, fp8):
    """Rows that clusters take by their lengths, among them equal ones, empty ones and lengths that are out of range:
    in any order each has the same bits."""
    lens = [4096, 17, 0, 300, 300, 2500, 1, 300, 4096, 64] + [20 * i for i in range(more)]
    rows = len(lens)
    step = Step(lens, [0] * rows, 64, hk=hk, fp8=fp8, seed=34)
    q = torch.randn(rows, hq, 128, generator=step.gen).half()
    before = torch.rand(rows, hk, 4096, generator=step.gen)
    given = np.array(lens)
    given[6], given[7] = -3, 5000                            # taken for 0 and 4096, and flagged
    full = step.tables.copy()
    full[7] = full[0]                                        # blocks for its 4096 tokens
    ws = ops.alloc_decode_weights_workspace(rows, hq, hk, 128, 4096, 64)
    results = []
    for seed in range(4):
        order = np.arange(rows) if seed == 0 else np.random.default_rng(seed).permutation(rows)
        a, err = step.gpu(block_tables=i32(full[order]), seq_lens=i32(given[order])), err_word()
        w, out = before[order].cuda(), torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        ops.decode_weights(out, w, q[order].cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, 4096,
                           ws, k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
        assert ops.check_error(err) == ERR_LEN
        back = np.argsort(order)
        results.append((out.cpu()[back], w.cpu()[back]))
    for out, w in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(w, results[0][1])
    out, w = results[0]
    ref = weights_ref(step, q, 0.0883, [1] * rows, [1] * rows)
    ref[6] = None
    for r in (6, 2):
        assert bool((out[r] == 0).all()) and torch.equal(w[r], before[r])
    w[7], ref[7] = before[7], None
    check_weights(step, w, before, ref, [1] * rows)


def test_decode_weights_of_bad_lengths_blocks_and_numbers(cuda_device):
    step = Step([100, 60, 300, 40], [0] * 4, 16, seed=13)
    q = torch.randn(4, 12, 128, generator=step.gen).half()
    q[3, 2, 5] = float("nan")
    before = torch.rand(4, 2, 300, generator=step.gen)
    t, lens = step.tables.copy(), [100, -4, 301, 40]                  # row 2 is clamped to 300
    t[0, 1] = step.nb                                                  # slots 16 .. 31 of row 0
    a, err = step.gpu(block_tables=i32(t), seq_lens=i32(lens)), err_word()
    ws = ops.alloc_decode_weights_workspace(4, 12, 2, 128, 300, 16)
    out, w = torch.zeros(4, 12, 128, dtype=torch.float16, device="cuda"), before.cuda()
    ops.decode_weights(out, w, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.0883, 300, ws,
                       dev_err=err)
    assert ops.check_error(err) == ERR_BLOCK | ERR_LEN
    assert torch.equal(w[1].cpu(), before[1])
    assert bool(torch.isnan(w[3, 0, :40]).all()) and bool(torch.isfinite(w[3, 1]).all())
    assert torch.equal(w[0, :, 16:32].cpu(), before[0, :, 16:32])      # they got nothing
    q[3, 2, 5] = 0
    ref = weights_ref(step, q, 0.0883, [1] * 4, [1] * 4, skip=[(0, i) for i in range(16, 32)])
    ref[1] = None
    w[3] = before[3].cuda()
    ref[3] = None
    check_weights(step, w, before, ref, [1] * 4)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("top", [900, 3000, 7000])
def test_decode_weights_keep_many_faint_tokens_in_the_output(cuda_device, top, fp8):
    """One token without a value, the others 2^-26 to 2^-28 of its weight and all of the output.  A weight is off by
    2^-11 of itself, and by 2^-32 of the largest below the fp16 numbers of eleven bits: the reference that weights are
    taken from lies 2^7 below the largest."""
    step = Step([top, top // 3], [0, 0], 16, fp8=fp8, seed=31)
    q = torch.zeros(2, 12, 128, dtype=torch.float16)
    q[:, :, 0] = 1
    keys = torch.zeros(step.k_pool.shape)
    values = torch.rand(step.v_pool.shape, generator=step.gen) * 300 + 100
    for r, n in enumerate(step.lens):
        at = step.slots(r)
        keys.view(-1, 2, 128)[at, :, 0] = -26. - 2 * (torch.arange(n) % 2)[:, None]
        keys.view(-1, 2, 128)[at[n // 2], :, 0] = 0
        values.view(-1, 2, 128)[at[n // 2]] = 0
    if fp8:
        step.k_scale, step.v_scale = torch.ones(2), torch.tensor([100., 50.])
        step.k_pool, step.v_pool = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (keys, values))
    else:
        step.k_pool, step.v_pool = keys.half(), (values * 100).half()
    scale = float(torch.tensor(np.log(2.0), dtype=torch.float32))
    ref = weights_ref(step, q, scale, [1, 1], [1, 1])
    before = torch.zeros(2, 2, top)
    a, err, w = step.gpu(), err_word(), before.cuda()
    out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    ops.decode_weights(out, w, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], scale, top,
                       ops.alloc_decode_weights_workspace(2, 12, 2, 128, top, 16), k_scale=a["k_scale"],
                       v_scale=a["v_scale"], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_weights(step, w, before, ref, [1, 1])
    for r, n in enumerate(step.lens):
        o, big, e = (x[:, 0] for x in ref[r][2])
        low = 2.0 ** -32 * step.values(step.v_pool, r, step.v_scale).abs().sum(0).repeat_interleave(6, 0)
        tol = H * o.abs() + (H + 2 * e + (8 + n) * U) * big + low + 2.0 ** -25
        assert bool((tol < 0.1 * o.abs()).all())                       # a fault of the faint tokens' own size shows
        check(out[r], o, tol, f"output of row {r}")


PROMPTS = [
    # cached, chunk, window, block, q heads, kv heads
    ([0], [1], None, 16, 12, 2),
    ([0, 5, 100, 0], [3, 1, 22, 0], None, 16, 12, 2),
    ([10, 0, 127, 128], [130, 300, 1, 64], None, 64, 12, 2),       # tiles and query blocks that end anywhere
    ([300, 1000], [200, 77], 32, 48, 12, 2),                       # the last 32 of a chunk
    ([300, 0, 7], [40, 500, 2], 1, 16, 12, 2),                     # the last one alone
    ([20000, 3], [6, 4], None, 64, 12, 2),                         # few queries over a long cache
    ([0, 64], [700, 260], None, 128, 32, 8),
    ([500, 31], [150, 90], None, 32, 28, 4),
    ([500, 31], [129, 250], None, 16, 4, 4),                       # a head a group
    ([257, 0], [100, 37], None, 16, 24, 1),                        # five queries a block
    ([9, 400], [70, 11], None, 16, 10, 2),
    ([50], [9], None, 16, 128, 1),                                 # a query a block
    ([60, 0], [9, 33], None, 112, 65, 1),                          # one and 63 rows of nothing
    ([37 * i % 400 for i in range(60)], [5 + i % 9 for i in range(60)], 7, 16, 12, 2),
    ([0, 0], [2000, 1100], None, 64, 12, 2),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prefill_weights_match_the_formula(cuda_device, case, fp8):
    """As decode's, with an exponent's further roundings: the logarithm of the sum is rounded
    twice, and so is its difference from the score: below U (2 |score| + 3 log2 L) of a
    weight, and constants within 4 U."""
    prefix, nodes, window, bs, hq, hk = PROMPTS[case]
    step = Step(prefix, nodes, bs, hk=hk, fp8=fp8, seed=600 + case)
    q = torch.randn(step.total, hq, 128, generator=step.gen).half()
    before = torch.rand(step.rows, hk, step.max_len + 3, generator=step.gen)
    used = [min(n, window or n) for n in nodes]
    ref = weights_ref(step, q, 0.0883, nodes, used, extra=lambda n, mag: 4 + 2 * mag + 3 * np.log2(n + 1))
    a, err = step.gpu(), err_word()
    ws = ops.alloc_prefill_weights_workspace(step.rows, step.total, hq, hk, 128, step.max_len, bs, window=window)
    outs = []
    for fill in (0, 255):                                             # whatever the workspace holds
        ws.fill_(fill)
        w = before.cuda()
        ops.prefill_weights(w, q.cuda(), a["k_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.0883,
                            step.max_len, ws, window=window, k_scale=a["k_scale"], dev_err=err)
        torch.cuda.synchronize()
        outs.append(w)
    assert int(err.item()) == 0
    assert torch.equal(*outs)                                         # the same bits every time
    check_weights(step, outs[0], before, ref, nodes)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_weights_of_bad_rows_blocks_and_unseen_numbers(cuda_device, fp8):
    """A row too long, a block out of range, queries and keys that are no numbers where
    nobody, or somebody, sees them."""
    step = Step([100, 60, 300, 40], [30, 9, 45, 33], 16, fp8=fp8, seed=14)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    before = torch.rand(4, 2, step.max_len, generator=step.gen)
    ws = ops.alloc_prefill_weights_workspace(4, step.total, 12, 2, 128, step.max_len, 16)
    err = err_word()

    def run(x, **kw):
        a, w = step.gpu(**kw), before.cuda()
        ops.prefill_weights(w, x.cuda(), a["k_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.0883,
                            step.max_len, ws, k_scale=a["k_scale"], dev_err=err)
        torch.cuda.synchronize()
        return w

    more = dict(extra=lambda n, mag: 4 + 2 * mag + 3 * np.log2(n + 1))
    clean = run(q)
    t, lens = step.tables.copy(), list(step.lens)
    lens[1] = step.max_len + 1
    t[0, 1] = -1                                                       # slots 16 .. 31 of row 0
    t[2, 20] = step.nb + 7                                             # slots 320 .. 335 of row 2
    got = run(q, block_tables=i32(t), seq_lens=i32(lens))
    assert ops.check_error(err) == ERR_BLOCK | ERR_LEN
    skip = [(0, i) for i in range(16, 32)] + [(2, i) for i in range(320, 336)]
    ref = weights_ref(step, q, 0.0883, step.nodes, step.nodes, skip=skip, **more)
    ref[1] = None
    check_weights(step, got, before, ref, step.nodes)
    assert torch.equal(got[3], clean[3])
    # a query that is no number: its tokens' sums in its head's group; the others keep their bits
    x = q.clone()
    x[5, 7, 3] = float("nan")                                          # row 0, query 5, KV head 1
    got = run(x)
    assert bool(torch.isnan(got[0, 1, :106]).all()) and bool(torch.isfinite(got[0, 1, 106:130]).all())
    same = torch.ones(4, 2, dtype=torch.bool)
    same[0, 1] = False
    assert torch.equal(got[same.cuda()], clean[same.cuda()])
    assert torch.equal(got[0, 1, 106:], clean[0, 1, 106:])             # no such query sees them
    # a key that is no number, seen by the last three queries of row 3 alone
    slot = step.slots(3)[70]
    step.k_pool.view(-1, 2, 128)[slot, 0] = 0x7F if fp8 else float("nan")
    got = run(q)
    assert bool(torch.isnan(got[3, 0, :73]).all())
    same = torch.ones(4, 2, dtype=torch.bool)
    same[3, 0] = False
    assert torch.equal(got[same.cuda()], clean[same.cuda()])
    assert ops.check_error(err) == 0


@pytest.mark.parametrize("chunk,done", [(40, True), (400, False)])
def test_prefill_weights_of_rows_that_name_the_same_queries(cuda_device, chunk, done):
    """Two rows of all the queries and two of less than none: as they come, or, where the
    workspace has no room for so many query blocks, nothing at all."""
    step = Step([0] * 4, [chunk] * 4, 16, seed=15)
    q = torch.randn(chunk, 12, 128, generator=step.gen).half().cuda()
    w = torch.rand(4, 2, chunk, generator=step.gen).cuda()
    before, err, a = w.clone(), err_word(), step.gpu()
    starts = torch.tensor([0, chunk, 0, chunk, 0], dtype=torch.int32)
    ws = ops.alloc_prefill_weights_workspace(4, chunk, 12, 2, 128, chunk, 16)
    ws.fill_(77)
    ops.prefill_weights(w, q, a["k_pool"], a["block_tables"], a["seq_lens"], starts.cuda(), 0.1, chunk, ws, dev_err=err)
    assert ops.check_error(err) == ERR_LEN
    for r in range(4):
        assert torch.equal(w[r], before[r]) == (r % 2 == 1 or not done)


def test_decode_and_prefill_weights_in_a_graph_on_another_stream(cuda_device):
    """Captured together over separate workspaces, replayed twice: the eager calls' bits."""
    step = Step([700, 30, 90], [100, 64, 1], 64, seed=16)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half().cuda()
    last = q[[99, 163, 164]].contiguous()
    a = step.gpu()
    wsp = ops.alloc_prefill_weights_workspace(3, step.total, 12, 2, 128, step.max_len, 64, window=16)
    wsd = ops.alloc_decode_weights_workspace(3, 12, 2, 128, step.max_len, 64)
    out = torch.zeros(3, 12, 128, dtype=torch.float16, device="cuda")
    w = torch.rand(3, 2, step.max_len, generator=step.gen).cuda()
    first = w.clone()

    def both(stream=None):
        ops.prefill_weights(w, q, a["k_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.09, step.max_len, wsp,
                            window=16, stream=stream)
        ops.decode_weights(out, w, last, a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.09,
                           step.max_len, wsd, stream=stream)

    both()
    torch.cuda.synchronize()
    want, want_out = w.clone(), out.clone()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            both()
    for _ in range(2):
        w.copy_(first)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, want) and torch.equal(out, want_out)


# ---- eviction ----

class Lists:
    """Rows of `lens` tokens in `layers` layers, with weights, recorded positions for
    the first `tracked` slots and the outcome that the definition gives."""

    def __init__(self, lens, budget, bs=16, layers=2, hk=2, d=128, fp8=False, sinks=0, recent=0, tracked=None,
                 seed=0, stride=None, weights=None, skipped=()):
        self.step = step = Step(lens, [0] * len(lens), bs, hk=hk, d=d, fp8=False, layers=layers, seed=seed)
        rng = np.random.default_rng(seed)
        self.lens, self.budget, self.sinks, self.recent, self.fp8 = list(lens), budget, sinks, recent, fp8
        self.layers, self.hk, self.d = layers, hk, d
        self.top = max(1, max(lens))
        stride = stride or self.top
        shape = (layers, len(lens), hk, stride)
        if fp8:
            step.k_pool, step.v_pool = (torch.randint(0, 256, step.k_pool.shape, generator=step.gen, dtype=torch.uint8)
                                        for _ in range(2))
        self.weights = np.exp(2 * rng.standard_normal(shape)).astype(np.float32) if weights is None else weights(rng, shape)
        self.tracked = [0] * len(lens) if tracked is None else tracked
        self.pos = np.full(shape, -77, dtype=np.int32)
        self.next = []
        for r, n in enumerate(lens):
            had = self.tracked[r] + (5 if self.tracked[r] else 0)
            for i in np.ndindex(layers, hk):
                self.pos[i[0], r, i[1], :self.tracked[r]] = rng.permutation(had)[:self.tracked[r]]
            self.next.append(had + n - self.tracked[r])
        self.want(skipped)

    def want(self, skipped=()):
        """Slots that each list's tokens move between, and the arrays afterwards."""
        self.w_after, self.p_after = self.weights.copy(), self.pos.copy()
        self.new = [min(n, self.budget) for n in self.lens]
        self.moves = []
        for i in np.ndindex(self.layers, len(self.lens), self.hk):
            r = i[1]
            n, keep = self.lens[r], self.new[r]
            if r in skipped:
                continue
            t = np.arange(n)
            pos = np.where(t < self.tracked[r], self.pos[i][:n], self.next[r] - n + t)
            w = self.weights[i][:n]
            safe = (pos < self.sinks) | (pos >= self.next[r] - self.recent)
            rank = np.where(safe, 2, np.isnan(w).astype(int))
            order = np.lexsort((t, -np.where(rank > 0, 0, w), -rank))
            stays = np.zeros(n, dtype=bool)
            stays[order[:keep]] = True
            to, frm = t[(t < keep) & ~stays], t[(t >= keep) & stays]
            assert len(to) == len(frm)
            at = t[:keep].copy()
            at[to] = frm
            self.w_after[i][:keep], self.p_after[i][:keep] = w[at], pos[at]
            self.moves.append((i, to, frm))

    def pools_after(self):
        s, out = self.step, []
        for pool in (s.k_pool, s.v_pool):
            p = pool.clone().view(self.layers, -1, self.hk, self.d)
            for (layer, r, h), to, frm in self.moves:
                if len(to):
                    slots = s.slots(r)
                    p[layer, slots[to], h] = pool.view(self.layers, -1, self.hk, self.d)[layer, slots[frm], h]
            out.append(p.view(pool.shape))
        return out

    def run(self, in_place=True, stream=None, err=None, bare=False, max_len=None, **kw):
        s = self.step
        g = dict(k_pool=s.k_pool.cuda(), v_pool=s.v_pool.cuda(), block_tables=i32(s.tables), seq_lens=i32(self.lens),
                 weights=torch.from_numpy(self.weights).cuda(), token_pos=torch.from_numpy(self.pos).cuda())
        g.update(kw)
        w, p = g["weights"], g["token_pos"]
        if not in_place:
            w, p = torch.full_like(w, -1), torch.full_like(p, -1)
        new = torch.full((len(self.lens),), -5, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        ops.evict(**g, budget=self.budget, max_seq_len=max_len or self.top, sinks=self.sinks, recent=self.recent,
                  tracked=None if bare else i32(self.tracked), next_pos=None if bare else i32(self.next),
                  weights_out=None if in_place else w, token_pos_out=None if in_place else p, new_seq_lens=new,
                  dev_err=err, stream=stream)
        torch.cuda.synchronize()
        return g["k_pool"], g["v_pool"], w, p, new

    def check(self, got, in_place=True, skipped=()):
        k, v, w, p, new = (x.cpu() for x in got)
        for name, x, y in zip("kv", (k, v), self.pools_after()):
            bits = torch.uint8 if self.fp8 else torch.int16
            assert torch.equal(x.view(bits), y.view(bits)), name
        for r, n in enumerate(self.new):
            assert int(new[r]) == (-5 if r in skipped else n)
            live = 0 if r in skipped else n
            for x, y, before in ((w.numpy(), self.w_after, self.weights), (p.numpy(), self.p_after, self.pos)):
                np.testing.assert_array_equal(x[:, r, :, :live].view(np.int32), y[:, r, :, :live].view(np.int32))
                rest = x[:, r, :, live:]
                assert (rest.view(np.int32) == before[:, r, :, live:].view(np.int32)).all() if in_place else (rest == -1).all()


EVICTS = [
    dict(lens=[1], budget=1),
    dict(lens=[2, 1, 0, 3], budget=1),
    dict(lens=[40, 17, 16, 15, 0, 33], budget=16),                       # above, at and below the budget
    dict(lens=[300, 257, 20], budget=256, sinks=4, recent=32, tracked=[256, 256, 0]),
    dict(lens=[1025] * 3, budget=1024, sinks=4, recent=64, tracked=[1024] * 3, layers=3),   # one token goes
    dict(lens=[700, 3000, 90], budget=77, bs=48, hk=4, sinks=7, recent=70),   # the protected fill the budget
    dict(lens=[700, 300], budget=100, d=64, hk=1, recent=100),
    dict(lens=[700, 300], budget=100, d=96),
    dict(lens=[90, 60], budget=50, d=256, layers=1),
    dict(lens=[90, 60], budget=50, d=640, layers=1),
    dict(lens=[4096, 4097, 511, 513], budget=512, bs=64),                # two blocks a list
    dict(lens=[16385, 30, 9000], budget=4100, bs=128, layers=1, sinks=3, recent=1000, tracked=[4100, 30, 4100]),
    dict(lens=[40000, 1], budget=33000, bs=64, layers=1, hk=1, d=16, sinks=4, recent=5),    # eight; most stay
    dict(lens=[100], budget=99, stride=130),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict_matches_the_definition(cuda_device, case, fp8):
    x = Lists(**EVICTS[case], fp8=fp8, seed=400 + case)
    for in_place in (True, False):
        err = err_word()
        got = x.run(in_place=in_place, err=err)
        assert int(err.item()) == 0
        x.check(got, in_place)


def ties(rng, shape):
    return rng.integers(0, 3, shape).astype(np.float32)


def odd_numbers(rng, shape):
    w = rng.standard_normal(shape).astype(np.float32)
    pick = rng.integers(0, 12, shape)
    for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42)):
        w[pick == i] = x
    return w


@pytest.mark.parametrize("weights", [ties, odd_numbers, lambda rng, shape: np.zeros(shape, np.float32),
                                     lambda rng, shape: 1 + 2.0 ** -23 * rng.integers(0, 700, shape).astype(np.float32)])
@pytest.mark.parametrize("lens,budget", [([50, 40], 39), ([3000, 2000], 1000), ([9000, 20000], 8000)])
def test_evict_orders_ties_zeros_and_what_is_no_number(cuda_device, weights, lens, budget):
    x = Lists(lens, budget, layers=1, d=16, sinks=2, recent=3, weights=weights, seed=budget)
    x.check(x.run())


# Lists too long for a small block, and so many that each has one large block, or a cluster of two with a
# large share each.
@pytest.mark.parametrize("lens,hk,layers", [([5000, 4097] + [4500] * 18, 4, 2), ([20000, 24576] + [6000] * 38, 4, 1),
                                            ([24577] + [5000] * 39, 4, 1), ([16500, 9000] + [4000] * 14, 4, 2)])
@pytest.mark.parametrize("weights", [None, odd_numbers, ties])
def test_evict_of_many_long_lists(cuda_device, lens, hk, layers, weights):
    x = Lists(lens, 3900, layers=layers, hk=hk, d=16, bs=64, sinks=2, recent=30, weights=weights, seed=len(lens))
    for in_place in (True, False):
        err = err_word()
        got = x.run(in_place=in_place, err=err)
        assert int(err.item()) == 0
        x.check(got, in_place)


# Lists of a small block, a short one and a large one, many of each.
PROTECTED = [([1500] * 60 + [2048, 600, 257], 256, 8, 4), ([4000] * 30 + [4096, 2100], 900, 4, 4),
             ([5000] * 40 + [6000], 1500, 4, 2)]


@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("lens,budget,layers,hk", PROTECTED)
def test_evict_where_exactly_the_protected_stay(cuda_device, lens, budget, layers, hk, sinks):
    """sinks + recent == budget, a sliding window: no list has a weight to choose by.  Many lists, often: warps
    must not run ahead of those that still read the counts of protected tokens."""
    x = Lists(lens, budget, layers=layers, hk=hk, d=16, bs=64, sinks=sinks, recent=budget - sinks, seed=budget)
    first = x.run()
    x.check(first)
    for _ in range(20):
        for a, b in zip(x.run(), first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("lens,budget,layers,hk", [([300, 90], 64, 2, 2), ([3000, 2600], 700, 2, 2), ([9000, 20000], 3000, 1, 2),
                                                   ([5000] * 40, 1500, 2, 4)])
def test_evict_of_more_protected_tokens_than_may_stay(cuda_device, lens, budget, layers, hk):
    """Recorded positions that repeat: the protected of the lowest slots stay."""
    x = Lists(lens, budget, layers=layers, hk=hk, d=16, bs=64, sinks=4, recent=10, tracked=[n - 20 for n in lens], seed=budget)
    rng = np.random.default_rng(budget)
    for r, n in enumerate(x.tracked):
        x.pos[:, r, :, :n] = rng.integers(0, 6, (layers, hk, n))
    x.want()
    for in_place in (True, False):
        x.check(x.run(in_place=in_place), in_place)


def test_evict_of_a_first_time_takes_slots_for_positions(cuda_device):
    x = Lists([100, 60, 300], 64, sinks=4, recent=20, seed=5)
    x.check(x.run(bare=True))


def test_evict_a_single_layer_has_lists_without_a_layer(cuda_device):
    x = Lists([100, 60, 300], 64, layers=1, sinks=4, recent=20, seed=6)
    s = x.step
    k, v, w, p, new = x.run(k_pool=s.k_pool[0].cuda(), v_pool=s.v_pool[0].cuda(),
                            weights=torch.from_numpy(x.weights[0]).cuda(), token_pos=torch.from_numpy(x.pos[0]).cuda())
    x.check((k[None], v[None], w[None], p[None], new))


def test_evict_skips_and_flags_bad_rows_and_blocks(cuda_device):
    x = Lists([100, 60, 300, 80], 64, recent=20, seed=7, skipped=(1, 2))
    err, lens = err_word(), [100, -1, 301, 80]
    got = x.run(seq_lens=i32(lens), err=err)
    assert ops.check_error(err) == ERR_LEN
    x.check(got, skipped=(1, 2))
    # the block of row 0's slots 16 .. 31 out of range: nothing moves into it, the lists' entries do
    x = Lists([100, 60], 64, recent=20, seed=7)
    t = x.step.tables.copy()
    lost = int(t[0, 1])
    t[0, 1] = x.step.nb
    got = x.run(block_tables=i32(t), err=err)
    assert ops.check_error(err) == ERR_BLOCK
    after = x.pools_after()
    for pool, want, was in zip(got[:2], after, (x.step.k_pool, x.step.v_pool)):
        want[:, lost] = was[:, lost]
        assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))
    np.testing.assert_array_equal(got[2].cpu().numpy(), x.w_after)
    np.testing.assert_array_equal(got[3].cpu().numpy(), x.p_after)


def test_evict_in_a_graph_on_another_stream(cuda_device):
    """Captured once, replayed on new contents; the same bits as an eager call."""
    xs = [Lists([3000, 70, 5000], 1000, sinks=4, recent=100, seed=s) for s in (8, 9)]
    g = {}
    s = xs[0].step
    args = dict(k_pool=s.k_pool.cuda(), v_pool=s.v_pool.cuda(), block_tables=i32(s.tables), seq_lens=i32(s.lens),
                weights=torch.from_numpy(xs[0].weights).cuda(), token_pos=torch.from_numpy(xs[0].pos).cuda())
    new, nxt = torch.zeros(3, dtype=torch.int32, device="cuda"), i32(xs[0].next)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            ops.evict(**args, budget=1000, max_seq_len=5000, sinks=4, recent=100, next_pos=nxt, new_seq_lens=new)
    for x in xs:
        for name, y in (("k_pool", x.step.k_pool), ("v_pool", x.step.v_pool), ("block_tables", i32(x.step.tables)),
                        ("weights", torch.from_numpy(x.weights)), ("token_pos", torch.from_numpy(x.pos))):
            args[name].copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        x.check((args["k_pool"], args["v_pool"], args["weights"], args["token_pos"], new))


# ---- the calls together ----

@pytest.mark.parametrize("fp8", [False, True])
def test_rows_kept_within_a_budget(cuda_device, fp8):
    """Two layers: prompts written, attended to and weighed by their last queries, cut to a
    budget; then steps of one token each, cut again every few.  Every slot holds the key and
    value of the position that its list records, bit for bit, each list is the definition's, and each
    step's output and weights are those of the tokens that are left."""
    prompt, budget, sinks, recent, bs, hq, hk, layers = [150, 40, 77], 64, 4, 16, 16, 12, 2, 2
    rows, steps, scale, window = 3, 9, 0.0883, 16
    top = max(prompt)
    cap = top + steps
    step = Step([0] * rows, [n + steps for n in prompt], bs, fp8=fp8, layers=layers, seed=700)
    gen = step.gen
    k_pool, v_pool = step.k_pool.cuda(), step.v_pool.cuda()
    tables = i32(step.tables)
    ks, vs = (None, None) if not fp8 else (step.k_scale.cuda(), step.v_scale.cuda())
    qw, kw = ((1 + 0.1 * torch.randn(128, generator=gen)).half().cuda() for _ in range(2))
    rates, err = ops.rope_rates(ops.rope_frequencies(128)), err_word()
    weights = torch.zeros(layers, rows, hk, cap, device="cuda")
    pos = torch.zeros(layers, rows, hk, cap, dtype=torch.int32, device="cuda")
    kept = {}                                   # (layer, row, head, position): key and value as stored

    def slots(r, t):
        t = np.asarray(t)
        return torch.from_numpy(step.tables[r, t // bs].astype(np.int64) * bs + t % bs).cuda()

    def stored(layer, r, h, t):
        s = slots(r, t)
        return k_pool[layer].view(-1, hk, 128)[s, h], v_pool[layer].view(-1, hk, 128)[s, h]

    def widened(x, scale_, h):
        return (x.view(torch.float8_e4m3fn).double() * scale_[h].double() if fp8 else x.double()).cpu()

    def append(layer, lens, counts, at):
        starts = np.concatenate([[0], np.cumsum(counts)])
        x = torch.randn(int(starts[-1]), hq + 2 * hk, 128, generator=gen).half().cuda()
        q = torch.empty(int(starts[-1]), hq, 128, dtype=torch.float16, device="cuda")
        ops.norm_rope_append(k_pool[layer], v_pool[layer], tables, i32(lens), i32(starts), x[:, hq:hq + hk],
                             x[:, hq + hk:], rates, kw, cap, q=x[:, :hq], q_out=q, q_weight=qw,
                             rope_positions=i32(at), k_scale=ks, v_scale=vs, dev_err=err)
        for r in range(rows):
            for h in range(hk):
                t = np.arange(lens[r] - counts[r], lens[r])
                for p, kk, vv in zip(at[starts[r]:], *stored(layer, r, h, t)):
                    kept[layer, r, h, int(p)] = (kk.clone(), vv.clone())
        return q, i32(starts)

    def evict(lens, tracked, nxt):
        want = []
        for i in np.ndindex(layers, rows, hk):
            r, n = i[1], lens[i[1]]
            t = np.arange(n)
            p = np.where(t < tracked[r], pos[i][:n].cpu().numpy(), nxt[r] - n + t)
            w = weights[i][:n].cpu().numpy()
            safe = (p < sinks) | (p >= nxt[r] - recent)
            stays = np.zeros(n, dtype=bool)
            stays[np.lexsort((t, -w, -safe.astype(int)))[:budget]] = True
            want.append((i, dict(zip(p[stays].tolist(), w[stays].tolist()))))
        new = torch.empty(rows, dtype=torch.int32, device="cuda")
        ops.evict(k_pool, v_pool, tables, i32(lens), weights, pos, budget, cap, sinks=sinks, recent=recent,
                  tracked=i32(tracked), next_pos=i32(nxt), new_seq_lens=new, dev_err=err)
        left = new.tolist()
        assert left == [min(n, budget) for n in lens]
        for i, keep in want:
            n = left[i[1]]
            p = pos[i][:n].tolist()
            assert dict(zip(p, weights[i][:n].tolist())) == keep
            for at, kk, vv in zip(p, *stored(*i, np.arange(n))):
                assert torch.equal(kk, kept[(*i, at)][0]) and torch.equal(vv, kept[(*i, at)][1])
        return left

    lens, nxt = list(prompt), list(prompt)
    total = sum(prompt)
    at = np.concatenate([np.arange(n) for n in prompt])
    ws = ops.alloc_prefill_weights_workspace(rows, total, hq, hk, 128, cap, bs, window=window)
    for layer in range(layers):
        q, starts = append(layer, lens, prompt, at)
        ops.prefill_weights(weights[layer], q, k_pool[layer], tables, i32(lens), starts, scale, cap, ws, window=window,
                            k_scale=ks, dev_err=err)
        given = weights[layer].sum(-1).cpu()     # every query gives each head's whole weight
        for r, n in enumerate(prompt):
            assert torch.allclose(given[r], torch.full((hk,), float(min(n, window) * hq // hk)), rtol=1e-4, atol=0)
    tracked = [0] * rows
    lens = tracked = evict(lens, tracked, nxt)
    ws = ops.alloc_decode_weights_workspace(rows, hq, hk, 128, cap, bs)
    for i in range(steps):
        lens, nxt = [n + 1 for n in lens], [n + 1 for n in nxt]
        for layer in range(layers):
            q, _ = append(layer, lens, [1] * rows, np.array(nxt) - 1)
            before, out = weights[layer].cpu().double(), torch.empty_like(q)
            ops.decode_weights(out, weights[layer], q, k_pool[layer], v_pool[layer], tables, i32(lens), scale, cap, ws,
                               k_scale=ks, v_scale=vs, dev_err=err)
            for r in range(rows):
                for h in range(hk):
                    kk, vv = stored(layer, r, h, np.arange(lens[r]))
                    kk, vv = widened(kk, ks, h), widened(vv, vs, h)
                    p = torch.softmax(q[r, 6 * h:6 * h + 6].double().cpu() @ kk.T * scale, -1)
                    w = before[r, h, :lens[r]]
                    w[-1] = 0
                    assert torch.allclose(weights[layer, r, h, :lens[r]].cpu().double(), w + p.sum(0), rtol=1e-4, atol=1e-6)
                    assert torch.allclose(out[r, 6 * h:6 * h + 6].double().cpu(), p @ vv, rtol=4e-3, atol=4e-3)
        if i % 4 == 3:
            lens = tracked = evict(lens, tracked, nxt)
    assert int(err.item()) == 0 and nxt == [n + steps for n in prompt]


def chain(fp8, seed):
    """A prompt's weights, its eviction, then steps of decode and eviction, queued on the current stream
    without a wait: each call reads what the one before has written.  Returns the call and its results."""
    step = Step([0, 0, 0], [300, 47, 180], 16, fp8=fp8, seed=seed)
    a = step.gpu()
    k0, v0 = a["k_pool"].clone(), a["v_pool"].clone()
    scales = dict(k_scale=a["k_scale"], v_scale=a["v_scale"])
    q = torch.randn(step.total, 12, 128, generator=step.gen).half().cuda()
    steps = [torch.randn(3, 12, 128, generator=step.gen).half().cuda() for _ in range(3)]
    w, pos = torch.zeros(3, 2, 300, device="cuda"), torch.zeros(3, 2, 300, dtype=torch.int32, device="cuda")
    lens = [torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(4)]
    nxt = i32([300, 47, 180])
    outs = [torch.zeros(3, 12, 128, dtype=torch.float16, device="cuda") for _ in range(3)]
    wsp = ops.alloc_prefill_weights_workspace(3, step.total, 12, 2, 128, 300, 16, window=40)
    wsd = ops.alloc_decode_weights_workspace(3, 12, 2, 128, 300, 16)
    torch.cuda.synchronize()

    def run(wait=lambda: None):
        a["k_pool"].copy_(k0), a["v_pool"].copy_(v0)
        w.zero_(), wait()
        ops.prefill_weights(w, q, a["k_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.09, 300, wsp, window=40,
                            k_scale=scales["k_scale"]), wait()
        at, tracked = a["seq_lens"], None
        for i, budget in enumerate((100, 60, 30)):
            ops.evict(a["k_pool"], a["v_pool"], a["block_tables"], at, w, pos, budget, 300, sinks=2, recent=9,
                      tracked=tracked, next_pos=nxt, new_seq_lens=lens[i]), wait()
            at = tracked = lens[i]
            ops.decode_weights(outs[i], w, steps[i], a["k_pool"], a["v_pool"], a["block_tables"], at, 0.09, 300, wsd,
                               **scales), wait()
    return run, [a["k_pool"], a["v_pool"], w, pos] + lens + outs


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_queued_one_behind_the_other_and_two_chains_at_once(cuda_device, fp8):
    """Without waits, on two streams at once and in a replayed graph: the bits of calls run one by one."""
    runs, wants = [], []
    for seed in (801, 802):
        run, results = chain(fp8, seed)
        run(torch.cuda.synchronize)
        wants.append([x.clone() for x in results])
        runs.append((run, results))
    streams = [torch.cuda.Stream() for _ in runs]
    graphs = []
    for (run, _), stream in zip(runs, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(stream), torch.cuda.graph(graphs[-1], stream=stream):
            run()
    torch.cuda.synchronize()
    for captured in (False, True):
        for _, results in runs:
            for x in results:
                x.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for (run, _), stream, graph in zip(runs, streams, graphs):
                with torch.cuda.stream(stream):
                    graph.replay() if captured else run()
        torch.cuda.synchronize()
        for (_, results), want in zip(runs, wants):
            for x, y in zip(results, want):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_calls_over_pools_past_32_bits(cuda_device):
    """The bits that the four calls give over a small pool, over pools of more than 2^31 elements."""
    rows, n, bs, hk = 2, 200, 64, 2
    per, far = (n + bs - 1) // bs, (2 ** 31) // (bs * hk * 128) + 100
    gen = torch.Generator().manual_seed(77)
    x = torch.randn(rows * n, 12 + 2 * hk, 128, generator=gen).half().cuda()
    norm = torch.rand(128, generator=gen).half().cuda()
    last = torch.randn(rows, 12, 128, generator=gen).half().cuda()
    lens, starts = i32([n] * rows), i32([0, n, 2 * n])
    rates = ops.rope_rates(ops.rope_frequencies(128))
    results = []
    for base in (0, far):
        pools = [torch.zeros(base + rows * per, bs, hk, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
        tables = i32(base + np.arange(rows * per).reshape(rows, per)[:, ::-1])
        w, pos = torch.zeros(rows, hk, n, device="cuda"), torch.zeros(rows, hk, n, dtype=torch.int32, device="cuda")
        q, out, new, err = torch.empty_like(x[:, :12]).contiguous(), torch.empty_like(last), torch.zeros_like(lens), err_word()
        ops.norm_rope_append(*pools, tables, lens, starts, x[:, 12:12 + hk], x[:, 12 + hk:], rates, norm, n, q=x[:, :12],
                             q_out=q, q_weight=norm, dev_err=err)
        ops.prefill_weights(w, q, pools[0], tables, lens, starts, 0.09, n,
                            ops.alloc_prefill_weights_workspace(rows, rows * n, 12, hk, 128, n, bs), dev_err=err)
        ops.evict(*pools, tables, lens, w, pos, 90, n, sinks=3, recent=20, new_seq_lens=new, dev_err=err)
        ops.decode_weights(out, w, last, *pools, tables, new, 0.09, n,
                           ops.alloc_decode_weights_workspace(rows, 12, hk, 128, n, bs), dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and new.tolist() == [90, 90]
        results.append([q, w, pos, out] + [p[base:].clone() for p in pools])
        del pools
    assert float(results[0][4].abs().max()) > 0
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---- bounded waits that run out ----

TIMEOUT = 8


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("top,rows", [(700, 160), (1024, 20), (6000, 20)])
@pytest.mark.parametrize("granule", [1, 3, 6, 11])
def test_decode_weights_give_up_and_the_next_call_is_as_ever(cuda_device, top, rows, granule, fp8):
    """Blocks alone, in clusters and of the even cut give up with copies in flight: the call ends, flags it, leaves
    the entries behind the rows alone, and the next one over the same workspace has the bits of the one before."""
    lens = [max(1, top - 31 * i) for i in range(rows)]
    step = Step(lens, [0] * rows, 64, fp8=fp8, seed=71)
    q = torch.randn(rows, 12, 128, generator=step.gen).half().cuda()
    before = torch.rand(rows, 2, top, generator=step.gen).cuda()
    a, err = step.gpu(), err_word()
    ws = ops.alloc_decode_weights_workspace(rows, 12, 2, 128, top, 64)

    def run():
        w, out = before.clone(), torch.zeros_like(q)
        ops.decode_weights(out, w, q, a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], 0.09, top, ws,
                           k_scale=a["k_scale"], v_scale=a["v_scale"], dev_err=err)
        torch.cuda.synchronize()
        return out, w

    want = run()
    assert int(err.item()) == 0
    try:
        ops.debug_set_weights_hooks(granule=granule)
        _, w = run()
    finally:
        ops.debug_set_weights_hooks()
    assert ops.check_error(err) == TIMEOUT
    for r, n in enumerate(lens):
        assert torch.equal(w[r, :, n:], before[r, :, n:])
    assert all(torch.equal(x, y) for x, y in zip(run(), want))
    assert int(err.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("jobs", [1, 2, 6, 10])
@pytest.mark.parametrize("role", ["copies", "products", "widening", "sums"])
def test_prefill_weights_give_up_and_the_next_call_is_as_ever(cuda_device, role, jobs, fp8):
    """Any of a block's roles gives up, at once or with tiles and products in flight: as decode's."""
    step = Step([900, 10, 300], [700, 1500, 33], 48, fp8=fp8, seed=72)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half().cuda()
    before = torch.rand(3, 2, step.max_len + 7, generator=step.gen).cuda()
    a, err = step.gpu(), err_word()
    ws = ops.alloc_prefill_weights_workspace(3, step.total, 12, 2, 128, step.max_len, 48)

    def run():
        w = before.clone()
        ops.prefill_weights(w, q, a["k_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.09, step.max_len, ws,
                            k_scale=a["k_scale"], dev_err=err)
        torch.cuda.synchronize()
        return w

    want = run()
    assert int(err.item()) == 0
    for fill in (None, 0, 255):
        if fill is not None:
            ws.fill_(fill)
        try:
            ops.debug_set_weights_hooks(role=role, jobs=jobs)
            w = run()
        finally:
            ops.debug_set_weights_hooks()
        assert ops.check_error(err) == (TIMEOUT if fp8 or role != "widening" else 0)
        for r, n in enumerate(step.lens):
            assert torch.equal(w[r, :, n:], before[r, :, n:])
        assert torch.equal(run(), want)
        assert int(err.item()) == 0


# ---- eviction and the block manager ----

def test_evicted_rows_go_on_over_their_blocks_and_a_finished_ones_go_round(cuda_device):
    """A row evicts, is truncated and goes on in the slots behind what stayed, over the blocks that it has; when it
    ends they go to another row, and nothing of the row beside it changes."""
    bs, hq, hk, budget, sinks, recent, cap, steps = 16, 12, 2, 48, 2, 8, 352, 30
    gen = torch.Generator().manual_seed(90)
    randn = lambda *shape: torch.randn(*shape, generator=gen).half()
    bm = BlockManager(36, bs, cap // bs)
    prompts = [300, 90]
    for seq, n in enumerate(prompts):
        bm.admit(seq, n, steps + 1)
    tables, lens = bm.tables([0, 1])
    pools = [randn(36, bs, hk, 128) for _ in range(2)]
    k_pool, v_pool = (x.cuda() for x in pools)
    weights = torch.rand(2, hk, cap, generator=gen)
    w, pos, err = weights.cuda(), torch.zeros(2, hk, cap, dtype=torch.int32, device="cuda"), err_word()

    def slots(table, t):
        t = np.asarray(t)
        return torch.from_numpy(table[t // bs].astype(np.int64) * bs + t % bs)

    def stored(r, n):
        return [p.cpu().view(-1, hk, 128)[slots(tables[r], np.arange(n))] for p in (k_pool, v_pool)]

    want = []                                               # per row: keys and values by slot
    for r, n in enumerate(prompts):
        rows = [p.view(-1, hk, 128)[slots(tables[r], np.arange(n))].clone() for p in pools]
        for h in range(hk):
            t = np.arange(n)
            safe = (t < sinks) | (t >= n - recent)
            stays = np.zeros(n, dtype=bool)
            stays[np.lexsort((t, -weights[r, h, :n].numpy(), -safe.astype(int)))[:budget]] = True
            to, frm = t[(t < budget) & ~stays], t[(t >= budget) & stays]
            for x in rows:
                x[to, h] = x[frm, h]
        want.append([x[:budget] for x in rows])
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    ops.evict(k_pool, v_pool, i32(tables), i32(lens), w, pos, budget, cap, sinks=sinks, recent=recent, new_seq_lens=new,
              dev_err=err)
    for seq, n in enumerate(new.tolist()):
        bm.truncate(seq, n)
    kept, lens = bm.tables([0, 1])
    assert lens.tolist() == [budget, budget] and np.array_equal(kept, tables)
    ws = ops.alloc_decode_weights_workspace(2, hq, hk, 128, cap, bs)
    for i in range(steps):
        at = [bm.append_slot(seq) for seq in (0, 1)]
        assert at == [(budget + i, None)] * 2
        k, v, q = randn(2, hk, 128), randn(2, hk, 128), randn(2, hq, 128)
        tables, lens = bm.tables([0, 1])
        ops.append(k_pool, v_pool, i32(tables), i32([p for p, _ in at]), k.cuda(), v.cuda(), dev_err=err)
        out = torch.empty(2, hq, 128, dtype=torch.float16, device="cuda")
        ops.decode_weights(out, w, q.cuda(), k_pool, v_pool, i32(tables), i32(lens), 0.0883, cap, ws, dev_err=err)
        torch.cuda.synchronize()
        for r in range(2):
            want[r] = [torch.cat([x, y[r:r + 1]]) for x, y in zip(want[r], (k, v))]
            for x, y in zip(stored(r, int(lens[r])), want[r]):
                assert torch.equal(x, y)
            for h in range(hk):
                kk, vv = (x[:, h].double() for x in want[r])
                p = torch.softmax(q[r, 6 * h:6 * h + 6].double() @ kk.T * 0.0883, -1)
                assert torch.allclose(out[r, 6 * h:6 * h + 6].double().cpu(), p @ vv, rtol=4e-3, atol=4e-3)
    assert np.array_equal(tables, kept)                     # thirty tokens more in the blocks that they had
    # row 0 ends; another one takes its blocks
    bm.free(0)
    assert bm.try_admit(2, 320, 1)
    table, n = bm.table(2)
    assert set(table[:20].tolist()) & set(kept[0][:20].tolist()) and not set(table[:20].tolist()) & set(kept[1][:8].tolist())
    k, v = randn(1, n, hk, 128), randn(1, n, hk, 128)
    ops.prefill_scatter(k_pool, v_pool, i32(table[None]), i32([0]), i32([0]), i32([n]), k.cuda(), v.cuda(), dev_err=err)
    torch.cuda.synchronize()
    for x, y in zip(stored(1, int(lens[1])), want[1]):
        assert torch.equal(x, y)
    for p, x in ((k_pool, k), (v_pool, v)):
        assert torch.equal(p.cpu().view(-1, hk, 128)[slots(table, np.arange(n))], x[0])
    assert int(err.item()) == 0


def test_a_first_call_inside_a_capture(cuda_device):
    """A fresh process whose first decode and prompt weights are captured: what a first call asks the device for
    may be asked there, and the replays give the eager calls' bits."""
    code = """
import torch
from paged_kv_cache_06_gb300 import ops
gen = torch.Generator().manual_seed(3)
rows, n, bs = 76, 900, 32
per = (n + bs - 1) // bs
k, v = (torch.randn(rows * per, bs, 2, 128, generator=gen).half().cuda() for _ in range(2))
tables = torch.arange(rows * per, dtype=torch.int32).view(rows, per).flip(1).contiguous().cuda()
lens = torch.full((rows,), n, dtype=torch.int32, device="cuda")
q = torch.randn(rows, 12, 128, generator=gen).half().cuda()
starts = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
first = torch.rand(rows, 2, n, generator=gen).cuda()
w, out = first.clone(), torch.zeros_like(q)
wsd = ops.alloc_decode_weights_workspace(rows, 12, 2, 128, n, bs)
wsp = ops.alloc_prefill_weights_workspace(rows, rows, 12, 2, 128, n, bs)
def both():
    ops.decode_weights(out, w, q, k, v, tables, lens, 0.09, n, wsd)
    ops.prefill_weights(w, q, k, tables, lens, starts, 0.09, n, wsp)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    both()
results = []
for run in (graph.replay, graph.replay, both):
    w.copy_(first)
    out.zero_()
    run()
    torch.cuda.synchronize()
    results.append((w.clone(), out.clone()))
assert float(results[0][1].abs().max()) > 0 and not torch.equal(results[0][0], first)
for r in results[1:]:
    assert torch.equal(r[0], results[0][0]) and torch.equal(r[1], results[0][1])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root, timeout=300).returncode == 0
