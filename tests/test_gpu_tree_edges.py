"""GPU tests of the drafted step's edges: numbers that are none, weights far
below a row's largest, bad rows, calls that start early, units cut between
blocks."""
import time

import numpy as np
import pytest
import torch

from paged_kv_cache_06_gb300 import ops
from test_gpu_tree_step import ERR_LEN, ERR_TIMEOUT, Step, check, err_word, i32, random_parents, seen_of, tree_ref, tree_run

pytestmark = pytest.mark.gpu

ERR_PLAN = 0x10

# prefix, nodes: whole units; units of two pieces (76 units of 64 granules over 152
# blocks); units of many pieces
CUTS = [([100, 7, 300], [9, 4, 12]), ([4090] * 38, [6] * 38), ([20000, 50], [9, 3])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,nodes", CUTS)
def test_a_query_that_is_no_number_has_none_for_an_answer(cuda_device, prefix, nodes, fp8):
    """However its unit is cut; and the other (node, head) rows keep their bits."""
    step = Step(prefix, nodes, 64, fp8=fp8, seed=41)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(nodes, 2), step.starts)
    want = tree_run(step, q, mask, 0.1)
    bad = [(0, 0, 5), (2, 7, 100), (step.total - 1, 11, 0)]
    for g, h, d in bad:
        q[g, h, d] = float("nan")
    got = tree_run(step, q, mask, 0.1)
    hit = torch.zeros(step.total, 12, dtype=torch.bool)
    for g, h, _ in bad:
        hit[g, h] = True
    assert bool(torch.isnan(got[hit.cuda()]).all())
    assert torch.equal(got[~hit.cuda()], want[~hit.cuda()])


@pytest.mark.parametrize("prefix,nodes", CUTS)
def test_cached_keys_that_are_no_numbers_reach_every_node(cuda_device, prefix, nodes):
    """A run of 1024 tokens (whole pieces among them) whose keys are NaN in one KV head."""
    step = Step(prefix, nodes, 64, seed=42)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(nodes, 2), step.starts)
    want = tree_run(step, q, mask, 0.1)
    a = step.prefix[0] // 4
    step.k_pool.view(-1, 2, 128)[step.slots(0, a, min(a + 1024, step.prefix[0])), 1] = float("nan")
    got = tree_run(step, q, mask, 0.1)
    n = nodes[0]
    assert bool(torch.isnan(got[:n, 6:]).all())
    assert torch.equal(got[:n, :6], want[:n, :6]) and torch.equal(got[n:], want[n:])


@pytest.mark.parametrize("prefix,nodes", CUTS)
def test_scales_that_are_no_numbers(cuda_device, prefix, nodes):
    """A KV head whose key or value scale is NaN has no numbers for answers; the other
    head keeps its bits."""
    step = Step(prefix, nodes, 64, fp8=True, seed=43)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    mask = ops.tree_mask(random_parents(nodes, 2), step.starts)
    want = tree_run(step, q, mask, 0.1)
    for name in ("k_scale", "v_scale"):
        sc = getattr(step, name).clone()
        sc[0] = float("nan")
        got = tree_run(step, q, mask, 0.1, **{name: sc.cuda()})
        assert bool(torch.isnan(got[:, :6]).all()), name
        assert torch.equal(got[:, 6:], want[:, 6:]), name


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cached,nodes", [(1000, 3), (4090, 6), (30000, 2)])
def test_weights_far_below_the_largest_count(cuda_device, cached, nodes, fp8):
    """One token in 128 has a weight of 1 and a value of 0, all others a weight of 2^-26
    and a large value: what they add up to is the answer.

    Weights are stored for their product as fp16 numbers 2^7 above the row's reference,
    so one below 2^-21 of it is off by 2^-32 of it at most; the rest as in tree_ref,
    whose bound for small weights is 2^-25."""
    bits = 26
    step = Step([cached], [nodes], 64, hk=1, fp8=fp8, seed=44)
    L = step.lens[0]
    big = torch.arange(L) % 128 == 40
    k = torch.zeros(L, 1, 128)
    k[big, 0, 0] = 1.0
    v = torch.where(big, 0.0, 448.0 if fp8 else 60000.0)[:, None, None].expand(L, 1, 128)
    for pool, x in ((step.k_pool, k), (step.v_pool, v)):
        x = x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.half()
        pool.view(-1, 1, 128)[step.slots(0)] = x
    if fp8:
        step.k_scale, step.v_scale = torch.ones(1), torch.full((1,), 134.0)
    q = torch.zeros(step.total, 4, 128, dtype=torch.float16)
    q[:, :, 0] = 1.0
    scale = bits * float(np.log(2.0))
    ref, tol = tree_ref(step, q, seen_of(step, None), scale)
    low = 2.0 ** -25 - 2.0 ** -32
    val = 60032.0 if fp8 else 60000.0
    n = L - int(big.sum())
    # tree_ref's bound for the small weights' roundings, less what 2^7 more leaves of it; every
    # node sees at least n - nodes of those tokens
    tol = tol - low * val * (n - nodes)
    # p|v| of a row is the row's answer, so its other terms stay
    got = tree_run(step, q, None, scale)
    assert float(ref.min()) > 0.05
    check(got, ref, tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_shares_given_up_are_merged_by_the_last_block(cuda_device, fp8):
    """Units of three pieces and more whose blocks wait for each other for next to no
    time: whoever arrives last does the others' shares, with the same bits, and the
    workspace is ready for the next call."""
    patience(fp8, (([20000, 50], [9, 3], (12, 2)), ([9000, 7000, 8000], [6, 4, 5], (4, 4)),
                   ([30000], [64], (12, 2))))


@pytest.mark.parametrize("fp8", [False, True])
def test_the_second_of_two_pieces_does_not_wait_for_the_first(cuda_device, fp8):
    """Units of two pieces whose second block hardly waits: whichever block stores last
    merges the two, with the fold's bits."""
    # 76 units over 152 blocks: every one in two halves
    folded, handed_over = patience(fp8, (([4090] * 38, [6] * 38, (12, 2)),))
    assert folded == 0 and (handed_over > 0 or fp8)  # over FP8 pools the second half is the longer one
    patience(fp8, (([2000] * 38, [40] * 38, (12, 2)), ([4000] * 19, [30] * 19, (32, 4)),
                   ([1500, 900, 3000] * 13, [12, 3, 22] * 13, (12, 2))))


def patience(fp8, batches):
    """The same bits however long blocks wait; how many blocks stored a last piece with the
    usual patience and with none (a partial is 2 x 128 + 128 x 128 floats, two a block)."""
    counts = [0, 0]

    def last_pieces(ws):
        return int((ws[192 * 32 * 4:].view(torch.float32).view(192, 2, -1)[:, 1] != 0).any(-1).sum())

    for prefix, nodes, heads in batches:
        step = Step(prefix, nodes, 64, hk=heads[1], fp8=fp8, seed=48)
        q = torch.randn(step.total, heads[0], 128, generator=step.gen).half()
        ws = ops.alloc_tree_workspace(step.rows, step.total, *heads, 128, 64)
        err = err_word()
        want = tree_run(step, q, None, 0.1, err, workspace=ws)
        counts[0] += last_pieces(ws)
        try:
            for help_ns in (1, 1, 1, 500, 2000, 1, 3000):
                ops.debug_set_tree_hooks(help_ns)
                assert torch.equal(tree_run(step, q, None, 0.1, err, workspace=ws), want), help_ns
        finally:
            ops.debug_set_tree_hooks()
        counts[1] += last_pieces(ws)
        assert torch.equal(tree_run(step, q, None, 0.1, err, workspace=ws), want)
        assert ops.check_error(err) == 0
        # the words by which blocks find each other are back at zero (they come before the partials)
        assert int(ws[:192 * 32 * 4].count_nonzero()) == 0
    return counts


@pytest.mark.parametrize("fp8", [False, True])
def test_a_block_that_gives_up_its_fold_waits_for_the_copy(cuda_device, fp8):
    """A block that gives up between issuing the copy of the other half and using it:
    the call ends soon, flags the error, and the next one on a zero-filled workspace
    is right."""
    prefix, nodes = CUTS[1]
    step = Step(prefix, nodes, 64, fp8=fp8, seed=49)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    ws = ops.alloc_tree_workspace(step.rows, step.total, 12, 2, 128, 64)
    err = err_word()
    want = tree_run(step, q, None, 0.1, err, workspace=ws)
    assert ops.check_error(err) == 0
    for _ in range(3):
        try:
            ops.debug_set_tree_hooks(0, True)
            t0 = time.perf_counter()
            got = tree_run(step, q, None, 0.1, err, workspace=ws)
            assert time.perf_counter() - t0 < 2.0
        finally:
            ops.debug_set_tree_hooks()
        assert ops.check_error(err) == ERR_TIMEOUT
        assert bool(torch.isnan(got).any())           # what the blocks left out
        ws.zero_()
        assert torch.equal(tree_run(step, q, None, 0.1, err, workspace=ws), want)
        assert ops.check_error(err) == 0


def test_a_refused_plan_keeps_the_streams_order(cuda_device):
    """Tree attention, a planned decode that starts early and refuses its plan, and a
    rotary append in place on the tree's output: the append waits for the tree."""
    step = Step([30000, 9000, 50], [9, 12, 3], 64, seed=46, fill=False)
    T, d = step.total, 128
    q = torch.randn(T, 12, d, generator=step.gen).half().cuda()
    k, v = (torch.randn(T, 2, d, generator=step.gen).half().cuda() for _ in range(2))
    rates = ops.rope_rates(ops.rope_frequencies(d))
    a = step.gpu()
    rows = (a["block_tables"], a["seq_lens"], a["q_start"])
    ws = ops.alloc_tree_workspace(3, T, 12, 2, d, 64)
    dws = ops.alloc_workspace(3, 12, 2, d, step.max_len, 64)
    plan = ops.alloc_plan(3, 12, 2, d, step.max_len, 64)
    ops.plan(plan, a["block_tables"], i32([16, 16, 16]), None, 12, 2, d, 64, step.nb, 16)
    z = torch.empty(3, 12, d, dtype=torch.float16, device="cuda")
    err = err_word()

    def go(wait):
        out = torch.full_like(q, float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):
            ops.tree_attention(out, q, a["k_pool"], a["v_pool"], *rows, 0.1, step.max_len, ws)
            wait()
            ops.decode_planned(z, q[:3], a["k_pool"], a["v_pool"], *rows[:2], 0.1, step.max_len, plan, dws, pdl=True,
                               dev_err=err)
            wait()
            ops.rope_append(a["k_pool"], a["v_pool"], *rows, k, v, rates, step.max_len, q=out, q_out=out)
            wait()
        torch.cuda.synchronize()
        assert ops.check_error(err) == ERR_PLAN
        return out

    want = go(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(go(lambda: None), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_what_a_call_reads_may_come_from_the_kernel_before_it(cuda_device, fp8):
    """Lengths from the commit, then starts, paths, tables, positions, rates and mask words
    that kernels of the same stream have just written: with a wait after each, without, and
    captured, the same bits."""
    hq, hk, d, rounds = 12, 2, 128, 6
    step = Step([300, 17, 2000, 60], [9, 4, 13, 6], 16, fp8=fp8, seed=47, fill=False)
    T, rows = step.total, step.rows
    x0 = torch.randn(T, hq, d, generator=step.gen).half().cuda()
    masks = [ops.tree_mask(random_parents(step.nodes, s), step.starts).cuda() for s in range(rounds)]
    rates = [ops.rope_rates(ops.rope_frequencies(d, base=10000.0 + 500 * s)) for s in range(rounds)]
    paths = [i32([[0, 2, 3 + s % 3, 8], [1, 3, -1, -1], [4, 5, 6 + s, 12], [s % 6, -1, -1, -1]]) for s in range(rounds)]
    counts = i32([4, 2, 4, 1])
    # the rows change places from round to round: starts, tables and lengths with them
    order = [torch.roll(torch.arange(rows), s).cuda() for s in range(rounds)]
    nodes = i32(step.nodes)

    def run(how):
        a = step.gpu()
        x, out = x0.clone(), torch.empty_like(x0)
        lens, nl = a["seq_lens"].clone(), torch.zeros(rows, dtype=torch.int32, device="cuda")
        tables, starts = torch.full_like(a["block_tables"], -1), torch.full_like(a["q_start"], -1)
        mask, rate, path, pos = (torch.full_like(t, -1) for t in (masks[0], rates[0], paths[0], x0[:, 0, 0].int()))
        plen = torch.full_like(counts, -1)
        ws = ops.alloc_tree_workspace(rows, T, hq, hk, d, 16)
        err = err_word()
        args = (tables, lens, starts)
        sc = dict(k_scale=a["k_scale"], v_scale=a["v_scale"])
        wait = torch.cuda.synchronize if how == "waits" else lambda: None

        def go():
            for s in range(rounds):
                o = order[s]
                starts.copy_(a["q_start"])
                starts[1:].copy_(torch.cumsum(nodes[o], 0))
                torch.index_select(a["block_tables"], 0, o, out=tables)
                torch.index_select(a["seq_lens"], 0, o, out=lens)
                mask.copy_(masks[s] if s % rows == 0 else mask)
                rate.copy_(rates[s])
                pos.fill_(100 * s)
                wait()
                ops.rope_append(a["k_pool"], a["v_pool"], *args, x[:, :hk], x[:, hk:2 * hk], rate, step.max_len,
                                q=x, q_out=out, rope_positions=pos, dev_err=err, **sc)
                wait()
                ops.tree_attention(x, out, a["k_pool"], a["v_pool"], *args, 0.09, step.max_len, ws,
                                   mask=mask if s % rows == 0 else None, dev_err=err, **sc)
                torch.index_select(paths[s], 0, o, out=path)
                torch.index_select(counts, 0, o, out=plen)
                wait()
                ops.tree_commit(a["k_pool"], a["v_pool"], *args, path, plen, step.max_len, new_seq_lens=nl, dev_err=err)
                # the committed tokens alone, as the next step's lengths and no new nodes but the last
                lens.copy_(nl)
                starts.copy_(torch.arange(rows + 1, device="cuda"))
                wait()
                ops.tree_attention(out[:rows], x[:rows], a["k_pool"], a["v_pool"], *args, 0.09, step.max_len, ws,
                                   dev_err=err, **sc)
                x[:rows].copy_(out[:rows])
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
        return [t.cpu().view(torch.uint8) for t in (x, out, nl, a["k_pool"], a["v_pool"])], x

    want, x = run("waits")
    assert bool(torch.isfinite(x).all())
    for how in ("stream", "stream", "graph"):
        for w, g in zip(want, run(how)[0]):
            assert torch.equal(w, g), how


def test_rows_that_overlap_beyond_all_bounds_are_refused(cuda_device):
    """Starts that rise and fall: every other row names all the nodes, and their work
    together passes 2^31 tile steps (512 rows x 8 KV heads x 256 M blocks of each of four
    planes x 3,125 granules).  Nothing is written; smaller ones are answered."""
    hq, hk, T, rows, L = 64, 8, 16384, 1024, 200000
    pool = torch.randn(1, 64, hk, 128, device="cuda").half()
    q = torch.zeros(T, hq, 128, dtype=torch.float16, device="cuda")
    q[:64] = torch.randn(64, hq, 128, device="cuda").half()
    ws = ops.alloc_tree_workspace(rows, T, hq, hk, 128, 64)
    tables = torch.zeros(rows, L // 64, dtype=torch.int32, device="cuda")
    err = err_word()

    def go(nodes, length, total):
        starts = torch.zeros(rows + 1, dtype=torch.int32)
        starts[1::2] = nodes
        out = torch.full((total, hq, 128), float("nan"), dtype=torch.float16, device="cuda")
        ops.tree_attention(out, q[:total], pool, pool, tables, torch.full((rows,), length, dtype=torch.int32).cuda(),
                           starts.cuda(), 0.1, L, ws, dev_err=err)
        assert ops.check_error(err) == ERR_LEN        # the rows between have fewer than no nodes
        return out

    assert bool(torch.isnan(go(T, L, T)).all())
    got = go(64, 300, 64)                             # every other row gives the same answers, but for roundings
    want = torch.empty_like(got)
    ops.tree_attention(want, q[:64], pool, pool, tables[:1], i32([300]), i32([0, 64]), 0.1, L, ws, dev_err=err)
    torch.cuda.synchronize()
    assert ops.check_error(err) == 0
    assert bool(((got - want).float().abs() <= 2e-3 + 2e-3 * want.float().abs()).all())


def test_rope_append_flags_rows_that_no_token_leads_to(cuda_device):
    """Rows without nodes, of falling starts, and behind total_q are looked at too."""
    step = Step([20, 9, 40], [6, 3, 2], 16, seed=45, fill=False)
    k, v = (torch.randn(11, 2, 128, generator=step.gen).half().cuda() for _ in range(2))
    rates = ops.rope_rates(ops.rope_frequencies(128))

    def go(lens, starts, total=11):
        a = step.gpu(seq_lens=i32(lens), q_start=i32(starts))
        err = err_word()
        ops.rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], k[:total], v[:total],
                        rates, step.max_len, dev_err=err)
        return ops.check_error(err)

    assert go([26, 12, 42], [0, 6, 9, 11]) == 0
    assert go([26, 12, 42], [0, 6, 6, 8]) == 0
    assert go([26, 1000, 42], [0, 6, 6, 8]) == ERR_LEN      # above the bound, without nodes
    assert go([26, -1, 42], [0, 6, 6, 8]) == ERR_LEN
    assert go([26, 12, 42], [0, 6, 2, 2]) == ERR_LEN        # fewer than no nodes
    assert go([26, 12, 42], [0, 6, 9, 11], total=6) == ERR_LEN   # nodes past total_q
    rows = 700                                               # more rows than the block has threads
    t = torch.zeros(rows, 1, dtype=torch.int32)
    for bad in (0, 255, 699):
        lens = torch.full((rows,), 1, dtype=torch.int32)
        lens[bad] = 17
        st = torch.zeros(rows + 1, dtype=torch.int32)
        st[-1] = 1
        if bad == rows - 1:
            st[1:] = 1
        a = step.gpu(block_tables=t.cuda(), seq_lens=lens.cuda(), q_start=st.cuda())
        err = err_word()
        ops.rope_append(a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], k[:1], v[:1], rates,
                        16, dev_err=err)
        assert ops.check_error(err) == ERR_LEN, bad


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_whose_offsets_pass_32_bits(cuda_device, fp8):
    """The last blocks of pools of more than 2^32 bytes: the same bits as in small pools."""
    bs, hk, d = 64, 2, 128
    step = Step([300, 40, 129], [9, 30, 5], bs, hk=hk, fp8=fp8, seed=50, fill=False)
    extra = (1 << 32) // (bs * hk * d * (1 if fp8 else 2)) + 3
    q = torch.randn(step.total, 12, d, generator=step.gen).half().cuda()
    k, v = (torch.randn(step.total, hk, d, generator=step.gen).half().cuda() for _ in range(2))
    mask = ops.tree_mask(random_parents(step.nodes, 6), step.starts).cuda()
    rates = ops.rope_rates(ops.rope_frequencies(d))
    paths = i32([[0, 3, 8], [2, 17, 29], [1, 4, -1]])

    def run(shift):
        a = step.gpu()
        kp, vp = a["k_pool"], a["v_pool"]
        if shift:
            kp, vp = (torch.empty((shift + step.nb, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in (kp, vp))
            kp[shift:], vp[shift:] = a["k_pool"], a["v_pool"]
        tables = torch.where(a["block_tables"] >= 0, a["block_tables"] + shift, -1).int()
        rows = (tables, a["seq_lens"], a["q_start"])
        sc = dict(k_scale=a["k_scale"], v_scale=a["v_scale"])
        err, nl = err_word(), torch.zeros(3, dtype=torch.int32, device="cuda")
        ws = ops.alloc_tree_workspace(3, step.total, 12, hk, d, bs)
        qo, out = torch.empty_like(q), torch.empty_like(q)
        ops.rope_append(kp, vp, *rows, k, v, rates, step.max_len, q=q, q_out=qo, dev_err=err, **sc)
        ops.tree_attention(out, qo, kp, vp, *rows, 0.1, step.max_len, ws, mask=mask, dev_err=err, **sc)
        ops.tree_commit(kp, vp, *rows, paths, i32([3, 3, 2]), step.max_len, new_seq_lens=nl, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return [x.cpu() for x in (qo, out, kp[shift:].view(torch.uint8), vp[shift:].view(torch.uint8), nl)]

    for a, b in zip(run(0), run(extra)):
        assert torch.equal(a, b)


def test_a_prompt_sized_chain_equals_prefill(cuda_device):
    """Chunks of hundreds to thousands of tokens without a mask, over empty and long caches,
    beside the prefill kernel (2e-3 + 2e-3 |ref| is its tolerance; both sides take half at most)."""
    step = Step([0, 500, 9000, 3], [2048, 1000, 700, 1500], 64, seed=51)
    q = torch.randn(step.total, 12, 128, generator=step.gen).half()
    a = step.gpu()
    out = torch.empty(step.total, 12, 128, dtype=torch.float16, device="cuda")
    ops.prefill(out, q.cuda(), a["k_pool"], a["v_pool"], a["block_tables"], a["seq_lens"], a["q_start"], 0.0883,
                step.max_len)
    err = err_word()
    got = tree_run(step, q, None, 0.0883, err)
    assert int(err.item()) == 0
    assert bool(((got - out).float().abs() <= 2e-3 + 2e-3 * out.float().abs()).all())


@pytest.mark.parametrize("rise", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("log2", [20, 23, 24, 25, 26, 27])
def test_scores_so_large_that_their_differences_round(cuda_device, log2, rise):
    """Finite scores of 2^20 to 2^27 (in powers of two of the weight) that grow along the
    row by a few units in the last place.  Roundings of the products decide which token
    counts, but every answer is a mean of the row's values: finite, and between the
    smallest and the largest of each dim."""
    step = Step([1700, 1000], [9, 4], 16, seed=52)
    q = torch.zeros(step.total, 12, 128, dtype=torch.float16)
    q[:, :, 0] = 4096.0
    q[:, :, 1] = 1.0
    kp = step.k_pool.view(-1, 2, 128)
    scale = 2.0 ** (log2 - 24) * float(np.log(2.0))
    for r in range(2):
        s = step.slots(r)
        kp[s] = 0
        kp[s, :, 0] = 4096.0                   # a score of 2^24 in units of the scale, more by `rise` from tile to tile
        kp[s, :, 1] = (rise * (torch.arange(len(s)) // 128)).half()[:, None]
    mask = ops.tree_mask(random_parents(step.nodes, 3), step.starts)
    got = tree_run(step, q, mask, scale).double().cpu()
    assert bool(torch.isfinite(got).all())
    for r in range(2):
        v = step.values(step.v_pool, r, None).repeat_interleave(6, 1)
        a = int(step.starts[r])
        x = got[a:a + step.nodes[r]]
        slack = 2.0 ** -9 * v.abs().amax(0)     # weights, sums and the output are rounded to 2^-11 each
        assert bool((x <= v.amax(0) + slack).all()) and bool((x >= v.amin(0) - slack).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,nodes,heads", [
    ([0, 354, 1856, 1777, 0, 3828], [86, 1, 72, 34, 43, 3], (32, 8)),   # a piece of three, then units of one tile
    ([40] * 300, [3] * 300, (12, 2)),                                  # four units of one tile a block
    ([30, 3000] * 60, [5, 2] * 60, (4, 4)),
])
def test_a_warp_that_stays_behind_at_a_units_end(cuda_device, prefix, nodes, heads, fp8):
    """The other softmax group may have no tile in the next unit and be at its end at once:
    what one warp still has to read of this unit's sums must be there."""
    step = Step(prefix, nodes, 64, hk=heads[1], fp8=fp8, seed=53)
    q = torch.randn(step.total, heads[0], 128, generator=step.gen).half()
    ws = ops.alloc_tree_workspace(step.rows, step.total, *heads, 128, 64)
    err = err_word()
    ref, tol = tree_ref(step, q, seen_of(step, None), 0.0883)
    try:
        for linger_ns in (20000, 3000, 0):
            ops.debug_set_tree_hooks(0, False, linger_ns)
            check(tree_run(step, q, None, 0.0883, err, workspace=ws), ref, tol, f"linger {linger_ns}")
    finally:
        ops.debug_set_tree_hooks()
    assert ops.check_error(err) == 0
