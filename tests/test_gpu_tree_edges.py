"""GPU tests of the drafted step's edges: numbers that are none, weights far
below a row's largest, bad rows, calls that start early, units cut between
blocks."""
import pytest
import torch

from paged_kv_cache_06_gb300 import ops
from test_gpu_tree_step import Step, random_parents, tree_run

pytestmark = pytest.mark.gpu

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
