"""Frequency arguments that are finite while what follows from them is not."""
import math

import pytest
import torch

from paged_kv_cache_06_gb300 import ops

INVALID = 1


@pytest.mark.parametrize("kw", [
    dict(base=1e300, scaling="base", factor=1e300),
    dict(base=10000.0, scaling="base", factor=1e308),
    dict(scaling="by_parts", factor=2.0, original_len=1e308, low=-1.7e308, high=1.7e308),
    dict(scaling="by_parts", factor=2.0, original_len=4096.0, low=-1e308, high=1e308),
])
def test_results_that_are_no_numbers_are_refused(kw):
    with pytest.raises(ops.PagedKVError) as e:
        ops.rope_frequencies(64, **kw)
    assert e.value.status == INVALID


def test_the_largest_arguments_that_are_not():
    f = ops.rope_frequencies(64, base=1e290, scaling="base", factor=1e10)
    assert bool(torch.isfinite(f).all()) and float(f[0]) == 1.0 and bool((f[1:] < f[:-1]).all())
    f = ops.rope_frequencies(64, scaling="by_parts", factor=4.0, original_len=1e308, low=0.0, high=1e308)
    assert bool(torch.isfinite(f).all()) and math.isclose(float(f[-1]), 10000.0 ** (-62 / 64) / 4, rel_tol=1e-3)
