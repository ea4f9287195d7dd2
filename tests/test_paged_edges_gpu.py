"""GPU tests of the paged cache and its attention where values or batch
arrays are unusual, against plain 64-bit forms (paged_ref.py).  Attention is
held to the tolerance of test_paged_gpu.py, whose docstring derives it."""
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import paged_ref as ref
from test_paged_gpu import DEV, E4M3, _check_attn, _normal

pytestmark = pytest.mark.gpu


def _quantised_cache(k, v):
    """An E4M3 cache of the bf16 pools k, v, as cache_append would write them,
    and its float64 values."""
    parts = []
    for x in (k, v):
        y, e = ref.quantise(x)
        parts.append((y.float().to(E4M3).to(DEV), (e + 127).to(torch.uint8).to(DEV)))
    (k8, ks), (v8, vs) = parts
    return dd.PagedCache(k8, v8, ks, vs), ref.values(k8, ks), ref.values(v8, vs)


@pytest.mark.parametrize("gain", [2.0 ** -96, 2.0 ** -106, 2.0 ** -114])
@pytest.mark.parametrize("D,new,past", [
    (128, (1, 1), (600, 300)),       # items taken whole
    (64, (1,), (5000,)),             # one row split over many CTAs
    (128, (4, 3), (2000, 90)),       # more than eight rows per kv head
])
def test_attention_e4m3_values_near_the_smallest_scale(gain, D, new, past):
    # scores close together, so that the softmax's sum is as large as it gets;
    # it has nothing to do with the scale of V
    pr = ref.problem(new, past, 16, seed=D)
    shape = (pr.pages, 2, 16, D)
    cache, k64, v64 = _quantised_cache(_normal(shape, 1), _normal(shape, 2, gain=gain))
    assert int(cache.v_scale.min()) < 40
    _check_attn(_normal((sum(new), 6, D), 3, gain=0.05), cache, k64, v64, pr)
