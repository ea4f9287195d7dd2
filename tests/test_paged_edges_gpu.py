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


def _led_by_zero_rows(pr, H, D, gain, lead, zeros, seed):
    """q, k, v where the positions `zeros` of every sequence have V = 0 and
    scores about `lead` nats above the others'."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randn((H, D), generator=g)
    k = (torch.randn((pr.pages, H, pr.ps, D), generator=g) * 0.3).to(torch.bfloat16)
    v = (torch.randn((pr.pages, H, pr.ps, D), generator=g) * gain).to(torch.bfloat16)
    along = (u * (lead * D ** 0.5 / (u * u).sum(-1, keepdim=True))).to(torch.bfloat16)
    for b, n in enumerate(pr.lens):
        for pos in zeros:
            if pos < n:
                page = int(pr.page_table[b, pos // pr.ps])
                k[page, :, pos % pr.ps] = along
                v[page, :, pos % pr.ps] = 0
    return u, k, v


@pytest.mark.parametrize("gain,lead", [
    (2.0 ** -6, 8.0), (2.0 ** -10, 4.0), (2.0 ** -10, 8.0), (2.0 ** -24, 8.0), (2.0 ** -40, 0.0),
])
@pytest.mark.parametrize("D,G,new,past,zeros", [
    (128, 2, (1, 1), (40, 300), (5,)),                  # items taken whole
    (64, 4, (1,), (6000,), (0, 3000, 5999)),            # a split row
    (128, 4, (3, 2), (100, 2500), (0, 17, 99, 1000)),   # more than eight rows per kv head
])
def test_attention_e4m3_zero_values_under_high_scores(gain, lead, D, G, new, past, zeros):
    # a row of V that is zero (stored with the scale 2^0) adds nothing to the
    # output, however much of the softmax it takes
    pr = ref.problem(new, past, 16, seed=D + G)
    u, k, v = _led_by_zero_rows(pr, 2, D, gain, lead, zeros, 5)
    cache, k64, v64 = _quantised_cache(k, v)
    q = u.repeat_interleave(G, 0)[None] + 0.05 * _normal((sum(new), 2 * G, D), 6, dtype=torch.float32)
    _check_attn(q.to(torch.bfloat16), cache, k64, v64, pr)


@pytest.mark.parametrize("new,past", [((1, 2), (70, 900)), ((5,), (3000,))])
def test_attention_e4m3_values_of_many_scales(new, past):
    # rows of V that are zero, or scaled by 2^-30 to 2^30, at random
    pr = ref.problem(new, past, 16, seed=9)
    g = torch.Generator().manual_seed(10)
    shape = (pr.pages, 2, 16, 128)
    v = torch.randn(shape, generator=g) * torch.exp2(60 * torch.rand(shape[:3], generator=g) - 30)[..., None]
    v[torch.rand(shape[:3], generator=g) < 0.2] = 0
    cache, k64, v64 = _quantised_cache(_normal(shape, 11), v.to(torch.bfloat16))
    _check_attn(_normal((sum(new), 6, 128), 12), cache, k64, v64, pr)
    # and nothing but zeros
    cache, k64, v64 = _quantised_cache(_normal(shape, 11), torch.zeros(shape, dtype=torch.bfloat16))
    out = _check_attn(_normal((sum(new), 6, 128), 12), cache, k64, v64, pr)
    assert (out == 0).all()
