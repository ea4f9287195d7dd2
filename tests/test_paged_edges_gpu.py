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


def _standing(cu, most):
    """The rows that stand: possible by themselves and behind those before."""
    end, rows = 0, []
    for q0, q1 in zip(cu[:-1], cu[1:]):
        rows.append(end <= q0 <= q1 <= most)
        end = q1 if rows[-1] else end
    return rows


BIG = 2 ** 31 - 1
OFFSETS = [
    [0, 9, 5, 8],        # a row past the end: the last one stands all the same
    [0, 8, 3, 6],        # a row inside the first one
    [-4, 2, 5, 8],
    [0, 3, -7, 8],
    [0, BIG, -BIG - 1, 8],
    [3, -BIG - 1, 5, 8],
    [2, 2, 4, 8, 1, 8],
    [8, 0, 8, 8],
]
FITTING = [[0, 3, 3, 8], [2, 4, 4, 7]]   # in order; packed rows of no sequence


def _spoilt_batch(cu, unit, total, before=0, seed=3):
    """A batch over the offsets, in units of `unit` tokens, behind `before`
    rows of one token each: (problem of the rows that stand, cu, lens, batch)."""
    def scaled(x):
        return before + x * unit if abs(x) < 1000 else x

    cu = list(range(before)) + [scaled(x) for x in cu]
    total = before + total * unit
    stands = _standing(cu, total)
    new = [q1 - q0 if ok else 0 for q0, q1, ok in zip(cu[:-1], cu[1:], stands)]
    lens = [7 + 3 * (b % 5) + n for b, n in enumerate(new)]
    pr = ref.problem(new, [x - n for x, n in zip(lens, new)], 8, seed=seed)
    pr.cu_new = torch.tensor(cu, dtype=torch.int32)
    batch = dd.PagedBatch(pr.page_table.to(DEV), pr.cu_new.to(DEV), pr.kv_len.to(DEV), total)
    return pr, total, all(stands), batch


@pytest.mark.parametrize("unit,before", [(1, 0), (40, 0), (1, 290), (1, 1100)])
@pytest.mark.parametrize("cu", OFFSETS + FITTING)
def test_offsets_out_of_order_leave_the_standing_rows(cu, unit, before):
    # append and attention agree on which rows those are, and touch no other's
    H, D = 2, 64
    pr, total, fine, batch = _spoilt_batch(cu, unit, 8, before)
    cache, k64, v64 = _quantised_cache(*(_normal((pr.pages, H, 8, D), i) for i in (1, 2)))
    cache = dd.PagedCache(k64.to(torch.bfloat16).to(DEV), v64.to(torch.bfloat16).to(DEV))
    x = _normal((total, 2 * H, D), 4)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, total, 2 * H))
    dd.cache_append(cache, batch, x[:, :H].to(DEV), x[:, H:].to(DEV), workspace=ws)
    _latched(ws, not fine)
    for b, n in enumerate(pr.new):
        t0 = int(pr.cu_new[b])
        for i in range(n):
            pos = pr.lens[b] - n + i
            at = int(pr.page_table[b, pos // 8]), slice(None), pos % 8
            k64[at], v64[at] = x[t0 + i, :H].double(), x[t0 + i, H:].double()
    assert torch.equal(cache.k.cpu().double(), k64) and torch.equal(cache.v.cpu().double(), v64)
    q = _normal((total, 2 * H, D), 5)
    for causal in (True, False):
        out = torch.full((total, 2 * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
        dd.paged_attn(q.to(DEV), cache, batch, causal=causal, out=out, workspace=ws)
        _latched(ws, not fine)
        want, _, mag = ref.attention(q, k64, v64, pr, D ** -0.5, causal)
        mine = torch.zeros(total, dtype=torch.bool)
        for b, n in enumerate(pr.new):
            mine[int(pr.cu_new[b]):int(pr.cu_new[b]) + n] |= n > 0
        out = out.cpu().double()
        err = (out - want).abs()[mine]
        tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * mag +
               2.0 ** -11 * want.abs().amax(-1, keepdim=True))[mine]
        assert (err <= tol).all()
        assert (out[~mine] == 7).all()


def _latched(ws, expected):
    if not expected:
        return dd.query_device_error(ws)
    with pytest.raises(dd.DDError) as err:
        dd.query_device_error(ws)
    assert err.value.status == 6  # DD_ERR_DEVICE_BOUNDS
    dd.query_device_error(ws)     # cleared by the query


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("cu", OFFSETS + FITTING)
def test_prefixes_out_of_order_leave_the_standing_rows(cu, kind):
    H, D, ps, total = 2, 64, 8, 10
    stands = _standing(cu, BIG)
    lens = [min(q1 - q0, total - q0) if ok and q0 < total else 0
            for q0, q1, ok in zip(cu[:-1], cu[1:], stands)]
    pr = ref.problem([0] * len(lens), lens, ps, seed=7)
    k, v = (_normal((pr.pages, H, ps, D), i) for i in (1, 2))
    cache, k64, v64 = _quantised_cache(k, v)
    if kind == "bf16":
        cache, k64, v64 = dd.PagedCache(k.to(DEV), v.to(DEV)), k.double(), v.double()
    # (one page at least per row: what a search gone astray would look up)
    width = max(pr.page_table.shape[1], 2)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    table[:, :pr.page_table.shape[1]] = pr.page_table.clamp(min=0)
    kp, vp = (torch.full((total, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = dd.new_workspace(256)
    dd.cache_read(cache, table.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV),
                  k_out=kp, v_out=vp, workspace=ws)
    _latched(ws, not all(stands))
    for out, pool in ((kp, k64), (vp, v64)):
        want = torch.full((total, H, D), 7.0, dtype=torch.float64)
        for b, n in enumerate(lens):
            if n:
                want[cu[b]:cu[b] + n] = ref.sequence(pool, pr, b, n).transpose(0, 1)
        assert torch.equal(out.double().cpu(), want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,new", [(64, 30), (128, 30), (64, 90), (128, 90)])
def test_attention_many_items_of_few_key_tiles(kind, D, new):
    # items of one to six key tiles, several to a CTA and some split between two,
    # with one query tile and with two: every call gives the same result
    H, B = 8, 30
    g = torch.Generator().manual_seed(D + new)
    past = torch.randint(0, 640, (B,), generator=g).tolist()
    pr = ref.problem((new,) * B, past, 16, seed=2)
    k, v = (_normal((pr.pages, H, 16, D), i) for i in (1, 2))
    cache, k64, v64 = _quantised_cache(k, v)
    if kind == "bf16":
        cache, k64, v64 = dd.PagedCache(k.to(DEV), v.to(DEV)), k.double(), v.double()
    q = _normal((new * B, 2 * H, D), 3)
    # (a wide spread of scores: references move along the keys)
    first = _check_attn(q, cache, k64, v64, pr, scale=0.6)
    batch = dd.PagedBatch(pr.page_table.to(DEV), pr.cu_new.to(DEV), pr.kv_len.to(DEV), new)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, new * B, 2 * H))
    dev = q.to(DEV)
    for _ in range(20):
        out, _ = dd.paged_attn(dev, cache, batch, scale=0.6, workspace=ws)
        assert torch.equal(out, first)
    dd.query_device_error(ws)


def test_rows_above_a_bound_of_none_are_latched():
    # max_new = 0 with new tokens: impossible rows, for append and attention alike
    H, D = 2, 64
    pr = ref.problem((2, 0, 1), (9, 5, 30), 8)
    cache = dd.new_paged_cache(pr.pages, 8, H, D)
    x = _normal((3, 2 * H, D), 1).to(DEV)
    batch = dd.PagedBatch(pr.page_table.to(DEV), pr.cu_new.to(DEV), pr.kv_len.to(DEV), 0)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, 3, 2 * H))
    dd.cache_append(cache, batch, x[:, :H], x[:, H:], workspace=ws)
    _latched(ws, True)
    assert (cache.k == 0).all() and (cache.v == 0).all()
    out = torch.full((3, 2 * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((3, 2 * H), 7.0, device=DEV)
    dd.paged_attn(x, cache, batch, out=out, lse=lse, workspace=ws)
    _latched(ws, True)
    assert (out == 7).all() and (lse == 7).all()
    # no new tokens at all: nothing wrong with that bound
    none = dd.PagedBatch(batch.page_table, torch.zeros_like(batch.cu_new), batch.kv_len, 0)
    dd.paged_attn(x, cache, none, out=out, lse=lse, workspace=ws)
    _latched(ws, False)
    assert (out == 7).all() and (lse == 7).all()
