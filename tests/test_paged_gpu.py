"""GPU tests of the paged cache (append, read back) and of the attention of
new tokens over it, against plain 64-bit forms (paged_ref.py).

Attention tolerance: the output is rounded to bf16 (off by at most 2^-8 of
its value), each probability is rounded to bf16 for the product with V (at
most 2^-8 of it), and a partial sum of a split row is held with 11 bits
against the row's largest value (2^-11).  So, with A = sum_j p_j |v_j|,
  |err| <= 2^-8 |O| + (2^-8 + 2^-12) A + 2^-11 max_d |O|,
where 2^-12 A covers the fp32 sums: exponents off by up to 2^-24 D sum|q k|
scale (about 1e-4 for unit normal inputs) and 2^-22 in 2^x.  The log-sum-exp
is fp32 throughout: |err| <= 1e-4 by the same sum."""
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import paged_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
BOUNDS = 6  # DD_ERR_DEVICE_BOUNDS


def _normal(shape, seed, gain=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def _pool(pr, H, D, kind, seed=1, gain=1.0):
    """A cache with every slot filled (on the device) and its float64 values."""
    k, v = (_normal((pr.pages, H, pr.ps, D), seed + i, gain) for i in range(2))
    if kind == "bf16":
        cache = dd.PagedCache(k.to(DEV), v.to(DEV))
    else:
        qs = [ref.quantise(x) for x in (k, v)]
        k8, v8 = (q[0].float().to(E4M3).to(DEV) for q in qs)
        ks, vs = ((q[1] + 127).to(torch.uint8).to(DEV) for q in qs)
        cache = dd.PagedCache(k8, v8, ks, vs)
    return cache, ref.values(cache.k, cache.k_scale), ref.values(cache.v, cache.v_scale)


def _batch(pr, max_new=None):
    return dd.PagedBatch(pr.page_table.to(DEV), pr.cu_new.to(DEV), pr.kv_len.to(DEV),
                         max(pr.new + [0]) if max_new is None else max_new)


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D,ps,new,past", [
    (8, 128, 16, (1, 1, 1), (0, 15, 16)),        # single tokens: first, last and first of a page
    (2, 64, 8, (37, 0, 5), (3, 9, 0)),           # a sequence without new tokens
    (1, 128, 64, (130,), (61,)),
    (3, 64, 512, (700, 1), (1, 511)),
])
def test_append_then_read(kind, H, D, ps, new, past):
    pr = ref.problem(new, past, ps, seed=ps + H)
    cache, _, _ = _pool(pr, H, D, kind, seed=3)
    before = [_bits(t) for t in (cache.k, cache.v)]
    T = sum(new)
    qkv = _normal((T, 3 * H, D), 7, gain=3.0)
    qkv[0, :, 0] = 448.0  # the largest code
    qkv[-1, H:] *= 2.0 ** -30
    qkv[T // 2, 2 * H] = 0.0
    dev = qkv.to(DEV)
    ws = dd.new_workspace(256)
    dd.cache_append(cache, _batch(pr), dev[:, H:2 * H], dev[:, 2 * H:], workspace=ws)
    dd.query_device_error(ws)
    touched = torch.zeros((pr.pages, H, ps), dtype=torch.bool)
    for which, (pool, scale, src) in enumerate(((cache.k, cache.k_scale, qkv[:, H:2 * H]),
                                                (cache.v, cache.v_scale, qkv[:, 2 * H:]))):
        want, e = ref.quantise(src) if kind == "e4m3" else (src.double(), None)
        t = 0
        for b, n in enumerate(new):
            for i in range(n):
                pos = past[b] + i
                page, slot = int(pr.page_table[b, pos // ps]), pos % ps
                touched[page, :, slot] = True
                assert torch.equal(pool[page, :, slot].float().double().cpu(), want[t])
                if e is not None:
                    assert torch.equal(scale[page, :, slot].cpu().double() - 127, e[t])
                t += 1
        after = _bits(pool).view(pr.pages, H, ps, -1)
        old = before[which].view(pr.pages, H, ps, -1)
        assert torch.equal(after[~touched], old[~touched])
    # reading back: the packed prefix, exact, rows outside it as they were
    lens = torch.tensor(pr.lens)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)
    total = int(cu[-1])
    kp, vp = (torch.full((total + 2, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    dd.cache_read(cache, pr.page_table.to(DEV), cu.to(DEV), k_out=kp, v_out=vp, workspace=ws)
    dd.query_device_error(ws)
    for out, pool, scale in ((kp, cache.k, cache.k_scale), (vp, cache.v, cache.v_scale)):
        v64 = ref.values(pool, scale)
        want = torch.cat([ref.sequence(v64, pr, b, n).transpose(0, 1)
                          for b, n in enumerate(pr.lens)])
        assert torch.equal(out[:total].double().cpu(), want)
        assert (out[total:] == 7).all()


def test_append_e4m3_extremes():
    # scales at both ends, halves between codes, infinities and NaN
    D, H, ps = 64, 1, 8
    rows = torch.zeros((8, H, D), dtype=torch.bfloat16)
    rows[0, 0, :4] = torch.tensor([3.3e38, -1e38, 1e30, float("inf")])
    rows[1, 0, :4] = torch.tensor([1e-38, -3e-39, 2.0 ** -133, 0.0])
    rows[2, 0, :3] = torch.tensor([float("nan"), float("-inf"), 5.0])
    rows[3, 0, :6] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11])
    rows[4, 0, :2] = torch.tensor([450.0, 449.0 / 256])
    rows[5, 0, :] = float("nan")
    rows[6, 0, 0] = -0.0
    rows[7, 0, 5] = -1.0
    pr = ref.problem((8,), (0,), ps)
    cache = dd.new_paged_cache(pr.pages, ps, H, D, E4M3)
    x = rows.to(DEV)
    ws = dd.new_workspace(256)
    dd.cache_append(cache, _batch(pr), x, x, workspace=ws)
    want, e = ref.quantise(rows)
    page = int(pr.page_table[0, 0])
    got = cache.k[page, 0].float().double().cpu()
    assert torch.equal(got.isnan(), want[:, 0].isnan())
    assert torch.equal(got.nan_to_num(0), want[:, 0].nan_to_num(0))
    assert torch.equal(cache.k_scale[page, 0].cpu().double() - 127, e[:, 0])
    assert torch.equal(_bits(cache.k), _bits(cache.v))
    kp, _ = dd.cache_read(cache, pr.page_table.to(DEV), torch.tensor([0, 8], dtype=torch.int32,
                                                                     device=DEV), total=8)
    back = want[:, 0] * 2.0 ** e
    assert torch.equal(kp[:, 0].double().cpu().nan_to_num(0), back.nan_to_num(0))


def test_cache_impossible_rows_and_pages_are_latched_and_skipped():
    H, D, ps = 2, 64, 8
    pr = ref.problem((4, 4, 4), (0, 6, 2), ps)
    cache = dd.new_paged_cache(pr.pages, ps, H, D)
    x = _normal((12, H, D), 5).to(DEV)
    ws = dd.new_workspace(256)
    table = pr.page_table.clone()
    table[1, 1] = pr.pages            # sequence 1's second page does not exist
    lens = pr.kv_len.clone()
    lens[2] = table.shape[1] * ps + 1  # longer than its table
    bad = dd.PagedBatch(table.to(DEV), pr.cu_new.to(DEV), lens.to(DEV), 4)
    dd.cache_append(cache, bad, x, x, workspace=ws)
    with pytest.raises(dd.DDError) as err:
        dd.query_device_error(ws)
    assert err.value.status == BOUNDS
    k = cache.k.cpu()
    assert torch.equal(k[table[0, 0], :, :4].transpose(0, 1), x[:4].cpu())
    assert torch.equal(k[table[1, 0], :, 6:8].transpose(0, 1), x[4:6].cpu())
    assert (k != 0).sum() == (x[:6] != 0).sum().item()
    # positions below zero are not stored (no error)
    lens[1], lens[2] = 2, 0
    some = dd.PagedBatch(pr.page_table.to(DEV), pr.cu_new.to(DEV), lens.to(DEV), 4)
    cache.k.zero_()
    dd.cache_append(cache, some, x, x, workspace=ws)
    dd.query_device_error(ws)
    k = cache.k.cpu()
    assert torch.equal(k[pr.page_table[1, 0], :, :2].transpose(0, 1), x[6:8].cpu())
    assert (k != 0).sum() == (x[[0, 1, 2, 3, 6, 7]] != 0).sum().item()
    # reading: rows of the missing page are left alone
    kp = torch.full((20, H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 4, 14, 14], dtype=torch.int32, device=DEV)
    dd.cache_read(cache, table.to(DEV), cu, k_out=kp, v_out=torch.empty_like(kp), workspace=ws)
    with pytest.raises(dd.DDError):
        dd.query_device_error(ws)
    assert (kp[12:] == 7).all() and (kp[:12] != 7).any()


def _check_attn(q, cache, k64, v64, pr, causal=True, scale=None, batch=None):
    D = q.shape[2]
    batch = _batch(pr) if batch is None else batch
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, q.shape[0], q.shape[1]))
    out, lse = dd.paged_attn(q.to(DEV), cache, batch, scale=scale, causal=causal, want_lse=True,
                             workspace=ws)
    dd.query_device_error(ws)
    scale = D ** -0.5 if scale is None else scale
    want, wlse, mag = ref.attention(q, k64, v64, pr, scale, causal)
    got = out.double().cpu()
    err = (got - want).abs()
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * mag +
           2.0 ** -11 * want.abs().amax(-1, keepdim=True))
    assert (err <= tol).all(), (err - tol).max()
    none = wlse.isinf()
    got_l = lse.double().cpu()
    assert torch.equal(got_l.isinf(), none)
    assert (got_l[none] < 0).all()
    assert (got_l[~none] - wlse[~none]).abs().max() <= 1e-4 if (~none).any() else True
    return out


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,ps,new,past,causal", [
    (2, 2, 128, 16, (1, 1, 1), (0, 127, 300), True),       # single tokens
    (1, 1, 64, 8, (1,), (5000,), True),                    # one row split over many keys
    (8, 2, 128, 64, (256,), (1000,), True),                # a block
    (2, 4, 128, 32, (70, 0, 1, 33), (100, 50, 0, 513), True),
    (2, 3, 64, 16, (129, 5), (0, 260), True),              # a prompt's first chunk; odd group
    (1, 8, 128, 128, (300,), (129,), False),               # every token sees every position
    (2, 7, 64, 256, (40, 3), (17, 900), False),
    (1, 16, 128, 512, (9,), (1023,), True),
])
def test_attention(kind, H, G, D, ps, new, past, causal):
    pr = ref.problem(new, past, ps, seed=H + G + D)
    cache, k64, v64 = _pool(pr, H, D, kind, seed=D + G)
    _check_attn(_normal((sum(new), H * G, D), 9), cache, k64, v64, pr, causal)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_sharp_and_wide_values(kind):
    # a softmax near one-hot, and V far from unit scale
    pr = ref.problem((64, 3), (400, 1000), 16)
    k, v = _normal((pr.pages, 2, 16, 128), 1), _normal((pr.pages, 2, 16, 128), 2, gain=1e6)
    if kind == "bf16":
        cache = dd.PagedCache(k.to(DEV), v.to(DEV))
    else:
        (k8, ke), (v8, ve) = ref.quantise(k), ref.quantise(v)
        cache = dd.PagedCache(k8.float().to(E4M3).to(DEV), v8.float().to(E4M3).to(DEV),
                              (ke + 127).to(torch.uint8).to(DEV), (ve + 127).to(torch.uint8).to(DEV))
    _check_attn(_normal((67, 4, 128), 3, gain=8.0), cache, ref.values(cache.k, cache.k_scale),
                ref.values(cache.v, cache.v_scale), pr)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_ignores_what_lies_past_the_length(kind, D):
    # NaN in every slot that no sequence owns, page ids past the length invalid
    pr = ref.problem((3, 1, 130), (10, 200, 77), 16)
    cache, k64, v64 = _pool(pr, 2, D, kind)
    owned = torch.zeros((pr.pages, 16), dtype=torch.bool)
    for b, n in enumerate(pr.lens):
        for pos in range(n):
            owned[pr.page_table[b, pos // 16], pos % 16] = True
    for pool in (cache.k, cache.v):
        if kind == "bf16":
            pool.masked_fill_(~owned[:, None, :, None].to(DEV), float("nan"))
        else:
            pool.view(torch.uint8).masked_fill_(~owned[:, None, :, None].to(DEV), 0x7f)
    if kind == "e4m3":
        for s in (cache.k_scale, cache.v_scale):
            s.masked_fill_(~owned[:, None].to(DEV), 255)
    _check_attn(_normal((134, 4, D), 4), cache, k64.nan_to_num(0), v64.nan_to_num(0), pr)
    _check_attn(_normal((134, 4, D), 5), cache, k64.nan_to_num(0), v64.nan_to_num(0), pr,
                causal=False)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_rows_that_see_nothing(causal):
    # lengths of zero, lengths below the new tokens, padded rows
    pr = ref.problem((5, 3, 200, 2), (-2, -3, -150, 4), 16)
    cache, k64, v64 = _pool(pr, 1, 128, "bf16")
    q = _normal((210, 2, 128), 6)
    out = _check_attn(q, cache, k64, v64, pr, causal)
    assert (out[5:8] == 0).all()
    # two more rows than the batch has: left as they were
    q2 = torch.cat([q, q[:2]]).to(DEV)
    o = torch.full((212, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((212, 2), 7.0, device=DEV)
    dd.paged_attn(q2, cache, _batch(pr), causal=causal, out=o, lse=lse)
    assert torch.equal(o[:210], out) and (o[210:] == 7).all() and (lse[210:] == 7).all()


def test_attention_takes_views_and_loose_bounds():
    # q inside a fused projection; max_new and the table wider than needed
    pr = ref.problem((6, 1), (30, 40), 8)
    cache, k64, v64 = _pool(pr, 2, 64, "bf16")
    fused = _normal((7, 8, 64), 8)
    table = torch.cat([pr.page_table, torch.full((2, 5), 2 ** 30, dtype=torch.int32)], 1)
    batch = dd.PagedBatch(table.to(DEV), pr.cu_new.to(DEV), pr.kv_len.to(DEV), 900)
    want = _check_attn(fused[:, 2:6], cache, k64, v64, pr)
    out, _ = dd.paged_attn(fused.to(DEV)[:, 2:6], cache, batch)
    assert (out.double() - want.double()).abs().max() <= 2.0 ** -6


def test_attention_latches_bad_pages_and_rows():
    pr = ref.problem((2, 3, 4), (100, 60, 20), 16)
    cache, k64, v64 = _pool(pr, 2, 128, "e4m3")
    q = _normal((9, 4, 128), 10)
    good = _check_attn(q, cache, k64, v64, pr)
    table, lens = pr.page_table.clone(), pr.kv_len.clone()
    table[0, 2] = -5
    lens[1] = -1
    batch = dd.PagedBatch(table.to(DEV), pr.cu_new.to(DEV), lens.to(DEV), 4)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, 9, 4))
    out, _ = dd.paged_attn(q.to(DEV), cache, batch, workspace=ws)
    with pytest.raises(dd.DDError) as err:
        dd.query_device_error(ws)
    assert err.value.status == BOUNDS
    assert torch.equal(out[5:], good[5:])


def test_attention_repeats_replays_and_follows_the_lengths():
    # one captured call serves other lengths; results do not depend on scheduling
    pr = ref.problem((1, 1, 1, 1), (900, 17, 400, 2000), 16)
    cache, k64, v64 = _pool(pr, 4, 128, "e4m3")
    q = _normal((4, 8, 128), 11).to(DEV)
    batch = _batch(pr)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, 4, 8))
    out = torch.empty_like(q)

    def call():
        dd.paged_attn(q, cache, batch, out=out, workspace=ws)

    call()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    batch.kv_len -= torch.tensor([1, 3, 300, 5], dtype=torch.int32, device=DEV)
    graph.replay()
    got = out.clone()
    pr.lens = batch.kv_len.cpu().tolist()
    want = _check_attn(q.cpu(), cache, k64, v64, pr, batch=batch)
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_wide_batch(kind):
    # more sequences than a CTA has threads, most of them short
    g = torch.Generator().manual_seed(1)
    new = torch.randint(0, 3, (900,), generator=g).tolist()
    past = torch.randint(0, 40, (900,), generator=g).tolist()
    pr = ref.problem(new, past, 8)
    cache, k64, v64 = _pool(pr, 1, 64, kind)
    _check_attn(_normal((sum(new), 2, 64), 12), cache, k64, v64, pr)


def test_paged_attention_equals_canvas_attention_on_the_packed_cache():
    # a canvas over a paged cache (causal = False) and dd_canvas_attn over the
    # same positions read back: the definitions agree within both tolerances
    pr = ref.problem((256,), (700,), 32)
    cache, k64, v64 = _pool(pr, 4, 128, "bf16")
    q = _normal((256, 8, 128), 13)
    out = _check_attn(q, cache, k64, v64, pr, causal=False)
    cu = torch.tensor([0, 956], dtype=torch.int32)
    kp, vp = dd.cache_read(cache, pr.page_table.to(DEV), cu.to(DEV), total=956)
    pre = torch.tensor([0, 700], dtype=torch.int32)
    o2, _ = dd.canvas_attn(q.to(DEV)[None], kp[None, 700:].contiguous(), vp[None, 700:].contiguous(),
                           kp[:700], vp[:700], pre.to(DEV), pre)
    diff = (o2[0].double() - out.double()).abs().max().item()
    assert diff <= 2.0 ** -6


def test_attention_wide_batch_with_long_chunks():
    # more sequences than the tensor-core kernel has threads, a few of them long
    g = torch.Generator().manual_seed(2)
    new = torch.randint(0, 2, (1000,), generator=g).tolist()
    past = torch.randint(0, 30, (1000,), generator=g).tolist()
    new[7], new[640], new[999] = 150, 20, 33
    pr = ref.problem(new, past, 8)
    cache, k64, v64 = _pool(pr, 1, 64, "bf16")
    _check_attn(_normal((sum(new), 2, 64), 14), cache, k64, v64, pr)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,new,past", [
    (2, 2, 128, (3, 2, 1, 0), (-1, -2, 0, 5)),  # few rows, some of which see nothing
    (1, 100, 64, (1, 3), (700, 5)),             # one kv head for a hundred query heads
    (1, 128, 128, (2,), (300,)),
    (2, 5, 128, (60, 1), (0, 2000)),            # one query tile, odd group
])
def test_attention_row_counts(kind, H, G, D, new, past):
    pr = ref.problem(new, past, 16, seed=G)
    cache, k64, v64 = _pool(pr, H, D, kind, seed=G)
    _check_attn(_normal((sum(new), H * G, D), 15), cache, k64, v64, pr)


def test_pool_beyond_32_bit_offsets():
    # pages whose first byte lies past 2^32: 8 heads of 64 x 128 bf16 take
    # 128 KB a page
    H, D, ps, pages = 8, 128, 64, 33000
    cache = dd.new_paged_cache(pages, ps, H, D)
    new, past = (70, 1), (0, 0)
    table = torch.tensor([[pages - 1, 32768], [32900, 0]], dtype=torch.int32)
    x = _normal((71, 3 * H, D), 16)
    dev = x.to(DEV)
    cu = torch.tensor([0, 70, 71], dtype=torch.int32)
    lens = torch.tensor([70, 1], dtype=torch.int32)
    batch = dd.PagedBatch(table.to(DEV), cu.to(DEV), lens.to(DEV), 70)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, 71, H))
    dd.cache_append(cache, batch, dev[:, H:2 * H], dev[:, 2 * H:], workspace=ws)
    out, lse = dd.paged_attn(dev[:, :H], cache, batch, want_lse=True, workspace=ws)
    kp, vp = dd.cache_read(cache, batch.page_table, batch.cu_new, total=71, workspace=ws)
    dd.query_device_error(ws)
    assert torch.equal(kp.cpu(), x[:, H:2 * H]) and torch.equal(vp.cpu(), x[:, 2 * H:])
    one, _ = dd.paged_attn(dev[70:, :H], cache, dd.PagedBatch(
        batch.page_table[1:], torch.tensor([0, 1], dtype=torch.int32, device=DEV),
        batch.kv_len[1:], 1))
    assert torch.equal(one[0].cpu(), x[70, 2 * H:])  # a single key: its value
    pr = ref.Problem(ps, torch.tensor([[1, 0], [2, 0]]), cu, lens, 3, list(new), [70, 1])
    pool = torch.zeros((2, 3, H, ps, D), dtype=torch.float64)
    for i in range(70):
        pool[:, 1 if i < 64 else 0, :, i % 64] = torch.stack([x[i, H:2 * H], x[i, 2 * H:]]).double()
    pool[:, 2, :, 0] = torch.stack([x[70, H:2 * H], x[70, 2 * H:]]).double()
    want, wlse, mag = ref.attention(x[:, :H], pool[0], pool[1], pr, D ** -0.5, True)
    err = (out.double().cpu() - want).abs()
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * mag +
           2.0 ** -11 * want.abs().amax(-1, keepdim=True))
    assert (err <= tol).all()
    assert (lse.double().cpu() - wlse).abs().max() <= 1e-4


def test_two_calls_at_once_on_their_own_streams():
    # long enough to overlap, one with few rows and one with many
    cases = []
    for new, past, kind in (((1,) * 8, (6000,) * 8, "e4m3"), ((200, 256), (4000, 3000), "bf16")):
        pr = ref.problem(new, past, 16, seed=len(new))
        H, D = 4, 128
        k, v = (torch.randn((pr.pages, H, 16, D), device=DEV).to(torch.bfloat16) for _ in range(2))
        cache = dd.PagedCache(k, v)
        if kind == "e4m3":
            s = torch.full((pr.pages, H, 16), 120, dtype=torch.uint8, device=DEV)
            cache = dd.PagedCache(k.to(E4M3), v.to(E4M3), s, s.clone())
        q = torch.randn((sum(new), 8, D), device=DEV).to(torch.bfloat16)
        batch = _batch(pr)
        ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, q.shape[0], 8))
        want, _ = dd.paged_attn(q, cache, batch, workspace=ws)
        cases.append((q, cache, batch, ws, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(5):
        for i, (q, cache, batch, ws, _) in enumerate(cases):
            outs[i].append(dd.paged_attn(q, cache, batch, workspace=ws, stream=streams[i])[0])
    torch.cuda.synchronize()
    for i, (_, _, _, ws, want) in enumerate(cases):
        dd.query_device_error(ws)
        assert all(torch.equal(o, want) for o in outs[i])


def test_captured_calls_that_share_a_workspace():
    # two graphs (few rows, many rows) replayed in turn on one workspace, with
    # calls of the other operators of the family between them
    pr1 = ref.problem((1,) * 5, (900, 40, 3000, 7, 128), 16, seed=1)
    pr2 = ref.problem((70, 130), (500, 1500), 16, seed=2)
    work = []
    for pr in (pr1, pr2):
        cache, _, _ = _pool(pr, 2, 64, "bf16")
        q = _normal((sum(pr.new), 4, 64), 17).to(DEV)
        work.append((q, cache, _batch(pr), torch.empty_like(q)))
    V = 1000
    logits = torch.randn((9, V), device=DEV)
    draft = [torch.randn((7, V), device=DEV), torch.zeros(7, dtype=torch.int32, device=DEV),
             torch.full((7,), 0.5, device=DEV),
             torch.tensor([0, 3, 7], dtype=torch.int32, device=DEV),
             torch.full((7,), 0.999, device=DEV), torch.tensor([0.2, 0.8], device=DEV)]
    n = max([dd.paged_attn_workspace_bytes(c, b, q.shape[0], 4) for q, c, b, _ in work] +
            [dd.verify_draft_workspace_bytes(2, 7, V)])
    ws = dd.new_workspace(n)
    graphs, want = [], []
    for q, cache, batch, out in work:
        dd.paged_attn(q, cache, batch, out=out, workspace=ws)
        want.append(out.clone())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                dd.paged_attn(q, cache, batch, out=out, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    first = None
    for _ in range(3):
        for i, graph in enumerate(graphs):
            work[i][3].zero_()
            graph.replay()
            assert torch.equal(work[i][3], want[i])
            o = dd.verify_draft(logits, *draft, workspace=ws)
            first = first or {k: t.clone() for k, t in o.items()}
            assert all(torch.equal(o[k], first[k]) for k in o)
    dd.query_device_error(ws)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [20, 200])
def test_timeout_is_reported_and_the_next_call_is_right(kind, new):
    # the tensor-core kernel stalls on a barrier that nothing completes, gives
    # up after 100 us and frees what it holds
    pr = ref.problem((new, 3), (700, 90), 16)
    cache, k64, v64 = _pool(pr, 2, 128, kind)
    q = _normal((new + 3, 4, 128), 18)
    batch = _batch(pr)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, new + 3, 4))
    dd.set_test_stall_ns(100_000)
    try:
        dd.paged_attn(q.to(DEV), cache, batch, workspace=ws)
        with pytest.raises(dd.DDError) as err:
            dd.query_device_error(ws)
    finally:
        dd.set_test_stall_ns(0)
    assert err.value.status == 5  # DD_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        _check_attn(q, cache, k64, v64, pr)


def test_outputs_belong_to_the_calls_stream():
    # memory freed on the current stream with work on it still pending is not
    # what a call on another stream gets for its outputs
    pr = ref.problem((3, 60), (100, 900), 16, seed=4)
    cache, _, _ = _pool(pr, 2, 64, "bf16")
    q, batch = _normal((63, 8, 64), 5).to(DEV), _batch(pr)
    ws = dd.new_workspace(dd.paged_attn_workspace_bytes(cache, batch, 63, 8))
    want, want_lse = dd.paged_attn(q, cache, batch, want_lse=True, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty_like(want), torch.empty_like(want_lse)]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in held:
        t.fill_(7)
    del held, t
    out, lse = dd.paged_attn(q, cache, batch, want_lse=True, workspace=ws, stream=side)
    torch.cuda.synchronize()
    dd.query_device_error(ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_batch_arrays_and_totals_may_change():
    pr = ref.problem((1, 4), (50, 200), 16, seed=6)
    cache, k64, v64 = _pool(pr, 2, 64, "bf16")
    q, batch = _normal((5, 4, 64), 7).to(DEV), _batch(pr)
    _check_attn(q.cpu(), cache, k64, v64, pr, batch=batch)
    # another tensor of lengths in place of the first, which is gone
    batch.kv_len = batch.kv_len - 3
    torch.full((2,), 1 << 28, dtype=torch.int32, device=DEV)
    pr.lens = batch.kv_len.cpu().tolist()
    _check_attn(q.cpu(), cache, k64, v64, pr, batch=batch)
    for name, bad in (("kv_len", batch.kv_len[:1]), ("cu_new", batch.cu_new.long()),
                      ("page_table", batch.page_table[0])):
        with pytest.raises(ValueError):
            setattr(batch, name, bad)
    # what one call was given does not change under it
    five, seven = batch._c(5), batch._c(7)
    assert (five.total_new, seven.total_new) == (5, 7)
    with pytest.raises(ValueError):
        dd.paged_attn(q.cpu(), cache, batch)
    with pytest.raises(AttributeError):
        cache.k = cache.v


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D,new,past", [
    (2, 128, (1, 1), (767, 1023)),           # the longest items that a CTA takes whole
    (2, 128, (1, 1), (768, 1024)),           # and one key more
    (1, 64, (1, 0, 2, 1), (1022, 4, 0, 3)),  # some sequences empty or without new tokens
    (37, 64, (1, 1, 0, 1), (20, 500, 9, 300)),   # as many items as there may be CTAs of one kind
    (60, 64, (1, 1, 3, 1, 1), (20, 500, 9, 300, 64)),  # more items than CTAs
])
def test_attention_items_taken_whole(kind, H, D, new, past):
    pr = ref.problem(new, past, 16, seed=H)
    cache, k64, v64 = _pool(pr, H, D, kind, seed=D)
    _check_attn(_normal((sum(new), 2 * H, D), 21), cache, k64, v64, pr)
