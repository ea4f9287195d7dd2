"""Refusals of the paged-cache, attention-over-cache and verification calls:
arguments are checked before any launch, so these need no GPU (the pointers
are never followed)."""
import ctypes

import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import paged_ref as ref
from block_discrete_diffusion_dd_b200 import build as libbuild

FAKE = 1 << 20
ODD = FAKE + 2
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return dd.load()


def _cache(pages=10, ps=16, H=8, D=128, dtype=dd.DD_BF16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return dd._PagedCacheC(pages, ps, H, D, dtype, k, v, ks, vs)


def _batch(B=2, pages=5, total=4, max_new=4, table=FAKE, cu=FAKE, lens=FAKE):
    return dd._PagedBatchC(B, pages, total, max_new, table, cu, lens)


def _append(lib, cache=None, batch=None, k=FAKE, ks=1024, v=FAKE, vs=1024, ws=FAKE, n=256):
    return lib.dd_cache_append(_cache() if cache is None else cache,
                               _batch() if batch is None else batch, k, ks, v, vs, ws, n, None)


def _attn(lib, cache=None, batch=None, hq=16, q=FAKE, qs=2048, scale=0.1, out=FAKE, ws=FAKE,
          n=1 << 40):
    return lib.dd_paged_attn(_cache() if cache is None else cache,
                             _batch() if batch is None else batch, hq, q, qs, scale, 1, out,
                             None, ws, n, None)


BAD_CACHES = [
    (_cache(pages=0), INVALID), (_cache(H=0), INVALID), (_cache(ps=0), INVALID),
    (_cache(ps=24), UNSUPPORTED), (_cache(ps=4), UNSUPPORTED), (_cache(ps=1024), UNSUPPORTED),
    (_cache(D=96), UNSUPPORTED), (_cache(dtype=7), INVALID), (_cache(dtype=dd.DD_F32), UNSUPPORTED),
    (_cache(k=None), INVALID), (_cache(v=ODD), INVALID), (_cache(pages=1 << 30), UNSUPPORTED),
    (_cache(dtype=dd.DD_E4M3, ks=None), INVALID), (_cache(dtype=dd.DD_E4M3, vs=ODD), INVALID),
]
BAD_BATCHES = [
    (_batch(B=-1), INVALID), (_batch(total=-1), INVALID), (_batch(max_new=-1), INVALID),
    (_batch(pages=0), INVALID), (_batch(pages=1 << 28), UNSUPPORTED), (_batch(table=None), INVALID),
    (_batch(cu=None), INVALID), (_batch(lens=None), INVALID),
]


@pytest.mark.parametrize("cache,code", BAD_CACHES)
def test_bad_caches(lib, cache, code):
    for call in (lambda: _append(lib, cache=cache), lambda: _attn(lib, cache=cache),
                 lambda: lib.dd_cache_read(cache, 2, 5, FAKE, FAKE, 4, FAKE, FAKE, FAKE, 256, None)):
        assert call() == code
        assert dd.last_error()


@pytest.mark.parametrize("batch,code", BAD_BATCHES)
def test_bad_batches(lib, batch, code):
    assert _append(lib, batch=batch) == code
    assert _attn(lib, batch=batch) == code
    assert dd.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(ks=1016), INVALID), (dict(vs=1028), INVALID), (dict(k=None), INVALID),
    (dict(v=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE),
    (dict(n=255), WORKSPACE),
    (dict(batch=_batch(total=1 << 28)), UNSUPPORTED),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code
    assert dd.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(hq=12), INVALID), (dict(hq=0), INVALID), (dict(hq=8 * 129, qs=8 * 129 * 128), UNSUPPORTED),
    (dict(qs=2040), INVALID), (dict(qs=2052), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(ws=None), WORKSPACE),
    (dict(n=0), WORKSPACE),
])
def test_attention_refusals(lib, kw, code):
    assert _attn(lib, **kw) == code
    assert dd.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(total=-1), INVALID), (dict(B=-1), INVALID), (dict(pages=0), INVALID),
    (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(out=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE),
])
def test_read_refusals(lib, kw, code):
    a = dict(B=2, pages=5, table=FAKE, cu=FAKE, total=4, out=FAKE, ws=FAKE, n=256)
    a.update(kw)
    st = lib.dd_cache_read(_cache(), a["B"], a["pages"], a["table"], a["cu"], a["total"], FAKE,
                           a["out"], a["ws"], a["n"], None)
    assert st == code
    assert dd.last_error()


def _verify(lib, tau=1.0, tau_d=1.0, dtype=0, B=2, T=4, V=100, z=FAKE, zs=100, d=FAKE, ds=100,
            tok=FAKE, cu=FAKE, u=FAKE, acc=FAKE, ws=FAKE, n=1 << 40):
    prm = dd.VerifyParams(tau, tau_d)
    return lib.dd_verify_draft(ctypes.byref(prm), dtype, B, T, V, z, zs, d, ds, tok, FAKE, cu,
                               FAKE, u, acc, FAKE, FAKE, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tau=0.0), INVALID), (dict(tau_d=float("inf")), INVALID), (dict(dtype=2), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(zs=99), INVALID),
    (dict(ds=99), INVALID), (dict(z=None), INVALID), (dict(z=ODD), INVALID), (dict(d=None), INVALID),
    (dict(tok=None), INVALID), (dict(cu=None), INVALID), (dict(u=None), INVALID),
    (dict(acc=None), INVALID), (dict(ws=None), WORKSPACE), (dict(n=256), WORKSPACE),
    (dict(B=1 << 30, V=1 << 20, zs=1 << 20, ds=1 << 20), UNSUPPORTED),
])
def test_verify_refusals(lib, kw, code):
    assert _verify(lib, **kw) == code
    assert dd.last_error()


def test_empty_calls_do_nothing(lib):
    none = _batch(B=0, total=0, table=None, cu=None, lens=None)
    assert _append(lib, batch=none, k=None, v=None, ws=None) == 0
    assert _append(lib, batch=_batch(total=0), k=None, v=None, ws=None) == 0
    assert _attn(lib, batch=none, q=None, out=None, ws=None) == 0
    assert _attn(lib, batch=_batch(total=0), q=None, out=None, ws=None) == 0
    assert lib.dd_cache_read(_cache(), 0, 5, None, None, 0, None, None, None, 0, None) == 0
    assert _verify(lib, B=0, T=0, z=None, d=None, tok=None, cu=None, u=None, acc=None, ws=None) == 0


def test_workspace_queries(lib):
    assert lib.dd_cache_workspace() == 256
    assert lib.dd_paged_attn_workspace(_cache(), _batch(), 16) >= 256
    assert lib.dd_paged_attn_workspace(_cache(D=96), _batch(), 16) == 0
    assert lib.dd_paged_attn_workspace(_cache(), _batch(B=-1), 16) == 0
    assert lib.dd_paged_attn_workspace(_cache(), _batch(), 12) == 0
    assert dd.verify_draft_workspace_bytes(2, 8, 1000) > 256
    assert dd.verify_draft_workspace_bytes(-1, 8, 1000) == 0
    assert dd.verify_draft_workspace_bytes(2, 8, 0) == 0


def test_python_checks():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dd.PagedCache(k, k)  # not on a GPU
    with pytest.raises(ValueError):
        dd.PagedBatch(torch.zeros((2, 3), dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                      torch.zeros(2, dtype=torch.int32), 1)
    x = torch.zeros((5, 3, 64), dtype=torch.bfloat16)
    cpu = torch.device("cpu")
    assert dd._packed(x, 3, 64, torch.bfloat16, cpu, "x") == 192
    assert dd._packed(x[:, :2], 2, 64, torch.bfloat16, cpu, "x") == 192
    assert dd._packed(x[:1, :2], 2, 64, torch.bfloat16, cpu, "x") == 128
    for bad in (x[:, :2], x.float(), x.transpose(1, 2), x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            dd._packed(bad, 3, 64, torch.bfloat16, cpu, "x")


def test_reference_quantiser_matches_torch():
    # the tests' reference, by code lookup, against torch's cast of the same scaled values
    x = torch.randn((50, 2, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    v, e = ref.quantise(x)
    y = x.float() * (2.0 ** -e.float())[..., None]
    assert torch.equal(y.to(torch.float8_e4m3fn).double(), v)
    assert (y.abs().amax(-1) <= 448).all() and (y.abs().amax(-1) > 224).all()


def test_sizes_that_indices_cannot_hold(lib):
    assert _verify(lib, V=(1 << 30) + 1, zs=1 << 31, ds=1 << 31) == UNSUPPORTED
    assert dd.verify_draft_workspace_bytes(1, 1, (1 << 30) + 1) == 0
    assert dd.verify_draft_workspace_bytes(1, 1, 1 << 30) > 0
    # 2 heads: one unit more than 2^30
    assert _append(lib, batch=_batch(total=(1 << 28) + 1)) == UNSUPPORTED
