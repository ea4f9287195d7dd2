"""The operators of a block's commit together, as a server uses them: the
prompts are appended to a paged cache, a block is drafted by the sampler, its
keys and values are appended, its tokens encoded causally over the cache, the
drafted tokens verified, the cache cut back to what was accepted, and read
back as the packed prefix of the next canvas.  Everything is enqueued on one
stream before the first value is looked at."""
import numpy as np
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import oracle
import paged_ref as ref
from parity import check_attn

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_commit_a_block(kind):
    B, H, Hq, D, ps, C, V = 2, 2, 4, 128, 16, 24, 3000
    lens = (37, 200)
    g = torch.Generator().manual_seed(5)

    def r(*shape):
        return torch.randn(shape, generator=g)

    def i32(xs):
        return torch.tensor(xs, dtype=torch.int32)

    need = [-(-(n + C + 1) // ps) for n in lens]
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    pages = torch.randperm(sum(need), generator=g).to(torch.int32)
    table[0, :need[0]], table[1, :need[1]] = pages[:need[0]], pages[need[0]:]
    prompt = r(sum(lens), 2 * H, D).to(torch.bfloat16)
    block = r(B * C, Hq + 2 * H, D).to(torch.bfloat16)  # q, k and v of the drafted tokens
    target = r(B * (C + 1), V) * 3
    rows = [b * (C + 1) + i for b in range(B) for i in range(C)]
    draft = (target[rows] + 0.2 * r(B * C, V)).to(torch.bfloat16)
    target = target.to(torch.bfloat16)
    u, us = torch.rand(B * C, generator=g), torch.rand(B, generator=g)

    cache = dd.new_paged_cache(sum(need), ps, H, D,
                               torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    cu_c = i32([0, C, 2 * C]).to(DEV)
    d = {k: v.to(DEV) for k, v in dict(table=table, prompt=prompt, block=block, target=target,
                                       draft=draft, u=u, us=us).items()}
    ws = dd.new_workspace(1 << 24)
    first = dd.PagedBatch(d["table"], i32(np.concatenate([[0], np.cumsum(lens)])).to(DEV),
                          i32(lens).to(DEV), max(lens))
    dd.cache_append(cache, first, d["prompt"][:, :H], d["prompt"][:, H:], workspace=ws)
    s = dd.sample_renoise(d["draft"], 1.0, 0.0, seed=3, step=0)
    more = dd.PagedBatch(d["table"], cu_c, first.kv_len + C, C)
    dd.cache_append(cache, more, d["block"][:, Hq:Hq + H], d["block"][:, Hq + H:], workspace=ws)
    out, lse = dd.paged_attn(d["block"][:, :Hq], cache, more, want_lse=True, workspace=ws)
    o = dd.verify_draft(d["target"], d["draft"], s["pred"], s["conf"], cu_c, d["u"], d["us"],
                        workspace=ws)
    kept = first.kv_len + o["accepted"]  # what the rejected drafts wrote is behind the length
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = kept.cumsum(0)
    kp, vp = dd.cache_read(cache, d["table"], cu, total=sum(lens) + B * C, workspace=ws)
    dd.query_device_error(ws)

    # the drafts and their verification
    acc, tok, prob = ref.verify(target, draft, s["pred"].cpu(), s["conf"].cpu(), cu_c.cpu(), u, us,
                                1.0, 1.0)
    assert torch.equal(o["accepted"].cpu(), acc) and torch.equal(o["tokens"].cpu(), tok)
    assert 0 < int(acc.sum()) < B * C
    # the cache's contents, and the block's attention over them
    k64, v64 = ref.values(cache.k, cache.k_scale), ref.values(cache.v, cache.v_scale)
    pr = ref.Problem(ps, table, cu_c.cpu(), more.kv_len.cpu(), sum(need), [C] * B,
                     [n + C for n in lens])
    at = np.concatenate([[0], np.cumsum(lens)])
    for b in range(B):
        want = torch.cat([prompt[at[b]:at[b + 1]], block[b * C:(b + 1) * C, Hq:]])
        for pool, half in ((k64, want[:, :H]), (v64, want[:, H:])):
            x = half.double()
            if kind == "e4m3":
                q, e = ref.quantise(half)
                x = q * 2.0 ** e[..., None]
            assert torch.equal(ref.sequence(pool, pr, b, lens[b] + C).transpose(0, 1), x)
    want, wlse, mag = ref.attention(block[:, :Hq], k64, v64, pr, D ** -0.5, True)
    err = (out.double().cpu() - want).abs()
    tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * mag +
           2.0 ** -11 * want.abs().amax(-1, keepdim=True))
    assert (err <= tol).all()
    assert (lse.double().cpu() - wlse).abs().max() <= 1e-4
    # the packed prefix, and the next canvas over it
    n = [lens[b] + int(acc[b]) for b in range(B)]
    assert cu.tolist() == [0, n[0], n[0] + n[1]]
    for out_p, pool in ((kp, k64), (vp, v64)):
        whole = torch.cat([ref.sequence(pool, pr, b, n[b]).transpose(0, 1) for b in range(B)])
        assert torch.equal(out_p[:sum(n)].double().cpu(), whole)
    q, kc, vc = (r(B, C, h, D).to(torch.bfloat16) for h in (Hq, H, H))
    canvas, _ = dd.canvas_attn(q.to(DEV), kc.to(DEV), vc.to(DEV), kp[:sum(n)], vp[:sum(n)], cu,
                               cu.cpu())
    want, _ = oracle.canvas_attn(q, kc, vc, kp[:sum(n)].cpu(), vp[:sum(n)].cpu(), cu.cpu().numpy(),
                                 D ** -0.5)
    check_attn(canvas, want, torch.bfloat16)
