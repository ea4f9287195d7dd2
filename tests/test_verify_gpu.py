"""GPU tests of dd_verify_draft against a plain 64-bit form (paged_ref.py).
Whole outputs are equal: decisions and draws are formed in 64 bits on both
sides.  target_prob is an fp32 rounding of a quotient whose sum is fp32 at
worst 2^-20 off (exponentials within 2^-22, arguments of up to 100 within
2^-24 of 1): relative error <= 2e-6."""
import numpy as np
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import paged_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _case(k, V, dtype, seed, noise=0.5, tau=1.0, tau_d=1.0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(k), len(k)
    target = torch.randn((T + B, V), generator=g) * std
    rows = [sum(k[:b]) + b + i for b in range(B) for i in range(k[b])]
    draft = (target[rows] + noise * torch.randn((T, V), generator=g)).to(dtype)
    target = target.to(dtype)
    q = torch.softmax(draft.double() / tau_d, -1)
    tok = torch.multinomial(q, 1, generator=g)[:, 0] if T else torch.zeros(0, dtype=torch.long)
    conf = q.gather(1, tok[:, None])[:, 0].float()
    cu = torch.tensor([0] + np.cumsum(k).tolist(), dtype=torch.int32)
    return dict(target_logits=target, draft_logits=draft, draft_tokens=tok.to(torch.int32),
                draft_conf=conf, cu_draft=cu, u_accept=torch.rand(T, generator=g),
                u_sample=torch.rand(B, generator=g)), tau, tau_d


def _run(c, tau, tau_d, outputs=None):
    B, T, V = c["u_sample"].numel(), c["draft_tokens"].numel(), c["target_logits"].shape[1]
    ws = dd.new_workspace(dd.verify_draft_workspace_bytes(B, T, V))
    o = dd.verify_draft(**{k: v if v.is_cuda else v.to(DEV) for k, v in c.items()},
                        temperature=tau, draft_temperature=tau_d, outputs=outputs, workspace=ws)
    dd.query_device_error(ws)
    return {k: v.cpu() for k, v in o.items()}


def _check(c, tau, tau_d):
    o = _run(c, tau, tau_d)
    acc, tok, prob = ref.verify(c["target_logits"], c["draft_logits"], c["draft_tokens"],
                                c["draft_conf"], c["cu_draft"], c["u_accept"], c["u_sample"],
                                tau, tau_d)
    assert torch.equal(o["accepted"], acc)
    assert torch.equal(o["tokens"], tok)
    if prob.numel():
        big = prob > 1e-30
        assert ((o["target_prob"].double() - prob).abs()[big] <= 2e-6 * prob[big]).all()
    return o


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k,V,noise,tau,tau_d", [
    ((4, 0, 7), 1000, 0.1, 1.0, 1.0),
    ((8,), 32001, 0.5, 0.8, 1.0),        # an odd vocabulary: rows off 16-byte boundaries
    ((1, 1, 1, 1, 1), 2, 1.0, 1.0, 1.0),
    ((3, 2), 1, 0.0, 1.0, 1.0),          # one entry: always accepted
    ((0, 0), 5000, 0.5, 1.0, 1.0),       # nothing drafted
    ((64, 33), 4097, 0.02, 0.4, 0.4),
    ((5, 6), 262144, 1.0, 1.0, 0.8),
])
def test_verify(dtype, k, V, noise, tau, tau_d):
    for seed in range(3):
        c, tau, tau_d = _case(k, V, dtype, 100 * V + seed, noise, tau, tau_d)
        _check(c, tau, tau_d)


def test_verify_strided_rows_and_flat_logits():
    # flat rows: as many equal borders as entries, and a near-tie at every one
    c, tau, tau_d = _case((6, 3), 30000, torch.float32, 5, noise=1e-3, std=1e-3)
    wide = torch.full((11, 30013), 50.0)
    wide[:, :30000] = c["target_logits"]
    wide_d = torch.full((9, 30007), 50.0)
    wide_d[:, :30000] = c["draft_logits"]
    want = _check(c, tau, tau_d)
    v = dict(c, target_logits=wide.to(DEV)[:, :30000], draft_logits=wide_d.to(DEV)[:, :30000])
    got = _run(v, tau, tau_d)
    assert all(torch.equal(got[x], want[x]) for x in got)


def test_verify_ties_and_certain_cases():
    V = 4
    z = torch.zeros((2, V))
    c = dict(target_logits=z, draft_logits=z[:1], draft_tokens=torch.tensor([1], dtype=torch.int32),
             draft_conf=torch.tensor([0.5]), cu_draft=torch.tensor([0, 1], dtype=torch.int32),
             u_accept=torch.tensor([0.5]), u_sample=torch.tensor([0.0]))
    o = _run(c, 1.0, 1.0)  # u conf = p exactly: refused; no residual: the target itself
    assert o["accepted"].tolist() == [0] and o["tokens"].tolist() == [0, -1]
    c["u_accept"] = torch.tensor([0.5 - 2.0 ** -25])
    c["u_sample"] = torch.tensor([0.75])  # the fourth quarter
    o = _run(c, 1.0, 1.0)
    assert o["accepted"].tolist() == [1] and o["tokens"].tolist() == [1, 3]
    assert o["target_prob"].tolist() == [0.25]


def test_verify_masked_vocabulary():
    # -inf logits have no mass; a target row of -inf only has no token at all
    c, tau, tau_d = _case((3, 2), 500, torch.bfloat16, 8, noise=2.0)
    c["target_logits"][:, 100:] = float("-inf")
    o = _check(c, tau, tau_d)
    assert (o["tokens"] < 100).all()
    c["target_logits"][0] = float("-inf")
    o = _run(c, tau, tau_d)
    assert o["accepted"][0] == 0 and o["tokens"][0] == -1 and o["target_prob"][0] == 0


def test_verify_impossible_rows_and_padding():
    c, tau, tau_d = _case((3, 2, 4), 300, torch.float32, 9)
    want = _run(c, tau, tau_d)
    # rows behind the last sequence: left as they were
    pad = dict(c, **{k: torch.cat([c[k], c[k][:2]]) for k in
                     ("draft_logits", "draft_tokens", "draft_conf", "u_accept", "target_logits")})
    o = dd.verify_draft_outputs(3, 11, DEV)
    for t in o.values():
        t.fill_(77)
    got = _run(pad, tau, tau_d, outputs=o)
    assert torch.equal(got["tokens"][:12], want["tokens"]) and (got["tokens"][12:] == 77).all()
    assert (got["target_prob"][9:] == 77).all()
    # a token outside the vocabulary is refused, a bad row skipped; both latched
    bad = {k: v.to(DEV) for k, v in c.items()}
    bad["draft_tokens"][3] = 300
    bad["cu_draft"][3] = 10
    ws = dd.new_workspace(dd.verify_draft_workspace_bytes(3, 9, 300))
    o = dd.verify_draft(**bad, workspace=ws)
    with pytest.raises(dd.DDError) as e:
        dd.query_device_error(ws)
    assert e.value.status == 6
    assert o["accepted"].tolist()[1:] == [0, 0]
    assert torch.equal(o["tokens"][:4].cpu(), want["tokens"][:4])


def test_verify_replays():
    c, tau, tau_d = _case((9, 4), 50000, torch.bfloat16, 10)
    dev = {k: v.to(DEV) for k, v in c.items()}
    ws = dd.new_workspace(dd.verify_draft_workspace_bytes(2, 13, 50000))
    o = dd.verify_draft_outputs(2, 13)
    dd.verify_draft(**dev, outputs=o, workspace=ws)
    want = {k: v.clone() for k, v in o.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            dd.verify_draft(**dev, outputs=o, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in o.values():
            t.fill_(-5)
        graph.replay()
        assert all(torch.equal(o[k], want[k]) for k in o)


def test_verify_follows_the_target_distribution():
    # speculative sampling leaves the target's law whatever the draft's: over
    # 4000 sequences of one drafted token, the first emitted token's counts
    # lie within 5 standard deviations of the target's probabilities
    B, V = 4000, 8
    g = torch.Generator().manual_seed(3)
    zt, zd = torch.randn(V, generator=g), torch.randn(V, generator=g)
    q = torch.softmax(zd.double(), 0)
    tok = torch.multinomial(q, B, replacement=True, generator=g)
    c = dict(target_logits=zt.repeat(2 * B, 1), draft_logits=zd.repeat(B, 1),
             draft_tokens=tok.to(torch.int32), draft_conf=q[tok].float(),
             cu_draft=torch.arange(B + 1, dtype=torch.int32),
             u_accept=torch.rand(B, generator=g), u_sample=torch.rand(B, generator=g))
    o = _run(c, 1.0, 1.0)
    p = torch.softmax(zt.double(), 0)
    n = torch.bincount(o["tokens"][0::2].long(), minlength=V).double()
    assert ((n - B * p).abs() <= 5 * (B * p * (1 - p)).sqrt()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_decides_near_ties_in_64_bits(dtype):
    # u conf within a few fp32 steps of p on either side, row after row: far
    # closer than the fp32 sums of the scan can tell
    k, V = (40, 40), 5000
    c, tau, tau_d = _case(k, V, dtype, 21, noise=0.3)
    p = torch.cat([torch.softmax(c["target_logits"][b * 41:b * 41 + 40].double(), -1)
                   for b in range(2)])
    p = p.gather(1, c["draft_tokens"][:, None].long())[:, 0]
    c["draft_conf"] = (p * 2).float()
    u = (p / c["draft_conf"].double()).float()
    steps = torch.arange(80) % 5 - 4  # -4 .. 0 steps of u: the last ones around the border
    bits = u.view(torch.int32) + steps.to(torch.int32)
    c["u_accept"] = bits.view(torch.float32)
    _check(c, tau, tau_d)


def test_verify_on_another_stream():
    c, tau, tau_d = _case((5, 9), 20000, torch.bfloat16, 22)
    want = _run(c, tau, tau_d)
    dev = {k: v.to(DEV) for k, v in c.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = dd.verify_draft(**dev, temperature=tau, draft_temperature=tau_d, stream=side)
    side.synchronize()
    assert all(torch.equal(o[x].cpu(), want[x]) for x in want)


@pytest.mark.parametrize("k,V", [
    ((9,), 262144), ((2, 3, 0), 99001),                   # few chunks of the drawn rows
    ((1, 2, 0, 3, 2), 65537), ((1,) * 75, 4099),          # many
])
def test_verify_draws_over_few_and_many_chunks(k, V):
    for seed in range(2):
        c, tau, tau_d = _case(k, V, torch.bfloat16, 7 * V + seed, 0.7, 1.0, 0.9)
        _check(c, tau, tau_d)
