"""GPU tests of dd_verify_draft where logits are unusual or decisions close,
against a plain 64-bit form (paged_ref.py): decisions and draws are equal,
target_prob is within the tolerance of test_verify_gpu.py."""
import math

import numpy as np
import pytest
import torch

import block_discrete_diffusion_dd_b200 as dd
import paged_ref as ref
from test_verify_gpu import DEV, _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -3e10, -1e12, -1e15, -1e20, -1e29, -3e38])
def test_verify_large_finite_masks(dtype, mask):
    # most of the vocabulary masked by a large finite value: whole chunks of it
    V = 50000
    c, tau, tau_d = _case((5, 3), V, dtype, 31, noise=0.3, tau=0.9, tau_d=0.9)
    keep = 7000
    for z in ("target_logits", "draft_logits"):
        c[z][:, keep:] = mask
    q = torch.softmax(c["draft_logits"].double() / tau_d, -1)
    tok = torch.multinomial(q, 1, generator=torch.Generator().manual_seed(4))
    c["draft_tokens"] = tok[:, 0].to(torch.int32)
    c["draft_conf"] = q.gather(1, tok)[:, 0].float()
    o = _check(c, tau, tau_d)
    assert o["accepted"].sum() > 0 and (o["tokens"] < keep).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verify_rows_of_extreme_logits(dtype):
    # rows of the type's lowest value (a mask that leaves nothing: uniform), or
    # of magnitudes whose scaled value is far beyond the fp32 exponents' reach
    low, V = torch.finfo(dtype).min, 3001
    for seed, fill in enumerate((low, -1e35, -4e30, 1e9, -2e9, 3e12, 1e38, 3e38)):
        c, tau, tau_d = _case((2, 1), V, dtype, 40 + seed, noise=0.3)
        c["target_logits"][:] = fill
        c["draft_logits"][:] = low
        c["draft_conf"][:] = 1 / V
        c["u_accept"] = torch.tensor([0.999, 0.5, 0.25])
        for r in range(5):  # a few lower entries
            c["target_logits"][r, r::7] = low if fill > 0 else 1.5 * fill if fill > -1e38 else fill
        c["draft_tokens"] = torch.tensor([1, 3, 10], dtype=torch.int32)
        for t in (0.25, 1.0, 2.0):
            _check(c, t, tau_d)


def _near_tie(tau, bar_u, bar_conf, off):
    """Three logits whose p(1) lies `off` (relative) above bar_u * bar_conf."""
    c = math.log2(math.e) / float(np.float32(tau))
    bar = math.log2(bar_u) + math.log2(bar_conf)
    x1 = np.float32((bar + 0.5) / c)
    Z = 2.0 ** (float(x1) * c - bar) / (1 + off)
    x2 = np.float32(math.log2(Z - 1) / c)
    z = torch.tensor([[0.0, x1, x2], [0.0, 0.0, 0.0]])
    p = 2.0 ** (float(x1) * c - bar) / (1 + 2.0 ** (float(x2) * c))  # over the bar
    return z, p - 1


# constants log2(e) / tau that fp32 holds worst (one too large, one too small), and 1.3
@pytest.mark.parametrize("tau", [1.4424631595611572, 1.4425914287567139, 1.3])
@pytest.mark.parametrize("off", [2e-6, -2e-6, 5e-7, -5e-7])
def test_verify_decides_tiny_probabilities_exactly(tau, off):
    # u conf at the smallest product of two fp32 numbers, p a hair from it
    u, conf = 2.0 ** -149, 2.0 ** -149
    z, got = _near_tie(tau, u, conf, off)
    assert off * got > 0 and abs(got) > 1e-7
    case = dict(target_logits=z, draft_logits=z[:1], draft_tokens=torch.tensor([1], dtype=torch.int32),
                draft_conf=torch.tensor([conf]), cu_draft=torch.tensor([0, 1], dtype=torch.int32),
                u_accept=torch.tensor([u]), u_sample=torch.tensor([0.5]))
    assert case["draft_conf"].item() == conf
    o = _run(case, float(np.float32(tau)), 1.0)
    assert o["accepted"].tolist() == [1 if off > 0 else 0]


def _standing(cu, most):
    """The rows that stand: possible by themselves and behind those before."""
    end, rows = 0, []
    for q0, q1 in zip(cu[:-1], cu[1:]):
        rows.append(end <= q0 <= q1 <= most)
        end = q1 if rows[-1] else end
    return rows


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("cu", [
    [0, 9, 5, 8],        # a row past the end: the last one stands all the same
    [0, 8, 3, 6],        # a row inside the first one
    [-4, 2, 5, 8],
    [0, 3, -7, 8],
    [0, BIG, -BIG - 1, 8],
    [2, 2, 4, 8, 1, 8],
    [8, 0, 8, 8],
    [2, 4, 4, 7],        # in order; packed rows of no sequence
])
@pytest.mark.parametrize("before,V", [(0, 700), (300, 50)])
def test_verify_offsets_out_of_order_leave_the_standing_rows(cu, before, V):
    cu = list(range(before)) + [before + x if abs(x) < 1000 else x for x in cu]
    T, B = before + 8, len(cu) - 1
    stands = _standing(cu, T)
    c, tau, tau_d = _case((T,) + (0,) * (B - 1), V, torch.float32, 51, noise=0.5)
    c["cu_draft"] = torch.tensor(cu, dtype=torch.int32)
    # each row that stands alone, as a batch of its own
    out = dict(accepted=torch.zeros(B, dtype=torch.int32),
               tokens=torch.full((T + B,), 77, dtype=torch.int32),
               target_prob=torch.full((T,), 77.0, dtype=torch.float64))
    for b in range(B):
        if stands[b]:
            d, t = slice(cu[b], cu[b + 1]), slice(cu[b] + b, cu[b + 1] + b + 1)
            out["accepted"][b:b + 1], out["tokens"][t], out["target_prob"][d] = ref.verify(
                c["target_logits"][t], c["draft_logits"][d], c["draft_tokens"][d],
                c["draft_conf"][d], [0, cu[b + 1] - cu[b]], c["u_accept"][d],
                c["u_sample"][b:b + 1], tau, tau_d)
    # states that an earlier call has left: every draft refused, then all accepted
    ws = dd.new_workspace(dd.verify_draft_workspace_bytes(B, T, V))
    dev = {k: v.to(DEV) for k, v in c.items()}
    for u in (1e30, 0.0):
        dd.verify_draft(**dict(dev, cu_draft=torch.tensor([0] + [T] * B, dtype=torch.int32, device=DEV),
                               u_accept=torch.full((T,), u, device=DEV)), workspace=ws)
        o = dd.verify_draft_outputs(B, T, DEV)
        for x in o.values():
            x.fill_(77)
        dd.verify_draft(**dev, outputs=o, workspace=ws)
        if all(stands):
            dd.query_device_error(ws)
        else:
            with pytest.raises(dd.DDError) as err:
                dd.query_device_error(ws)
            assert err.value.status == 6  # DD_ERR_DEVICE_BOUNDS
        assert torch.equal(o["accepted"].cpu(), out["accepted"])
        assert torch.equal(o["tokens"].cpu(), out["tokens"])
        mine = out["target_prob"] != 77
        got = o["target_prob"].cpu().double()
        assert ((got - out["target_prob"]).abs()[mine] <= 2e-6 * out["target_prob"][mine]).all()
        assert (got[~mine] == 77).all()
