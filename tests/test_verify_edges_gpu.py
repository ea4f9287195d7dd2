"""GPU tests of dd_verify_draft where logits are unusual or decisions close,
against a plain 64-bit form (paged_ref.py): decisions and draws are equal,
target_prob is within the tolerance of test_verify_gpu.py."""
import math

import numpy as np
import pytest
import torch

from test_verify_gpu import _case, _check, _run

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
