"""Plain 64-bit forms of the paged-cache and verification operators, on the
CPU, written from their definitions with loops over sequences; and a builder
of small paged problems."""
from __future__ import annotations

import dataclasses
import math

import torch


def e4m3_values():
    """The non-negative finite E4M3 values (bias 7, three mantissa bits)."""
    vals = [m * 2.0 ** -9 for m in range(8)]
    vals += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(vals[:-1], dtype=torch.float64)  # the last code is NaN


def quantise(x: torch.Tensor):
    """bf16 [..., D] -> (E4M3 values in float64, exponent e): halves go to
    the code with the even mantissa, found by looking codes up."""
    x = x.double()
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    e = torch.zeros_like(a)
    for idx in (a > 0).nonzero():
        i = tuple(idx.tolist())
        m, ex = math.frexp(a[i].item())
        e[i] = min(120, max(-120, ex - 9 + (m > 0.875)))
    y = x * torch.pow(torch.tensor(2.0, dtype=torch.float64), -e)[..., None]
    codes = e4m3_values()
    mag = torch.where(y.isfinite(), y.abs(), 0.0)
    mag = torch.where(e[..., None] == 120, mag.clamp(max=240), mag)  # products stay finite in bf16
    hi = torch.searchsorted(codes, mag).clamp(max=codes.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag - codes[lo], codes[hi] - mag
    even_lo = lo % 2 == 0
    pick = torch.where((dl < dh) | ((dl == dh) & even_lo), lo, hi)
    out = torch.copysign(codes[pick], y)
    return torch.where(y.isfinite(), out, torch.nan), e


@dataclasses.dataclass
class Problem:
    ps: int
    page_table: torch.Tensor
    cu_new: torch.Tensor
    kv_len: torch.Tensor
    pages: int
    new: list
    lens: list


def problem(new, past, ps, seed=0, spare=3) -> Problem:
    """Pages in random order; entries past a sequence's length are -1."""
    g = torch.Generator().manual_seed(seed)
    lens = [p + n for p, n in zip(past, new)]
    need = [-(-max(x, 0) // ps) for x in lens]
    table = torch.full((len(new), max(need + [1])), -1, dtype=torch.int32)
    pool = torch.randperm(sum(need) + spare, generator=g).to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n]
        at += n
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32)
    return Problem(ps, table, cu, torch.tensor(lens, dtype=torch.int32), pool.numel(), list(new),
                   lens)


def values(k, scale):
    """A pool's values in float64."""
    k = k.cpu()
    if scale is None:
        return k.double()
    return k.float().double() * 2.0 ** (scale.cpu().double() - 127)[..., None]


def sequence(pool64, pr: Problem, b: int, n: int):
    """[heads, n, D]: the first n positions of sequence b."""
    pages = pr.page_table[b, :-(-n // pr.ps)].long()
    return pool64[pages].transpose(0, 1).flatten(1, 2)[:, :n]


def attention(q, k64, v64, pr: Problem, scale: float, causal: bool):
    """(out, lse, bound): bound[t, h, d] = sum_j p_j |v_jd|."""
    T, Hq, D = q.shape
    H = k64.shape[1]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    mag = torch.zeros((T, Hq, D), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(pr.new):
        L, t0 = pr.lens[b], int(pr.cu_new[b])
        if n == 0 or L <= 0:
            continue
        k, v = sequence(k64, pr, b, L), sequence(v64, pr, b, L)
        ends = (L - n + torch.arange(n) + 1).clamp(min=0) if causal else torch.full((n,), L)
        hidden = torch.arange(L)[None] >= ends[:, None]
        for h in range(Hq):
            s = q[t0:t0 + n, h].double() @ k[h // G].T * scale
            s = s.masked_fill(hidden, -math.inf)
            some = ends > 0
            p = torch.softmax(s[some], -1)
            out[t0:t0 + n, h][some] = p @ v[h // G]
            mag[t0:t0 + n, h][some] = p @ v[h // G].abs()
            lse[t0:t0 + n, h][some] = torch.logsumexp(s[some], -1)
    return out, lse, mag


def verify(target, draft, tok, conf, cu, u, us, tau, tau_d):
    """accepted, tokens, target_prob."""
    B, V = len(cu) - 1, target.shape[1]
    T = tok.numel()
    accepted, tokens = [], torch.full((T + B,), -1, dtype=torch.int32)
    prob = torch.zeros(T, dtype=torch.float64)

    def soft(z, t):
        return torch.softmax(z.double() / t, -1)

    for b in range(B):
        q0, k = int(cu[b]), int(cu[b + 1] - cu[b])
        p = [soft(target[q0 + b + i], tau) for i in range(k + 1)]
        n = k
        for i in reversed(range(k)):
            prob[q0 + i] = p[i][int(tok[q0 + i])]
            if float(u[q0 + i]) * float(conf[q0 + i]) >= prob[q0 + i]:
                n = i
        w = p[n]
        if n < k:
            r = (w - soft(draft[q0 + n], tau_d)).clamp(min=0)
            w = r if r.sum() > 0 else w
        cum = w.cumsum(0)
        past = (cum > float(us[b]) * cum[-1]).nonzero()
        nxt = int(past[0]) if len(past) else int((w > 0).nonzero()[-1])
        accepted.append(n)
        tokens[q0 + b:q0 + b + n] = tok[q0:q0 + n]
        tokens[q0 + b + n] = nxt
    return torch.tensor(accepted, dtype=torch.int32), tokens, prob
