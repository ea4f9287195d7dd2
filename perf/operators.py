"""What the serving operators around a block compute and how much of it there
is: appending new keys and values to a paged cache (as bf16, or as E4M3 with
a power-of-two scale per token and head), reading a paged cache back as the
packed prefix, attention of a chunk of new tokens over the paged cache, and
verification of drafted tokens against the target's probabilities.

`run` computes each operator in plain torch operations, or, where `own` is
true, through the package's entry points.  `exact` computes it again from the
definition in 64 bits.  Lengths follow from the case alone; contents follow
from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 32 sequences: a decoding step's cache write
        dict(name="append_token_b32_e4m3", op="append", batch=32, new_lo=1, new_hi=1, past_lo=512,
             past_hi=4096, heads_kv=8, head_dim=128, page=16, kind="e4m3", lens=1),
        # the prompts of 8 sequences written at once
        dict(name="append_prompt_b8_e4m3", op="append", batch=8, new_lo=512, new_hi=16384,
             past_lo=0, past_hi=0, heads_kv=8, head_dim=128, page=64, kind="e4m3", lens=2),
        # one sequence's cache laid out as the packed prefix of a canvas
        dict(name="read_b1_L4096_e4m3", op="read", batch=1, past_lo=4096, past_hi=4096, heads_kv=8,
             head_dim=128, page=16, kind="e4m3", lens=3),
        # the ragged prefixes of 8 canvases
        dict(name="read_ragged_b8_bf16", op="read", batch=8, past_lo=512, past_hi=16384, heads_kv=8,
             head_dim=128, page=32, kind="bf16", lens=4),
        # the smallest decoding step: latency counts
        dict(name="attn_token_b2_d64", op="attn", batch=2, new_lo=1, new_hi=1, past_lo=130,
             past_hi=700, heads_q=8, heads_kv=2, head_dim=64, page=16, kind="bf16", causal=True,
             lens=5),
        # one sequence with a long past: its single query row has to be split over the keys
        dict(name="attn_token_b1_L65536", op="attn", batch=1, new_lo=1, new_hi=1, past_lo=65535,
             past_hi=65535, heads_q=16, heads_kv=8, head_dim=128, page=32, kind="bf16",
             causal=True, lens=6),
        # a decoding step of a full server, over an 8-bit cache
        dict(name="attn_token_b64_e4m3", op="attn", batch=64, new_lo=1, new_hi=1, past_lo=512,
             past_hi=16384, heads_q=16, heads_kv=8, head_dim=128, page=16, kind="e4m3",
             causal=True, lens=7),
        # a finished block of 256 tokens encoded causally into its sequence
        dict(name="attn_block_b1_L4096", op="attn", batch=1, new_lo=256, new_hi=256, past_lo=4096,
             past_hi=4096, heads_q=16, heads_kv=8, head_dim=128, page=64, kind="bf16",
             causal=True, lens=8),
        # the blocks of 8 sequences over ragged 8-bit caches
        dict(name="attn_block_ragged_b8_e4m3", op="attn", batch=8, new_lo=200, new_hi=256,
             past_lo=512, past_hi=16384, heads_q=16, heads_kv=8, head_dim=128, page=16,
             kind="e4m3", causal=True, lens=9),
        # a chunk of two long prompts
        dict(name="attn_prompt_b2", op="attn", batch=2, new_lo=1500, new_hi=2048, past_lo=6000,
             past_hi=8192, heads_q=16, heads_kv=8, head_dim=128, page=128, kind="bf16",
             causal=True, lens=10),
        # eight drafted tokens of one sequence
        dict(name="verify_b1_k8", op="verify", batch=1, draft_lo=8, draft_hi=8, vocab=262144,
             kind="bf16", tau=1.0, draft_tau=1.0, noise=0.5, lens=11),
        # drafts of up to 64 tokens for each of 8 sequences
        dict(name="verify_b8_k64", op="verify", batch=8, draft_lo=33, draft_hi=64, vocab=262144,
             kind="bf16", tau=0.8, draft_tau=0.8, noise=0.05, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "verify"])
    while True:
        case = dict(op=op, lens=rng.randrange(1 << 20))
        if op == "verify":
            k = _log_int(rng, 1, 64)
            case.update(batch=_log_int(rng, 1, 16), draft_lo=max(1, k // 2), draft_hi=k,
                        vocab=_log_int(rng, 1000, 262144), kind=rng.choice(["bf16", "f32"]),
                        tau=rng.choice([0.4, 0.8, 1.0]), draft_tau=rng.choice([0.8, 1.0]),
                        noise=rng.choice([0.05, 0.5, 2.0]))
            most = {"bytes": 2.0e8}
        else:
            past = _log_int(rng, 1, 65536)
            case.update(batch=_log_int(rng, 1, 64), past_lo=past // 4, past_hi=past,
                        heads_kv=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([64, 128]),
                        page=rng.choice([8, 16, 32, 64, 128]), kind=rng.choice(["bf16", "e4m3"]))
            most = {"bytes": 3.0e8}
            if op != "read":
                new = 1 if op == "attn" and rng.random() < 0.4 else _log_int(rng, 1, 2048)
                case.update(new_lo=max(1, new // 2), new_hi=new)
            if op == "attn":
                case.update(heads_q=case["heads_kv"] * rng.choice([1, 2, 3, 4, 8]),
                            causal=rng.random() < 0.7)
                most = {"bytes": 1.0e9, "flops": 2.0e11}
        w = work(case)
        pool = 0 if op == "verify" else sum(_past(case)) * case["heads_kv"] * case["head_dim"]
        if all(w[x] <= most[x] for x in most) and pool <= 6e8:
            return case


def _ints(case, what, lo, hi):
    rng = random.Random("%s/%d" % (what, case["lens"]))
    return [rng.randint(lo, hi) for _ in range(case["batch"])]


def _past(case):
    return _ints(case, "past", case["past_lo"], case["past_hi"])


def _new(case):
    return _ints(case, "new", case["new_lo"], case["new_hi"]) if "new_lo" in case else \
        [0] * case["batch"]


def _drafts(case):
    return _ints(case, "draft", case["draft_lo"], case["draft_hi"])


def work(case):
    if case["op"] == "verify":
        # the target's rows and one draft row per sequence; a maximum, an exponential and a sum each
        k = _drafts(case)
        rows = sum(k) + 2 * case["batch"]
        es = 2 if case["kind"] == "bf16" else 4
        return {"bytes": rows * case["vocab"] * es + 16 * rows, "flops": 3 * rows * case["vocab"]}
    past, new = _past(case), _new(case)
    H, D = case["heads_kv"], case["head_dim"]
    row = 2 * H * D * 2                                        # a bf16 token, keys and values
    held = row if case["kind"] == "bf16" else 2 * H * (D + 1)  # as the cache holds it
    if case["op"] == "append":
        return {"bytes": sum(new) * (row + held), "flops": 4 * sum(new) * H * D}
    if case["op"] == "read":
        return {"bytes": sum(past) * (row + held), "flops": 2 * sum(past) * H * D}
    Hq = case["heads_q"]
    seen = sum(n * p + (n * (n + 1) // 2 if case["causal"] else n * n) for p, n in zip(past, new))
    return {"bytes": sum(p + n for p, n in zip(past, new)) * held + sum(new) * Hq * (4 * D + 4),
            "flops": 4 * Hq * D * seen}


# ------------------------------------------------------------------ inputs
def _i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


def _cum(xs):
    return _i32([0] + torch.tensor(xs).cumsum(0).tolist())


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + case["lens"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    st = dict(case)
    st["rows"] = st.pop("batch")
    if case["op"] == "verify":
        # logits as the sampler's workloads have them (a spike over normal ones); the draft's
        # are the target's with an error, so that most drafted tokens are accepted
        k, B, V = _drafts(case), case["batch"], case["vocab"]
        T = sum(k)
        dt = torch.bfloat16 if case["kind"] == "bf16" else torch.float32
        target = normal(T + B, V).mul_(3)
        target[torch.arange(T + B, device=DEV),
               torch.randint(0, V, (T + B,), generator=g, device=DEV)] += 8
        of_draft = [r for r in range(T + B)]
        for end in reversed([sum(k[:b + 1]) + b for b in range(B)]):
            del of_draft[end]
        draft = (target[torch.tensor(of_draft, dtype=torch.long, device=DEV)] +
                 normal(T, V).mul_(case["noise"])).to(dt)
        target = target.to(dt)
        z = draft.float() / case["draft_tau"]
        e = torch.empty_like(z).exponential_(generator=g)
        tok = (z - e.log_()).argmax(-1) if T else torch.zeros(0, dtype=torch.long, device=DEV)
        del e
        conf = (z.gather(1, tok[:, None])[:, 0] - torch.logsumexp(z, 1)).exp()
        st.update(target=target, draft=draft, draft_tokens=tok.to(torch.int32),
                  draft_conf=conf.float(), cu_draft=_cum(k),
                  u_accept=torch.rand(T, generator=g, device=DEV),
                  u_sample=torch.rand(B, generator=g, device=DEV))
        if own:
            import block_discrete_diffusion_dd_b200 as dd
            st["ws"] = dd.new_workspace(dd.verify_draft_workspace_bytes(B, T, V))
            st["outputs"] = dd.verify_draft_outputs(B, T, DEV)
        return st

    past, new = _past(case), _new(case)
    B, H, D, ps = case["batch"], case["heads_kv"], case["head_dim"], case["page"]
    # pages of a pool in no order, as a server that has run for a while hands them out
    need = [-(-(p + n) // ps) for p, n in zip(past, new)]
    width = max(need + [1])
    pool = torch.randperm(sum(need) + 3, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, :need[b]] = pool[at:at + need[b]]
        at += need[b]
    pages = pool.numel()
    # tokens of different size: each has a scale of its own
    k, v = (torch.randn((pages, H, ps, D), generator=g, device=DEV, dtype=torch.bfloat16) *
            normal(pages, 1, ps, 1).mul_(0.5).exp_().to(torch.bfloat16) for _ in range(2))
    st.update(table=table, cu_new=_cum(new), kv_len=_i32([p + n for p, n in zip(past, new)]),
              cu_past=_cum(past), max_new=max(new + [0]), longest=max(p + n for p, n in zip(past, new)),
              total=sum(new), total_past=sum(past), k_scale=None, v_scale=None)
    if case["kind"] == "e4m3":
        k, st["k_scale"] = _quantised(k)
        v, st["v_scale"] = _quantised(v)
    st.update(k=k, v=v)
    T = sum(new)
    if case["op"] == "append":
        # views of a fused projection's output, as a model's layer has them
        qkv = normal(T, 4 * H, D).to(torch.bfloat16)
        st.update(k_new=qkv[:, 2 * H:3 * H], v_new=qkv[:, 3 * H:])
    if case["op"] == "attn":
        st["q"] = normal(T, case["heads_q"], D).to(torch.bfloat16)
    if own:
        import block_discrete_diffusion_dd_b200 as dd
        st["cache"] = dd.PagedCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        st["batch"] = dd.PagedBatch(table, st["cu_new"], st["kv_len"], st["max_new"])
        nbytes = 256
        if case["op"] == "attn":
            nbytes = dd.paged_attn_workspace_bytes(st["cache"], st["batch"], T, case["heads_q"])
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty((T, case["heads_q"]), dtype=torch.float32, device=DEV)
        if case["op"] == "read":
            st["k_out"], st["v_out"] = (torch.empty((sum(past), H, D), dtype=torch.bfloat16,
                                                    device=DEV) for _ in range(2))
        st["ws"] = dd.new_workspace(nbytes)
    return st


# ------------------------------------------------------------- plain forms
def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _quantised(x):
    """bf16 [..., D] -> E4M3 codes and the scale's exponent byte: the smallest
    power of two 2^e with max|x| <= 448 2^e, kept as e + 127 (e = 0 for zeros)."""
    x = x.float()
    m, ex = torch.frexp(torch.where(x.isfinite(), x.abs(), 0.0).amax(-1))  # max = m 2^ex
    e = torch.where(m > 0, ex - 9 + (m > 0.875).int(), 0).clamp(-120, 120)
    y = x * _pow2(-e)[..., None]
    return (torch.where(y.isfinite(), y, torch.nan).to(torch.float8_e4m3fn),
            (e + 127).to(torch.uint8))


def _held(x, scale):
    """What the cache holds, in 32 bits."""
    return x.float() if scale is None else x.float() * _pow2(scale.int() - 127)[..., None]


def _rows(cu, total):
    """Batch row and place in it of each of the packed rows."""
    at = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu.long(), at, right=True) - 1
    return b, at - cu.long()[b]


def _slots(st, b, pos):
    ps = st["page"]
    return st["table"][b, pos // ps].long(), pos % ps


def _append(st):
    b, i = _rows(st["cu_new"], st["total"])
    n = (st["cu_new"][1:] - st["cu_new"][:-1]).long()
    page, slot = _slots(st, b, st["kv_len"].long()[b] - n[b] + i)
    if st["kind"] == "bf16":
        st["k"][page, :, slot] = st["k_new"]
        st["v"][page, :, slot] = st["v_new"]
        return {"k": st["k"], "v": st["v"]}
    k, ks = _quantised(st["k_new"])
    v, vs = _quantised(st["v_new"])
    st["k"].view(torch.uint8)[page, :, slot] = k.view(torch.uint8)
    st["v"].view(torch.uint8)[page, :, slot] = v.view(torch.uint8)
    st["k_scale"][page, :, slot] = ks
    st["v_scale"][page, :, slot] = vs
    return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _gathered(st, x, scale, page, slot):
    codes = x if scale is None else x.view(torch.uint8)
    got = codes[page, :, slot]
    return got if scale is None else _held(got.view(torch.float8_e4m3fn), scale[page, :, slot])


def _read(st):
    b, i = _rows(st["cu_past"], st["total_past"])
    page, slot = _slots(st, b, i)
    return {"k": _gathered(st, st["k"], st["k_scale"], page, slot).to(torch.bfloat16),
            "v": _gathered(st, st["v"], st["v_scale"], page, slot).to(torch.bfloat16)}


def _attn(st):
    B, H, D, Hq, n = st["rows"], st["heads_kv"], st["head_dim"], st["heads_q"], st["max_new"]
    L, ps, G = st["longest"], st["page"], st["heads_q"] // st["heads_kv"]
    dev_kv = st["kv_len"].long()
    count = (st["cu_new"][1:] - st["cu_new"][:-1]).long()
    # keys and values of every sequence, padded to the longest: [B, H, L, D]
    table = st["table"][:, :-(-L // ps)].long().clamp(min=0)
    k, v = (_held(st[x], st[x + "_scale"])[table].transpose(1, 2).reshape(B, H, -1, D)[:, :, :L]
            for x in ("k", "v"))
    b, i = _rows(st["cu_new"], st["total"])
    q = torch.zeros((B, n, Hq, D), device=DEV)
    q[b, i] = st["q"].float()
    s = torch.matmul(q.reshape(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D),
                     k.transpose(-1, -2)).mul_(D ** -0.5).view(B, H, n, G, L)
    key = torch.arange(L, device=DEV)
    ends = dev_kv[:, None].expand(B, n)
    if st["causal"]:
        ends = ends - count[:, None] + torch.arange(n, device=DEV) + 1
    hidden = key >= ends[:, :, None]
    s.masked_fill_(hidden[:, None, :, None, :], -torch.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((key < dev_kv[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.reshape(B, H, n * G, L), v).view(B, H, n, G, D) / \
        torch.where(total > 0, total, 1.0)
    lse = (m + total.log())[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)[b, i].to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, n, Hq)[b, i]}


def _softmax64(z, tau):
    z = z.double() / tau
    z = (z - z.amax(-1, keepdim=True)).exp_()
    return z.div_(z.sum(-1, keepdim=True))


def _verify(st):
    B, V = st["rows"], st["vocab"]
    cu = st["cu_draft"].long()
    k = cu[1:] - cu[:-1]
    T = st["draft_tokens"].numel()
    b, i = _rows(st["cu_draft"], T)
    row = torch.arange(T, device=DEV) + b  # each sequence has one target row more than drafts
    p_all = _softmax64(st["target"], st["tau"])
    p = p_all[row, st["draft_tokens"].long()]
    refused = st["u_accept"].double() * st["draft_conf"].double() >= p
    accepted = k.clone().scatter_reduce_(0, b, torch.where(refused, i, k[b]), "amin")
    at = accepted + cu[:-1]
    target = p_all[at + torch.arange(B, device=DEV)]
    some = accepted < k
    draft = _softmax64(st["draft"][at.clamp(max=max(T - 1, 0))], st["draft_tau"]) if T else target
    rest = torch.where(some[:, None], (target - draft).clamp(min=0), target)
    rest = torch.where((rest.sum(-1) > 0)[:, None], rest, target)
    cum = rest.cumsum(-1)
    bar = st["u_sample"].double() * cum[:, -1]
    last = V - 1 - rest.gt(0).flip(-1).int().argmax(-1)
    nxt = torch.minimum((cum <= bar[:, None]).sum(-1), last)
    tokens = torch.full((T + B,), -1, dtype=torch.int32, device=DEV)
    tokens[row] = torch.where(i < accepted[b], st["draft_tokens"], -1)
    tokens[at + torch.arange(B, device=DEV)] = nxt.to(torch.int32)
    return {"accepted": accepted.to(torch.int32), "tokens": tokens, "target_prob": p.float()}


def run(state):
    if own:
        import block_discrete_diffusion_dd_b200 as dd
        if state["op"] == "append":
            dd.cache_append(state["cache"], state["batch"], state["k_new"], state["v_new"],
                            workspace=state["ws"])
            held = {"k": state["k"], "v": state["v"]}
            if state["kind"] == "e4m3":
                held.update(k_scale=state["k_scale"], v_scale=state["v_scale"])
            return held
        if state["op"] == "read":
            k, v = dd.cache_read(state["cache"], state["table"], state["cu_past"],
                                 k_out=state["k_out"], v_out=state["v_out"],
                                 workspace=state["ws"])
            return {"k": k, "v": v}
        if state["op"] == "attn":
            out, lse = dd.paged_attn(state["q"], state["cache"], state["batch"],
                                     causal=state["causal"], out=state["out"], lse=state["lse"],
                                     workspace=state["ws"])
            return {"out": out, "lse": lse}
        o = dd.verify_draft(state["target"], state["draft"], state["draft_tokens"],
                            state["draft_conf"], state["cu_draft"], state["u_accept"],
                            state["u_sample"], state["tau"], state["draft_tau"],
                            outputs=state["outputs"], workspace=state["ws"])
        return {"accepted": o["accepted"], "tokens": o["tokens"], "target_prob": o["target_prob"]}
    return {"append": _append, "read": _read, "attn": _attn, "verify": _verify}[state["op"]](state)


# ------------------------------------------------- the definitions, 64 bits
def _pow2_64(n):
    return ((n.long() + 1023) << 52).view(torch.float64)


def _code64(x):
    """The E4M3 values (in 64 bits) and exponents of x [..., D]: halves to even."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a / 448.0))
    e = torch.where(a > 0, e, torch.zeros_like(e))
    e = torch.where(a > 448 * _pow2_64(e), e + 1, e)
    e = torch.where((a > 0) & (a <= 448 * _pow2_64(e - 1)), e - 1, e)
    y = x * _pow2_64(-e)[..., None]
    m, ex = torch.frexp(y)  # |y| = m 2^ex, m in [1/2, 1): three bits behind the leading one
    step = _pow2_64(ex.clamp(min=-5) - 4)
    return torch.round(y / step) * step, e


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        k, out = _drafts(case), []
        t0 = d0 = 0
        for n in k:
            z = st["target"][t0:t0 + n].double() / case["tau"]
            x = st["draft_tokens"][d0:d0 + n].long()
            out.append((z.gather(1, x[:, None])[:, 0] - torch.logsumexp(z, 1)).exp())
            t0, d0 = t0 + n + 1, d0 + n
        return {"accepted": None, "tokens": None, "target_prob": torch.cat(out)}
    past, new, ps = _past(case), _new(case), case["page"]
    if case["op"] == "append":
        held = {x: st[x].double() for x in ("k", "v")}
        for x in ("k", "v"):
            y, e = st[x + "_new"].double(), None
            if case["kind"] == "e4m3":
                y, e = _code64(y)
            t = 0
            for b in range(case["batch"]):
                pos = torch.arange(past[b], past[b] + new[b], device=DEV)
                held[x][st["table"][b].long()[pos // ps], :, pos % ps] = y[t:t + new[b]]
                t += new[b]
        if case["kind"] == "e4m3":
            held.update(k_scale=None, v_scale=None)
        return held
    length = past if case["op"] == "read" else [p + n for p, n in zip(past, new)]
    whole = {}
    for x in ("k", "v"):
        whole[x] = st[x].double()
        if case["kind"] == "e4m3":
            whole[x] = whole[x] * _pow2_64(st[x + "_scale"].long() - 127)[..., None]

    def of(x, b):  # [heads, tokens, D]
        pages = st["table"][b, :-(-length[b] // ps)].long()
        return whole[x][pages].transpose(0, 1).flatten(1, 2)[:, :length[b]]

    if case["op"] == "read":
        return {x: torch.cat([of(x, b).transpose(0, 1) for b in range(case["batch"])])
                for x in ("k", "v")}
    H, G = case["heads_kv"], case["heads_q"] // case["heads_kv"]
    outs, lses, t = [], [], 0
    for b in range(case["batch"]):
        q = st["q"][t:t + new[b]].double().unflatten(1, (H, G))
        t += new[b]
        k, v = of("k", b), of("v", b)
        o, l = [], []
        for h in range(H):
            s = torch.einsum("igd,jd->igj", q[:, h], k[h]) / math.sqrt(case["head_dim"])
            if case["causal"]:
                i = torch.arange(new[b], device=DEV)[:, None, None]
                j = torch.arange(length[b], device=DEV)
                s = s.masked_fill(j > past[b] + i, -math.inf)
            l.append(torch.logsumexp(s, -1))
            o.append(torch.einsum("igj,jd->igd", torch.softmax(s, -1), v[h]))
        outs.append(torch.stack(o, 1).flatten(1, 2))
        lses.append(torch.stack(l, 1).flatten(1, 2))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
