"""Speed and accuracy cases of the operators around a verify call of a batch with a shared prompt:
attention over a shared prefix and each sequence's own cache, rotary positions with the append of
new rows to the cache, and log probabilities of given tokens.

``run`` computes a case in plain torch operations, or, where ``own`` is true, through
``long_context_speculative_split_gb300.ops``.  ``exact`` computes it once more in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _prefix(name, B, T, Hq, Hkv, D, P, cap, dtype):
    return dict(name=name, op="prefix_attn", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, cap=cap, dtype=dtype)


def _rope(name, B, T, Hq, Hkv, D, rot, cap, dtype, interleaved, base, scaling, factor, offset, ragged):
    return dict(name=name, op="rope_append", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, cap=cap, dtype=dtype,
                interleaved=interleaved, base=base, scaling=scaling, factor=factor, offset=offset, ragged=ragged)


def _logp(name, B, T, V, top, dtype, padded):
    return dict(name=name, op="token_logprobs", B=B, T=T, V=V, top=top, dtype=dtype, padded=padded)


def listed():
    return [
        # the tiny float32 configuration of the tests, verify rows over a short shared prompt: latency
        _prefix("prefix_tiny_f32", 2, 4, 4, 1, 64, 512, 300, "f32"),
        # four requests decoding one token each just after a shared system prompt: latency
        _prefix("prefix_decode_b4", 4, 1, 32, 8, 128, 2000, 128, "bf16"),
        # an odd mid-size batch: three query heads a KV head, head_dim 64, odd lengths
        _prefix("prefix_odd_b45", 45, 3, 24, 8, 64, 5001, 777, "bf16"),
        # a verify round of a batch of 32 over a shared 8k context with ragged own caches
        _prefix("prefix_verify_b32", 32, 4, 32, 8, 128, 8192, 512, "bf16"),
        # the benchmark's batch and context with the context shared: 128 x 5 rows over 32k keys
        _prefix("prefix_verify_b128", 128, 5, 32, 8, 128, 32768, 1024, "bf16"),
        # one verify round's new rows, behind a shared prefix, banded scaling for a long context
        _rope("rope_verify_b128", 128, 5, 32, 8, 128, 128, 64, "bf16", False, 500000.0, "llama3", 8.0, 32768, False),
        # partial rotary with interleaved pairs, float32, odd row count
        _rope("rope_partial_f32", 3, 333, 8, 2, 64, 32, 400, "f32", True, 10000.0, "ntk", 4.0, 0, True),
        # prefill of four ragged prompts
        _rope("rope_prefill_b4", 4, 8192, 32, 8, 128, 128, 8192, "bf16", False, 10000.0, "yarn", 16.0, 0, True),
        # one request's verify rows with 20 alternatives each: latency
        _logp("logprobs_verify_b1", 1, 4, 128256, 20, "f32", False),
        # an odd vocabulary, rows that start off a 16-byte boundary
        _logp("logprobs_odd_v50257", 37, 1, 50257, 3, "bf16", False),
        # the committed tokens of a batch-128 round: -1 after each sequence's last token
        _logp("logprobs_verify_b128", 128, 5, 128256, 8, "f32", True),
        # scoring of prompts
        _logp("logprobs_score_b2", 2, 1024, 128256, 20, "bf16", False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefix_attn", "rope_append", "token_logprobs"])
    if op == "prefix_attn":
        if rng.random() < 0.2:
            return {k: v for k, v in _prefix("", _log_int(rng, 1, 6), rng.randint(1, 6), 4, rng.choice([1, 2, 4]),
                                             rng.choice([64, 128]), _log_int(rng, 32, 1200), _log_int(rng, 16, 400),
                                             "f32").items() if k != "name"}
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
        B, T = _log_int(rng, 1, 128), rng.randint(1, 8)
        P, cap = _log_int(rng, 64, 32768), _log_int(rng, 16, 1024)
        while B * T * Hkv * G * P * D > 128 * 5 * 32 * 32768 * 128:
            P = max(64, P // 2)
        return {k: v for k, v in _prefix("", B, T, Hkv * G, Hkv, D, P, cap, "bf16").items() if k != "name"}
    if op == "rope_append":
        D, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 8]), rng.choice([1, 3, 4])
        rot = rng.choice([D, D, D // 2, D // 4])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            B, T = _log_int(rng, 1, 256), rng.randint(1, 8)
        else:
            B, T = rng.randint(1, 4), _log_int(rng, 16, 4096)
        cap = T + rng.randint(0, 64)
        scaling = rng.choice(["none", "linear", "ntk", "llama3", "yarn"])
        return {k: v for k, v in _rope("", B, T, Hkv * G, Hkv, D, rot, cap, dtype, rng.random() < 0.5,
                                       rng.choice([10000.0, 500000.0]), scaling, float(rng.choice([2, 4, 8, 16])),
                                       _log_int(rng, 1, 1000000), rng.random() < 0.5).items() if k != "name"}
    V, dtype = _log_int(rng, 1000, 262144), rng.choice(["bf16", "f32"])
    B, T = _log_int(rng, 1, 128), rng.randint(1, 8)
    while B * T * V * 4 > 2048 * 128256 * 2:
        B = max(1, B // 2)
    return {k: v for k, v in _logp("", B, T, V, rng.choice([0, 1, 5, 8, 20, 32]), dtype, rng.random() < 0.5).items()
            if k != "name"}


# ---------------------------------------------------------------------------- inputs
def _own_lengths(case, seed):
    """Own-cache rows of each sequence: ragged in [max(T, cap / 4), cap]."""
    g = torch.Generator().manual_seed(seed * 7919 + 5)
    lo = max(case["T"], case["cap"] // 4)
    hi = max(case["cap"], lo)
    return torch.randint(lo, hi + 1, (case["B"],), generator=g).to(torch.int32)


def _heavy_keys(shape, gen, dtype):
    """Keys ~ N(0, 1) with about 1 % of the rows scaled by 8."""
    k = torch.randn(shape, generator=gen, device=DEV).to(dtype)
    heavy = torch.rand(shape[:-1], generator=gen, device=DEV) < 0.01
    return torch.where(heavy[..., None], k * 8, k)


def _frequencies(case):
    """Angles per position of the rotary pairs (64 bits), and the factor on cos and sin."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "llama3":  # long waves slowed down, short ones kept, a ramp between
        waves = 8192 * inv / (2 * math.pi)  # turns over the original length
        keep = ((waves - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return inv * (keep + (1 - keep) / f), 1.0
    if case["scaling"] == "yarn":
        def index(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
        slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return inv * (1 - slow) + inv / f * slow, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _scaling(case):
    """The same as an argument of ops.rope_table."""
    return {"none": None, "linear": dict(kind="linear", factor=case["factor"]),
            "ntk": dict(kind="ntk", factor=case["factor"]),
            "llama3": dict(kind="llama3", factor=case["factor"], low_freq_factor=1.0, high_freq_factor=4.0,
                           original_len=8192),
            "yarn": dict(kind="yarn", factor=case["factor"], original_len=4096, beta_fast=32.0, beta_slow=1.0),
            }[case["scaling"]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "prefix_attn":
        B, T, Hq, Hkv, D, P, cap = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "P", "cap"))
        cap = max(cap, T)
        dt = TYPES[case["dtype"]]
        s["q"] = torch.randn((B, T, Hq, D), generator=gen, device=DEV).to(dt)
        s["k_prefix"] = _heavy_keys((Hkv, P, D), gen, dt)
        s["v_prefix"] = torch.randn((Hkv, P, D), generator=gen, device=DEV).to(dt)
        s["k"] = _heavy_keys((B, Hkv, cap, D), gen, dt)
        s["v"] = torch.randn((B, Hkv, cap, D), generator=gen, device=DEV).to(dt)
        s["prefix_len"] = torch.full((1,), P, dtype=torch.int32, device=DEV)
        s["kv_len"] = _own_lengths(case, seed).to(DEV)
        if own:
            from long_context_speculative_split_gb300 import mgd, ops
            s["ws"] = ops.workspace(mgd.mgd_prefix_workspace_size(B, T, Hq, Hkv, D, P, cap), torch.device(DEV))
            s["out"] = torch.empty((B, T, Hq, D), dtype=dt, device=DEV)
            s["lse"] = torch.empty((B, T, Hq), dtype=torch.float32, device=DEV)
    elif case["op"] == "rope_append":
        B, T, Hq, Hkv, D, cap = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "cap"))
        dt = TYPES[case["dtype"]]
        # one projection's output, split by heads as views
        qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=gen, device=DEV).to(dt)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["k"] = torch.zeros((B, Hkv, cap, D), dtype=dt, device=DEV)
        s["v"] = torch.zeros((B, Hkv, cap, D), dtype=dt, device=DEV)
        g = torch.Generator().manual_seed(seed * 104729 + 3)
        n = torch.randint(max(1, T // 2), T + 1, (B,), generator=g) if case["ragged"] else torch.full((B,), T)
        before = torch.randint(0, cap - T + 1, (B,), generator=g)
        s["new_len"] = n.to(torch.int32).to(DEV)
        s["kv_len"] = (before + n).to(torch.int32).to(DEV)
        s["pos_offset"] = torch.full((1,), case["offset"], dtype=torch.int32, device=DEV)
        inv, mag = _frequencies(case)
        s["inv_freq"], s["magnitude"] = inv.to(DEV), mag
        s["q_out"] = torch.zeros((B, T, Hq, D), dtype=dt, device=DEV)
        if own:
            from long_context_speculative_split_gb300 import mgd, ops
            s["table"] = ops.rope_table(case["rot"], case["base"], _scaling(case), device=torch.device(DEV))
            s["ws"] = ops.workspace(mgd.mgd_rope_workspace_size(B), torch.device(DEV))
    else:
        B, T, V, K = (case[n] for n in ("B", "T", "V", "top"))
        s["logits"] = (torch.randn((B, T, V), generator=gen, device=DEV) * 3).to(TYPES[case["dtype"]])
        # tokens of a model: mostly likely ones (the highest of a few random entries)
        near = torch.randint(0, V, (B, T, 64), generator=gen, device=DEV)
        best = s["logits"].gather(2, near).float().argmax(2, keepdim=True)
        tok = near.gather(2, best)[..., 0].to(torch.int32)
        if case["padded"]:
            keep = torch.randint(1, T + 1, (B, 1), generator=gen, device=DEV)
            tok = torch.where(torch.arange(T, device=DEV)[None, :] < keep, tok, torch.full_like(tok, -1))
        s["tokens"] = tok
        if own:
            from long_context_speculative_split_gb300 import mgd, ops
            s["ws"] = ops.workspace(mgd.mgd_logprobs_workspace_size(B * T, V, K), torch.device(DEV))
            s["out"] = dict(logprob=torch.empty((B, T), device=DEV), entropy=torch.empty((B, T), device=DEV),
                            rank=torch.empty((B, T), dtype=torch.int32, device=DEV),
                            top_ids=torch.empty((B, T, K), dtype=torch.int32, device=DEV),
                            top_logprobs=torch.empty((B, T, K), device=DEV))
    return s


# ---------------------------------------------------------------------------- plain forms
def _plain_prefix(s):
    B, T, Hq, Hkv, D = (s[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    dt = s["q"].dtype
    q = s["q"].float().view(B, T, Hkv, G, D).permute(2, 0, 1, 3, 4)            # [Hkv, B, T, G, D]
    P, cap = s["k_prefix"].shape[1], s["k"].shape[2]
    sp = (q.reshape(Hkv, B * T * G, D) @ s["k_prefix"].float().transpose(1, 2)) * scale
    sp = sp.masked_fill(torch.arange(P, device=DEV) >= s["prefix_len"], float("-inf"))
    so = (q.permute(1, 0, 2, 3, 4).reshape(B, Hkv, T * G, D) @ s["k"].float().transpose(2, 3)) * scale
    last = s["kv_len"][:, None] - T + torch.arange(T, device=DEV)              # [B, T] last visible own row
    hide = torch.arange(cap, device=DEV)[None, None] > last[..., None]         # [B, T, cap]
    so = so.masked_fill(hide[:, None, :, None].expand(B, 1, T, G, cap).reshape(B, 1, T * G, cap), float("-inf"))
    mp = sp.amax(-1).view(Hkv, B, T * G).transpose(0, 1)                       # [B, Hkv, TG]
    m = torch.maximum(mp, so.amax(-1))
    ep = torch.exp(sp - m.transpose(0, 1).reshape(Hkv, B * T * G, 1))
    eo = torch.exp(so - m[..., None])
    z = ep.sum(-1).view(Hkv, B, T * G).transpose(0, 1) + eo.sum(-1)
    o = (ep @ s["v_prefix"].float()).view(Hkv, B, T * G, D).transpose(0, 1) + eo @ s["v"].float()
    o = (o / z[..., None]).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (m + torch.log(z)).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return {"out": o.to(dt), "lse": lse}


def _rows(s):
    """Per new row: whether it exists, its cache row and its position."""
    n, L = s["new_len"].long()[:, None], s["kv_len"].long()[:, None]
    t = torch.arange(s["T"], device=DEV)[None]
    at = L - n + t
    return t < n, at, at + s["pos_offset"].long()


def _plain_rope(s):
    rot, half = s["rot"], s["rot"] // 2
    live, at, pos = _rows(s)
    angle = pos.double()[..., None] * s["inv_freq"]
    cos = (angle.cos() * s["magnitude"]).float()[:, :, None]                   # [B, T, 1, rot / 2]
    sin = (angle.sin() * s["magnitude"]).float()[:, :, None]

    def turn(x):
        f = x.float()
        a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if s["interleaved"] else (f[..., :half], f[..., half:rot])
        c, d = a * cos - b * sin, a * sin + b * cos
        y = torch.stack((c, d), -1).flatten(-2) if s["interleaved"] else torch.cat((c, d), -1)
        return torch.cat((y, f[..., rot:]), -1).to(x.dtype)

    b, t = live.nonzero(as_tuple=True)
    s["q_out"][b, t] = turn(s["q"])[b, t]
    s["k"][b, :, at[b, t]] = turn(s["k_new"])[b, t]
    s["v"][b, :, at[b, t]] = s["v_new"][b, t]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_logprobs(s):
    x, tok, K, V = s["logits"].float(), s["tokens"].long(), s["top"], s["V"]
    live = tok >= 0
    t = tok.clamp(min=0)[..., None]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    xt = x.gather(-1, t)
    logp = (xt - lse)[..., 0]
    ent = (torch.log(z) - (e * (x - m)).sum(-1, keepdim=True) / z)[..., 0]
    j = torch.arange(V, device=DEV)
    rank = ((x > xt).sum(-1) + ((x == xt) & (j < t)).sum(-1)).to(torch.int32)
    # order by (value, lowest index first) as one 64-bit whole number
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * (1 << 32) + ((1 << 32) - 1 - j)
    ids = torch.topk(order, K, -1).indices if K else torch.zeros((*tok.shape, 0), dtype=torch.int64, device=DEV)
    top = x.gather(-1, ids) - lse
    zero, no = torch.zeros_like(logp), live[..., None]
    return {"logprob": torch.where(live, logp, zero), "entropy": torch.where(live, ent, zero),
            "rank": torch.where(live, rank, torch.full_like(rank, -1)),
            "top_ids": torch.where(no, ids, torch.full_like(ids, -1)).to(torch.int32),
            "top_logprobs": torch.where(no, top, torch.full_like(top, float("-inf")))}


# ---------------------------------------------------------------------------- the framework's calls
def _own_run(s):
    from long_context_speculative_split_gb300 import ops
    if s["op"] == "prefix_attn":
        out, lse = ops.prefix_attn(s["q"], s["k_prefix"], s["v_prefix"], s["prefix_len"], s["k"], s["v"], s["kv_len"],
                                   ws=s["ws"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if s["op"] == "rope_append":
        q = ops.rope_append(s["q"], s["k_new"], s["v_new"], s["table"], s["k"], s["v"], s["kv_len"],
                            new_len=s["new_len"], pos_offset=s["pos_offset"], interleaved=s["interleaved"],
                            q_out=s["q_out"], ws=s["ws"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    return ops.token_logprobs(s["logits"], s["tokens"], top=s["top"], ws=s["ws"], out=s["out"])


def run(state):
    if own:
        return _own_run(state)
    return {"prefix_attn": _plain_prefix, "rope_append": _plain_rope, "token_logprobs": _plain_logprobs}[state["op"]](
        state)


# ---------------------------------------------------------------------------- 64 bits
def _exact_prefix(s):
    B, T, Hq, Hkv, D = (s[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    out = torch.empty((B, T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, T, Hq), dtype=torch.float64, device=DEV)
    P, lens = int(s["prefix_len"]), s["kv_len"].tolist()
    kp, vp = s["k_prefix"][:, :P].double(), s["v_prefix"][:, :P].double()
    for b in range(B):
        for h in range(Hkv):
            keys = torch.cat((kp[h], s["k"][b, h, :lens[b]].double()))
            vals = torch.cat((vp[h], s["v"][b, h, :lens[b]].double()))
            x = torch.einsum("tgd,jd->tgj", s["q"][b, :, h * G:(h + 1) * G].double(), keys) / D ** 0.5
            for t in range(T - 1):  # the last row sees every key
                x[t, :, P + lens[b] - T + t + 1:] = -math.inf
            l = torch.logsumexp(x, -1)
            lse[b, :, h * G:(h + 1) * G] = l
            out[b, :, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", (x - l[..., None]).exp(), vals)
    return {"out": out, "lse": lse}


def _exact_rope(s):
    half = s["rot"] // 2
    pairs = torch.arange(half, device=DEV)
    first, second = (2 * pairs, 2 * pairs + 1) if s["interleaved"] else (pairs, pairs + half)
    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    new, total, off = s["new_len"].tolist(), s["kv_len"].tolist(), int(s["pos_offset"])
    for b in range(s["B"]):
        n, start = new[b], total[b] - new[b]
        pos = torch.arange(start + off, start + off + n, dtype=torch.float64, device=DEV)
        unit = torch.polar(torch.full((n, half), s["magnitude"], dtype=torch.float64, device=DEV),
                           pos[:, None] * s["inv_freq"][None])[:, None]
        for src, put in ((s["q"], "q"), (s["k_new"], "k")):
            x = src[b, :n].double()
            y = torch.complex(x[..., first], x[..., second]) * unit
            x = x.index_copy(-1, first, y.real).index_copy(-1, second, y.imag)
            if put == "q":
                q[b, :n] = x
            else:
                k[b, :, start:start + n] = x.transpose(0, 1)
        v[b, :, start:start + n] = s["v_new"][b, :n].double().transpose(0, 1)
    return {"q": q, "k": k, "v": v}


def _exact_logprobs(s):
    B, T, K = s["B"], s["T"], s["top"]
    f = torch.float64
    logp, ent = torch.zeros((B, T), dtype=f, device=DEV), torch.zeros((B, T), dtype=f, device=DEV)
    top = torch.full((B, T, K), -math.inf, dtype=f, device=DEV)
    for b in range(B):
        for t in range(T):
            tok = int(s["tokens"][b, t])
            if tok < 0:
                continue
            lp = torch.log_softmax(s["logits"][b, t].double(), 0)
            logp[b, t] = lp[tok]
            ent[b, t] = -(lp.exp() * lp).sum()
            if K:
                top[b, t] = lp.topk(K).values
    return {"logprob": logp, "entropy": ent, "rank": None, "top_ids": None, "top_logprobs": top}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"prefix_attn": _exact_prefix, "rope_append": _exact_rope, "token_logprobs": _exact_logprobs}[s["op"]](s)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "prefix_attn":
        B, T, Hq, Hkv, D, P = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "P"))
        esz = 2 if case["dtype"] == "bf16" else 4
        lo = max(T, case["cap"] // 4)
        rows = B * (lo + max(case["cap"], lo)) / 2  # mean own rows
        nbytes = 2 * B * T * Hq * D * esz + 4 * B * T * Hq + 2 * Hkv * P * D * esz + 2 * Hkv * rows * D * esz
        return {"bytes": nbytes, "flops": 4 * D * Hq * T * (B * P + rows - B * (T - 1) / 2)}
    if case["op"] == "rope_append":
        esz = 2 if case["dtype"] == "bf16" else 4
        n = (max(1, case["T"] // 2) + case["T"]) / 2 if case["ragged"] else case["T"]
        heads = case["Hq"] + 2 * case["Hkv"]
        turned = case["Hq"] + case["Hkv"]
        return {"bytes": 2 * case["B"] * n * heads * case["D"] * esz, "flops": 3 * case["B"] * n * turned * case["rot"]}
    rows = case["B"] * ((case["T"] + 1) / 2 if case["padded"] else case["T"])
    esz = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": rows * case["V"] * esz + rows * (16 + 8 * case["top"]), "flops": 6 * rows * case["V"]}
