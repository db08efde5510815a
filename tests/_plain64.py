"""Plain float64 forms of shared-prefix attention, rotary positions and token log probabilities
(torch, on the inputs' device), written from the definitions in include/mgd.h: what the GPU results of those calls are
compared with.  Test infrastructure only."""
import math

import torch


def prefix_attention(q, kp, vp, plen, k, v, kv_len, scale):
    """q [B,T,Hq,D]; kp, vp [Hkv,P,D] with plen rows in use; own k, v [B,Hkv,cap,D] -> out, lse (float64)."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((B, T, Hq), dtype=torch.float64, device=q.device)
    q, kp, vp, k, v = (x.double() for x in (q, kp, vp, k, v))
    for b in range(B):
        L = int(kv_len[b])
        for h in range(Hkv):
            keys, vals = torch.cat((kp[h, :plen], k[b, h, :L])), torch.cat((vp[h, :plen], v[b, h, :L]))
            for t in range(T):
                n = plen + L - T + t + 1
                s = q[b, t, h * G:(h + 1) * G] @ keys[:n].T * scale
                m = s.amax(-1, keepdim=True)
                e = (s - m).exp()
                z = e.sum(-1, keepdim=True)
                out[b, t, h * G:(h + 1) * G] = e @ vals[:n] / z
                lse[b, t, h * G:(h + 1) * G] = (m + z.log())[:, 0]
    return out, lse


def rope_radians(rot, base, scaling=None):
    """Angle per position of each pair (python floats) and the magnitude."""
    kind = None if scaling is None else scaling["kind"]
    f = None if scaling is None else scaling["factor"]
    if kind == "ntk":
        base = base * f ** (rot / (rot - 2))
    inv, mag = [base ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if kind == "linear":
        inv = [x / f for x in inv]
    if kind == "llama3":
        lo, hi, n = scaling["low_freq_factor"], scaling["high_freq_factor"], scaling["original_len"]
        new = []
        for x in inv:
            wave = 2 * math.pi / x
            if wave < n / hi:
                new.append(x)
            elif wave > n / lo:
                new.append(x / f)
            else:
                smooth = (n / wave - lo) / (hi - lo)
                new.append((1 - smooth) * x / f + smooth * x)
        inv = new
    if kind == "yarn":
        def dim(turns):
            return rot * math.log(scaling["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(dim(scaling["beta_fast"])), 0)
        hi = min(math.ceil(dim(scaling["beta_slow"])), rot - 1)
        new = []
        for i, x in enumerate(inv):
            ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            new.append(x / f * ramp + x * (1 - ramp))
        inv, mag = new, 0.1 * math.log(f) + 1.0
    return inv, mag


def rope(x, pos, inv, mag, interleaved):
    """x [..., H, D] float64, pos [...] whole numbers: every head turned by its row's position."""
    half = len(inv)
    y = x.double().clone()
    ang = pos.double()[..., None] * torch.tensor(inv, dtype=torch.float64, device=x.device)
    c, s = (ang.cos() * mag)[..., None, :], (ang.sin() * mag)[..., None, :]
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    a, b = x.double()[..., i0], x.double()[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    return y


def token_logprobs(x, tok, K):
    """One row x [V] (any float type), token tok >= 0 -> (logprob, entropy, rank, ids, logprobs) as python values."""
    x = x.double()
    V = x.numel()
    if bool((x.isnan() | (x == math.inf)).any()) or not bool((x > -math.inf).any()):
        return math.nan, math.nan, -1, [-1] * K, [-math.inf] * K
    d = x - x.max()
    lp = d - d.exp().sum().log()  # not x - (max + log sum): a row of float32's lowest value would absorb the sum
    p = lp.exp()
    ent = -float((p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum())
    j = torch.arange(V, device=x.device)
    rank = int((x > x[tok]).sum() + ((x == x[tok]) & (j < tok)).sum())
    order = torch.sort(-(x + 0.0), stable=True).indices[:K]
    ids, lps = [], []
    for i in order.tolist():
        ok = float(x[i]) > -math.inf
        ids.append(i if ok else -1)
        lps.append(float(lp[i]) if ok else -math.inf)
    ids += [-1] * (K - len(ids))
    lps += [-math.inf] * (K - len(lps))
    return float(lp[tok]), ent, rank, ids, lps
