"""Plain float64 forms of the attention layers' operators, from their definitions."""
import math

import torch

F64 = torch.float64


def channel_order(rot, interleaved):
    """The rotated channels, pair by pair."""
    if interleaved:
        return torch.arange(rot)
    return torch.arange(rot).reshape(2, rot // 2).T.flatten()


def qknorm(x, positions, freqs, weight=None, interleaved=False, eps=1e-6):
    """x [tokens, heads, d] float64 (any device), positions [tokens]."""
    n = x
    if weight is not None:
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight
    rot = 0 if freqs is None else 2 * freqs.numel()
    if rot == 0:
        return n
    order = channel_order(rot, interleaved).to(x.device)
    ang = (positions.to(F64)[:, None] * freqs)[:, None]
    a, b = n[..., order[0::2]], n[..., order[1::2]]
    out = n.clone()
    out[..., order[0::2]] = a * torch.cos(ang) - b * torch.sin(ang)
    out[..., order[1::2]] = a * torch.sin(ang) + b * torch.cos(ang)
    return out


def encode(x, kind):
    """(values that the cache stands for, bytes) of rows [..., d] in float64; kind e4m3 or int8."""
    top = 448.0 if kind == "e4m3" else 127.0
    bad = ~torch.isfinite(x).all(-1)
    x = torch.where(bad[..., None], 0.0, x)
    most = x.abs().amax(-1)
    e = torch.full(most.shape, -126.0, dtype=F64, device=x.device)
    for p in range(-126, 130):  # the smallest power that is large enough
        e = torch.where(most > top * 2.0 ** (p - 1), float(p), e) if p > -126 else e
    y = x * torch.exp2(-e)[..., None]
    if kind == "int8":
        code = torch.round(y)
    else:
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        code = torch.round(y / step) * step
    value = torch.where(bad[..., None], math.nan, code * torch.exp2(e)[..., None])
    return value, torch.where(bad, 255, (e + 127).long())


def rows(pool, scale, pages, page, n):
    """The first n places of a sequence, [heads, n, d] float64; places without a page are NaN."""
    out = torch.full((pool.shape[1], n, pool.shape[3]), math.nan, dtype=F64)
    for p in range(n):
        col = p // page
        if col >= len(pages) or not 0 <= pages[col] < pool.shape[0]:
            continue
        x = pool[pages[col], :, p % page].float().to(F64)
        if scale is not None:
            byte = scale[pages[col], :, p % page]
            power = torch.where(byte == 255, math.nan, torch.exp2(byte.to(F64) - 127))
            x = x * power[:, None]
        out[:, p] = x
    return out


def attn(q, cache, pages, lens, scale, window=0):
    """q [B,T,Hq,d] (CPU); places whose page is missing are unseen.  Returns out, lse."""
    B, T, Hq, d = q.shape
    kp, vp, ks, vs = cache
    G, page = kp.shape[1], kp.shape[2]
    rep = Hq // G
    out = torch.zeros(B, T, Hq, d, dtype=F64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=F64)
    cap = pages.shape[1] * page
    for b in range(B):
        n = int(lens[b])
        ids = pages[b].tolist()
        have = max(0, min(n, cap))
        k, v = rows(kp, ks, ids, page, have), rows(vp, vs, ids, page, have)
        there = torch.tensor([0 <= ids[p // page] < kp.shape[0] for p in range(have)], dtype=torch.bool)
        for t in range(T):
            hi = n - T + t + 1
            at = torch.arange(have)
            seen = there & (at < hi)
            if window:
                seen &= at >= hi - window
            if not seen.any():
                continue
            for h in range(Hq):
                s = (k[h // rep][seen] @ q[b, t, h].to(F64)) * scale
                out[b, t, h] = torch.softmax(s, 0) @ v[h // rep][seen]
                lse[b, t, h] = torch.logsumexp(s, 0)
    return out, lse


def fixed(p):
    """Whole multiples of 2^-44, to nearest (ties to even), as Python integers."""
    out = []
    for x in p.tolist():
        x = 0.0 if not x > 0 else min(x, 1.0)
        out.append(round(x * 2.0 ** 44))  # the product is exact, round() is to nearest even
    return out


def verify(p, q, drafts, u, counts=None):
    """Lists of tokens and counts; every sum in Python integers."""
    B, K1, V = p.shape
    K = K1 - 1
    toks, commit = [], []
    for b in range(B):
        have = K if counts is None else int(counts[b])
        if have < -1 or have > K:
            have = -1
        row = [-1] * K1
        if have < 0:
            toks.append(row)
            commit.append(0)
            continue
        kept = 0
        while kept < have:
            d = int(drafts[b, kept])
            if not 0 <= d < V:
                break
            qd = 1.0 if q is None else float(q[b, kept, d])
            if not float(u[b, kept]) * qd < float(p[b, kept, d]):  # exact in doubles
                break
            row[kept] = d
            kept += 1
        w = full = fixed(p[b, kept])
        if kept < have:
            if q is not None:
                less = fixed(q[b, kept])
            else:
                less = [0] * V
                if 0 <= int(drafts[b, kept]) < V:
                    less[int(drafts[b, kept])] = 1 << 44
            w = [max(x - y, 0) for x, y in zip(w, less)]
            if sum(w) == 0:
                w = full
        total = sum(w)
        if total > 0:
            m = int(min(max(float(u[b, K]), 0.0), 1 - 2.0 ** -24) * 2 ** 24)
            left, run = m * total >> 24, 0
            for i, x in enumerate(w):
                run += x
                if run > left:
                    row[kept] = i
                    break
        toks.append(row)
        commit.append(kept + 1)
    return torch.tensor(toks, dtype=torch.int32), torch.tensor(commit, dtype=torch.int32)
