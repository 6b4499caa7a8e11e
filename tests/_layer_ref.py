"""Plain float64 forms of the operators around the recurrence, token by token or
row by row on the CPU, and the element-wise comparison of their tests."""
import torch

F64 = torch.float64


def close(got, ref, *, rel, rms=0.0, what=""):
    """|got - ref| <= rel |ref| + rms * rms(ref), element by element."""
    got, ref = got.detach().cpu().to(F64), ref.detach().cpu().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not ref.numel():
        return
    bound = rel * ref.abs() + rms * ref.square().mean().sqrt() + 1e-30
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.3f} times the bound"


def spans(B, T, lens):
    """(first flat token, length) of each sequence."""
    if lens is None:
        return [(n * T, T) for n in range(B)]
    at, out = 0, []
    for n in lens:
        out.append((at, n))
        at += n
    return out


def conv(x, w, b=None, *, silu=False, lens=None, init=None):
    """(y, final_state) in float64; differentiable."""
    D, W = w.shape
    flat = x.reshape(-1, D).to(F64)
    ys, last = [], []
    for n, (at, ln) in enumerate(spans(*x.shape[:2], lens)):
        before = torch.zeros(W - 1, D, dtype=F64) if init is None else init[n].to(F64)
        whole = torch.cat([before, flat[at:at + ln]])
        u = sum(whole[j:j + ln] * w[:, j].to(F64) for j in range(W))
        if b is not None:
            u = u + b.to(F64)
        ys.append(u * torch.sigmoid(u) if silu else u)
        last.append(whole[ln:])
    y = torch.cat(ys).reshape(x.shape) if ys else flat.reshape(x.shape)
    return y, torch.stack(last) if last else torch.zeros(0, W - 1, D, dtype=F64)


def scan(x, dt, A, B, C, D=None, *, bias=None, softplus=False, lens=None, h0=None, keep=None):
    """(y, hT) in float64; ``keep`` gives the token count after which each state is taken."""
    n, T, H, dx = x.shape
    G, ds = B.shape[2:]
    rep = H // G
    X, Dt = x.reshape(-1, H, dx).to(F64), dt.reshape(-1, H).to(F64)
    Bf = B.reshape(-1, G, ds).to(F64).repeat_interleave(rep, 1)
    Cf = C.reshape(-1, G, ds).to(F64).repeat_interleave(rep, 1)
    if softplus:
        Dt = torch.logaddexp(Dt + (0 if bias is None else bias.to(F64)), torch.zeros((), dtype=F64))
    a = torch.exp(Dt * A.to(F64))
    ys, last = [None] * X.shape[0], []
    for i, (at, ln) in enumerate(spans(n, T, lens)):
        S = torch.zeros(H, ds, dx, dtype=F64) if h0 is None else h0[i].to(F64)
        end = S
        for k in range(ln):
            t = at + k
            S = a[t][:, None, None] * S + Bf[t][:, :, None] * (Dt[t][:, None] * X[t])[:, None, :]
            y = (S * Cf[t][:, :, None]).sum(1)
            ys[t] = y if D is None else y + D.to(F64)[:, None] * X[t]
            if keep is None or keep[i] == k + 1:
                end = S
        last.append(end)
    y = torch.stack(ys).reshape(x.shape) if ys else X.reshape(x.shape)
    return y, torch.stack(last) if last else torch.zeros(0, H, ds, dx, dtype=F64)


def norm(x, *, weight=None, gate=None, act="sigmoid", first=False, residual=None, scale=1.0,
         res_scale=None, out_weight=None, eps=1e-6):
    """(r, y) in float64; differentiable."""
    unit = lambda v: v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    z = 1.0
    if gate is not None:
        g = gate.to(F64)
        z = torch.sigmoid(g) if act == "sigmoid" else g * torch.sigmoid(g)
    v = x.to(F64) * z if first else x.to(F64)
    m = v if weight is None else unit(v) * weight.to(F64)
    if not first:
        m = m * z
    r = scale * m
    if res_scale is not None:
        r = r * res_scale.to(F64)
    if residual is not None:
        r = r + residual.to(F64)
    return r, None if out_weight is None else unit(r) * out_weight.to(F64)
