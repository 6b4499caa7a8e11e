"""Cases, inputs and plain forms of the operators around the recurrence.

Three operators, each with the forms that a user calls:

* ``conv``: the short causal convolution over the tokens of each channel (prompt, step, gradient);
* ``scan``: the selective state-space scan with one decay per head (prompt, step);
* ``norm``: RMS norms before and after a block, fused with its gate and its residual scale
  (forward, gradient).

``run`` computes a case either in its plain form (elementary torch operations in float32, rounded
once at the end) or, where ``own`` is true, through the library's entry points.  ``exact`` gives the
results from the definitions in float64.
"""
import itertools
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def lengths(case):
    """Tokens of each sequence: fixed, or (packed) drawn uniformly from [lo, hi] by the case's own seed."""
    if case["packed"]:
        r = random.Random(case["lens_seed"])
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    return [case["t"]] * case["n"]


def conv_case(name, form, n, t, d, width, dtype, packed=False, lo=0, hi=0, lens_seed=0):
    return {"name": name, "op": "conv", "form": form, "n": n, "t": t, "d": d, "width": width, "dtype": dtype,
            "packed": packed, "lo": lo, "hi": hi, "lens_seed": lens_seed}


def scan_case(name, form, n, t, h, g, ds, dx, dtype, packed=False, lo=0, hi=0, lens_seed=0, commit=False):
    return {"name": name, "op": "scan", "form": form, "n": n, "t": t, "h": h, "g": g, "ds": ds, "dx": dx, "dtype": dtype,
            "packed": packed, "lo": lo, "hi": hi, "lens_seed": lens_seed, "commit": commit}


def norm_case(name, form, rows, heads, d, dtype, gate, first, sandwich):
    return {"name": name, "op": "norm", "form": form, "rows": rows, "heads": heads, "d": d, "dtype": dtype, "gate": gate,
            "first": first, "sandwich": sandwich}


def listed():
    return [
        # q, k and v (32 heads of 128 each) of the packed prefill batch: 16 requests' prompts
        conv_case("conv_prompt_packed", "prompt", 16, 0, 12288, 4, "bf16", True, 128, 8192, 1002),
        # one token of each of 1024 running sequences, the same channels
        conv_case("conv_step_pool", "step", 1024, 1, 12288, 4, "bf16"),
        # a training step's gradients over the fixed-length batch
        conv_case("conv_train", "train", 4, 4096, 12288, 4, "bf16"),
        # the tiny float32 workload: a short prompt, where launches and latency count
        scan_case("scan_prompt_tiny", "prompt", 1, 256, 2, 1, 64, 64, "f32"),
        # the fixed-length prefill batch
        scan_case("scan_prompt_batch", "prompt", 4, 4096, 32, 4, 128, 128, "bf16"),
        # the packed prefill batch on heads of 64 channels, continued from earlier states
        scan_case("scan_prompt_packed", "prompt", 16, 0, 64, 8, 128, 64, "bf16", True, 128, 8192, 1002),
        # one long document of an odd number of tokens: few chains, a long axis
        scan_case("scan_prompt_long", "prompt", 1, 131071, 32, 1, 128, 128, "bf16"),
        # one token of each of 1024 running sequences: the state pool is read and written once
        scan_case("scan_step_pool", "step", 1024, 1, 32, 4, 128, 128, "bf16"),
        # 8 drafted tokens of 5 sequences, of which each keeps a prefix
        scan_case("scan_step_draft", "step", 5, 8, 32, 4, 128, 128, "bf16", commit=True),
        # the sandwich around a block for 8 decoding sequences: the smallest call
        norm_case("norm_serve", "forward", 8, 1, 4096, "bf16", "", False, True),
        # the gated output norm of the fixed-length batch: 32 heads of 128
        norm_case("norm_heads", "forward", 16384, 32, 128, "bf16", "sigmoid", False, False),
        # a training step's gradients of the sandwich with a gate
        norm_case("norm_train", "train", 16384, 1, 4096, "bf16", "silu", True, True),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["conv", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    packed = rng.random() < 0.5
    if op == "conv":
        form = rng.choice(["prompt", "step", "train"])
        d, width = rng.choice([8, 8, 1]) * log(16, 1536), rng.choice([2, 3, 4])
        if form == "step":
            c = conv_case("", form, log(1, 1024), rng.choice([1, 1, 2, 5, 8]), d, width, dtype)
        else:
            n = log(1, 16)
            hi = max(2, min(8192, log(3, 16384) if n > 4 else log(3, 32768)))
            c = conv_case("", form, n, min(hi, 16384 // n), d, width, dtype, packed, max(1, hi // 32), min(hi, 65536 // n),
                          rng.randrange(1 << 20))
    elif op == "scan":
        form = rng.choice(["prompt", "prompt", "step"])
        ds, dx = rng.choice([64, 128, 128]), rng.choice([64, 128])
        g = rng.choice([1, 2, 4])
        h = g * rng.choice([1, 2, 3, 5, 8])
        if form == "step":
            c = scan_case("", form, log(1, 700), rng.choice([1, 1, 2, 5, 8]), h, g, ds, dx, dtype, commit=rng.random() < 0.4)
        else:
            n = log(1, 16)
            hi = max(2, log(3, 2048 if dtype == "f32" else 16384))
            c = scan_case("", form, n, max(1, min(hi, 16384 // n)), h, g, ds, dx, dtype, packed, max(1, hi // 32),
                          max(1, min(hi, 32768 // n)), rng.randrange(1 << 20))
    else:
        form = rng.choice(["forward", "train"])
        heads = rng.choice([1, 1, 2, 7, 32])
        d = rng.choice([64, 128, 192]) if heads > 1 else rng.choice([8, 1]) * log(64, 768)
        rows = log(1, max(2, min(16384, (1 << 25) // (heads * d))))
        c = norm_case("", form, rows, heads, d, dtype, rng.choice(["", "sigmoid", "silu"]), rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def offsets(lens):
    return [0] + list(itertools.accumulate(lens))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    f = dict(device=DEV, dtype=torch.float32, generator=gen)
    s = {"case": case}
    if case["op"] == "norm":
        rows, heads, d = case["rows"], case["heads"], case["d"]
        shape = (rows, heads, d) if heads > 1 else (rows, d)
        s["x"] = torch.randn(shape, **f).to(dt)
        s["w"] = 1 + 0.1 * torch.randn(d, **f)
        s["gate"] = torch.randn(shape, **f).to(dt) if case["gate"] else None
        s["res"] = s["ls"] = s["ow"] = None
        if case["sandwich"]:
            s["res"] = (2 * torch.randn(shape, **f)).to(dt)
            s["ls"] = 0.5 + 0.1 * torch.randn(d, **f)
            s["ow"] = 1 + 0.1 * torch.randn(d, **f)
        if case["form"] == "train":
            s["dr"] = torch.randn(shape, **f).to(dt)
            s["dy"] = torch.randn(shape, **f).to(dt) if case["sandwich"] else None
        return s
    lens = lengths(case)
    n, total = len(lens), sum(lens)
    lead = (1, total) if case["packed"] else (n, case["t"])
    s["lens"] = lens
    cu = offsets(lens)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV) if case["packed"] else None
    # where each token sits: its sequence and its place in it (the plain forms' plan)
    s["seq"] = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(lens, device=DEV), output_size=total)
    s["first"] = torch.tensor(cu[:-1], device=DEV)
    s["len"] = torch.tensor(lens, device=DEV)
    s["pos"] = torch.arange(total, device=DEV) - s["first"][s["seq"]]
    if case["op"] == "conv":
        d, k = case["d"], case["width"]
        s["x"] = torch.randn(*lead, d, **f).to(dt)
        s["w"] = torch.randn(d, k, **f) * k ** -0.5
        s["b"] = 0.1 * torch.randn(d, **f)
        s["init"] = torch.randn(n, k - 1, d, **f).to(dt)
        if case["form"] == "train":
            s["init"] = None
            s["dy"] = torch.randn(*lead, d, **f).to(dt)
        return s
    h, g, ds, dx = case["h"], case["g"], case["ds"], case["dx"]
    s["x"] = torch.randn(*lead, h, dx, **f).to(dt)
    s["B"] = (torch.randn(*lead, g, ds, **f) * ds ** -0.25).to(dt)
    s["C"] = (torch.randn(*lead, g, ds, **f) * ds ** -0.25).to(dt)
    s["dt"] = torch.randn(*lead, h, **f).to(dt)
    s["dtb"] = -2 + torch.randn(h, **f)
    s["A"] = -torch.exp(torch.rand(h, **f) * 2.77)  # decay rates in [-16, -1]
    s["D"] = 1 + 0.1 * torch.randn(h, **f)
    s["h0"] = 0.1 * torch.randn(n, h, ds, dx, **f)
    s["commit"] = None
    if case["commit"]:
        s["commit"] = torch.randint(0, case["t"] + 1, (n,), device=DEV, generator=gen, dtype=torch.int32)
    if case["form"] == "prompt":
        # the plain form's chunks: which token each place of each chunk holds (or none)
        q = 128
        per = [-(-x // q) for x in lens]
        cseq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(per, device=DEV), output_size=sum(per))
        cfirst = torch.tensor(offsets(per)[:-1], device=DEV)
        at = (torch.arange(sum(per), device=DEV) - cfirst[cseq])[:, None] * q + torch.arange(q, device=DEV)
        s["valid"] = at < s["len"][cseq][:, None]
        s["tok"] = torch.where(s["valid"], s["first"][cseq][:, None] + at, 0)
        s["cseq"], s["cfirst"], s["clast"] = cseq, cfirst, cfirst + torch.tensor(per, device=DEV) - 1
        s["back"] = (cfirst[s["seq"]] * q + s["pos"])
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def run_own(s):
    import kda_delta_rule_fwd_gb300 as kda
    c = s["case"]
    if c["op"] == "conv":
        if c["form"] == "prompt":
            return kda.conv_fwd(s["x"], s["w"], s["b"], activation="silu", cu_seqlens=s["cu"], init_state=s["init"])
        if c["form"] == "step":
            return kda.conv_step(s["x"], s["w"], s["init"], s["b"], activation="silu"), s["init"]
        return kda.conv_bwd(s["x"], s["w"], s["dy"], s["b"], activation="silu", cu_seqlens=s["cu"])[:3]
    if c["op"] == "scan":
        if c["form"] == "prompt":
            return kda.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["dtb"], dt_softplus=True,
                                cu_seqlens=s["cu"], h0=s["h0"], out_dtype=s["x"].dtype)
        y = kda.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"], D=s["D"], dt_bias=s["dtb"], dt_softplus=True,
                          num_commit=s["commit"], out_dtype=s["x"].dtype)
        return y, s["h0"]
    kw = dict(weight=s["w"], gate=s["gate"], gate_act=c["gate"] or "sigmoid", gate_first=c["first"], residual=s["res"],
              scale=0.5, res_scale=s["ls"], out_weight=s["ow"])
    if c["form"] == "forward":
        return kda.norm_fwd(s["x"], **kw)
    return kda.norm_bwd(s["x"], s["dr"], s["dy"], **kw)


def run(s):
    if own:
        return run_own(s)
    return PLAIN[s["case"]["op"], s["case"]["form"]](s)


# ---------------------------------------------------------------------------
# plain forms: float32, one rounding at the end
# ---------------------------------------------------------------------------
def taps(s, j):
    """Input j of each token's window, [tokens, d]: from the tokens, from the state before the first one, or zero."""
    k, d = s["w"].shape[1], s["w"].shape[0]
    x = s["x"].reshape(-1, d).float()
    back = torch.arange(x.shape[0], device=DEV) - (k - 1) + j
    inside = (s["pos"] - (k - 1) + j >= 0)[:, None]
    early = 0.0
    if s["init"] is not None:
        early = s["init"].float()[s["seq"], (s["pos"] + j).clamp(max=k - 2)]
    return torch.where(inside, x[back.clamp(min=0)], early)


def conv_pre(s):
    return sum(s["w"][:, j] * taps(s, j) for j in range(s["w"].shape[1])) + s["b"]


def conv_last(s):
    """The last k - 1 inputs of each sequence, those of the earlier state where it is shorter."""
    k, d = s["w"].shape[1], s["w"].shape[0]
    p = s["len"][:, None] - (k - 1) + torch.arange(k - 1, device=DEV)
    x = s["x"].reshape(-1, d)[(s["first"][:, None] + p).clamp(min=0)]
    old = torch.gather(s["init"], 1, (p + k - 1).clamp(max=k - 2)[..., None].expand(-1, -1, d))
    return torch.where((p >= 0)[..., None], x, old)


def conv_prompt(s):
    u = conv_pre(s)
    y = u / (1 + torch.exp(-u))
    return y.to(s["x"].dtype).reshape(s["x"].shape), conv_last(s)


def conv_step(s):
    k, t = s["w"].shape[1], s["x"].shape[1]
    x = torch.cat([s["init"], s["x"]], 1)
    f = x.float()
    u = sum(s["w"][:, j] * f[:, j:j + t] for j in range(k)) + s["b"]
    y = u / (1 + torch.exp(-u))
    s["init"].copy_(x[:, t:])
    return y.to(s["x"].dtype), s["init"]


def conv_train(s):
    k, d = s["w"].shape[1], s["w"].shape[0]
    u = conv_pre(s)
    g = 1 / (1 + torch.exp(-u))
    du = s["dy"].reshape(-1, d).float() * (g * (1 + u * (1 - g)))
    n = du.shape[0]

    def part(j):  # what the outputs k - 1 - j tokens later give to each token's gradient
        ahead = torch.arange(n, device=DEV) + (k - 1 - j)
        inside = (s["pos"] + (k - 1 - j) < s["len"][s["seq"]])[:, None]
        return s["w"][:, j] * torch.where(inside, du[ahead.clamp(max=n - 1)], 0.0)

    dx = sum(part(j) for j in range(k))
    dw = torch.stack([(du * taps(s, j)).sum(0) for j in range(k)], 1)
    return dx.to(s["x"].dtype).reshape(s["x"].shape), dw, du.sum(0)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def sums_between(a):
    """[..., n] -> [..., n + 1, n + 1]: the sum of a[j .. i-1] at (i, j), j <= i, each summed by itself."""
    n = a.shape[-1]
    m = torch.arange(n + 1, device=DEV)
    x = torch.cat([torch.zeros_like(a[..., :1]), a], -1)[..., :, None] * (m[:, None] > m[None, :])
    return torch.cumsum(x, -2)


def scan_prompt(s):
    c = s["case"]
    h, g, ds, dx = c["h"], c["g"], c["ds"], c["dx"]
    rep = h // g
    tok, valid = s["tok"], s["valid"]
    nc, q = tok.shape
    x = s["x"].reshape(-1, h, dx).float()[tok]
    b = s["B"].reshape(-1, g, ds).float()[tok]
    cc = s["C"].reshape(-1, g, ds).float()[tok]
    dt = softplus(s["dt"].reshape(-1, h).float() + s["dtb"])[tok] * valid[..., None]
    la = (dt * s["A"]).permute(0, 2, 1)  # [chunks, heads, q]
    xw = (x * dt[..., None]).permute(0, 2, 1, 3)  # [chunks, heads, q, dx]
    cum = torch.cumsum(la, -1)
    m = torch.arange(q, device=DEV)
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(m[:, None] < m[None, :], -math.inf))
    cb = torch.einsum("cign,cjgn->cgij", cc, b).repeat_interleave(rep, 1)
    y = torch.matmul(cb * decay, xw)
    bh = b.permute(0, 2, 1, 3).repeat_interleave(rep, 1)  # [chunks, heads, q, ds]
    ch = cc.permute(0, 2, 1, 3).repeat_interleave(rep, 1)
    after = torch.flip(torch.cumsum(torch.flip(la, [-1]), -1), [-1]) - la  # decay from each token to its chunk's end
    local = torch.matmul((bh * torch.exp(after)[..., None]).transpose(-1, -2), xw)  # [chunks, heads, ds, dx]
    # states at the chunks' starts: decayed sums over the earlier chunks of the same sequence
    tot = cum[..., -1].transpose(0, 1)  # [heads, chunks]
    between = sums_between(tot)  # [heads, nc + 1, nc + 1]
    i = torch.arange(nc, device=DEV)
    same = (s["cseq"][:, None] == s["cseq"][None, :]) & (i[:, None] > i[None, :])
    mix = torch.exp(between[:, :nc, 1:].masked_fill(~same, -math.inf))
    start = torch.matmul(mix, local.transpose(0, 1).reshape(h, nc, ds * dx)).reshape(h, nc, ds, dx)
    since = torch.gather(between[:, :nc], 2, s["cfirst"][s["cseq"]][None, :, None].expand(h, -1, 1))
    start = start + torch.exp(since)[..., None] * s["h0"].transpose(0, 1)[:, s["cseq"]]
    start = start.transpose(0, 1)
    y = y + torch.matmul(ch * torch.exp(cum)[..., None], start)
    y = y.permute(0, 2, 1, 3) + s["D"][:, None] * x
    y = y.reshape(nc * q, h, dx)[s["back"]].reshape(s["x"].shape)
    last = s["clast"]
    end = torch.exp(tot.transpose(0, 1)[last])[..., None, None] * start[last] + local[last]
    return y.to(s["x"].dtype), end


def scan_step(s):
    c = s["case"]
    rep = c["h"] // c["g"]
    x = s["x"].float()
    dt = softplus(s["dt"].float() + s["dtb"])
    a = torch.exp(dt * s["A"])
    b = s["B"].float().repeat_interleave(rep, 2)
    cc = s["C"].float().repeat_interleave(rep, 2)
    state, kept, ys = s["h0"], s["h0"], []
    for t in range(c["t"]):
        state = a[:, t, :, None, None] * state + b[:, t, :, :, None] * (dt[:, t, :, None] * x[:, t])[:, :, None, :]
        ys.append((cc[:, t, :, :, None] * state).sum(2) + s["D"][:, None] * x[:, t])
        if s["commit"] is not None:
            kept = torch.where((s["commit"] == t + 1)[:, None, None, None], state, kept)
    s["h0"].copy_(state if s["commit"] is None else kept)
    return torch.stack(ys, 1).to(s["x"].dtype), s["h0"]


EPS = 1e-6
SCALE = 0.5


def act(name, z):
    g = 1 / (1 + torch.exp(-z))
    return g if name == "sigmoid" else z * g


def dact(name, z):
    g = 1 / (1 + torch.exp(-z))
    return g * (1 - g) if name == "sigmoid" else g * (1 + z * (1 - g))


def rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def norm_parts(s):
    """The branch's input to its norm, that norm's result, the gated branch and its sum with the residual."""
    c = s["case"]
    x = s["x"].float()
    z = act(c["gate"], s["gate"].float()) if c["gate"] else None
    v = x * z if c["gate"] and c["first"] else x
    m = v * rms(v) * s["w"]
    b = m * z if c["gate"] and not c["first"] else m
    r = SCALE * b
    if c["sandwich"]:
        r = s["res"].float() + s["ls"] * r
    return x, z, v, m, b, r


def norm_forward(s):
    *_, r = norm_parts(s)
    y = (r * rms(r) * s["ow"]).to(s["x"].dtype) if s["case"]["sandwich"] else None
    return r.to(s["x"].dtype), y


def rms_grad(dy, x, w):
    """Gradients of x * rms(x) * w for x and, summed over the rows, for w."""
    k = rms(x)
    n = x * k
    p = dy * w
    return k * (p - n * (p * n).mean(-1, keepdim=True)), (dy * n).reshape(-1, x.shape[-1]).sum(0)


def norm_train(s):
    c, t = s["case"], s["x"].dtype
    x, z, v, m, b, r = norm_parts(s)
    dr = s["dr"].float()
    dow = dls = dres = dgate = None
    if c["sandwich"]:
        more, dow = rms_grad(s["dy"].float(), r, s["ow"])
        dr = dr + more
        dres = dr.to(t)
        dls = (SCALE * dr * b).reshape(-1, c["d"]).sum(0)
        db = SCALE * s["ls"] * dr
    else:
        db = SCALE * dr
    dz = None
    dm = db
    if c["gate"] and not c["first"]:
        dz, dm = db * m, db * z
    dv, dw = rms_grad(dm, v, s["w"])
    dx = dv
    if c["gate"] and c["first"]:
        dz, dx = dv * x, dv * z
    if c["gate"]:
        dgate = (dz * dact(c["gate"], s["gate"].float())).to(t)
    return dx.to(t), dgate, dres, dw, dls, dow


PLAIN = {("conv", "prompt"): conv_prompt, ("conv", "step"): conv_step, ("conv", "train"): conv_train,
         ("scan", "prompt"): scan_prompt, ("scan", "step"): scan_step,
         ("norm", "forward"): norm_forward, ("norm", "train"): norm_train}


# ---------------------------------------------------------------------------
# work and exact results
# ---------------------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["heads"] * case["d"]
        fwd = 1 + bool(case["gate"]) + (3 if case["sandwich"] else 1)  # x, gate, residual in; r and y out
        if case["form"] == "forward":
            return {"bytes": n * e * fwd, "flops": n * (20 if case["sandwich"] else 10)}
        # x, gate, residual, dr, dy in; dx, dgate, dresidual out
        return {"bytes": n * e * (3 + 2 * bool(case["gate"]) + 3 * case["sandwich"]), "flops": n * (50 if case["sandwich"] else 25)}
    lens = lengths(case)
    n, tokens = len(lens), sum(lens)
    if case["op"] == "conv":
        d, k = case["d"], case["width"]
        state = 2 * n * (k - 1) * d * e
        if case["form"] == "train":
            return {"bytes": 3 * tokens * d * e + 8 * d * (k + 1), "flops": tokens * d * (6 * k + 10)}
        return {"bytes": 2 * tokens * d * e + state + 4 * d * (k + 1), "flops": tokens * d * (2 * k + 5)}
    h, g, ds, dx = case["h"], case["g"], case["ds"], case["dx"]
    flow = tokens * e * (2 * h * dx + 2 * g * ds + h)
    # each token updates a head's state and reads it: 2 multiply-adds per element
    return {"bytes": flow + 2 * 4 * n * h * ds * dx, "flops": tokens * h * 4 * ds * dx}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(s)
    return exact_conv(s) if case["op"] == "conv" else exact_scan(s)


def exact_norm(s):
    c = s["case"]
    need = c["form"] == "train"
    v = {k: s[k].double().requires_grad_(need) for k in ("x", "gate", "res", "w", "ls", "ow") if s[k] is not None}
    unit = lambda u: u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    gate = 1.0
    if c["gate"]:
        gate = torch.sigmoid(v["gate"]) if c["gate"] == "sigmoid" else torch.nn.functional.silu(v["gate"])
    b = unit(v["x"] * gate) * v["w"] if c["first"] else unit(v["x"]) * v["w"] * gate
    r, y = 0.5 * b, None
    if c["sandwich"]:
        r = v["res"] + v["ls"] * r
        y = unit(r) * v["ow"]
    if not need:
        return r, y
    loss = (r * s["dr"].double()).sum()
    if y is not None:
        loss = loss + (y * s["dy"].double()).sum()
    loss.backward()
    return tuple(v[k].grad if k in v else None for k in ("x", "gate", "res", "w", "ls", "ow"))


def exact_conv(s):
    c = s["case"]
    k, d = c["width"], c["d"]
    need = c["form"] == "train"
    x, w, b = (s[n].double().requires_grad_(need) for n in ("x", "w", "b"))
    flat = x.reshape(-1, d)
    if need:
        dy = s["dy"].double().reshape(-1, d)
    at, ys, last = 0, [], []
    total = [torch.zeros_like(t) for t in (x, w, b)]
    for i, n in enumerate(s["lens"]):
        seq = flat[at:at + n]
        before = s["init"][i].double() if s["init"] is not None else torch.zeros(k - 1, d, dtype=torch.float64, device=DEV)
        whole = torch.cat([before, seq], 0)
        u = sum(whole[j:j + n] * w[:, j] for j in range(k)) + b
        y = torch.nn.functional.silu(u)
        last.append(whole[n:])
        if need:  # one sequence's graph at a time
            for t, more in zip(total, torch.autograd.grad((y * dy[at:at + n]).sum(), (x, w, b), retain_graph=True)):
                t += more
        else:
            ys.append(y)
        at += n
    if need:
        return tuple(total)
    return torch.cat(ys, 0).reshape(s["x"].shape), torch.stack(last, 0)


def exact_scan(s):
    """Token by token, all sequences at once: past a sequence's end its state is left as it is."""
    c = s["case"]
    h, g, ds, dx = c["h"], c["g"], c["ds"], c["dx"]
    n, most = len(s["lens"]), max(s["lens"])
    steps = torch.arange(most, device=DEV)[:, None]
    inside = steps < s["len"]  # [most, n]
    at = torch.where(inside, s["first"] + steps, 0)
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    delta = torch.logaddexp(s["dt"].reshape(-1, h).double() + s["dtb"].double(), zero)[at] * inside[..., None]
    a = torch.exp(delta * s["A"].double()).reshape(most, n, g, h // g, 1, 1)
    x = s["x"].reshape(-1, h, dx)[at].double()
    xw = (x * delta[..., None]).reshape(most, n, g, h // g, 1, dx)
    b = s["B"].reshape(-1, g, ds)[at].double().reshape(most, n, g, 1, ds, 1)
    cc = s["C"].reshape(-1, g, ds)[at].double().reshape(most, n, g, 1, 1, ds)
    state = s["h0"].double().reshape(n, g, h // g, ds, dx)
    end, y = state, torch.empty(most, n, g, h // g, 1, dx, dtype=torch.float64, device=DEV)
    state = state.clone()
    for t in range(most):
        state.mul_(a[t]).addcmul_(b[t], xw[t])
        torch.matmul(cc[t], state, out=y[t])
        if s["commit"] is not None:
            end = torch.where((s["commit"] == t + 1)[:, None, None, None, None], state, end)
    y = y.reshape(most, n, h, dx) + s["D"].double()[:, None] * x
    out = torch.empty(sum(s["lens"]), h, dx, dtype=torch.float64, device=DEV)
    out[at[inside]] = y[inside]
    end = state if s["commit"] is None else end
    return out.reshape(s["x"].shape), end.reshape(n, h, ds, dx)
