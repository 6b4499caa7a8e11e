"""Cases, inputs and plain forms of the attention layers' operators in a hybrid stack.

Four operators, each with the forms that a user calls:

* ``qknorm``: norms of queries and keys per head with the position's rotation (forward, gradient);
* ``cache``: writing keys and values into a paged cache, in their type or in 8 bits, and reading them back
  (whole prompts, a few tokens of each running sequence);
* ``attn``: 1 to 8 new tokens of each sequence over its paged cache;
* ``verify``: drafted tokens against the target's probabilities, from given random numbers.

``run`` computes a case either in its plain form (elementary torch operations in float32, rounded
once at the end; angles in float64, sums of probabilities in exact fixed point) or, where ``own`` is
true, through the library's entry points.  ``exact`` gives the results from the definitions in float64.
"""
import itertools
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "int8": 1}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def lengths(case):
    """New tokens (cache) or keys (attn) of each sequence, drawn from [lo, hi] by the case's own seed."""
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def qknorm_case(name, form, tokens, hq, hk, d, rot, pairs, dtype, far):
    return {"name": name, "op": "qknorm", "form": form, "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "pairs": pairs, "dtype": dtype, "far": far}


def cache_case(name, n, lo, hi, before, h, d, page, dtype, kind, lens_seed):
    return {"name": name, "op": "cache", "form": "write_read", "n": n, "lo": lo, "hi": hi, "before": before, "h": h, "d": d,
            "page": page, "dtype": dtype, "kind": kind, "lens_seed": lens_seed}


def attn_case(name, n, t, lo, hi, hq, h, d, page, dtype, kind, window, lens_seed):
    return {"name": name, "op": "attn", "form": "step", "n": n, "t": t, "lo": lo, "hi": hi, "hq": hq, "h": h, "d": d,
            "page": page, "dtype": dtype, "kind": kind, "window": window, "lens_seed": lens_seed}


def verify_case(name, n, k, v, dtype, ragged, certain):
    return {"name": name, "op": "verify", "form": "sample", "n": n, "k": k, "v": v, "dtype": dtype, "ragged": ragged,
            "certain": certain}


def listed():
    return [
        # one token of 8 running sequences: 32 heads of queries, 8 of keys, far into their documents
        qknorm_case("qknorm_serve", "forward", 8, 32, 8, 128, 128, "halves", "bf16", 131072),
        # the fixed-length prefill batch, 4 x 4096 tokens
        qknorm_case("qknorm_prompt", "forward", 16384, 32, 8, 128, 128, "halves", "bf16", 4096),
        # a training step's gradients of the same, half of each head rotated, in adjacent pairs
        qknorm_case("qknorm_train", "train", 16384, 32, 8, 128, 64, "adjacent", "bf16", 4096),
        # the packed prefill batch's keys and values into 8-bit pages and back, behind shared prefixes
        cache_case("cache_prompt_e4m3", 16, 128, 8192, 512, 8, 128, 64, "bf16", "e4m3", 1002),
        # one token of each of 1024 running sequences
        cache_case("cache_step_int8", 1024, 1, 1, 5000, 8, 128, 64, "bf16", "int8", 1003),
        # a pool of 256 running sequences over 8-bit caches of the packed batch's lengths
        attn_case("attn_pool_e4m3", 256, 1, 128, 8192, 32, 8, 128, 64, "bf16", "e4m3", 0, 1004),
        # one long document of an odd number of tokens: few rows, a long axis
        attn_case("attn_long", 1, 1, 131071, 131071, 32, 8, 128, 64, "bf16", "bf16", 0, 1005),
        # 8 drafted tokens of 16 sequences, small pages
        attn_case("attn_draft_int8", 16, 8, 128, 32768, 32, 8, 128, 16, "bf16", "int8", 0, 1006),
        # the tiny float32 workload: two heads of 64, short caches
        attn_case("attn_tiny", 2, 1, 100, 256, 2, 2, 64, 16, "f32", "f32", 0, 1007),
        # 3 drafted tokens of 4 sequences: a latency-bound call over an odd vocabulary
        verify_case("verify_serve", 4, 3, 50257, "f32", False, False),
        # 7 drafted tokens of a pool of 256 sequences
        verify_case("verify_pool", 256, 7, 131072, "f32", True, False),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["qknorm", "cache", "attn", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    seed = rng.randrange(1 << 20)
    if op == "qknorm":
        d = rng.choice([64, 96, 128, 128, 256])
        hk = rng.choice([1, 2, 5, 8])
        hq = hk * rng.choice([1, 2, 4, 7])
        tokens = log(1, min(16384, (1 << 26) // ((hq + hk) * d)))
        c = qknorm_case("", rng.choice(["forward", "train"]), tokens, hq, hk, d, rng.choice([d, d, d // 2]),
                        rng.choice(["halves", "adjacent"]), dtype, log(100, 1 << 20))
    elif op == "cache":
        h, d, page = rng.choice([1, 2, 5, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        kind = rng.choice([dtype, "e4m3", "int8"])
        n = log(1, 1024)
        hi = log(1, max(2, min(8192, 65536 // n)))
        c = cache_case("", n, max(1, hi // 8), hi, rng.choice([0, log(1, 5000)]), h, d, page, dtype, kind, seed)
    elif op == "attn":
        h, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
        kind = rng.choice([dtype, "e4m3", "int8"])
        hq, t, n = h * rng.choice([1, 2, 4, 7, 8]), rng.choice([1, 1, 2, 5, 8]), log(1, 256)
        # half of the 8-bit pool's keys and values at most
        most = (1 << 30) // (n * h * d * 2 * SIZE[kind]) // (4 if dtype == "f32" else 1)
        hi = log(t + 1, max(t + 2, min(131072, most)))
        c = attn_case("", n, t, max(t, hi // 32), hi, hq, h, d, page, dtype, kind, rng.choice([0, 0, log(1, 4096)]), seed)
    else:
        n, v = log(1, 256), rng.choice([1, 8]) * log(125, 16384)
        c = verify_case("", n, rng.choice([1, 2, 3, 5, 7]), v, dtype, rng.random() < 0.5, rng.random() < 0.25)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def offsets(lens):
    return [0] + list(itertools.accumulate(lens))


def paged(s, case, total, gen):
    """A pool of pages, more than the sequences need, and each sequence's pages in no order."""
    n, page = len(total), case["page"]
    most = max(-(-x // page) for x in total)
    pool = n * most + 3
    ids = torch.randperm(pool, device=DEV, generator=gen)[:n * most].to(torch.int32)
    s["pages"] = ids.reshape(n, most)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    s["total"] = total
    shape, kind = (pool, case["h"], page, case["d"]), KINDS[case["kind"]]
    out = []
    for _ in range(2):
        if case["kind"] in ("bf16", "f32"):
            out.append((torch.randn(shape, device=DEV, generator=gen).to(kind), None))
        else:  # codes as written from normal values: the largest of a row near the type's largest
            top = 448 if case["kind"] == "e4m3" else 127
            code = torch.empty(shape, dtype=kind, device=DEV)
            for i in range(0, pool, 4096):
                x = torch.randn((min(4096, pool - i), *shape[1:]), device=DEV, generator=gen)
                x = (x * (top / 5)).clamp(-top, top)
                code[i:i + 4096] = (torch.round(x) if case["kind"] == "int8" else x).to(kind)
            byte = (120 if case["kind"] == "e4m3" else 122) + torch.randint(0, 2, shape[:3], device=DEV, generator=gen)
            out.append((code, byte.to(torch.uint8)))
    s["cache"] = (out[0][0], out[1][0], out[0][1], out[1][1])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    f = dict(device=DEV, dtype=torch.float32, generator=gen)
    s = {"case": case}
    if case["op"] == "qknorm":
        n, d = case["tokens"], case["d"]
        for name, h in (("q", case["hq"]), ("k", case["hk"])):
            s[name] = torch.randn(n, h, d, **f).to(dt)
            s[name + "w"] = 1 + 0.1 * torch.randn(d, **f)
            if case["form"] == "train":
                s["d" + name] = torch.randn(n, h, d, **f).to(dt)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
        s["freqs"] = 10000.0 ** (-2 * i / case["rot"])
        if n <= 1024:  # single tokens anywhere in their documents, else prompts one after the other
            s["pos"] = torch.randint(0, case["far"], (n,), device=DEV, generator=gen, dtype=torch.int32)
        else:
            s["pos"] = (torch.arange(n, device=DEV) % case["far"]).to(torch.int32)
        return s
    if case["op"] == "verify":
        n, k, v = case["n"], case["k"], case["v"]
        logits = 2 * torch.randn(n, k + 1, v, **f)
        s["p"] = torch.softmax(logits, -1).to(dt)
        near = torch.softmax(logits[:, :k] + 0.5 * torch.randn(n, k, v, **f), -1)
        del logits
        s["drafts"] = torch.multinomial(near.reshape(n * k, v), 1, generator=gen).reshape(n, k).to(torch.int32)
        s["q"] = near.to(dt)
        if case["certain"]:  # drafted without probabilities (copied from the text): often the target's likely token
            top = s["p"][:, :k].argmax(-1).to(torch.int32)
            s["drafts"] = torch.where(torch.rand(n, k, **f) < 0.8, top, s["drafts"])
            s["q"] = None
        s["u"] = torch.rand(n, k + 1, **f)
        s["counts"] = None
        if case["ragged"]:
            s["counts"] = torch.randint(0, k + 1, (n,), device=DEV, generator=gen, dtype=torch.int32)
        return s
    lens = lengths(case)
    n = len(lens)
    if case["op"] == "cache":
        cu = offsets(lens)
        total = cu[-1]
        paged(s, case, [x + case["before"] for x in lens], gen)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["k"] = torch.randn(1, total, case["h"], case["d"], **f).to(dt)
        s["v"] = torch.randn(1, total, case["h"], case["d"], **f).to(dt)
        # where each token goes (the plain form's plan)
        seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(lens, device=DEV), output_size=total)
        s["seq"] = seq
        s["at"] = torch.arange(total, device=DEV) - torch.tensor(cu[:-1], device=DEV)[seq] + case["before"]
        return s
    paged(s, case, lens, gen)
    s["q"] = torch.randn(n, case["t"], case["hq"], case["d"], **f).to(dt)
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def run_own(s):
    import kda_delta_rule_fwd_gb300 as kda
    c = s["case"]
    if c["op"] == "qknorm":
        kw = dict(q_weight=s["qw"], k_weight=s["kw"], interleaved=c["pairs"] == "adjacent", eps=EPS)
        if c["form"] == "forward":
            return kda.qknorm_fwd(s["q"], s["k"], s["pos"], s["freqs"], **kw)
        return kda.qknorm_bwd(s["q"], s["k"], s["dq"], s["dk"], s["pos"], s["freqs"], **kw)
    if c["op"] == "cache":
        cache = kda.KVCache(*s["cache"])
        kda.cache_write(s["k"], s["v"], cache, s["pages"], s["lens"], cu_seqlens=s["cu"])
        return kda.cache_read(cache, s["pages"], s["lens"], s["k"].shape[1], cu_seqlens=s["cu"], dtype=s["k"].dtype)
    if c["op"] == "attn":
        return kda.attn_step(s["q"], kda.KVCache(*s["cache"]), s["pages"], s["lens"], window=c["window"])
    return kda.draft_verify(s["p"], s["q"], s["drafts"], s["u"], num_draft=s["counts"])


def run(s):
    if own:
        return run_own(s)
    return PLAIN[s["case"]["op"], s["case"]["form"]](s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def rotation(s):
    a = s["pos"].double()[:, None] * s["freqs"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def split(case, x):
    """The two members of each pair, and the channels that stay."""
    r = case["rot"]
    if case["pairs"] == "halves":
        return x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]


def merge(case, a, b, rest):
    both = torch.cat([a, b], -1) if case["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([both, rest], -1)


def qknorm_forward(s):
    cos, sin = rotation(s)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        f = x.float()
        a, b, rest = split(s["case"], f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w)
        out.append(merge(s["case"], a * cos - b * sin, a * sin + b * cos, rest).to(x.dtype))
    return tuple(out)


def qknorm_train(s):
    cos, sin = rotation(s)
    dx, dw = [], []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        f = x.float()
        k = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        n = f * k
        a, b, rest = split(s["case"], dy.float())
        g = merge(s["case"], a * cos + b * sin, b * cos - a * sin, rest)
        p = g * w
        dx.append((k * (p - n * (p * n).mean(-1, keepdim=True))).to(x.dtype))
        dw.append((g * n).sum((0, 1)))
    return (*dx, *dw)


def power(b):
    """2^(b - 127) from its byte."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def encode(x, kind):
    """Codes and bytes of rows: the smallest power of two that brings a row into the type's range."""
    f = x.float()
    part, e = torch.frexp(f.abs().amax(-1))  # part in [1/2, 1)
    top, shift = (0.875, 9) if kind == "e4m3" else (127 / 128, 7)
    e = (e - shift + (part > top).to(torch.int32)).clamp(min=-126)
    e = torch.where(part == 0, -126, e)
    y = f * ((127 - e) << 23).view(torch.float32)[..., None]
    y = torch.round(y) if kind == "int8" else y
    return y.to(KINDS[kind]), (e + 127).to(torch.uint8)


def cache_write_read(s):
    c = s["case"]
    page = s["pages"][s["seq"], s["at"] // c["page"]].long()
    off = s["at"] % c["page"]
    out = []
    for i, x in enumerate((s["k"], s["v"])):
        held, scale = s["cache"][i], s["cache"][i + 2]
        if scale is None:
            held[page, :, off] = x[0].to(held.dtype)
            out.append(held[page, :, off].to(x.dtype)[None])
            continue
        code, b = encode(x[0], c["kind"])
        held.view(torch.uint8)[page, :, off] = code.view(torch.uint8)
        scale[page, :, off] = b
        back = held.view(torch.uint8)[page, :, off].view(held.dtype).float() * power(scale[page, :, off])[..., None]
        out.append(back.to(x.dtype)[None])
    return tuple(out)


def attn_step(s):
    c = s["case"]
    n, t, h, d, page = c["n"], c["t"], c["h"], c["d"], c["page"]
    rep = c["hq"] // h
    most = max(s["total"])
    some = max(1, (1 << 29) // (most * h * d))
    outs = []
    for i in range(0, n, some):
        ids = s["pages"][i:i + some, :-(-most // page)].long()
        m, keys = ids.shape[0], ids.shape[1] * page

        def rows(held, scale):
            x = held.view(torch.uint8)[ids].view(held.dtype).float() if scale is not None else held[ids].float()
            if scale is not None:
                x = x * power(scale[ids])[..., None]
            return x.permute(0, 2, 1, 3, 4).reshape(m, h, keys, d)

        q = s["q"][i:i + some].float().reshape(m, t, h, rep, d).permute(0, 2, 1, 3, 4).reshape(m, h, t * rep, d)
        sc = torch.matmul(q, rows(s["cache"][0], s["cache"][2]).transpose(-1, -2)) * d ** -0.5
        at = torch.arange(keys, device=DEV)
        last = s["lens"][i:i + some, None].long() - t + torch.arange(t, device=DEV)  # [m, t]
        seen = at <= last[..., None]
        if c["window"]:
            seen &= at > last[..., None] - c["window"]
        sc = sc.reshape(m, h, t, rep, keys).masked_fill(~seen[:, None, :, None], -math.inf)
        top = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
        inside = (at < s["lens"][i:i + some, None])[:, None, :, None]
        v = torch.where(inside, rows(s["cache"][1], s["cache"][3]), 0.0)
        o = torch.matmul(p.reshape(m, h, t * rep, keys), v)
        z = p.sum(-1).reshape(m, h, t * rep, 1)
        o = torch.where(z > 0, o / z, 0.0).reshape(m, h, t, rep, d).permute(0, 2, 1, 3, 4)
        outs.append(o.reshape(m, t, c["hq"], d).to(s["q"].dtype))
    return torch.cat(outs, 0)


def fixed(p):
    """Probabilities as whole multiples of 2^-44."""
    return torch.round(p.double().clamp(0, 1) * 2.0 ** 44).to(torch.int64)


def verify_sample(s):
    c = s["case"]
    n, k = c["n"], c["k"]
    d = s["drafts"].long()
    have = s["counts"].long() if s["counts"] is not None else torch.full((n,), k, device=DEV)
    pd = torch.gather(s["p"][:, :k], 2, d[..., None])[..., 0].double()
    qd = torch.gather(s["q"], 2, d[..., None])[..., 0].double() if s["q"] is not None else torch.ones_like(pd)
    ok = (s["u"][:, :k].double() * qd < pd) & (torch.arange(k, device=DEV) < have[:, None])
    kept = torch.cumprod(ok.long(), 1).sum(1)
    at = torch.arange(n, device=DEV)
    p = fixed(s["p"][at, kept])
    w = p
    row = kept.clamp(max=k - 1)
    if s["q"] is not None:
        less = fixed(s["q"][at, row])
    else:
        less = torch.zeros_like(p).scatter_(1, d[at, row][:, None], 1 << 44)
    w = torch.where((kept < have)[:, None], (p - less).clamp(min=0), p)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    total = w.sum(1)
    m = (s["u"][:, k].double() * 2 ** 24).long()
    place = m * (total >> 24) + ((m * (total & (2 ** 24 - 1))) >> 24)
    more = (torch.cumsum(w, 1) <= place[:, None]).sum(1)
    i = torch.arange(k + 1, device=DEV)
    pad = torch.cat([d, d[:, :1]], 1)
    tokens = torch.where(i < kept[:, None], pad, torch.where(i == kept[:, None], more[:, None], -1))
    return tokens.to(torch.int32), (kept + 1).to(torch.int32)


PLAIN = {("qknorm", "forward"): qknorm_forward, ("qknorm", "train"): qknorm_train,
         ("cache", "write_read"): cache_write_read, ("attn", "step"): attn_step, ("verify", "sample"): verify_sample}


# ---------------------------------------------------------------------------
# work and exact results
# ---------------------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "qknorm":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["d"]
        if case["form"] == "forward":
            return {"bytes": 2 * n * e + 4 * case["tokens"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 4 * case["tokens"], "flops": 18 * n}
    if case["op"] == "verify":
        # the drafts' own probabilities, and the rows of the one place where a token is drawn
        rows = case["n"] * case["v"] * (1 if case["certain"] else 2)
        return {"bytes": rows * e + 20 * case["n"] * (case["k"] + 1), "flops": 4 * rows}
    lens = lengths(case)
    row = case["h"] * (case["d"] * SIZE[case["kind"]] + (case["kind"] in ("e4m3", "int8")))  # a token's keys (or values), held
    if case["op"] == "cache":
        n = 2 * sum(lens)
        return {"bytes": 2 * n * (case["h"] * case["d"] * e + row), "flops": 4 * n * case["h"] * case["d"]}
    t, w = case["t"], case["window"]
    keys = sum(min(x, w + t - 1) if w else x for x in lens)
    seen = sum(min(x - t + 1 + j, w) if w else x - t + 1 + j for x in lens for j in range(t))
    return {"bytes": 2 * keys * row + 2 * len(lens) * t * case["hq"] * case["d"] * e, "flops": 4 * seen * case["hq"] * case["d"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qknorm": exact_qknorm, "cache": exact_cache, "attn": exact_attn, "verify": exact_verify}[case["op"]](s)


def exact_qknorm(s):
    c = s["case"]
    need = c["form"] == "train"
    r = c["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["pos"].double(), s["freqs"]))[:, None]
    order = torch.arange(r, device=DEV)
    if c["pairs"] == "halves":
        order = order.reshape(2, r // 2).T.flatten()  # the channels, pair by pair
    back = torch.argsort(order)
    out = []
    for name in ("q", "k"):
        x, w = s[name].double().requires_grad_(need), s[name + "w"].double().requires_grad_(need)
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        z = torch.view_as_complex(y[..., order].unflatten(-1, (r // 2, 2))) * turn
        y = torch.cat([torch.view_as_real(z).flatten(-2)[..., back], y[..., r:]], -1)
        out.append(torch.autograd.grad((y * s["d" + name].double()).sum(), (x, w)) if need else y)
    if need:
        return out[0][0], out[1][0], out[0][1], out[1][1]
    return tuple(out)


def exact_cache(s):
    c = s["case"]
    out = []
    for x in (s["k"], s["v"]):
        x = x.double()
        if c["kind"] in ("bf16", "f32"):
            out.append(x.to(KINDS[c["kind"]]).double())
            continue
        top = 448.0 if c["kind"] == "e4m3" else 127.0
        most = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -200) / top))
        e = torch.where(most > top * torch.exp2(e), e + 1, e)  # where the logarithm was rounded across
        e = torch.where(most <= top * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
        y = x * torch.exp2(-e)
        if c["kind"] == "int8":
            step = torch.ones_like(y)
        else:  # 3 bits below the leading one, and no finer than 2^-9
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        out.append(torch.round(y / step) * step * torch.exp2(e))
    return tuple(out)


def exact_attn(s):
    c = s["case"]
    t, rep, page, d = c["t"], c["hq"] // c["h"], c["page"], c["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)

    def rows(held, scale, ids, n):
        x = held.view(torch.uint8)[ids].view(held.dtype) if scale is not None else held[ids]
        x = x.to(torch.float64 if held.dtype != torch.float8_e4m3fn else torch.float32).double()
        if scale is not None:
            x = x * torch.exp2(scale[ids].double() - 127)[..., None]
        return x.transpose(1, 2).reshape(-1, c["h"], d)[:n].transpose(0, 1)

    for i, n in enumerate(s["total"]):
        ids = s["pages"][i, :-(-n // page)].long()
        k = rows(s["cache"][0], s["cache"][2], ids, n)
        v = rows(s["cache"][1], s["cache"][3], ids, n)
        for j in range(t):
            hi = n - t + 1 + j
            lo = max(0, hi - c["window"]) if c["window"] else 0
            q = s["q"][i, j].double().reshape(c["h"], rep, d)
            p = torch.softmax(torch.einsum("hrd,hkd->hrk", q, k[:, lo:hi]) / math.sqrt(d), -1)
            out[i, j] = torch.einsum("hrk,hkd->hrd", p, v[:, lo:hi]).reshape(c["hq"], d)
    return out


def exact_verify(s):
    """One sequence after the other, from float64 probabilities."""
    c = s["case"]
    k = c["k"]
    tokens = torch.full((c["n"], k + 1), -1, dtype=torch.int32)
    commit = torch.zeros(c["n"], dtype=torch.int32)
    for b in range(c["n"]):
        drafts, u = s["drafts"][b].tolist(), s["u"][b].double().tolist()
        have = k if s["counts"] is None else int(s["counts"][b])
        kept = 0
        while kept < have:
            d = drafts[kept]
            q = 1.0 if s["q"] is None else float(s["q"][b, kept, d])
            if not u[kept] * q < float(s["p"][b, kept, d]):
                break
            tokens[b, kept] = d
            kept += 1
        w = s["p"][b, kept].double()
        if kept < have:
            if s["q"] is not None:
                rest = torch.relu(w - s["q"][b, kept].double())
            else:
                rest = w.clone()
                rest[drafts[kept]] = 0
            w = rest if float(rest.sum()) > 0 else w
        up = torch.cumsum(w, 0)
        tokens[b, kept] = int(torch.searchsorted(up, u[k] * up[-1:], right=True).clamp(max=int((w > 0).nonzero()[-1])))
        commit[b] = kept + 1
    return tokens.to(DEV), commit.to(DEV)
