"""GPU parity of the operators around the recurrence (convolution, scan, norms)
against plain float64 forms, at the sizes and boundaries where they can go wrong.

Tolerances, element by element (see _layer_ref.close), from the arithmetic:
* float32 results of a few float32 operations (convolution, norms): each rounds by
  2^-24 of its operands; sums of up to 8192 terms in trees and the fast exponential
  and division stay under 50 such roundings of the result's scale: 3e-6, doubled for
  the parts that cancel: rel 6e-6, rms 6e-6.
* bf16 results: half an ulp, 2^-9 of the result, on top of that: rel 2^-8, rms 6e-6.
* scan in float32: the state and the output are sums over the tokens and the state
  rows, whose terms cancel: 1e-4 of the rms, the package's float32 bound.
* scan on bf16 inputs: the package's bound for bf16 inputs, 1e-2 of the rms, on y
  (operands rounded to bf16 inside); the state keeps 16 bits of each update, 1e-4.
* sums over rows or tokens (parameter gradients): float32 sums in fixed order,
  n 2^-24 in the worst case and far less in a tree: rms 3e-5.
"""
import itertools

import pytest
import torch

import _layer_ref as ref
from _layer_ref import close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TIGHT = {F32: dict(rel=6e-6, rms=6e-6), BF: dict(rel=2.0 ** -8, rms=6e-6)}
SCAN_Y = {F32: dict(rel=0, rms=1e-4), BF: dict(rel=2.0 ** -8, rms=1e-2)}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def cu_of(lens):
    return torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32, device=DEV)


def cut(t, wide, at):
    """The same values as a column slice of a wider, NaN-filled tensor."""
    lead, inner = t.shape[:2], t.shape[2:]
    n = inner.numel()
    big = torch.full((*lead, wide), float("nan"), dtype=t.dtype, device=DEV)
    big[..., at:at + n] = t.reshape(*lead, n).to(DEV)
    return big[..., at:at + n].unflatten(-1, inner) if len(inner) > 1 else big[..., at:at + n]


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------
CONV_LENS = [None, [1, 0, 2, 3, 0, 64, 65, 0, 130], [0, 0, 5], [700]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [8, 1032, 37])
@pytest.mark.parametrize("lens", CONV_LENS)
def test_conv(kda, dtype, W, D, lens):
    g = gen(W * 1000 + D)
    B, T = (3, 77) if lens is None else (1, sum(lens))
    N = B if lens is None else len(lens)
    silu, with_bias, with_init = D != 37, W != 3, W != 2
    x, w = rnd(g, B, T, D, dtype=dtype), rnd(g, D, W)
    b = rnd(g, D) if with_bias else None
    init = rnd(g, N, W - 1, D, dtype=dtype) if with_init else None
    dev = lambda t: None if t is None else t.to(DEV)
    cu = None if lens is None else cu_of(lens)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    act = "silu" if silu else None
    y, fin = kda.conv_fwd(dev(x), dev(w), dev(b), activation=act, cu_seqlens=cu,
                          init_state=dev(init), workspace=ws)
    ry, rf = ref.conv(x, w, b, silu=silu, lens=lens, init=init)
    close(y, ry, what="y", **TIGHT[dtype])
    assert torch.equal(fin.cpu().to(torch.float64), rf), "the state is a copy of inputs"
    assert kda.read_device_status(ws) == kda.KDA_OK
    # gradients
    dy, df = rnd(g, B, T, D, dtype=dtype), rnd(g, N, W - 1, D, dtype=dtype)
    ps = [t.to(torch.float64).requires_grad_() if t is not None else None for t in (x, w, b, init)]
    ry, rf = ref.conv(ps[0], ps[1], ps[2], silu=silu, lens=lens, init=ps[3])
    ((ry * dy.double()).sum() + (rf * df.double()).sum()).backward()
    dx, dw, db, di = kda.conv_bwd(dev(x), dev(w), dev(dy), dev(b), activation=act, cu_seqlens=cu,
                                  init_state=dev(init), dfinal=dev(df), want_dinit=True)
    close(dx, ps[0].grad, what="dx", **TIGHT[dtype])
    close(dw, ps[1].grad, rel=6e-6, rms=3e-5, what="dw")
    if with_bias:
        close(db, ps[2].grad, rel=6e-6, rms=3e-5, what="db")
    else:
        assert db is None
    if with_init:
        close(di, ps[3].grad, what="dinit", **TIGHT[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("D", [40, 2048, 13])
def test_conv_step(kda, dtype, T, D):
    g = gen(T + D)
    N, W = 5, 2 + T % 3
    x, w, b = rnd(g, N, T, D, dtype=dtype).to(DEV), rnd(g, D, W).to(DEV), rnd(g, D).to(DEV)
    init = rnd(g, N, W - 1, D, dtype=dtype).to(DEV)
    state = init.clone()
    y = kda.conv_step(x, w, state, b, activation="silu")
    ry, rf = ref.conv(x.cpu(), w.cpu(), b.cpu(), silu=True, init=init.cpu())
    close(y, ry, what="y", **TIGHT[dtype])
    assert torch.equal(state.cpu().double(), rf)
    # commit counts: outputs of every token, the state of the kept prefix
    keep = torch.tensor([0, T, T // 2, 1, max(0, T - 1)], dtype=torch.int32, device=DEV)
    kept = init.clone()
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    y2 = kda.conv_step(x, w, kept, b, activation="silu", num_commit=keep, workspace=ws)
    assert torch.equal(y2, y) and kda.read_device_status(ws) == kda.KDA_OK
    for n, k in enumerate(keep.tolist()):
        one = init[n:n + 1].clone()
        if k:
            kda.conv_step(x[n:n + 1, :k].contiguous(), w, one, b, activation="silu")
        assert torch.equal(kept[n:n + 1], one)
    again = init.clone()
    assert kda.conv_step(x, w, again, b, num_commit=keep, want_out=False) is None
    assert torch.equal(again, kept)
    # a count outside 0..T is reported and leaves its state alone
    bad = keep.clone()
    bad[1], bad[2] = T + 1, -1
    other = init.clone()
    kda.conv_step(x, w, other, b, activation="silu", num_commit=bad, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(other[1:3], init[1:3]) and torch.equal(other[3:], kept[3:])


def test_conv_prompt_then_steps(kda):
    """A prompt's state continues in single tokens exactly as one longer prompt."""
    g = gen(5)
    x, w, b = rnd(g, 2, 40, 64, dtype=BF).to(DEV), rnd(g, 64, 4).to(DEV), rnd(g, 64).to(DEV)
    whole, end = kda.conv_fwd(x, w, b, activation="silu")
    part, state = kda.conv_fwd(x[:, :30].contiguous(), w, b, activation="silu")
    rest = [kda.conv_step(x[:, t:t + 1].contiguous(), w, state, b, activation="silu")
            for t in range(30, 40)]
    assert torch.equal(torch.cat([part, *rest], 1), whole) and torch.equal(state, end)


@pytest.mark.parametrize("at", [0, 3, 8])
def test_conv_strided_and_poisoned(kda, at):
    """A column slice of a wider tensor gives the same bits, and what is outside it (NaN here),
    like NaN in a neighbouring sequence, is never used."""
    g = gen(6)
    lens = [33, 7, 50]
    x, w = rnd(g, 1, 90, 48, dtype=BF).to(DEV), rnd(g, 48, 4).to(DEV)
    cu = cu_of(lens)
    y, s = kda.conv_fwd(x, w, cu_seqlens=cu)
    y2, s2 = kda.conv_fwd(cut(x.cpu(), 48 + 16, at), w, cu_seqlens=cu)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    dy = rnd(g, 1, 90, 48, dtype=BF).to(DEV)
    for a, b in zip(kda.conv_bwd(x, w, dy, cu_seqlens=cu)[:2],
                    kda.conv_bwd(cut(x.cpu(), 48 + 16, at), w, dy, cu_seqlens=cu)[:2]):
        assert torch.equal(a, b)
    bad = x.clone()
    bad[:, 33:40] = float("nan")
    y3, s3 = kda.conv_fwd(bad, w, cu_seqlens=cu)
    assert torch.equal(y3[:, :33], y[:, :33]) and torch.equal(y3[:, 40:], y[:, 40:])
    assert torch.equal(s3[[0, 2]], s[[0, 2]]) and y3[:, 33:40].isnan().all()
    dx = kda.conv_bwd(x, w, dy, cu_seqlens=cu, activation="silu")[0]
    dx3 = kda.conv_bwd(bad, w, dy, cu_seqlens=cu, activation="silu")[0]
    assert torch.equal(dx3[:, :33], dx[:, :33]) and torch.equal(dx3[:, 40:], dx[:, 40:])


# ---------------------------------------------------------------------------
# scan
# ---------------------------------------------------------------------------
def scan_inputs(seed, B, T, H, G, ds, dx, dtype, N, fast=False):
    g = gen(seed)
    x = rnd(g, B, T, H, dx, dtype=dtype)
    Bm, C = (rnd(g, B, T, G, ds, dtype=dtype, std=ds ** -0.25) for _ in range(2))
    dt = rnd(g, B, T, H, dtype=dtype, std=4.0 if fast else 1.0)
    A = -torch.exp(torch.rand(H, generator=g) * (5 if fast else 2.77))
    return dict(x=x, dt=dt, A=A, B=Bm, C=C, D=rnd(g, H), bias=rnd(g, H) - 2,
                h0=rnd(g, N, H, ds, dx))


def scan_call(kda, v, *, cu=None, softplus=True, **kw):
    d = {k: t.to(DEV) for k, t in v.items()}
    return kda.scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"],
                        dt_bias=d["bias"] if softplus else None, dt_softplus=softplus,
                        cu_seqlens=cu, h0=d["h0"], **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ds,dx", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("B,T,lens", [(2, 1, None), (1, 63, None), (2, 64, None), (1, 65, None),
                                      (2, 129, None), (1, 200, None),
                                      (1, 0, [1, 0, 17, 64, 0, 66, 128, 30])])
def test_scan(kda, dtype, ds, dx, B, T, lens):
    G, H = (2, 6) if ds == 128 else (1, 3)
    T = T if lens is None else sum(lens)
    N = B if lens is None else len(lens)
    v = scan_inputs(ds + dx + T, B, T, H, G, ds, dx, dtype, N)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    y, hT = scan_call(kda, v, cu=None if lens is None else cu_of(lens), out_dtype=dtype,
                      workspace=ws)
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"],
                      softplus=True, lens=lens, h0=v["h0"])
    assert kda.read_device_status(ws) == kda.KDA_OK
    close(y, ry, what="y", **SCAN_Y[dtype])
    close(hT, rh, rel=0, rms=1e-4, what="hT")
    # the other output type: the same values, rounded or not
    other = BF if dtype == F32 else F32
    y2, h2 = scan_call(kda, v, cu=None if lens is None else cu_of(lens), out_dtype=other)
    assert torch.equal(h2, hT)
    assert torch.equal(y2.to(BF), y.to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_strong_and_zero_decay(kda, dtype):
    """Steps from 0 (softplus far below: the state is kept) to hundreds (it is forgotten)."""
    v = scan_inputs(3, 2, 150, 4, 2, 128, 64, dtype, 2, fast=True)
    v["dt"][:, 20:40] = -200.0
    v["dt"][:, 60:64] = 300.0
    v["A"][1] = 0.0
    v["A"][2] = -1e4
    y, hT = scan_call(kda, v, out_dtype=dtype)
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"],
                      softplus=True, h0=v["h0"])
    for h in range(4):  # heads differ by orders of magnitude: each against its own scale
        close(y[:, :, h], ry[:, :, h], what=f"y {h}", **SCAN_Y[dtype])
        close(hT[:, h], rh[:, h], rel=0, rms=1e-4, what=f"hT {h}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_plain_steps_and_defaults(kda, dtype):
    """dt as given (no softplus), no skip, no start state, no final state wanted."""
    v = scan_inputs(4, 1, 100, 2, 1, 64, 64, dtype, 1)
    v["dt"] = v["dt"].abs() * 0.1
    d = {k: t.to(DEV) for k, t in v.items()}
    y, hT = kda.scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], output_final_state=False,
                         out_dtype=dtype)
    assert hT is None
    ry, _ = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"])
    close(y, ry, what="y", **SCAN_Y[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_strided_and_poisoned(kda, dtype):
    """Slices of one projection [x | B | C | dt], at any alignment, and NaN in the sequence between."""
    lens = [70, 10, 90]
    v = scan_inputs(7, 1, 170, 4, 2, 64, 64, dtype, 3)
    cu = cu_of(lens)
    y, hT = scan_call(kda, v, cu=cu, out_dtype=dtype)
    for pad in (8, 3):
        s = dict(v)
        for k, at in (("x", pad), ("B", 0), ("C", pad), ("dt", 1)):
            s[k] = cut(v[k], v[k].shape[2:].numel() + 16, at)
        y2, h2 = scan_call(kda, s, cu=cu, out_dtype=dtype)
        if pad == 8:
            assert torch.equal(y2, y) and torch.equal(h2, hT)
        else:  # an unaligned slice may take another path
            close(y2, y, what="y", **SCAN_Y[dtype])
            close(h2, hT, rel=0, rms=1e-4, what="hT")
    for k in ("x", "B", "C", "dt"):
        bad = {n: t.clone() for n, t in v.items()}
        bad[k][:, 70:80] = float("nan")
        y3, h3 = scan_call(kda, bad, cu=cu, out_dtype=dtype)
        assert torch.equal(y3[:, :70], y[:, :70]) and torch.equal(y3[:, 80:], y[:, 80:]), k
        assert torch.equal(h3[[0, 2]], hT[[0, 2]]), k


def test_scan_state_in_place(kda):
    v = scan_inputs(8, 2, 90, 2, 1, 128, 128, BF, 2)
    y, hT = scan_call(kda, v, out_dtype=BF)
    d = {k: t.to(DEV) for k, t in v.items()}
    y2, h2 = kda.scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"],
                          dt_softplus=True, h0=d["h0"], hT=d["h0"], out_dtype=BF)
    assert h2 is d["h0"] and torch.equal(h2, hT) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ds,dx", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_scan_step(kda, dtype, ds, dx, T):
    N, H, G = 4, 6, 3
    v = scan_inputs(T + ds + dx, N, T, H, G, ds, dx, dtype, N)
    d = {k: t.to(DEV) for k, t in v.items()}
    call = lambda state, **kw: kda.scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], state,
                                             D=d["D"], dt_bias=d["bias"], dt_softplus=True, **kw)
    state = d["h0"].clone()
    y = call(state)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"])
    ry, rh = ref.scan(*args, bias=v["bias"], softplus=True, h0=v["h0"])
    # every product and sum in float32: the package's float32 bound holds for both input types
    close(y, ry, rel=0, rms=1e-4, what="y")
    close(state, rh, rel=0, rms=1e-4, what="state")
    keep = torch.tensor([0, T, T // 2, 1], dtype=torch.int32, device=DEV)
    kept = d["h0"].clone()
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    y2 = call(kept, num_commit=keep, workspace=ws, out_dtype=BF)
    assert torch.equal(y2, y.to(BF)) and kda.read_device_status(ws) == kda.KDA_OK
    _, rk = ref.scan(*args, bias=v["bias"], softplus=True, h0=v["h0"], keep=keep.tolist())
    close(kept, rk, rel=0, rms=1e-4, what="kept")
    assert torch.equal(kept[0], d["h0"][0]) and torch.equal(kept[1], state[1])
    again = d["h0"].clone()
    assert call(again, num_commit=keep, want_out=False) is None and torch.equal(again, kept)
    bad = torch.tensor([T + 1, T, -1, 1], dtype=torch.int32, device=DEV)
    other = d["h0"].clone()
    call(other, num_commit=bad, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(other[[0, 2]], d["h0"][[0, 2]]) and torch.equal(other[[1, 3]], kept[[1, 3]])


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
NORMS = {
    "plain": dict(w=1),
    "gated": dict(w=1, gate="sigmoid"),
    "gate first": dict(w=1, gate="silu", first=True),
    "no norm": dict(gate="silu", res=1),
    "pre": dict(res=1, ow=1),
    "sandwich": dict(w=1, res=1, ls=1, ow=1, scale=0.5),
    "all after": dict(w=1, gate="silu", res=1, ls=1, ow=1, scale=0.5),
    "all first": dict(w=1, gate="sigmoid", first=True, res=1, ls=1, ow=1, scale=-1.5),
}


@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 64), (5, 127), (33, 128), (7, 192), (4, 1000),
                                    (2, 1024), (3, 4096), (2, 4099), (2, 8192), (700, 96)])
@pytest.mark.parametrize("kind", list(NORMS))
def test_norm(kda, dtype, rdtype, rows, d, kind):
    o = NORMS[kind]
    g = gen(rows * 10000 + d)
    x = rnd(g, rows, d, dtype=dtype)
    v = dict(weight=1 + rnd(g, d, std=0.2) if "w" in o else None,
             gate=rnd(g, rows, d, dtype=dtype, std=2.0) if "gate" in o else None,
             residual=rnd(g, rows, d, dtype=rdtype) if "res" in o else None,
             res_scale=1 + rnd(g, d, std=0.2) if "ls" in o else None,
             out_weight=1 + rnd(g, d, std=0.2) if "ow" in o else None)
    act, first, scale = o.get("gate", "sigmoid"), o.get("first", False), o.get("scale", 1.0)
    dev = lambda t: None if t is None else t.to(DEV)
    kw = dict({k: dev(t) for k, t in v.items()}, gate_act=act, gate_first=first, scale=scale,
              eps=1e-5, res_dtype=rdtype)
    r, y = kda.norm_fwd(dev(x), **kw)
    ps = {k: t.double().requires_grad_() for k, t in dict(v, x=x).items() if t is not None}
    rr, ry = ref.norm(ps["x"], **{k: ps.get(k) for k in v}, act=act, first=first, scale=scale,
                      eps=1e-5)
    assert r.dtype == rdtype
    close(r, rr, what="r", **TIGHT[rdtype])
    if "ow" in o:
        close(y, ry, what="y", **TIGHT[dtype])
        r2, y2 = kda.norm_fwd(dev(x), want_r=False, **kw)
        assert r2 is None and torch.equal(y2, y)
    else:
        assert y is None
    dr, dy = rnd(g, rows, d, dtype=rdtype), rnd(g, rows, d, dtype=dtype) if "ow" in o else None
    loss = (rr * dr.double()).sum() + (0 if dy is None else (ry * dy.double()).sum())
    loss.backward()
    got = kda.norm_bwd(dev(x), dev(dr), dev(dy), **kw)
    # rows of one or a few channels: 1 - n^2 / d cancels down to eps, and so do the bits
    few = 50 if d < 8 else 1
    for name, a in zip(("x", "gate", "residual", "weight", "res_scale", "out_weight"), got):
        if name not in ps:
            assert a is None
            continue
        t = a.dtype
        tol = dict(rel=6e-6, rms=3e-5) if name in ("weight", "res_scale", "out_weight") else TIGHT[t]
        close(a, ps[name].grad, what=f"d{name}", rel=tol["rel"] * few, rms=tol["rms"] * few)


@pytest.mark.parametrize("at", [0, 5, 8])
@pytest.mark.parametrize("heads", [1, 3])
def test_norm_strided(kda, at, heads):
    """x and gate as column slices of a wider projection: the same bits as dense copies."""
    g = gen(at)
    d = 64
    x, gate = (rnd(g, 2, 9, heads, d, dtype=BF) for _ in range(2))
    if heads == 1:
        x, gate = x[:, :, 0], gate[:, :, 0]
    w = (1 + rnd(g, d, std=0.2)).to(DEV)
    dr = rnd(g, *x.shape, dtype=BF).to(DEV)
    a, _ = kda.norm_fwd(x.to(DEV), weight=w, gate=gate.to(DEV))
    xs, gs = cut(x, heads * d + 24, at), cut(gate, heads * d + 8, 0)
    b, _ = kda.norm_fwd(xs, weight=w, gate=gs)
    close(b, a, what="r", **TIGHT[BF])
    for p, q in zip(kda.norm_bwd(x.to(DEV), dr, weight=w, gate=gate.to(DEV)),
                    kda.norm_bwd(xs, dr, weight=w, gate=gs)):
        if p is not None:
            close(q, p, what="grad", rel=2.0 ** -7, rms=1e-4)


def test_norm_residual_in_place(kda):
    g = gen(9)
    x, h = rnd(g, 40, 512, dtype=BF).to(DEV), rnd(g, 40, 512).to(DEV)
    w, ow = (1 + rnd(g, 512, std=0.2)).to(DEV), (1 + rnd(g, 512, std=0.2)).to(DEV)
    r, y = kda.norm_fwd(x, weight=w, residual=h, out_weight=ow)
    r2, y2 = kda.norm_fwd(x, weight=w, residual=h, out_weight=ow, r=h)
    assert r2 is h and torch.equal(r, h) and torch.equal(y, y2)


# ---------------------------------------------------------------------------
# all of them
# ---------------------------------------------------------------------------
def test_gradients_against_differences(kda):
    """Directional derivatives: the gradient along a random direction against central differences
    of the plain float64 form (step 1e-4: the differences err by about 1e-8 of the loss's scale,
    the float32 gradients by 1e-5)."""
    g = gen(11)
    B, T, D, W = 1, 60, 24, 4
    lens = [20, 3, 37]
    p = dict(x=rnd(g, B, T, D), w=rnd(g, D, W), b=rnd(g, D))
    dy = rnd(g, B, T, D)
    grads = kda.conv_bwd(p["x"].to(DEV), p["w"].to(DEV), dy.to(DEV), p["b"].to(DEV),
                         activation="silu", cu_seqlens=cu_of(lens))
    f = lambda q: (ref.conv(q["x"], q["w"], q["b"], silu=True, lens=lens)[0] * dy.double()).sum()
    along(f, p, dict(zip(("x", "w", "b"), grads)), g)
    R, d = 12, 80
    p = dict(x=rnd(g, R, d), weight=1 + rnd(g, d, std=0.2), gate=rnd(g, R, d),
             residual=rnd(g, R, d), res_scale=rnd(g, d), out_weight=rnd(g, d))
    dr, dy2 = rnd(g, R, d), rnd(g, R, d)
    for first in (False, True):
        got = kda.norm_bwd(p["x"].to(DEV), dr.to(DEV), dy2.to(DEV), gate_act="silu",
                           gate_first=first, scale=0.7,
                           **{k: t.to(DEV) for k, t in p.items() if k != "x"})

        def f(q):
            r, y = ref.norm(q["x"], act="silu", first=first, scale=0.7,
                            **{k: t for k, t in q.items() if k != "x"})
            return (r * dr.double()).sum() + (y * dy2.double()).sum()
        along(f, p, dict(zip(("x", "gate", "residual", "weight", "res_scale", "out_weight"), got)), g)


def along(f, p, grads, g):
    for name, t in p.items():
        v = rnd(g, *t.shape).double()
        h = 1e-4
        plus, minus = (f({**{k: q.double() for k, q in p.items()}, name: t.double() + s * h * v})
                       for s in (1, -1))
        diff = ((plus - minus) / (2 * h)).item()
        mine = (grads[name].cpu().double() * v).sum().item()
        scale = (grads[name].cpu().double() * v).square().sum().sqrt().item()
        assert abs(diff - mine) <= 1e-4 * scale, (name, diff, mine, scale)


def test_repeatable_and_other_streams(kda):
    """The same bits again, and on another stream (whose outputs belong to it)."""
    g = gen(12)
    x, w, dy = rnd(g, 2, 500, 256, dtype=BF).to(DEV), rnd(g, 256, 4).to(DEV), rnd(g, 2, 500, 256, dtype=BF).to(DEV)
    one = kda.conv_bwd(x, w, dy, activation="silu")[:2]
    xn, wn, drn = x.reshape(-1, 256), w[:, 0].contiguous(), dy.reshape(-1, 256)
    two = kda.norm_bwd(xn, drn, weight=wn)
    v = scan_inputs(13, 1, 300, 4, 2, 128, 128, BF, 1)
    three = scan_call(kda, v, out_dtype=BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = (kda.conv_bwd(x, w, dy, activation="silu", stream=s)[:2],
             kda.norm_bwd(xn, drn, weight=wn, stream=s), scan_call(kda, v, out_dtype=BF))
    torch.cuda.synchronize()
    for a, b in zip((one, two, three), again):
        for p, q in zip(a, b):
            assert p is q is None or torch.equal(p, q)


def test_malformed_offsets_are_reported(kda):
    """Offsets that do not rise from 0 to T: every access stays inside, the status says so."""
    g = gen(14)
    x, w = rnd(g, 1, 50, 16, dtype=BF).to(DEV), rnd(g, 16, 4).to(DEV)
    v = {k: t.to(DEV) for k, t in scan_inputs(1, 1, 50, 2, 1, 64, 64, BF, 2).items()}
    for cu in ([0, 60, 50], [0, 30, 20], [5, 20, 50], [0, 20, 49]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
        kda.conv_fwd(x, w, cu_seqlens=c, workspace=ws)
        assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS, cu
        kda.conv_bwd(x, w, x, cu_seqlens=c, workspace=ws)
        assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS, cu
        kda.scan_fwd(v["x"], v["dt"], v["A"], v["B"], v["C"], cu_seqlens=c, workspace=ws)
        assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS, cu


def test_no_tokens(kda):
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=DEV)
    w = torch.ones(16, 4, device=DEV)
    y, s = kda.conv_fwd(e(2, 0, 16), w)
    assert y.shape == (2, 0, 16) and not s.any()
    dx, dw, _, _ = kda.conv_bwd(e(2, 0, 16), w, e(2, 0, 16))
    assert dx.numel() == 0 and not dw.any()
    h0 = torch.randn(2, 2, 64, 64, device=DEV)
    one = torch.ones(2, device=DEV)
    y, hT = kda.scan_fwd(e(2, 0, 2, 64), e(2, 0, 2), -one, e(2, 0, 1, 64), e(2, 0, 1, 64), h0=h0)
    assert torch.equal(hT, h0)
    y, hT = kda.scan_fwd(e(0, 5, 2, 64), e(0, 5, 2), -one, e(0, 5, 1, 64), e(0, 5, 1, 64))
    assert hT.shape == (0, 2, 64, 64)
    r, _ = kda.norm_fwd(e(0, 64), weight=torch.ones(64, device=DEV))
    assert r.shape == (0, 64)
    got = kda.norm_bwd(e(0, 64), e(0, 64), weight=torch.ones(64, device=DEV))
    assert not got[3].any()
