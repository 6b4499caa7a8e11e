"""The operators around the recurrence at their edges: malformed offsets, steps that forget all,
values that are not finite.  Tolerances as in test_layer where a test does not derive its own."""
import pytest
import torch

import _layer_ref as ref
from _layer_ref import close
from test_layer import BF, DEV, F32, SCAN_Y, TIGHT, cu_of, gen, rnd, scan_call, scan_inputs

pytestmark = pytest.mark.gpu


def inside(t):
    """The same values in the middle of a buffer of NaN, 300 rows of the last dimension on each side."""
    d = t.shape[-1]
    big = torch.full((t.numel() // d + 600, d), float("nan"), dtype=t.dtype, device=DEV)
    mid = big[300:300 + t.numel() // d]
    mid.copy_(t.reshape(-1, d))
    return mid.view(t.shape)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [16, 13])
@pytest.mark.parametrize("cu", [[100, 150], [5, 20, 150], [70, 70, 150], [0, 150, 20], [0, 30, 20, 150],
                                [150, 0, 150], [0, 20, 149]])
def test_malformed_offsets_stay_inside_the_states(kda, dtype, D, cu):
    """Offsets that do not rise from 0 to T: no row outside the start states (or the cotangents of
    the final ones) is read, so the NaN around them reaches no result; the status reports them."""
    g = gen(21)
    T, W, N = 150, 4, len(cu) - 1
    x, w, dy = rnd(g, 1, T, D, dtype=dtype).to(DEV), rnd(g, D, W).to(DEV), rnd(g, 1, T, D, dtype=dtype).to(DEV)
    init, df = (inside(rnd(g, N, W - 1, D, dtype=dtype)) for _ in range(2))
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    y, s = kda.conv_fwd(x, w, cu_seqlens=c, init_state=init, activation="silu", workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS
    assert torch.isfinite(y).all() and torch.isfinite(s).all()
    dx, dw, _, di = kda.conv_bwd(x, w, dy, cu_seqlens=c, init_state=init, dfinal=df, want_dinit=True,
                                 activation="silu", workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS
    assert torch.isfinite(dw).all() and torch.isfinite(di).all()


@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,d", [(5, 64), (1, 128), (9, 256), (3, 37), (601, 96)])
def test_norm_without_eps(kda, dtype, rdtype, rows, d):
    """eps = 0 with rows that do not fill the last block: no part of a block without a row counts."""
    g = gen(rows + d)
    x, dr, dy = rnd(g, rows, d, dtype=dtype), rnd(g, rows, d, dtype=rdtype), rnd(g, rows, d, dtype=dtype)
    v = dict(weight=1 + rnd(g, d, std=0.2), gate=rnd(g, rows, d, dtype=dtype),
             residual=rnd(g, rows, d, dtype=rdtype), res_scale=1 + rnd(g, d, std=0.2),
             out_weight=1 + rnd(g, d, std=0.2))
    ps = {k: t.double().requires_grad_() for k, t in dict(v, x=x).items()}
    rr, ry = ref.norm(ps["x"], **{k: ps[k] for k in v}, eps=0.0)
    ((rr * dr.double()).sum() + (ry * dy.double()).sum()).backward()
    dev = {k: t.to(DEV) for k, t in v.items()}
    r, y = kda.norm_fwd(x.to(DEV), eps=0.0, **dev)
    close(r, rr, what="r", **TIGHT[rdtype])
    close(y, ry, what="y", **TIGHT[dtype])
    got = kda.norm_bwd(x.to(DEV), dr.to(DEV), dy.to(DEV), eps=0.0, **dev)
    for name, a in zip(("x", "gate", "residual", "weight", "res_scale", "out_weight"), got):
        sums = name in ("weight", "res_scale", "out_weight")
        close(a, ps[name].grad, what=f"d{name}", **(dict(rel=6e-6, rms=3e-5) if sums else TIGHT[a.dtype]))


def within(got, ref_, size, tol, what):
    """|got - ref| <= tol * size, element by element; `size` is the sum of the terms' magnitudes."""
    got, ref_ = got.detach().cpu().double(), ref_.detach().cpu().double()
    assert got.shape == ref_.shape and torch.isfinite(got).all(), what
    worst = ((got - ref_).abs() / (tol * size + 1e-30)).max().item()
    assert worst <= 1, f"{what}: {worst:.3f} times the bound"


def scan_sizes(v, **kw):
    """y and hT of the magnitudes: what the roundings of single terms are relative to."""
    return ref.scan(v["x"].abs(), v["dt"], v["A"], v["B"].abs(), v["C"].abs(), v["D"].abs(),
                    bias=v["bias"], softplus=True, h0=v["h0"].abs(), **kw)


# float32 outputs of bf16 prompts, relative to the magnitudes of an output's terms.  Each term has
# one operand of two bf16 parts (2^-18); sums of up to 64 + 128 float32 terms, as much again; the
# exponent of a decay by 2^-20, computed in float32, is off by 20 times a few 2^-24 (2^-17; stronger
# decays leave less of the term than that): together 2^-16.
SCAN_Y_TERMS = 2.0 ** -16


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dx", [64, 128])
@pytest.mark.parametrize("at", [0, 10, 31, 40, 55])
def test_scan_after_steps_that_forget(kda, dtype, dx, at):
    """Steps in the middle of a chunk that leave nothing of the state, with ordinary tokens after
    them; the last head's log decay is past float32's range."""
    v = scan_inputs(3, 2, 150, 6, 2, 128, dx, dtype, 2, fast=True)
    v["dt"][:, 20:30] = -200.0
    v["dt"][:, at:at + 4] = 300.0
    v["dt"][:, 64 + at] = 100.0
    for h, a in enumerate((-2.0, 0.0, -1e4, -148.0, -16.0, -3e38)):
        v["A"][h] = a
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"], softplus=True,
                      h0=v["h0"])
    size, _ = scan_sizes(v)
    for out in (BF, F32):
        y, hT = scan_call(kda, v, out_dtype=out)
        for h in range(6):
            close(y[:, :, h], ry[:, :, h], what=f"y {h}", **SCAN_Y[BF if BF in (dtype, out) else F32])
            close(hT[:, h], rh[:, h], rel=0, rms=1e-4, what=f"hT {h}")
            if out == F32:
                within(y[:, :, h], ry[:, :, h], size[:, :, h], SCAN_Y_TERMS, f"y {h}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dx,H,G", [(64, 3, 1), (64, 4, 2), (128, 2, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_scan_of_a_value_that_is_not_finite(kda, dtype, out, dx, H, G, bad):
    """Such a value of one token reaches no earlier token, no other sequence, and (of x and dt) no
    other channel or head; what the definition makes of it is not finite."""
    B, T, at, h, ch = 2, 150, 70, 1, 37
    v = scan_inputs(5, B, T, H, G, 128, dx, dtype, B)
    y, hT = scan_call(kda, v, out_dtype=out)
    for k in ("x", "x first", "x last", "dt", "B", "C"):
        t = {"x first": 64, "x last": 127}.get(k, at)
        w = {n: u.clone() for n, u in v.items()}
        if k.startswith("x"):
            w["x"][1, t, h, ch] = bad
        else:
            w[k][1, t, h if k == "dt" else 0] = float("nan")
        y2, h2 = scan_call(kda, w, out_dtype=out)
        assert torch.equal(y2[0], y[0]) and torch.equal(h2[0], hT[0]), k
        assert torch.equal(y2[1, :t], y[1, :t]), k
        if k.startswith("x"):
            assert not torch.isfinite(y2[1, t:, h, ch]).any() and not torch.isfinite(h2[1, h, :, ch]).any(), k
            y2[1, t:, h, ch], h2[1, h, :, ch] = y[1, t:, h, ch], hT[1, h, :, ch]
        elif k == "dt":
            assert not torch.isfinite(y2[1, t:, h]).any() and not torch.isfinite(h2[1, h]).any(), k
            y2[1, t:, h], h2[1, h] = y[1, t:, h], hT[1, h]
        else:
            n = H // G
            assert not torch.isfinite(y2[1, t, :n]).any(), k
            if k == "C":
                y2[1, t, :n] = y[1, t, :n]
            else:
                assert not torch.isfinite(h2[1, :n]).any()
                y2[1, t:, :n], h2[1, :n] = y[1, t:, :n], hT[1, :n]
        assert torch.equal(y2, y) and torch.equal(h2, hT), k


def test_workspace_on_the_host_is_refused(kda):
    """Before anything is launched."""
    x, w, A = torch.zeros(1, 8, 16, device=DEV), torch.zeros(16, 4, device=DEV), torch.zeros(2, device=DEV)
    xs, b = torch.zeros(1, 8, 2, 64, device=DEV), torch.zeros(1, 8, 1, 64, device=DEV)
    state = torch.zeros(1, 2, 64, 64, device=DEV)
    one = torch.ones(16, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: kda.conv_fwd(x, w, workspace=ws), lambda: kda.conv_bwd(x, w, x, workspace=ws),
                 lambda: kda.conv_step(x, w, torch.zeros(1, 3, 16, device=DEV), workspace=ws),
                 lambda: kda.scan_fwd(xs, xs[..., 0].contiguous(), A, b, b, workspace=ws),
                 lambda: kda.scan_step(xs, xs[..., 0].contiguous(), A, b, b, state, workspace=ws),
                 lambda: kda.norm_bwd(x, x, weight=one, workspace=ws)):
        with pytest.raises(ValueError, match="workspace"):
            call()


@pytest.mark.parametrize("ds,dx", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("B,T,lens", [(2, 200, None), (1, 2200, None), (1, 0, [1, 0, 64, 130, 63])])
def test_scan_float32_outputs_of_bf16_prompts(kda, ds, dx, B, T, lens):
    """Before any rounding to bf16: the read-out's and M's operands hold 16 bits."""
    T = T if lens is None else sum(lens)
    v = scan_inputs(T + ds, B, T, 2, 1, ds, dx, BF, B if lens is None else len(lens))
    y, _ = scan_call(kda, v, cu=None if lens is None else cu_of(lens), out_dtype=F32)
    ry, _ = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"], softplus=True,
                     lens=lens, h0=v["h0"])
    within(y, ry, scan_sizes(v, lens=lens)[0], SCAN_Y_TERMS, "y")


@pytest.mark.parametrize("ds,dx", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_scan_keeps_every_bit_of_an_update(kda, ds, dx):
    """The state after two tokens, relative to its two terms: the weight of the first one (an
    exponential, 2^-22) and a few float32 roundings, 2^-20.  Updates of two bf16 parts would be off by
    up to 2^-18."""
    v = scan_inputs(31 + ds, 2, 2, 4, 2, ds, dx, BF, 2)
    v["dt"] = v["dt"].abs() * 0.5
    v["A"] = -0.5 - 0.5 * torch.rand(4, generator=gen(32))
    d = {k: t.to(DEV) for k, t in v.items()}
    _, hT = kda.scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"])
    _, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"])
    size = ref.scan(v["x"].abs(), v["dt"], v["A"], v["B"].abs(), v["C"])[1]
    within(hT, rh, size, 2.0 ** -20, "hT")


def test_every_entry_point_runs_on_the_stream_it_is_given(kda):
    """Inputs that another stream writes late: calls made with that stream see them, others would
    see the NaN that was there."""
    g = gen(33)
    up = lambda *s, **kw: rnd(g, *s, **kw).to(DEV)
    x, w, dy = up(2, 200, 256, dtype=BF), up(256, 4), up(2, 200, 256, dtype=BF)
    conv = dict(x=x, w=w, dy=dy, state=up(2, 3, 256, dtype=BF))
    step = dict(conv, x=x[:, :3].contiguous(), state=conv["state"])
    bf, f32 = ({k: t.to(DEV) for k, t in scan_inputs(34, 1, 2200, 2, 1, 128, 64, dt, 1).items()}
               for dt in (BF, F32))
    one = {k: t[:, :5].contiguous() if t.dim() > 1 and k != "h0" else t for k, t in bf.items()}
    norm = dict(x=x, gate=dy, dr=up(2, 200, 256, dtype=BF), dy=up(2, 200, 256, dtype=BF), w=up(256))
    scan = lambda f, i, *state, **kw: f(i["x"], i["dt"], i["A"], i["B"], i["C"], *state, D=i["D"],
                                        dt_bias=i["bias"], dt_softplus=True, **kw)
    calls = [
        (conv, lambda i, s: kda.conv_fwd(i["x"], i["w"], init_state=i["state"], stream=s)),
        (step, lambda i, s: (kda.conv_step(i["x"], i["w"], i["state"], stream=s), i["state"])),
        (conv, lambda i, s: kda.conv_bwd(i["x"], i["w"], i["dy"], activation="silu", stream=s)[:2]),
        (bf, lambda i, s: scan(kda.scan_fwd, i, h0=i["h0"], hT=i["h0"], out_dtype=BF, stream=s)),
        (f32, lambda i, s: scan(kda.scan_fwd, i, h0=i["h0"], stream=s)),
        (one, lambda i, s: (scan(kda.scan_step, i, i["h0"], stream=s), i["h0"])),
        (norm, lambda i, s: kda.norm_fwd(i["x"], weight=i["w"], gate=i["gate"], out_weight=i["w"], stream=s)),
        (norm, lambda i, s: kda.norm_bwd(i["x"], i["dr"], i["dy"], weight=i["w"], gate=i["gate"],
                                         out_weight=i["w"], stream=s)[:2]),
    ]
    side = torch.cuda.Stream()
    for k, (inputs, call) in enumerate(calls):
        expect = call({n: t.clone() for n, t in inputs.items()}, None)
        late = {n: torch.full_like(t, float("nan")) for n, t in inputs.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
            for n, t in inputs.items():
                late[n].copy_(t)
        got = call(late, side)
        side.synchronize()
        for a, b in zip(got, expect):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("N", [1024, 1025, 2100])
def test_scan_of_many_sequences(kda, N):
    """More sequences than the planning block has threads, most of them empty or of one or two
    tokens, with one that is cut into segments behind them."""
    g = gen(N)
    lens = torch.randint(0, 3, (N,), generator=g).tolist()
    lens[N - 40] = 1500
    v = scan_inputs(N, 1, sum(lens), 1, 1, 64, 64, BF, N)
    v["h0"] *= 3
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    y, hT = scan_call(kda, v, cu=cu_of(lens), out_dtype=F32, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_OK
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"], softplus=True,
                      lens=lens, h0=v["h0"])
    close(y, ry, what="y", **SCAN_Y[BF])
    close(hT, rh, rel=0, rms=1e-4, what="hT")
    empty = [i for i, n in enumerate(lens) if n == 0]
    assert torch.equal(hT[empty].cpu(), v["h0"][empty])
