"""The operators around the recurrence at their edges: malformed offsets, steps that forget all,
values that are not finite.  Tolerances as in test_layer where a test does not derive its own."""
import pytest
import torch

import _layer_ref as ref
from _layer_ref import close
from test_layer import BF, DEV, F32, TIGHT, gen, rnd

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
