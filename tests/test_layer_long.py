"""GPU parity of the operators around the recurrence where their work is divided otherwise than in
the small cases: scans in segments, many chains, many tiles, rows of many lengths, and offsets past
32 bits.  Tolerances as in test_layer."""
import pytest
import torch

import _layer_ref as ref
import test_layer as small
from _layer_ref import close
from test_layer import BF, DEV, F32, SCAN_Y, cu_of, gen, rnd, scan_call, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,ds,dx,B,T,lens", [
    (2, 1, 128, 128, 1, 2200, None), (3, 1, 128, 64, 2, 1500, None), (2, 2, 64, 64, 1, 1025, None),
    (2, 1, 128, 128, 1, 0, [1900, 0, 70, 1100]), (3, 1, 64, 64, 1, 0, [5, 1300, 2, 1300])])
def test_scan_in_segments(kda, H, G, ds, dx, B, T, lens):
    """Few chains of many tokens: several segments at once."""
    T = T if lens is None else sum(lens)
    N = B if lens is None else len(lens)
    v = scan_inputs(T + dx, B, T, H, G, ds, dx, BF, N)
    v["A"][0] = -0.01  # a head that remembers the segments before
    v["h0"] *= 3
    y, hT = scan_call(kda, v, cu=None if lens is None else cu_of(lens), out_dtype=BF)
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"],
                      softplus=True, lens=lens, h0=v["h0"])
    close(y, ry, what="y", **SCAN_Y[BF])
    close(hT, rh, rel=0, rms=1e-4, what="hT")
    d = {k: t.to(DEV) for k, t in v.items()}
    y2, _ = kda.scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], dt_bias=d["bias"],
                         dt_softplus=True, cu_seqlens=None if lens is None else cu_of(lens),
                         h0=d["h0"], hT=d["h0"], out_dtype=BF)
    assert torch.equal(y2, y) and torch.equal(d["h0"], hT), "the states in place"


@pytest.mark.parametrize("ds,dx", [(64, 64), (128, 128)])
def test_scan_of_many_float32_chains(kda, ds, dx):
    """Enough chains for blocks of 32 columns; the same values as a call of few of them."""
    v = scan_inputs(ds, 48, 37, 4, 2, ds, dx, F32, 48)
    y, hT = scan_call(kda, v)
    ry, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], bias=v["bias"],
                      softplus=True, h0=v["h0"])
    close(y, ry, what="y", **SCAN_Y[F32])
    close(hT, rh, rel=0, rms=1e-4, what="hT")
    few = {k: t[-1:] if t.dim() > 1 else t for k, t in v.items()}
    y1, h1 = scan_call(kda, few)
    close(y1, y[-1:], what="y of few", **SCAN_Y[F32])
    close(h1, hT[-1:], rel=0, rms=1e-4, what="hT of few")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,lens", [(8, [4100]), (264, [2900, 0, 1, 1300]), (37, [2500])])
def test_conv_of_many_tiles(kda, dtype, D, lens):
    small.test_conv(kda, dtype, 4, D, lens)


@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,d", [(9000, 40), (3000, 256), (2100, 320), (1000, 777), (700, 1352),
                                    (500, 2560), (200, 4104), (170, 6144), (160, 8192)])
@pytest.mark.parametrize("kind", ["gated", "all first"])
def test_norm_of_many_rows(kda, dtype, rdtype, rows, d, kind):
    """More rows than are resident at once, for every division of a row among threads."""
    small.test_norm(kda, dtype, rdtype, rows, d, kind)


def test_offsets_past_32_bits(kda):
    """The last tokens of tensors of more than 2^31 elements, bit for bit those of a small call."""
    g = torch.Generator(device=DEV).manual_seed(3)
    fill = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=DEV).normal_(generator=g)
    D, T = 12288, 180_000
    w = fill(D, 4, dtype=F32)
    x, dy = fill(1, T, D), fill(1, T, D)
    y, s = kda.conv_fwd(x, w, activation="silu")
    y1, s1 = kda.conv_fwd(x[:, -103:], w, activation="silu")
    assert torch.equal(y[:, -100:], y1[:, 3:]) and torch.equal(s, s1)
    del y
    dx = kda.conv_bwd(x, w, dy, activation="silu")[0]
    dx1 = kda.conv_bwd(x[:, -103:], w, dy[:, -103:].contiguous(), activation="silu")[0]
    assert torch.equal(dx[:, -100:], dx1[:, 3:])
    del dx
    # rows of 4096 in the same memory
    xn, dn, wn = x.view(-1, 4096), dy.view(-1, 4096), w[:4096, 0].contiguous()
    r, _ = kda.norm_fwd(xn, weight=wn)
    assert torch.equal(r[-9:], kda.norm_fwd(xn[-9:], weight=wn)[0])
    del r
    dx = kda.norm_bwd(xn, dn, weight=wn)[0]
    assert torch.equal(dx[-9:], kda.norm_bwd(xn[-9:], dn[-9:], weight=wn)[0])
    del dx, xn, dn, dy
    # a prompt of 32 heads of 128, and a short sequence behind it
    T = x.numel() // 4096
    xs = x.view(1, T, 32, 128)
    dt, B, C = fill(1, T, 32), fill(1, T, 1, 128), fill(1, T, 1, 128)
    A = -torch.arange(1, 33, dtype=F32, device=DEV) / 8
    cu = torch.tensor([0, T - 65, T], dtype=torch.int32, device=DEV)
    y, hT = kda.scan_fwd(xs, dt, A, B, C, dt_softplus=True, cu_seqlens=cu, out_dtype=BF)
    tail = [t[:, -65:] for t in (xs, dt, B, C)]
    y1, h1 = kda.scan_fwd(tail[0], tail[1], A, tail[2], tail[3], dt_softplus=True, out_dtype=BF)
    assert torch.equal(y[:, -65:], y1) and torch.equal(hT[1:], h1)
    del x, xs, y, hT
    # single tokens over a pool of states
    N = 4200
    state = fill(N, 32, 128, 128, dtype=F32)
    kept = state[-2:].clone()
    step = (fill(N, 1, 32, 128), fill(N, 1, 32), fill(N, 1, 1, 128), fill(N, 1, 1, 128))
    y = kda.scan_step(step[0], step[1], A, step[2], step[3], state, dt_softplus=True)
    last = [t[-2:] for t in step]
    y1 = kda.scan_step(last[0], last[1], A, last[2], last[3], kept, dt_softplus=True)
    assert torch.equal(y[-2:], y1) and torch.equal(state[-2:], kept)
    del state
    pool = fill(61_000, 3, D)
    kept, xs = pool[-2:].clone(), fill(61_000, 1, D)
    y = kda.conv_step(xs, w, pool, activation="silu")
    y1 = kda.conv_step(xs[-2:], w, kept, activation="silu")
    assert torch.equal(y[-2:], y1) and torch.equal(pool[-2:], kept)
