"""Attention of new tokens over values that are infinite or NaN where a token sees them: each gives its
channel what it is, wherever it stands and however small its weight, and leaves the other channels alone.

Tolerances of those: as in the other tests of attention, 2^-13 of the largest value in bf16 and 2^-15 in
float32, and the output's rounding (2^-8, 2^-24); with scores of up to 480, which 2^-24 of them moves by
2^-15, four times as much, as a weight is off by e^x - 1 < 2^-14 and 64 products add to it.
"""
import math

import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def check(kda, q, k, v, lens, page, window=0, scale=0.125, factor=1):
    """k, v [B,most,heads,64] with values that are not finite; the expected result from finite ones."""
    n, most, heads, d = k.shape
    mp = -(-most // page)
    pages = torch.randperm(n * mp, generator=torch.Generator().manual_seed(5)).reshape(n, mp).to(torch.int32)
    cache = kda.kv_cache(n * mp, page, heads, d, dtype=k.dtype)
    full = torch.full((n,), most, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32)
    kda.cache_write(k.cuda(), v.cuda(), cache, pages.cuda(), full)
    got, lse = kda.attn_step(q.cuda(), cache, pages.cuda(), ln.cuda(), window=window, scale=scale, want_lse=True)
    kda.cache_write(k.cuda(), torch.where(torch.isfinite(v), v, torch.zeros((), dtype=v.dtype)).cuda(), cache, pages.cuda(), full)
    want, wl = ref.attn(q, tuple(None if t is None else t.cpu() for t in cache), pages, ln, scale, window)
    T, rep = q.shape[1], q.shape[2] // heads
    extra = torch.zeros_like(want)
    for b in range(n):
        for t in range(T):
            hi = lens[b] - T + t + 1
            lo = max(0, hi - window) if window else 0
            x = v[b, lo:max(hi, lo)].to(F64)
            x = torch.where(torch.isfinite(x), 0.0, x).sum(0)
            extra[b, t] = x.repeat_interleave(rep, 0)
    own = extra != 0  # NaN too
    got = got.cpu().to(F64)
    assert torch.equal(got[own].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0), extra[own].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0))
    f32 = q.dtype is torch.float32
    tol = want.abs() * (2.0 ** -24 if f32 else 2.0 ** -8) + factor * (2.0 ** -15 if f32 else 2.0 ** -13) * want.abs().max()
    assert ((got - want).abs() <= tol)[~own].all()
    assert ((lse.cpu().to(F64) - wl).abs()[wl > -math.inf] <= 2.0 ** -12 * factor).all()
    return own


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,rep", [(1, 4), (4, 4), (8, 4), (8, 9)])
@pytest.mark.parametrize("page,most", [(16, 2100), (64, 512), (4, 300)])
def test_seen_infinities(kda, page, most, T, rep, dtype):
    """Of either sign, of both, NaN, at the first place, inside, at the ends of the seen range, in a later
    drafted token; over caches in parts and over short tables, with a window and without."""
    g = torch.Generator().manual_seed(1)
    lens = [most, most // 3, 9, T]
    k, v = (torch.randn(4, most, 2, 64, generator=g).to(TYPES[dtype]) for _ in range(2))
    q = torch.randn(4, T, 2 * rep, 64, generator=g).to(TYPES[dtype])
    inf = math.inf
    for b, n in enumerate(lens):
        for place, head, ch, x in ((0, 0, 0, inf), (0, 1, 1, -inf), (n // 2, 0, 9, inf), (n // 2 + 1, 0, 17, -inf),
                                   (n // 3, 1, 33, inf), (n // 2, 1, 33, -inf), (n - 1, 0, 63, inf), (n - 1, 1, 62, -inf),
                                   (max(n - T, 0), 0, 40, inf), (n // 4, 0, 50, math.nan), (max(n - 20, 0), 1, 8, inf)):
            v[b, place, head, ch] = x
    own = check(kda, q, k, v, lens, page)
    assert own[0, :, :, [0, 9, 50]].any()
    check(kda, q, k, v, lens, page, window=20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("page", [16, 2])
def test_infinities_without_weight(kda, page, T, dtype):
    """Scores that rise and fall by hundreds along the cache: an infinity stays, though its weight is 0 in
    float32, in the place's own part and against all others."""
    n = 1200
    g = torch.Generator().manual_seed(2)
    up = torch.linspace(-60, 60, n).bfloat16().float()
    v = torch.randn(2, n, 1, 64, generator=g)
    for i, p in enumerate((0, 63, 64, 400, 700, 1100, n - T)):
        v[:, p, 0, 2 * i] = math.inf
        v[:, p, 0, 2 * i + 1] = -math.inf
    k = torch.zeros(2, n, 1, 64)
    k[0, :, 0, 0], k[1, :, 0, 0] = up, up.flip(0)
    q = torch.zeros(2, T, 2, 64)
    q[..., 0, 0], q[..., 1, 0] = 8.0, -8.0
    dt = TYPES[dtype]
    own = check(kda, q.to(dt), k.to(dt), v.to(dt), [n, n], page, scale=1.0, factor=4)
    assert own[:, -1, :, :14].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 8])
def test_all_values_infinite(kda, T, dtype):
    """Every value, over one part and over many."""
    g = torch.Generator().manual_seed(3)
    k = torch.randn(2, 900, 2, 64, generator=g).to(TYPES[dtype])
    q = torch.randn(2, T, 8, 64, generator=g).to(TYPES[dtype])
    v = torch.full((2, 900, 2, 64), -math.inf).to(TYPES[dtype])
    assert check(kda, q, k, v, [900, 30], 16).all()
    v[0, 3, 1, 5] = math.inf
    check(kda, q, k, v, [900, 30], 16)
