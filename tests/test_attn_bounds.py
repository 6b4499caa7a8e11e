"""Attention of new tokens against float64 for every number of query rows, with bounds that a place too many or too
few passes: of 333 places each has about 1/333 of the weight.

Tolerances.  Queries, keys and values are normal numbers: sum |q k| scale is at most 2^4, a single product at most
2 (3.5 sizes each, over sqrt 64).  bf16 queries: exact products, added in up to 8 steps of 17 numbers, each of which
the tensor cores may cut at 2^-23 of the largest, a partial sum of at most 8 units: 8 x 17 x 2^-23 x 8 < 2^-12.9 in the
worst case, 2^-13 with one cut in 20 as large.  float32 queries: the cuts of 16 products of at most 2 in 8 steps,
2^-23 x 2 x 128 = 2^-15, float32 additions of partial sums, 8 x 2^-24 x 8, and the query's 22 bits, 2^-22 x 2^4: below
2^-14.  These bound lse (of at most 16, whose roundings are 2^-20 each) and, twice over (the weight, the sum of weights),
each weight relatively, so that the output is off by as much of sum p |v|; to it come half a step of the weights' own
bits (2^-17 over bf16 caches, 2^-12 over codes, less than 2^-22 for float32 queries), up to 2^7 float32 additions of
sum p |v| (2^-17) and the output's rounding.
"""
import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FORMS = [("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "int8"), ("f32", "f32"), ("f32", "e4m3"), ("f32", "int8")]


def held(pool, scale, ids):
    """A sequence's pages as [heads, places, d] in float64."""
    x = (pool.view(torch.uint8)[ids].view(pool.dtype).float() if scale is not None else pool[ids]).to(F64)
    if scale is not None:
        x = x * torch.exp2(scale[ids].to(F64) - 127)[..., None]
    return x.transpose(0, 1).flatten(1, 2)


def exact(q, cache, pages, lens, scale, window=0):
    """out, lse and sum p |v| in float64."""
    B, T, hq, d = q.shape
    out, spread = (torch.zeros(B, T, hq, d, dtype=F64, device="cuda") for _ in range(2))
    lse = torch.full((B, T, hq), -torch.inf, dtype=F64, device="cuda")
    for b, n in enumerate(lens):
        k, v = held(cache.k, cache.k_scale, pages[b].long()), held(cache.v, cache.v_scale, pages[b].long())
        for t in range(T):
            hi = n - T + t + 1
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            s = torch.einsum("grd,gkd->grk", q[b, t].to(F64).unflatten(0, (k.shape[0], -1)), k[:, lo:hi]) * scale
            p = torch.softmax(s, -1)
            out[b, t] = torch.einsum("grk,gkd->grd", p, v[:, lo:hi]).flatten(0, 1)
            spread[b, t] = torch.einsum("grk,gkd->grd", p, v[:, lo:hi].abs()).flatten(0, 1)
            lse[b, t] = torch.logsumexp(s, -1).flatten()
    return out, lse, spread


def compare(kda, dtype, kind, lens, T, rep, d, page, cap, window, seed):
    g = torch.Generator().manual_seed(seed)
    n, mp = len(lens), cap // page
    pages = torch.randperm(n * mp, generator=g).reshape(n, mp).to(torch.int32).cuda()
    pools = []
    for _ in range(2):
        x = torch.randn(n * mp, 2, page, d, generator=g).clamp(-3.5, 3.5)
        if kind in ("f32", "bf16"):
            pools.append((x.to(TYPES[kind]).cuda(), None))
        else:
            value, byte = ref.encode(x.to(F64), kind)
            code = (value * torch.exp2(127 - byte.to(F64))[..., None]).float().to(TYPES[kind])
            pools.append((code.cuda(), byte.to(torch.uint8).cuda()))
    cache = kda.KVCache(pools[0][0], pools[1][0], pools[0][1], pools[1][1])
    q = torch.randn(n, T, 2 * rep, d, generator=g).clamp(-3.5, 3.5).to(TYPES[dtype]).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, lse = kda.attn_step(q, cache, pages, ln, window=window, want_lse=True)
    want, wl, spread = exact(q, cache, pages, lens, d ** -0.5, window)
    f32 = dtype == "f32"
    score = 2.0 ** -14 if f32 else 2.0 ** -13
    none = wl == -torch.inf
    assert torch.equal(lse == -torch.inf, none) and not got[none].any()
    assert ((lse.to(F64) - wl).abs() <= score + 2.0 ** -18)[~none].all(), (lse.to(F64) - wl)[~none].abs().max()
    weight = 2.0 ** -22 if f32 else 2.0 ** -17 if kind == "bf16" else 2.0 ** -12
    tol = want.abs() * (2.0 ** -24 if f32 else 2.0 ** -8) + spread * (2 * score + weight + 2.0 ** -17)
    err = (got.to(F64) - want).abs()
    assert (err <= tol).all(), (err / spread.clamp(min=1e-9)).max()


@pytest.mark.parametrize("dtype,kind", FORMS)
@pytest.mark.parametrize("T,rep", [(1, 1), (1, 8), (2, 7), (3, 5), (4, 4), (5, 4), (8, 4), (7, 5), (8, 8), (8, 9), (8, 16), (5, 27)])
def test_rows(kda, T, rep, dtype, kind):
    """1 to 135 rows per key-value head, over parts and over short tables."""
    for d in (64, 128):
        compare(kda, dtype, kind, [333, 120, T, 0], T, rep, d, 32, 352, 0, 1)
        compare(kda, dtype, kind, [333, 120, 2001, 5], T, rep, d, 32, 2016, 0, 2)


@pytest.mark.parametrize("dtype,kind", FORMS)
@pytest.mark.parametrize("page", [1, 8, 16, 128])
def test_windows_and_pages(kda, page, dtype, kind):
    for window in (1, 63, 64, 65, 200):
        compare(kda, dtype, kind, [333, 120, 1030, 9, 0], 3, 4, 64, page, 1152, window, 3)
        compare(kda, dtype, kind, [333, 120, 256, 9, 0], 8, 3, 64, page, 384, window, 4)


@pytest.mark.parametrize("dtype,kind", FORMS)
def test_every_length(kda, dtype, kind):
    """Lengths from 0 to past two tiles, one sequence each."""
    compare(kda, dtype, kind, list(range(0, 263)), 2, 2, 64, 16, 272, 0, 5)
    compare(kda, dtype, kind, list(range(0, 263)), 2, 2, 64, 16, 1024, 100, 6)
