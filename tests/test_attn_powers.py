"""Attention of new tokens over 8-bit caches whose rows have very different powers of two.

Tolerances.  Scores are sums of 64 products with sum |q k| scale below 2^4.  bf16 queries: every product is exact,
the sums in float32 are off by at most 66 steps of 2^-23 of them (2^-13, of lse and relatively of a weight).
float32 queries: 22 bits of the query (2^-22 of the sum), 16 cut-off additions of single products and four of
partial sums, at most 2^-17 together; taken twice (a weight and the sum of weights), and once more for the sums of
the values: 2^-15 of the sum of p |v|; lse, of at most 32 in size, within 2^-16.  A weight times its row's power
is off by half a step of 11 bits (bf16 queries, 2^-12) or of 22 (float32, less than 2^-16), and by 2^-25 where it
lies below f16's normal numbers, with the row's largest at 2^9 or more: 2^-34 of the largest such product for
each place, times a code below 2^9.  The largest product's row holds a code of 2^6 or more, so that it is at most
2^-6 of the largest of the sums of p |v|: 2^-31 of that sum for each of up to 1500 places, 2^-20.
"""
import math

import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FORMS = [("bf16", "e4m3"), ("bf16", "int8"), ("f32", "e4m3"), ("f32", "int8")]
ROWS = [(1, 4), (4, 4), (8, 4), (8, 8)]  # 4, 16, 32 and 64 query rows per key-value head


def state(lens, T, rep, page, dtype, kind, seed, most=None):
    """q [B,T,2 rep,64], a cache of two heads, its table and lengths, on the CPU; channel 0 of every query is 8
    and of every key 0, so that a key's channel 0 moves its score for all queries alike."""
    g = torch.Generator().manual_seed(seed)
    n, mp = len(lens), -(-(most or max(lens)) // page)
    pages = torch.randperm(n * mp + 3, generator=g)[:n * mp].reshape(n, mp).to(torch.int32)
    q = torch.randn(n, T, 2 * rep, 64, generator=g)
    q[..., 0] = 8.0
    pools = []
    for which in range(2):
        x = torch.randn(n * mp + 3, 2, page, 64, generator=g)
        if which == 0:
            x[..., 0] = 0.0
        value, byte = ref.encode(x.to(F64), kind)
        pools.append((value * torch.exp2(127 - byte.to(F64))[..., None], byte.to(torch.uint8)))
    cache = (pools[0][0].float().to(KINDS[kind]), pools[1][0].float().to(KINDS[kind]), pools[0][1], pools[1][1])
    return q.to(TYPES[dtype]), cache, pages, torch.tensor(lens, dtype=torch.int32)


def attend(kda, q, cache, pages, lens, window=0):
    out, lse = kda.attn_step(q.cuda(), kda.KVCache(*(t.cuda() for t in cache)), pages.cuda(), lens.cuda(), window=window,
                             want_lse=True)
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype,kind", FORMS)
@pytest.mark.parametrize("T,rep", ROWS)
@pytest.mark.parametrize("page", [4, 16, 64])
def test_powers_of_rows_that_nobody_sees(kda, page, T, rep, dtype, kind):
    """Finite rows of any power before every token's window, behind the length and in later drafted tokens
    leave every bit of the output as it is."""
    lens, w = [200, 450, 130], 20
    q, cache, pages, ln = state(lens, T, rep, page, dtype, kind, 1, most=1200)
    for cols, window in ((pages, w), (pages[:, :512 // page].contiguous(), w), (pages, 0)):  # split, a block per item
        want, wl = attend(kda, q, cache, cols, ln, window)
        for byte in (150, 170, 200, 254):
            spoiled = [t.clone() for t in cache]
            for b, n in enumerate(lens):
                first = max(0, n - T + 1 - window) if window else 0
                for p in [*range(max(0, first - 130), first), *range(n, n + 40)]:
                    at = int(pages[b, p // page]), p % page
                    spoiled[2][at[0], :, at[1]] = byte
                    spoiled[3][at[0], :, at[1]] = byte
            got, gl = attend(kda, q, spoiled, cols, ln, window)
            assert torch.equal(got, want) and torch.equal(gl, wl), (byte, window)
            if T > 1:  # the last drafted token's value: for itself alone
                for b, n in enumerate(lens):
                    spoiled[3][int(pages[b, (n - 1) // page]), :, (n - 1) % page] = byte
                got, gl = attend(kda, q, spoiled, cols, ln, window)
                assert torch.equal(got[:, :-1], want[:, :-1]) and torch.equal(gl[:, :-1], wl[:, :-1]), (byte, window)


@pytest.mark.parametrize("dtype,kind", FORMS)
@pytest.mark.parametrize("T,rep", ROWS)
@pytest.mark.parametrize("power,key", [(14, -60.0), (24, -60.0), (44, -60.0), (100, -120.0)])
def test_powers_of_rows_without_weight(kda, power, key, T, rep, dtype, kind):
    """A seen row of large power whose weight (e^-60, e^-120) leaves nothing of it takes no precision from the
    others: over caches in parts and over short tables, as the first row of a tile and as the newest."""
    lens = [333, 120, 1500, 9]
    q, cache, pages, ln = state(lens, T, rep, 16, dtype, kind, 2)
    cache = [t.clone() for t in cache]
    for b, places in enumerate(([0, 131], [119 - T], [64, 700, 1499 - T], [0])):
        for p in places:
            at = int(pages[b, p // 16]), p % 16
            key_row = torch.zeros(2, 64, dtype=F64)
            key_row[:, 0] = key
            value, byte = ref.encode(key_row, kind)
            cache[0][at[0], :, at[1]] = (value * torch.exp2(127 - byte.to(F64))[:, None]).float().to(KINDS[kind])
            cache[2][at[0], :, at[1]] = byte.to(torch.uint8)
            cache[3][at[0], :, at[1]] += power
    sizes = (cache[0], cache[1].float().abs().to(KINDS[kind]), *cache[2:])
    for some in ((0, 1, 2, 3), (0, 1, 3)):  # with and without the long one
        i = list(some)
        m = max(1, -(-int(ln[i].max()) // 16))
        cols = pages[i, :m].contiguous()
        got, lse = attend(kda, q[i], cache, cols, ln[i])
        want, wl = ref.attn(q[i], cache, cols, ln[i], 0.125)
        spread, _ = ref.attn(q[i], sizes, cols, ln[i], 0.125)
        f32 = dtype == "f32"
        tol = want.abs() * (2.0 ** -24 if f32 else 2.0 ** -8) + spread * (2.0 ** -15 if f32 else 2.0 ** -12 + 2.0 ** -13)
        assert ((got.to(F64) - want).abs() <= tol + 2.0 ** -20 * spread.amax(-1, keepdim=True)).all(), \
            ((got.to(F64) - want).abs() / spread).max()
        assert ((lse.to(F64) - wl).abs() <= (2.0 ** -16 if f32 else 2.0 ** -13)).all()


@pytest.mark.parametrize("dtype,kind", FORMS)
@pytest.mark.parametrize("T,rep", [(1, 4), (8, 4)])
def test_powers_from_end_to_end(kda, T, rep, dtype, kind):
    """Values of all sizes from 2^-76 to 2^117, one size to a sequence, and rows of zeros between them: the output is as
    exact for each."""
    n = 90
    q, cache, pages, ln = state([n] * 8, T, rep, 16, dtype, kind, 3)
    cache = [t.clone() for t in cache]
    for b, byte in enumerate((46, 55, 70, 90, 127, 160, 200, 235)):
        for col in pages[b].tolist():
            cache[3][col] = cache[3][col] - 120 + byte
            cache[1][col, :, 5::7] = torch.zeros(1).to(KINDS[kind])
            cache[3][col, :, 5::7] = 1
    got, lse = attend(kda, q, cache, pages, ln)
    up = [torch.exp2(torch.tensor(120.0 - x, dtype=F64)) for x in (46, 55, 70, 90, 127, 160, 200, 235)]
    want, wl = ref.attn(q, cache, pages, ln, 0.125)
    spread, _ = ref.attn(q, (cache[0], cache[1].float().abs().to(KINDS[kind]), *cache[2:]), pages, ln, 0.125)
    f32 = dtype == "f32"
    for b in range(8):  # compared at the size of the others
        err, size, sp = ((x[b].to(F64) * up[b]) for x in (got.to(F64) - want, want.abs(), spread))
        assert (err.abs() <= size * (2.0 ** -24 if f32 else 2.0 ** -8) + sp * (2.0 ** -15 if f32 else 2.0 ** -12 + 2.0 ** -13)).all(), b
    assert ((lse.to(F64) - wl).abs() <= (2.0 ** -16 if f32 else 2.0 ** -13)).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_lse_where_all_values_are_zero(kda, kind):
    """Rows of zeros have the smallest power: outputs of zeros, and lse as for any values."""
    q, cache, pages, ln = state([700, 30], 2, 4, 16, "bf16", kind, 4)
    none = (cache[0], torch.zeros_like(cache[1].float()).to(KINDS[kind]), cache[2], torch.full_like(cache[3], 1))
    got, lse = attend(kda, q, none, pages, ln)
    assert not got.any()
    assert ((lse.to(F64) - ref.attn(q, none, pages, ln, 0.125)[1]).abs() <= 2.0 ** -13).all()
    assert math.isfinite(lse.sum())
