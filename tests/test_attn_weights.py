"""The bits with which weights enter the products: up to 8 query rows per key-value head the output is the rounding
of the exact result, but where that lies next to a tie.

Scores are exact (four products of small whole multiples of 1/4, scale 1/8, below 6 in powers of two): a weight is off by
2^-21 through its exponent's rounding and 2^-22 through the exponential; sums of at most 6 weights, 17 cut-off additions
(2^-23 each) and the quotient: below 2^-18 of the sum of p |v|.  Weights of 16 bits (bf16 caches) add 2^-17, of 22 bits
(codes) nothing that counts; 11 bits would add 2^-12 and fail for every 30th output.
"""
import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,rep", [(1, 1), (1, 4), (1, 8), (2, 4), (2, 3)])
@pytest.mark.parametrize("cap", [16, 1024])
def test_few_places(kda, cap, T, rep, d, kind):
    g = torch.Generator().manual_seed(1)
    n, mp = 96, cap // 16
    pool = 2 * n
    lens = torch.randint(T, 7, (n,), generator=g, dtype=torch.int32)
    pages = torch.randint(0, pool, (n, mp), generator=g, dtype=torch.int32)
    pages[:, 0] = torch.randperm(pool, generator=g)[:n]
    q = torch.zeros(n, T, 2 * rep, d)
    q[..., 3:60:16] = torch.randint(-16, 17, (n, T, 2 * rep, 4), generator=g) / 4
    k = torch.zeros(n, 16, 2, d)
    k[..., 3:60:16] = torch.randint(-2, 3, (n, 16, 2, 4), generator=g).float()
    v = torch.randn(n, 16, 2, d, generator=g)
    cache = kda.kv_cache(pool, 16, 2, d, dtype=KINDS[kind])
    full = torch.full((n,), 16, dtype=torch.int32)
    kda.cache_write(k.bfloat16().cuda(), v.bfloat16().cuda(), cache, pages.cuda(), full.cuda())
    got = kda.attn_step(q.bfloat16().cuda(), cache, pages.cuda(), lens.cuda(), scale=0.125).cpu().to(F64)
    held = tuple(None if t is None else t.cpu() for t in cache)
    sizes = (held[0], held[1].float().abs().to(KINDS[kind]), *held[2:])
    want, _ = ref.attn(q.bfloat16(), held, pages, lens, 0.125)
    spread, _ = ref.attn(q.bfloat16(), sizes, pages, lens, 0.125)
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -60))) - 8)
    slack = 2.0 ** -18 + (2.0 ** -17 if kind == "bf16" else 0.0)
    assert ((got - want).abs() <= half * (1 + 2.0 ** -8) + slack * spread).all(), ((got - want).abs() - half).max()
