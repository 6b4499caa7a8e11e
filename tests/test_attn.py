"""The attention layers' operators against plain float64 forms.

Tolerances.  A rounding to a type of p bits is off by at most eps / 2 of the value (bf16 2^-8, float32
2^-24).  Norms: a sum of up to 256 squares in float32, its root, two products and the rotation's two
products and sum stay within 16 roundings (2^-20) of the pair's size, the angle within 2^-22; written
values are rounded once more.  Attention: scores are sums of up to 128 products in float32, at most
about 128 / 2 roundings of sum |q k| scale, which moves a weight by that much relatively; the weights'
own rounding is 2^-17 at most where they enter 16-bit products (bf16 caches), and the sums of weights
add 2^-20: taken together 2^-13 of the largest value in bf16 (sum |q k| scale up to 8) and 2^-15 in
float32, and the output's rounding.  Over 8-bit caches a bf16 query's weights are f16, 11 bits: each is
off by 2^-12 of itself at most, the sum of p v by 2^-12 of the sum of p |v| (computed beside the
reference).  Cache rows and drawn tokens are exact.
"""
import math

import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------------------
# norms with rotation
# ---------------------------------------------------------------------------
def qk_inputs(tokens, hq, hk, d, rot, dtype, seed, far=1 << 20):
    g = gen(seed)
    q, k = (torch.randn(tokens, h, d, generator=g).to(TYPES[dtype]) for h in (hq, hk))
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(2))
    pos = torch.randint(-far, far, (tokens,), generator=g, dtype=torch.int32)
    freqs = 10000.0 ** (-2 * torch.arange(rot // 2, dtype=F64) / max(rot, 1))
    return q, k, wq, wk, pos, freqs


QK_SIZES = [(1, 1, 1, 2, 2), (5, 3, 1, 64, 64), (9, 4, 2, 128, 128), (3, 32, 8, 128, 64), (7, 2, 1, 96, 48),
            (4, 5, 3, 256, 256), (2, 1, 7, 250, 90), (33, 2, 2, 64, 0), (6, 2, 1, 34, 6), (700, 7, 2, 128, 128),
            (11, 1, 1, 72, 40), (300, 8, 1, 256, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("size", QK_SIZES)
def test_qknorm(kda, size, inter, dtype):
    tokens, hq, hk, d, rot = size
    q, k, wq, wk, pos, freqs = qk_inputs(*size, dtype, 1)
    got = kda.qknorm_fwd(dev(q), dev(k), dev(pos), dev(freqs), q_weight=dev(wq), k_weight=dev(wk), interleaved=inter)
    for y, x, w in zip(got, (q, k), (wq, wk)):
        want = ref.qknorm(x.to(F64), pos, freqs, w.to(F64), inter)
        assert y.dtype == x.dtype and y.shape == x.shape
        err = (y.cpu().to(F64) - want).abs()
        assert (err <= want.abs() * ROUND[x.dtype] + 2.0 ** -19 * want.abs().max()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("size", QK_SIZES)
def test_qknorm_gradient(kda, size, inter, dtype):
    """dx: like the forward, with the mean's sum; the weights': a sum over rows, each row's term within
    2^-19, added in float32 by threads that keep at most rows / 4 of them (the order is a tree: 2^-19 of
    the sum of sizes is well above)."""
    tokens, hq, hk, d, rot = size
    q, k, wq, wk, pos, freqs = qk_inputs(*size, dtype, 2)
    g = gen(3)
    dq, dk = (torch.randn(x.shape, generator=g).to(x.dtype) for x in (q, k))
    got = kda.qknorm_bwd(dev(q), dev(k), dev(dq), dev(dk), dev(pos), dev(freqs), q_weight=dev(wq), k_weight=dev(wk),
                         interleaved=inter)
    for x, w, dy, dx, dw in ((q, wq, dq, got[0], got[2]), (k, wk, dk, got[1], got[3])):
        xd, wd = x.to(F64).requires_grad_(), w.to(F64).requires_grad_()
        y = ref.qknorm(xd, pos, freqs, wd, inter)
        gx, gw = torch.autograd.grad((y * dy.to(F64)).sum(), (xd, wd))
        # sizes of what cancels in dx: 1 / rms times the row's cotangent
        size_x = (dy.to(F64).abs().amax(-1, keepdim=True) * 2 + gx.abs().amax(-1, keepdim=True)) \
            * torch.rsqrt(x.to(F64).square().mean(-1, keepdim=True) + 1e-6)
        assert ((dx.cpu().to(F64) - gx).abs() <= gx.abs() * ROUND[x.dtype] + 2.0 ** -18 * size_x).all()
        size_w = (dy.to(F64).abs().amax() * x.to(F64).abs().amax()) * tokens * x.shape[1]
        assert dw.dtype == torch.float32
        assert ((dw.cpu().to(F64) - gw).abs() <= 2.0 ** -18 * size_w / max(1, math.sqrt(tokens * x.shape[1]) / 4)).all()


def test_qknorm_gradient_by_differences(kda):
    """Central differences of the float32 forward along a random direction: the forward is smooth at this
    scale, h^2 / 6 times the third derivative is below 1e-3 of the gradient, the forward's rounding
    (2^-21 of about 900 unit terms, random signs) over h = 1/64 below 2e-3."""
    q, k, wq, wk, pos, freqs = (dev(t) for t in qk_inputs(3, 2, 1, 64, 64, "f32", 4))
    g = torch.Generator(device="cuda").manual_seed(5)
    dq, dk, vq, vk = (torch.randn(t.shape, device="cuda", generator=g) for t in (q, k, q, k))
    uq, uk = (torch.randn(64, device="cuda", generator=g) for _ in range(2))
    gr = kda.qknorm_bwd(q, k, dq, dk, pos, freqs, q_weight=wq, k_weight=wk)
    h = 1 / 64

    def loss(s):
        a, b = kda.qknorm_fwd(q + s * vq, k + s * vk, pos, freqs, q_weight=wq + s * uq, k_weight=wk + s * uk)
        return ((a.double() * dq).sum() + (b.double() * dk).sum()).item()
    slope = (loss(h) - loss(-h)) / (2 * h)
    want = sum((a.double() * b).sum().item() for a, b in zip(gr, (vq, vk, uq, uk)))
    assert abs(slope - want) <= 1e-2 * max(1.0, abs(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_qknorm_views_parts_and_places(kda, dtype):
    """Column slices of one projection (even and odd offsets), no weights, no rotation, no k, in place,
    the farthest positions."""
    t, hq, hk, d = 13, 4, 2, 64
    q, k, wq, wk, pos, freqs = qk_inputs(t, hq, hk, d, d, dtype, 6)
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, -2 ** 31, 0
    want_q = ref.qknorm(q.to(F64), pos, freqs, wq.to(F64))
    want_k = ref.qknorm(k.to(F64), pos, freqs, wk.to(F64))

    def check(y, want, extra=1.0):
        err = (y.cpu().to(F64) - want).abs()
        assert (err <= want.abs() * ROUND[q.dtype] + extra * 2.0 ** -19 * want.abs().max()).all()
    a = dict(q_weight=dev(wq), k_weight=dev(wk))
    for off in (0, 8, 1):
        p = torch.zeros(t, (hq + hk) * d + 24 + off, dtype=q.dtype, device="cuda")
        qs = p[:, off:off + hq * d].unflatten(-1, (hq, d))
        ks = p[:, off + hq * d + 8:off + hq * d + 8 + hk * d].unflatten(-1, (hk, d))
        qs.copy_(q)
        ks.copy_(k)
        y, z = kda.qknorm_fwd(qs, ks, dev(pos), dev(freqs), **a)
        check(y, want_q)
        check(z, want_k)
    y, z = kda.qknorm_fwd(dev(q)[None], None, dev(pos)[None], dev(freqs), q_weight=dev(wq))
    assert z is None and y.shape == (1, t, hq, d)
    check(y[0], want_q)
    x = dev(q).clone()
    y, _ = kda.qknorm_fwd(x, None, dev(pos), dev(freqs), q_weight=dev(wq), q_out=x)
    assert y is x
    check(x, want_q)
    y, z = kda.qknorm_fwd(dev(q), dev(k), dev(pos), dev(freqs))
    check(y, ref.qknorm(q.to(F64), pos, freqs))
    y, z = kda.qknorm_fwd(dev(q), dev(k), None, None, **a)
    check(z, ref.qknorm(k.to(F64), pos, None, wk.to(F64)))
    dq, dk, dwq, dwk = kda.qknorm_bwd(dev(q), dev(k), dev(q), dev(k), dev(pos), dev(freqs))
    assert dwq is None and dwk is None
    check(dq, ref.qknorm(q.to(F64), -pos.long(), freqs))  # without a norm: the rotation back
    e, _ = kda.qknorm_fwd(dev(q)[:0], dev(k)[:0], dev(pos)[:0], dev(freqs), **a)
    assert e.shape == (0, hq, d)
    *_, dwq, dwk = kda.qknorm_bwd(dev(q)[:0], dev(k)[:0], dev(q)[:0], dev(k)[:0], dev(pos)[:0], dev(freqs), **a)
    assert not dwq.any() and not dwk.any()


# ---------------------------------------------------------------------------
# paged cache
# ---------------------------------------------------------------------------
def table(n, max_pages, pool, seed):
    return torch.randperm(pool, generator=gen(seed))[:n * max_pages].reshape(n, max_pages).to(torch.int32)


def wild(shape, dtype, seed):
    """Rows of very different sizes, with zeros, ties, powers of two, the type's ends and values that
    are not finite."""
    g = gen(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-40, 40, shape[:-1], generator=g).float())[..., None]
    f = x.reshape(-1, shape[-1])
    i = torch.arange(f.shape[0])
    f[i % 11 == 1] = 0.0
    f[i % 11 == 2] = torch.arange(shape[-1]).float() - 63.5
    f[i % 11 == 3] = torch.exp2(torch.randint(-30, 2, (shape[-1],), generator=g).float())
    f[i % 11 == 4, 0] = math.inf
    f[i % 11 == 5, 1] = math.nan
    f[i % 11 == 6] *= 2.0 ** -100
    f[i % 11 == 7, 2] = 3e38
    f[i % 11 == 8] = 448.0
    f[i % 11 == 9] = 127.0 * 2.0 ** -20
    return f.reshape(shape).to(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16), (128, 1)])
def test_cache_round_trip(kda, dtype, kind, d, page):
    h, T, n = 3, 7, 5
    mp = -(-70 // page)
    lens = torch.tensor([7, 70, 33, 3, 0], dtype=torch.int32)  # the last two hold fewer tokens than come
    k, v = (wild((n, T, h, d), TYPES[dtype], s) for s in (1, 2))
    pages = table(n, mp, n * mp + 2, 3)
    cache = kda.kv_cache(n * mp + 2, page, h, d, dtype=KINDS[kind])
    before = []
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(17)
            before.append(t.clone())
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    kda.cache_write(dev(k), dev(v), cache, dev(pages), dev(lens), workspace=ws)
    assert kda.read_device_status(ws) == 0
    touched = torch.zeros(n * mp + 2, page, dtype=torch.bool)
    for b in range(n):
        for t in range(T):
            p = int(lens[b]) - T + t
            if p < 0:
                continue
            at = int(pages[b, p // page]), p % page
            touched[at] = True
            for pool, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
                row = x[b, t].to(F64)
                got = pool[at[0], :, at[1]].cpu()
                if kind in ("e4m3", "int8"):
                    want, byte = ref.encode(row, kind)
                    assert torch.equal(scale[at[0], :, at[1]].cpu().long(), byte)
                    val = got.float().to(F64) * torch.exp2(byte.to(F64) - 127)[:, None]
                    bad = byte == 255
                    assert torch.equal(val[~bad], want[~bad])
                    assert not got.view(torch.uint8)[bad].any()
                else:
                    assert torch.equal(got.view(torch.uint8), x[b, t].to(got.dtype).view(torch.uint8)) \
                        or torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(x[b, t].to(got.dtype).float()))
    for t, was in zip((x for x in cache if x is not None), before):
        keep = (~touched).cuda()
        a, b = (y.view(torch.uint8).transpose(1, 2)[keep] for y in (t, was))
        assert torch.equal(a, b)  # every other row as it was
    for out in (torch.float32, torch.bfloat16):
        rk, rv = kda.cache_read(cache, dev(pages), dev(lens), T, dtype=out, workspace=ws)
        assert kda.read_device_status(ws) == 0
        for y, x in ((rk, k), (rv, v)):
            want = x.to(KINDS[kind]).to(F64) if kind in ("f32", "bf16") else ref.encode(x.to(F64), kind)[0]
            for b in range(n):
                for t in range(T):
                    if int(lens[b]) - T + t < 0:
                        want[b, t] = 0
            want = want.to(torch.float32).to(out)
            assert torch.equal(torch.nan_to_num(y.cpu().float()), torch.nan_to_num(want.float()))
            assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_cache_packed_views_and_bad_places(kda, kind):
    """Packed sequences (one empty), slices of a projection at odd offsets, pools with a stride between
    pages, rows behind the last sequence, pages outside the pool, lengths past the table."""
    h, d, page, lens_new = 2, 64, 16, [5, 0, 21, 2]
    cu = torch.tensor([0, 5, 5, 26, 28], dtype=torch.int32)
    total = torch.tensor([5, 9, 40, 2], dtype=torch.int32)
    mp, pool = 3, 14
    pages = table(4, mp, pool, 5)
    both = torch.zeros(pool, 2, h, page, d, dtype=KINDS[kind], device="cuda")
    sc = [None, None] if kind == "bf16" else [torch.zeros(pool, h, page, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = kda.KVCache(both[:, 0], both[:, 1], *sc)
    x = torch.randn(1, 28, 2 * h * d + 3, generator=gen(6)).bfloat16()
    for off in (0, 3):
        p = dev(x)
        k, v = (p[..., o:o + h * d].unflatten(-1, (h, d)) for o in (off, off + h * d))
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        kda.cache_write(k, v, cache, dev(pages), dev(total), cu_seqlens=dev(cu), workspace=ws)
        assert kda.read_device_status(ws) == 0
        rk, rv = kda.cache_read(cache, dev(pages), dev(total), 28, cu_seqlens=dev(cu))
        for y, z in ((rk, k), (rv, v)):
            want = z.cpu() if kind == "bf16" else ref.encode(z.cpu().to(F64), kind)[0].bfloat16()
            assert torch.equal(y.cpu(), want)
    # rows behind the last sequence stay; short offsets are reported
    short = torch.tensor([0, 5, 5, 20, 22], dtype=torch.int32)
    mark = torch.full((1, 28, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    mv = mark.clone()
    kda.cache_read(cache, dev(pages), dev(total), 28, cu_seqlens=dev(short), k=mark, v=mv, workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_BAD_SEQLENS
    assert (mark[:, 22:] == 7).all() and (mv[:, 22:] == 7).all() and not (mark[:, :22] == 7).all()
    # a page outside the pool, a length past the table
    bad = pages.clone()
    bad[2, 1], bad[3, 0] = pool, -1
    was = both.clone()
    kda.cache_write(k, v, cache, dev(bad), dev(total), cu_seqlens=dev(cu), workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(was.view(torch.uint8), both.view(torch.uint8))  # the same values where they went
    rk, _ = kda.cache_read(cache, dev(bad), dev(total), 28, cu_seqlens=dev(cu), workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert not rk[0, 26:].any() and rk[0, :5].any()
    far = torch.tensor([5, 9, 2 ** 31 - 1, 49], dtype=torch.int32)
    kda.cache_write(k, v, cache, dev(pages), dev(far), cu_seqlens=dev(cu), workspace=ws)
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# attention of new tokens
# ---------------------------------------------------------------------------
def attn_inputs(kda, lens, T, hq, hk, d, page, dtype, kind, seed, max_pages=None):
    n = len(lens)
    mp = max_pages or max(1, -(-max(lens) // page))
    pool = n * mp + 2
    g = gen(seed)
    pages = table(n, mp, pool, seed + 1)
    q = torch.randn(n, T, hq, d, generator=g).to(TYPES[dtype])
    pools = []
    for _ in range(2):
        x = torch.randn(pool, hk, page, d, generator=g)
        if kind in ("f32", "bf16"):
            pools.append((x.to(KINDS[kind]), None))
        else:
            val, byte = ref.encode(x.to(F64), kind)
            code = (val * torch.exp2(127 - byte.to(F64))[..., None]).float().to(KINDS[kind])
            pools.append((code, byte.to(torch.uint8)))
    cache = (pools[0][0], pools[1][0], pools[0][1], pools[1][1])
    return q, cache, pages, torch.tensor(lens, dtype=torch.int32)


def attn_check(kda, q, cache, pages, lens, window=0, scale=None, status=0):
    got, lse = kda.attn_step(dev(q), kda.KVCache(*map(dev, cache)), dev(pages), dev(lens), window=window, scale=scale,
                             want_lse=True)
    want, want_lse = ref.attn(q, cache, pages, lens, q.shape[-1] ** -0.5 if scale is None else scale, window)
    assert got.dtype == q.dtype and got.shape == q.shape
    tol = 2.0 ** -13 if q.dtype is torch.bfloat16 else 2.0 ** -15
    top = want.abs().nan_to_num().max().clamp(min=1e-3)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    err = (got.cpu().to(F64) - want).abs().nan_to_num()
    spread = 0.0
    if cache[2] is not None and q.dtype is torch.bfloat16:
        sizes = cache[1].float().abs().to(cache[1].dtype)
        spread = ref.attn(q, (cache[0], sizes, *cache[2:]), pages, lens,
                          q.shape[-1] ** -0.5 if scale is None else scale, window)[0].nan_to_num()
    assert (err <= want.abs().nan_to_num() * ROUND[q.dtype] + tol * top + 2.0 ** -12 * spread).all(), err.max()
    gone = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, gone)
    assert not got.cpu()[gone].any()
    diff = (lse.cpu().to(F64) - want_lse)[~gone].abs().nan_to_num()
    assert (diff <= 1e-3).all()
    return got, lse


ATTN = [  # lens, T, hq, hk, d, page, window
    ([1], 1, 1, 1, 64, 16, 0), ([5, 1, 64, 65], 1, 4, 2, 128, 16, 0), ([200, 63, 128, 1], 1, 8, 1, 128, 64, 0),
    ([17, 300], 8, 8, 2, 64, 32, 0), ([90, 8, 3, 0], 8, 14, 2, 128, 16, 0), ([700], 1, 2, 2, 64, 128, 0),
    ([700, 2], 2, 7, 7, 128, 64, 100), ([130, 64, 65, 1], 5, 16, 1, 64, 8, 3), ([1000], 8, 32, 2, 128, 64, 37),
    ([0, 0], 1, 4, 4, 128, 16, 0), ([257] * 5, 3, 12, 2, 64, 1, 0), ([64, 128, 192], 1, 20, 1, 128, 2, 64)]


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("f32", "e4m3"), ("f32", "int8"), ("bf16", "bf16"),
                                        ("bf16", "e4m3"), ("bf16", "int8")])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(map(str, c[1:])))
def test_attn(kda, case, dtype, kind):
    lens, T, hq, hk, d, page, window = case
    args = attn_inputs(kda, lens, T, hq, hk, d, page, dtype, kind, 7)
    attn_check(kda, *args, window=window)


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3")])
def test_attn_what_is_not_seen(kda, dtype, kind):
    """NaN and infinities behind the lengths, in other rows of a page, before the window, and in keys and
    values of later drafted tokens reach no token that does not see them; those that do get NaN."""
    lens, T, hq, hk, d, page, w = [70, 5, 130], 4, 8, 2, 64, 16, 20
    q, cache, pages, ln = attn_inputs(kda, lens, T, hq, hk, d, page, dtype, kind, 8, max_pages=10)
    cache = [None if t is None else t.clone() for t in cache]

    def spoil(b, p, which, what):
        at = int(pages[b, p // page]), p % page
        if kind == "e4m3":
            cache[which + 2][at[0], :, at[1]] = 255
            cache[which].view(torch.uint8)[at[0], :, at[1]] = 0
        else:
            cache[which][at[0], :, at[1]] = what
    for b, n in enumerate(lens):
        for p in range(n, pages.shape[1] * page):
            spoil(b, p, 0, math.nan)
            spoil(b, p, 1, math.inf if p % 2 else math.nan)
    attn_check(kda, q, cache, pages, ln)
    for b, n in enumerate(lens):  # before every token's window
        for p in range(0, n - T + 1 - w):
            spoil(b, p, 0, math.inf)
            spoil(b, p, 1, math.nan)
    got, _ = attn_check(kda, q, cache, pages, ln, window=w)
    assert torch.isfinite(got).all()
    # the newest token of the first, the oldest in the first token's window of the third
    spoil(0, 69, 1, math.nan)
    spoil(2, 130 - T + 1 - w, 1, math.nan)
    got, _ = attn_check(kda, q, cache, pages, ln, window=w)
    assert torch.isnan(got[0, 3]).all() and torch.isfinite(got[0, :3]).all()
    assert torch.isnan(got[2, 0]).all() and torch.isfinite(got[2, 1:]).all()
    spoil(0, 68, 0, math.nan)
    got, _ = attn_check(kda, q, cache, pages, ln, window=w)
    assert torch.isnan(got[0, 2:]).all() and torch.isfinite(got[0, :2]).all()


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "int8")])
def test_attn_missing_pages_and_lengths(kda, dtype, kind):
    """Pages outside the pool are unseen and reported, as are lengths past the table; negative lengths
    are empty."""
    q, cache, pages, ln = attn_inputs(kda, [100, 40, 64], 2, 4, 2, 64, 16, dtype, kind, 9, max_pages=7)
    pages[0, 2], pages[1, 0] = 10 ** 6, -5
    shape_ws = lambda: torch.empty(kda.attn.attn_workspace_size(kda.attn._attn_shape(
        dev(q), tuple(map(dev, cache)), dev(pages), dev(ln), None, 0)), dtype=torch.uint8, device="cuda")
    attn_check(kda, q, cache, pages, ln)
    for lens, status in (([100, 40, 64], kda.KDA_ERR_INVALID_ARG), ([30, 0, 64], 0), ([30, 0, 113], kda.KDA_ERR_INVALID_ARG),
                         ([-3, 0, 1], 0)):
        ws = shape_ws()
        lens = torch.tensor(lens, dtype=torch.int32)
        out = kda.attn_step(dev(q), kda.KVCache(*map(dev, cache)), dev(pages), dev(lens), workspace=ws)
        assert kda.read_device_status(ws) == status, lens
        want = ref.attn(q, cache, pages, lens, 64 ** -0.5)[0]
        assert ((out.cpu().to(F64) - want).abs() <= want.abs() * ROUND[q.dtype] + 2.0 ** -13 * 4).all()


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "int8")])
def test_attn_long_splits_repeat(kda, dtype, kind):
    """Long caches in many parts, sharp and flat scores, a strided q; the same bits twice."""
    n, T, hq, hk, d, page = 3, 2, 8, 2, 128, 64
    lens = [20011, 1, 9000]
    q, cache, pages, ln = attn_inputs(kda, lens, T, hq, hk, d, page, dtype, kind, 10)
    for scale in (0.0, 0.05, 3.0, -1.0):
        pad = torch.zeros(n, T, hq * d + 24, dtype=q.dtype)
        pad[..., 8:8 + hq * d] = q.flatten(2)
        qs = pad.cuda()[..., 8:8 + hq * d].unflatten(-1, (hq, d))
        c = kda.KVCache(*map(dev, cache))
        a, la = kda.attn_step(qs, c, dev(pages), dev(ln), scale=scale, want_lse=True)
        b, lb = kda.attn_step(qs, c, dev(pages), dev(ln), scale=scale, want_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)
        k = torch.stack([x.double() for x in rows_gpu(c.k, c.k_scale, dev(pages)[0], lens[0])])
        v = torch.stack([x.double() for x in rows_gpu(c.v, c.v_scale, dev(pages)[0], lens[0])])
        for t in range(T):
            m = lens[0] - T + t + 1
            s = torch.einsum("grd,gkd->grk", qs[0, t].double().reshape(hk, hq // hk, d), k[:, :m]) * scale
            want = torch.einsum("grk,gkd->grd", torch.softmax(s, -1), v[:, :m]).reshape(hq, d)
            # sharp scores: up to 128 roundings of |q k| scale, about 2^-17 x 100 x 3
            tol = (2.0 ** -13 if q.dtype is torch.bfloat16 else 2.0 ** -15) * (4 if abs(scale) >= 1 else 1)
            err = (a[0, t].double() - want).abs()
            spread = 0.0
            if cache[2] is not None and q.dtype is torch.bfloat16:
                spread = torch.einsum("grk,gkd->grd", torch.softmax(s, -1), v[:, :m].abs()).reshape(hq, d)
            assert (err <= want.abs() * ROUND[q.dtype] + tol * want.abs().max().clamp(min=0.1)
                    + 2.0 ** -12 * spread).all(), (scale, err.max())
            assert ((la[0, t].double() - torch.logsumexp(s, -1).flatten()).abs() <= 1e-3).all()


def rows_gpu(pool, scale, ids, n):
    x = pool.view(torch.uint8)[ids.long()].view(pool.dtype).float() if scale is not None else pool[ids.long()].float()
    if scale is not None:
        x = x * torch.exp2(scale[ids.long()].float() - 127)[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


# ---------------------------------------------------------------------------
# verification of drafts
# ---------------------------------------------------------------------------
def probs(B, K, V, seed, dtype=torch.float32, sharp=2.0):
    g = gen(seed)
    x = sharp * torch.randn(B, K + 1, V, generator=g)
    p = torch.softmax(x, -1)
    q = torch.softmax(x[:, :K] + torch.randn(B, K, V, generator=g), -1)
    drafts = torch.stack([torch.multinomial(q[b], 1, generator=g)[:, 0] for b in range(B)]) if K else torch.zeros(B, 0)
    return p.to(dtype), q.to(dtype), drafts.to(torch.int32), torch.rand(B, K + 1, generator=g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (3, 1, 2), (5, 4, 37), (2, 7, 128), (4, 3, 1000), (3, 31, 129), (2, 2, 50257),
                                   (33, 3, 4099)])
def test_verify(kda, B, K, V, dtype):
    p, q, d, u = probs(B, K, V, 11, TYPES[dtype])
    for qq, counts in ((q, None), (None, None), (q, torch.arange(B, dtype=torch.int32) % (K + 2) - 1)):
        got = kda.draft_verify(dev(p), dev(qq), dev(d), dev(u), num_draft=dev(counts))
        want = ref.verify(p, qq, d, u, counts)
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_verify_ends(kda):
    """Equal rows (all kept), impossible drafts, nothing left of p - q, ends of the random numbers,
    NaN, negative and large values, tokens outside the vocabulary, idle rows."""
    B, K, V = 8, 2, 300
    p, q, d, u = probs(B, K, V, 12)
    q[0] = p[0, :K]                      # kept whatever u < 1 says
    u[0] = 1 - 2.0 ** -24
    p[1, 0, int(d[1, 0])] = 0            # refused at 0 < 0
    u[1] = 0.0
    q[2, 0] = 1.0                        # nothing left: p itself
    u[2, 0] = 1 - 2.0 ** -24
    p[3, :, ::2] = math.nan
    p[4, :, 5] = -1.0
    p[4, :, 7] = 3.0
    d[5, 0] = V                          # outside: refused and reported
    d[6, 1] = -1
    p[7] = 0.0                           # nothing to draw from
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    got = kda.draft_verify(dev(p), dev(q), dev(d), dev(u), workspace=ws)
    want = ref.verify(p, q, d, u)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert got[1][0] == K + 1 and got[0][7, 0] == -1
    counts = torch.tensor([2, 1, 0, -1, 3, -7, 2, 2], dtype=torch.int32)
    got = kda.draft_verify(dev(p), dev(q), dev(d), dev(u), num_draft=dev(counts), workspace=ws)
    want = ref.verify(p, q, d, u, counts)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    assert kda.read_device_status(ws) == kda.KDA_ERR_INVALID_ARG  # 3 and -7
    got = kda.draft_verify(dev(p[:3]), dev(q[:3]), dev(d[:3]), dev(u[:3]), workspace=ws)
    assert kda.read_device_status(ws) == 0


def test_verify_follows_the_distribution(kda):
    """Drawn over an even grid of random numbers, each token comes as often as its weight says, to one
    step of the grid at each end."""
    V, n = 7, 4096
    p = torch.softmax(torch.randn(1, 1, V, generator=gen(13)), -1)
    u = ((torch.arange(n) + 0.5) / n)[:, None].float()
    got, commit = kda.draft_verify(dev(p.expand(n, 1, V).contiguous()), None, dev(torch.zeros(n, 0, dtype=torch.int32)), dev(u))
    assert (commit == 1).all()
    freq = torch.bincount(got[:, 0].long().cpu(), minlength=V) / n
    assert ((freq - p[0, 0]).abs() <= 2 / n).all()


# ---------------------------------------------------------------------------
# graphs, streams
# ---------------------------------------------------------------------------
def test_graph_replay_and_streams(kda):
    """All four captured into one graph on a stream of the caller's; replayed on new inputs and lengths."""
    B, T, hq, hk, d, page, V = 3, 2, 4, 2, 64, 16, 500
    q, k, wq, wk, pos, freqs = (dev(t) for t in qk_inputs(B * T, hq, hk, d, d, "bf16", 14))
    v = torch.randn_like(k)
    cache = kda.kv_cache(3 * 6, page, hk, d, dtype=torch.float8_e4m3fn)
    for t in cache:
        t.view(torch.uint8).fill_(100)
    pages, lens = dev(table(3, 6, 18, 15)), torch.tensor([2, 50, 90], dtype=torch.int32, device="cuda")
    p, qq, dr, u = (dev(t) for t in probs(B, T - 1, V, 16))

    def step():
        a, b = kda.qknorm_fwd(q.view(B, T, hq, d), k.view(B, T, hk, d), pos.view(B, T), freqs, q_weight=wq, k_weight=wk)
        kda.cache_write(b, v.view(B, T, hk, d), cache, pages, lens)
        o = kda.attn_step(a, cache, pages, lens)
        r = kda.cache_read(cache, pages, lens, T)
        return (o, *r, *kda.draft_verify(p, qq, dr, u))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = step()
    for seed, ln in ((17, [40, 3, 96]), (18, [1, 0, 2])):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        lens.copy_(torch.tensor(ln))
        u.copy_(torch.rand(u.shape, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,kind", [("f32", "f32"), ("f32", "int8"), ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("T,rep,d,page,copies", [(1, 4, 128, 16, 1), (3, 5, 64, 64, 1), (8, 4, 128, 32, 1), (8, 9, 64, 4, 1), (2, 3, 64, 16, 8)])
def test_attn_short_tables(kda, dtype, kind, T, rep, d, page, copies):
    """Tables of up to 512 places take a block per item, longer ones are split: the same inputs under tables of
    256 and 512 places and of a page more, with pages that are not in the pool behind the lengths."""
    lens = [256, 0, 1, 255, T - 1, -3, 100, 17] * copies
    for cap, more in ((256, []), (512, [512, 257]), (512 + page, [512, 511])):
        q, cache, pages, ln = attn_inputs(kda, lens + more, T, 2 * rep, 2, d, page, dtype, kind, 21, max_pages=cap // page)
        for b, n in enumerate(ln.tolist()):
            pages[b, -(-max(n, 0) // page):] = -1 if b % 2 else 2 ** 30
        attn_check(kda, q, cache, pages, ln)
        attn_check(kda, q, cache, pages, ln, window=33)


@pytest.mark.parametrize("page", [1, 16, 64])
def test_attn_short_tables_report(kda, page):
    """With a workspace the status, without one none is kept: places past the table and pages not in the pool
    that a token sees, and none that it does not; a workspace with no sequences; too small ones refused."""
    q, cache, pages, ln = attn_inputs(kda, [512, 200, 0], 2, 4, 2, 64, page, "bf16", "int8", 22)
    q, cache, pages = dev(q), kda.KVCache(*map(dev, cache)), dev(pages)
    ws = torch.full((64,), -1, dtype=torch.int32, device="cuda")
    bad = pages.clone()
    bad[1, 63 // page] = 10 ** 6
    for lens, table_, window, status in (
            ([512, 200, 0], pages, 0, 0), ([513, 200, 0], pages, 0, kda.KDA_ERR_INVALID_ARG), ([512, 200, 0], pages, 0, 0),
            ([512, 200, 0], bad, 0, kda.KDA_ERR_INVALID_ARG), ([512, 0, 200], bad, 0, 0), ([512, 200, -9], bad, 8, 0),
            ([512, 64, 1], bad, 8, kda.KDA_ERR_INVALID_ARG)):
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = kda.attn_step(q, cache, table_, lens, window=window, workspace=ws)
        assert kda.read_device_status(ws) == status, (lens, window)
        assert torch.equal(kda.attn_step(q, cache, table_, lens, window=window), got)
    ws.fill_(-1)
    assert kda.attn_step(q[:0], cache, pages[:0], lens[:0], workspace=ws).shape == q[:0].shape
    assert kda.read_device_status(ws) == 0
    with pytest.raises(RuntimeError):
        kda.attn_step(q, cache, pages, lens, workspace=ws[:32])
