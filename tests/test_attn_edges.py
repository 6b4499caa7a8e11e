"""The attention layers' operators together and at their edges: the speculative decoding example,
two graphs that share a workspace, pools and batches past 2^31 elements, streams, buffers of the
caller's, rows of all sizes."""
import os
import sys

import pytest
import torch

import _attn_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8, torch.bfloat16])
def test_hybrid_decode(kda, kind):
    """Rounds of drafts and single tokens go through bf16 stages of their own shapes: six roundings in a
    row (2^-9 of values up to about 4 rms each, with the products' growth) and, in 8 bits, codes that may
    fall to the neighbour (2^-4 of one row's part): 1e-1 of the rms."""
    import hybrid_decode
    a, b, pairs, kept = hybrid_decode.run(cache_dtype=kind)
    assert kept >= 6 * 3 * 2  # the sequences whose drafts are certain
    assert torch.equal(a.lens, b.lens)
    assert ((a.state - b.state).abs().max() / b.state.square().mean().sqrt()).item() <= 5e-2
    for x, y in pairs:
        if y.numel():
            assert torch.isfinite(x).all()
            assert ((x - y).abs().max() / y.square().mean().sqrt()).item() <= 1e-1


def attn_state(kda, n, hq, hk, d, page, most, kind, seed, T=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-most // page)
    cache = kda.kv_cache(n * per, page, hk, d, dtype=kind)
    pages = torch.randperm(n * per, device="cuda", generator=g).to(torch.int32).reshape(n, per)
    k, v = (torch.randn(n, most, hk, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    full = torch.full((n,), most, dtype=torch.int32, device="cuda")
    kda.cache_write(k, v, cache, pages, full)
    q = torch.randn(n, T, hq, d, device="cuda", generator=g).bfloat16()
    return q, cache, pages, full, k, v


def test_two_graphs_share_a_workspace(kda):
    """Two captured calls of different splits with one workspace, replayed by turns and with garbage in it
    between: each gives what it gives alone."""
    q, cache, pages, full, _, _ = attn_state(kda, 3, 8, 2, 128, 16, 5000, torch.int8, 1)
    short = torch.tensor([7, 0, 300], dtype=torch.int32, device="cuda")
    size = max(kda.attn.attn_workspace_size(kda.attn._attn_shape(q, cache, pages, full, None, 0)), 1 << 20)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [kda.attn_step(q, cache, pages, n, window=w) for n, w in ((full, 0), (short, 40))]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for n, w in ((full, 0), (short, 40)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(kda.attn_step(q, cache, pages, n, window=w, workspace=ws))
        graphs.append(graph)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        for i in (0, 1, 1, 0):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], want[i]), (fill, i)


def test_streams_and_own_buffers(kda):
    """Calls on a stream of the caller's, into its buffers; results as on the current stream."""
    q, cache, pages, full, k, v = attn_state(kda, 2, 4, 2, 64, 16, 700, torch.float8_e4m3fn, 2, T=3)
    s = torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    torch.cuda.synchronize()
    r = kda.attn_step(q, cache, pages, full, out=out, lse=lse, stream=s)
    s.synchronize()
    want, wl = kda.attn_step(q, cache, pages, full, want_lse=True)
    assert r[0] is out and r[1] is lse and torch.equal(out, want) and torch.equal(lse, wl)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    got = kda.cache_read(cache, pages, full, 700, k=rk, v=rv, stream=s)
    s.synchronize()
    assert got[0] is rk and all(torch.equal(a, b) for a, b in zip(got, kda.cache_read(cache, pages, full, 700)))
    w = torch.ones(64, device="cuda")
    freqs = torch.ones(32, dtype=F64, device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3)
    a, _ = kda.qknorm_fwd(q, None, pos, freqs, q_weight=w, stream=s)
    g = kda.qknorm_bwd(q, None, q, None, pos, freqs, q_weight=w, stream=s)
    s.synchronize()
    assert torch.equal(a, kda.qknorm_fwd(q, None, pos, freqs, q_weight=w)[0])
    assert torch.equal(g[2], kda.qknorm_bwd(q, None, q, None, pos, freqs, q_weight=w)[2])
    p = torch.softmax(torch.randn(5, 1, 999, device="cuda"), -1)
    tok, com = torch.empty(5, 1, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    none, u = torch.empty(5, 0, dtype=torch.int32, device="cuda"), torch.rand(5, 1, device="cuda")
    torch.cuda.synchronize()
    t = kda.draft_verify(p, None, none, u, tokens=tok, num_commit=com, stream=s)
    s.synchronize()
    assert t[0] is tok and t[1] is com and torch.equal(tok, kda.draft_verify(p, None, none, u)[0])


@pytest.mark.parametrize("T,rep", [(1, 1), (1, 8), (2, 7), (3, 5), (4, 4), (5, 4), (8, 4), (7, 5), (8, 8), (8, 9), (8, 16), (5, 27)])
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_rows_of_all_sizes(kda, kind, T, rep):
    """1 to 135 query rows per key-value head: every tile shape, rows cut into chunks; a step of T
    tokens gives what T steps of one token give.  Both round weights at most at 2^-12 and the output at
    2^-8: values of at most 4 differ by 2^-7 x 4."""
    dt = {"bf16": torch.bfloat16, "int8": torch.int8}[kind]
    q, cache, pages, full, _, _ = attn_state(kda, 2, 2 * rep, 2, 128, 32, 333, dt, 3, T=T)
    lens = torch.tensor([333, 120], dtype=torch.int32, device="cuda")
    got = kda.attn_step(q, cache, pages, lens)
    for t in range(T):
        one = kda.attn_step(q[:, t:t + 1].contiguous(), cache, pages, lens - (T - 1 - t))
        assert ((got[:, t:t + 1].float() - one.float()).abs() <= 2.0 ** -5).all()


@pytest.mark.parametrize("T", [1, 8])
def test_scores_that_grow_along_the_cache(kda, T):
    """Scores from far below 0 to far above it, rising and falling along the cache: the base of the weights
    has to follow by hundreds of powers of two, and in 8 bits the values' own powers differ by 2^40."""
    n, d, page = 1200, 64, 16
    g = torch.Generator().manual_seed(4)
    up = torch.linspace(-60, 60, n)
    for order in (up, up.flip(0), up[torch.randperm(n, generator=g)]):
        k = torch.zeros(1, n, 1, d)
        k[0, :, 0, 0] = order
        v = torch.randn(1, n, 1, d, generator=g) * torch.exp2(torch.randint(-20, 20, (1, n, 1, 1), generator=g).float())
        q = torch.zeros(1, T, 2, d)
        q[..., 0, 0], q[..., 1, 0] = 8.0, -8.0  # scores of +-480 in natural units
        for dtype, kind in ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float8_e4m3fn), (torch.float32, torch.int8),
                            (torch.float32, torch.float32)):
            cache = kda.kv_cache(n // page, page, 1, d, dtype=kind)
            pages = torch.arange(n // page, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
            lens = torch.tensor([n], dtype=torch.int32, device="cuda")
            kda.cache_write(k.cuda().to(dtype), v.cuda().to(dtype), cache, pages, lens)
            got, lse = kda.attn_step(q.cuda().to(dtype), cache, pages, lens, scale=1.0, want_lse=True)
            cpu = tuple(None if t is None else t.cpu() for t in cache)
            want, wl = ref.attn(q.to(dtype), cpu, pages.cpu(), lens.cpu(), 1.0)
            spread = ref.attn(q.to(dtype), (cpu[0], cpu[1].float().abs().to(cpu[1].dtype), *cpu[2:]), pages.cpu(), lens.cpu(), 1.0)[0]
            # scores of 480: 2^-24 of them moves a weight by 2^-15
            tol = spread * (2.0 ** -11 if dtype is torch.bfloat16 else 2.0 ** -13) + want.abs() * (2.0 ** -8 if dtype is torch.bfloat16 else 0)
            assert ((got.cpu().to(F64) - want).abs() <= tol + 1e-30).all(), (kind, dtype)
            assert ((lse.cpu().to(F64) - wl).abs() <= 2e-4 * wl.abs()).all()


def test_pools_past_31_bits(kda):
    """Pages whose elements lie past 2^31: write, read and attend at the pool's end."""
    h, d, page = 8, 128, 64
    num = (1 << 31) // (h * d * page) + 40
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    cache = kda.kv_cache(num, page, h, d, dtype=torch.int8)
    n, T = 2, 300
    pages = torch.stack([torch.arange(num - 5, num), torch.arange(num - 25, num - 20)]).to(torch.int32).cuda()
    lens = torch.tensor([T, T], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(n, T, h, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    kda.cache_write(k, v, cache, pages, lens)
    rk, rv = kda.cache_read(cache, pages, lens, T)
    assert torch.equal(rk.cpu().to(F64), ref.encode(k.cpu().to(F64), "int8")[0])
    q = torch.randn(n, 1, 16, d, device="cuda", generator=g).bfloat16()
    got = kda.attn_step(q, cache, pages, lens)
    small = kda.KVCache(*(t[num - 25:].clone() for t in cache))
    del cache
    assert torch.equal(got, kda.attn_step(q, small, pages - (num - 25), lens))


def test_batches_past_31_bits(kda):
    """Norms over more than 2^31 elements and probabilities past 2^31: the last rows as alone."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    tokens, heads, d = (1 << 31) // (32 * 128) + 7, 32, 128
    q = torch.empty(tokens, heads, d, dtype=torch.bfloat16, device="cuda").normal_()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    freqs = torch.ones(64, dtype=F64, device="cuda") / 7
    w = torch.ones(d, device="cuda")
    y, _ = kda.qknorm_fwd(q, None, pos, freqs, q_weight=w)
    tail, _ = kda.qknorm_fwd(q[-9:].clone(), None, pos[-9:].clone(), freqs, q_weight=w)
    assert torch.equal(y[-9:], tail)
    del q, y
    V, B, K = 131072, 2056, 7
    p = torch.rand(B, K + 1, V, dtype=torch.bfloat16, device="cuda")
    drafts = torch.randint(0, V, (B, K), dtype=torch.int32, device="cuda")
    u = torch.rand(B, K + 1, device="cuda")
    got = kda.draft_verify(p, None, drafts, u)
    tail = kda.draft_verify(p[-3:].clone(), None, drafts[-3:].clone(), u[-3:].clone())
    assert torch.equal(got[0][-3:], tail[0]) and torch.equal(got[1][-3:], tail[1])


def test_repeatable_gradients_and_many_sequences(kda):
    """The weights' gradients repeat bit for bit; more sequences than the splitting block has threads."""
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, dq, dk = (torch.randn(3001, h, 64, device="cuda", generator=g).bfloat16() for h in (5, 2, 5, 2))
    pos = torch.arange(3001, dtype=torch.int32, device="cuda")
    freqs = torch.ones(16, dtype=F64, device="cuda")
    w = torch.ones(64, device="cuda")
    a, b = (kda.qknorm_bwd(q, k, dq, dk, pos, freqs, q_weight=w, k_weight=w) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    n = 1500
    q, cache, pages, full, _, _ = attn_state(kda, n, 4, 1, 64, 16, 48, torch.bfloat16, 7)
    lens = (torch.arange(n, device="cuda") % 49).to(torch.int32)
    got = kda.attn_step(q, cache, pages, lens)
    for i in (0, 1, 48, 777, 1499):
        one = kda.attn_step(q[i:i + 1].contiguous(), cache, pages[i:i + 1].contiguous(), lens[i:i + 1].contiguous())
        assert ((got[i].float() - one[0].float()).abs() <= 2.0 ** -5).all()
    assert not got[0].any()


@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.int8), (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,rep", [(1, 3), (4, 7), (8, 5)])
def test_odd_bases(kda, dtype, kind, T, rep):
    """q, out and lse one element off every alignment give the same bits, over whole items and parts."""
    q, cache, pages, full, _, _ = attn_state(kda, 2, 2 * rep, 2, 64, 16, 3000, kind, 8, T=T)
    q = q.to(dtype)
    lens = torch.tensor([3000, 90], dtype=torch.int32, device="cuda")
    want, wl = kda.attn_step(q, cache, pages, lens, want_lse=True)
    flat = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
    flat[1:] = q.flatten()
    out = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
    lse = torch.zeros(wl.numel() + 1, device="cuda")
    kda.attn_step(flat[1:].view(q.shape), cache, pages, lens, out=out[1:].view(q.shape), lse=lse[1:].view(wl.shape))
    assert torch.equal(out[1:].view(q.shape), want) and torch.equal(lse[1:].view(wl.shape), wl)
    wide = torch.zeros(2, T, 2 * rep * 64 + 3, dtype=dtype, device="cuda")
    wide[..., 1:-2] = q.flatten(2)
    assert torch.equal(kda.attn_step(wide[..., 1:-2].unflatten(-1, (2 * rep, 64)), cache, pages, lens), want)


def test_drawing_without_drafts(kda):
    """K = 0: a token from p, with drafts left out."""
    p = torch.softmax(torch.randn(9, 1, 77, device="cuda"), -1)
    u = torch.rand(9, 1, device="cuda")
    got, commit = kda.draft_verify(p, None, None, u)
    want = ref.verify(p.cpu(), None, torch.zeros(9, 0, dtype=torch.int32), u.cpu())
    assert torch.equal(got.cpu(), want[0]) and (commit == 1).all()
    with pytest.raises(ValueError, match="drafts"):
        kda.draft_verify(torch.cat([p, p], 1), None, None, torch.rand(9, 2, device="cuda"))


@pytest.mark.parametrize("T,rep", [(1, 3), (8, 4)])
def test_largest_windows(kda, T, rep):
    """Windows up to 2^31 - 1 that reach before the first place are no windows; sequences shorter than the
    new tokens among them."""
    q, cache, pages, _, _, _ = attn_state(kda, 4, 2 * rep, 2, 64, 16, 600, torch.int8, 7, T=T)
    lens = torch.tensor([600, 0, 3, 77], dtype=torch.int32, device="cuda")
    want, lse = kda.attn_step(q, cache, pages, lens, want_lse=True)
    for w in (600, 2**31 - 600, 2**31 - 1):
        got, l = kda.attn_step(q, cache, pages, lens, window=w, want_lse=True)
        assert torch.equal(got, want) and torch.equal(l, lse)
