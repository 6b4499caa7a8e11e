"""Refusals of the attention layers' operators, on a machine without a GPU: the C entry points
reject bad arguments before any CUDA call is made, and the binding rejects tensors that it cannot
pass on."""
import pytest
import torch

FAKE = 1 << 32  # an aligned, never-dereferenced stand-in for a device pointer


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    import kda_delta_rule_fwd_gb300 as m
    from kda_delta_rule_fwd_gb300 import attn
    return m, attn, m.load()


def call(f, shape, n, size=1 << 40, ws=FAKE, **at):
    """f(shape, n pointers, workspace, bytes, stream) with FAKE pointers, ``at`` by position."""
    return f(shape, *[at.get(f"p{i}", FAKE) for i in range(n)], ws, size, None)


def test_qknorm_arguments(lib):
    m, attn, L = lib
    bad, odd, wsp = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE

    def shape(**kw):
        d = dict(tokens=4, q_heads=4, k_heads=2, d=64, rot=64, dtype=m.KDA_BF16, interleaved=0, eps=1e-6, ldq=0, ldk=0)
        return attn.QKNormShape(**{**d, **kw})

    def fwd(s, **k):
        return L.kda_qknorm_fwd(s, *[k.get(f"p{i}", FAKE) for i in range(8)], None)
    for s, want in ((dict(tokens=-1), bad), (dict(q_heads=0), bad), (dict(k_heads=-1), bad), (dict(d=63), bad),
                    (dict(d=0), bad), (dict(d=258), odd), (dict(rot=3), bad), (dict(rot=66), bad), (dict(rot=-2), bad),
                    (dict(dtype=7), bad), (dict(eps=-1.0), bad), (dict(eps=float("nan")), bad), (dict(ldq=255), bad),
                    (dict(ldk=127), bad), (dict(tokens=1 << 40), bad), (dict(q_heads=65537), bad), (dict(k_heads=65537), bad)):
        assert fwd(shape(**s)) == want, s
    assert fwd(None) == bad
    for i in (0, 1, 2, 3, 6, 7):
        assert fwd(shape(), **{f"p{i}": None}) == bad, i
    assert fwd(shape(), p0=FAKE + 1) == bad and fwd(shape(), p2=FAKE + 2) == bad and fwd(shape(), p3=FAKE + 4) == bad
    bwd = lambda s, **k: call(L.kda_qknorm_bwd, s, 12, **k)
    for i in (0, 1, 2, 3, 4, 5, 8, 9):
        assert bwd(shape(), **{f"p{i}": None}) == bad, i
    assert bwd(shape(), p6=None) == bad and bwd(shape(), p7=None) == bad  # a gradient without its weight
    assert bwd(shape(), ws=None) == wsp and bwd(shape(), ws=FAKE + 16) == wsp
    assert bwd(shape(), size=L.kda_qknorm_bwd_workspace_size(shape()) - 1) == wsp
    assert L.kda_qknorm_bwd_workspace_size(None) == 0


def test_cache_arguments(lib):
    m, attn, L = lib
    bad, odd, wsp = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE

    def shape(**kw):
        d = dict(B=2, T=3, num_seqs=0, heads=2, d=64, page=16, max_pages=4, num_pages=8, dtype=m.KDA_BF16, cache=2, ldk=0,
                 ldv=0, ldpage=0)
        return attn.CacheShape(**{**d, **kw})
    for f, nul in ((L.kda_cache_write, (0, 1, 3, 4, 5, 6, 7, 8)), (L.kda_cache_read, (1, 2, 3, 4, 5, 6))):
        w = f is L.kda_cache_write
        go = lambda s, **k: call(f, s, 9, **{("p2" if w else "p0"): None, **k})
        for s, want in ((dict(B=-1), bad), (dict(T=-1), bad), (dict(heads=0), bad), (dict(d=96), odd), (dict(d=0), bad),
                        (dict(page=0), bad), (dict(page=24), odd), (dict(page=1 << 17), odd), (dict(max_pages=0), bad),
                        (dict(num_pages=0), bad), (dict(dtype=3), bad), (dict(cache=4), bad), (dict(ldk=127), bad),
                        (dict(ldpage=2047), bad), (dict(ldpage=2049), bad), (dict(cache=1), bad)):  # scales of a bf16 cache
            assert go(shape(**s)) == want, s
        assert go(None) == bad
        for i in nul:
            assert go(shape(), **{f"p{i}": None}) == bad, i
        assert go(shape(), **{("p5" if w else "p3"): FAKE + 8}) == bad  # pools: 16 bytes
        assert go(shape(), **{("p3" if w else "p1"): FAKE + 2}) == bad
        assert go(shape(), ws=FAKE + 16) == wsp and go(shape(), size=255) == wsp
        packed = {"p2" if w else "p0": FAKE}
        assert go(shape(), **packed) == bad  # packed batches have B = 1
        assert go(shape(B=1, num_seqs=0), **packed) == bad
    assert call(L.kda_cache_read, shape(), 9, p0=None, p7=None, p8=None) == bad  # nothing to read into


def test_attn_arguments(lib):
    m, attn, L = lib
    bad, odd, wsp = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE

    def shape(**kw):
        d = dict(B=2, T=1, q_heads=4, kv_heads=2, d=128, page=64, max_pages=4, num_pages=8, dtype=m.KDA_BF16, cache=2,
                 scale=0.1, window=0, ldq=0, ldpage=0)
        return attn.AttnShape(**{**d, **kw})
    go = lambda s, **k: call(L.kda_attn_step, s, 9, **k)
    for s, want in ((dict(B=-1), bad), (dict(T=0), odd), (dict(T=9), odd), (dict(q_heads=3), bad), (dict(kv_heads=0), bad),
                    (dict(d=96), odd), (dict(page=48), odd), (dict(max_pages=0), bad), (dict(num_pages=0), bad),
                    (dict(dtype=5), bad), (dict(cache=9), bad), (dict(cache=0), odd), (dict(scale=float("nan")), bad),
                    (dict(window=-1), bad), (dict(ldq=511), bad), (dict(ldpage=1), bad)):
        assert go(shape(**s)) == want, s
        assert L.kda_attn_workspace_size(shape(**s)) == 0, s
    assert go(None) == bad and L.kda_attn_workspace_size(None) == 0
    for i in (0, 1, 2, 3, 4, 5, 6, 7):
        assert go(shape(), **{f"p{i}": None}) == bad, i
    assert go(shape(cache=1)) == bad  # scales of a bf16 cache
    assert go(shape(), p0=FAKE + 1) == bad and go(shape(), p1=FAKE + 8) == bad and go(shape(), p8=FAKE + 2) == bad
    assert go(shape(), p3=FAKE + 8) == bad and go(shape(), p4=FAKE + 1) == bad  # scales: 16 bytes
    size = L.kda_attn_workspace_size(shape())
    assert size >= 256
    assert go(shape(), ws=None) == wsp and go(shape(), ws=FAKE + 32) == wsp and go(shape(), size=size - 1) == wsp


def test_verify_arguments(lib):
    m, attn, L = lib
    bad, odd, wsp = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE
    shape = lambda **kw: attn.VerifyShape(**{**dict(B=2, K=3, V=100, dtype=m.KDA_F32), **kw})
    go = lambda s, **k: call(L.kda_draft_verify, s, 7, **k)
    for s, want in ((dict(B=-1), bad), (dict(K=-1), bad), (dict(K=32), odd), (dict(V=0), bad), (dict(V=1 << 19), odd),
                    (dict(dtype=2), bad)):
        assert go(shape(**s)) == want, s
    assert go(None) == bad
    for i in (0, 2, 4, 5, 6):
        assert go(shape(), **{f"p{i}": None}) == bad, i
    assert go(shape(), p0=FAKE + 2) == bad and go(shape(), p4=FAKE + 1) == bad
    assert go(shape(), ws=FAKE + 8) == wsp and go(shape(), size=16) == wsp


def test_binding_refuses(lib):
    m, attn, L = lib
    q = torch.zeros(2, 1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.qknorm_fwd(q, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.cache_write(q, q, m.kv_cache(2, 16, 4, 64, device="cpu"), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.cache_read(m.kv_cache(2, 16, 4, 64, device="cpu"), None, None, 1)
    with pytest.raises(ValueError, match="CUDA"):
        m.attn_step(q, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.draft_verify(q[0], None, None, None)
    with pytest.raises(TypeError, match="cache holds"):
        m.kv_cache(2, 16, 4, 64, dtype=torch.float16, device="cpu")
    if torch.cuda.is_available():
        return
    # the checks themselves need no device
    f = torch.zeros(32, dtype=torch.float64)
    pos = torch.zeros(2, dtype=torch.int32)
    go = lambda q=q, k=None, p=pos, f=f, w=None, kw=None: attn._qknorm_shape(q, k, p, f, w, kw, False, 1e-6)
    assert (go().tokens, go().rot, go().ldq) == (2, 64, 0)
    for match, kind, kw in (("float32 or bfloat16", TypeError, dict(q=q.half())), ("heads, d", ValueError, dict(q=q[0, 0])),
                            ("freqs", TypeError, dict(f=f.float())), ("positions", ValueError, dict(p=pos.long())),
                            ("positions", ValueError, dict(p=pos[:1])), ("needs positions", ValueError, dict(p=None)),
                            ("q_weight", ValueError, dict(w=torch.zeros(63))), ("k must have", ValueError, dict(k=q[0])),
                            ("shape", ValueError, dict(k=q[:1])),
                            ("one stride", ValueError, dict(q=torch.zeros(2, 1, 64, 4).transpose(-1, -2)))):
        with pytest.raises(kind, match=match):
            go(**kw)
    assert go(q=torch.zeros(2, 1, 300)[..., 4:260].unflatten(-1, (4, 64))).ldq == 300
    cache = m.kv_cache(5, 16, 4, 64, dtype=torch.int8, device="cpu")
    pages, lens = torch.zeros(2, 3, dtype=torch.int32), pos
    go = lambda c=cache, q=q, p=pages, n=lens: attn._attn_shape(q, c, p, n, None, 0)
    assert (go().page, go().max_pages, go().num_pages, go().cache) == (16, 3, 5, 3)
    wide = m.kv_cache(5, 16, 4, 64, device="cpu")
    for match, kind, kw in (("k_scale", ValueError, dict(c=cache._replace(k_scale=None))),
                            ("only an 8-bit", ValueError, dict(c=wide._replace(v_scale=cache.v_scale))),
                            ("q's type", TypeError, dict(c=wide)), ("channels", ValueError, dict(q=q[..., :32])),
                            ("k as v", TypeError, dict(c=cache._replace(v=wide.v))),
                            ("num_pages", ValueError, dict(c=cache._replace(v=cache.v[:4]))),
                            ("between them", ValueError, dict(c=cache._replace(k=cache.k.transpose(1, 2).contiguous().transpose(1, 2)))),
                            ("pages", ValueError, dict(p=pages[:1])), ("pages", ValueError, dict(p=pages.long())),
                            ("lens", ValueError, dict(n=lens[:1])), ("lens", ValueError, dict(n=lens.long())),
                            ("B, T", ValueError, dict(q=q[0]))):
        with pytest.raises(kind, match=match):
            go(**kw)
    both = torch.zeros(5, 2, 4, 16, 64, dtype=torch.int8)
    assert go(c=m.KVCache(both[:, 0], both[:, 1], cache.k_scale, cache.v_scale)).ldpage == 2 * 4 * 16 * 64


def test_numbers_that_the_structs_would_cut_off(lib, monkeypatch):
    """A window or a length of 2^32 + 5 is refused, not taken as 5."""
    m, attn, _ = lib
    cache = m.kv_cache(5, 16, 4, 64, device="cpu")
    q, pages, lens = torch.zeros(2, 1, 4, 64).bfloat16(), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for w, want in ((None, 0), (0, 0), (5, 5), (2**31 - 1, 2**31 - 1)):
        assert attn._attn_shape(q, cache, pages, lens, None, w).window == want
    for w in (-1, 2**31, 2**32 + 5):
        with pytest.raises(ValueError, match="window"):
            attn._attn_shape(q, cache, pages, lens, None, w)
    monkeypatch.setattr(attn, "_elsewhere", lambda x, stream: False)
    for T in (-1, 2**31, 2**32 + 5):
        with pytest.raises(ValueError, match="T must"):
            m.cache_read(cache, pages, lens, T)


def test_attn_status_left_out(lib):
    """A short table's workspace holds the status alone: it may be left out, but not be of the wrong size."""
    m, attn, L = lib

    def shape(max_pages, B=0):
        return attn.AttnShape(B=B, T=1, q_heads=4, kv_heads=2, d=128, page=64, max_pages=max_pages, num_pages=8,
                              dtype=m.KDA_BF16, cache=2, scale=0.1, window=0, ldq=0, ldpage=0)
    for pages, B in ((4, 2), (8, 2), (9, 0)):
        assert L.kda_attn_workspace_size(shape(pages, B)) == 256
    assert L.kda_attn_workspace_size(shape(9, 2)) > 256
    go = lambda s, ws, size: L.kda_attn_step(s, *[FAKE] * 9, ws, size, None)
    assert go(shape(9, 2), None, 0) == go(shape(4), FAKE, 0) == go(shape(4), FAKE, 255) == go(shape(4), None, 256) \
        == go(shape(4), FAKE + 8, 256) == m.KDA_ERR_WORKSPACE
    assert call(L.kda_attn_step, shape(4, 2), 9, p4=None) == m.KDA_ERR_INVALID_ARG
    # checked, and nothing to launch
    assert L.kda_attn_step(shape(4), *[FAKE] * 3, None, None, *[FAKE] * 4, None, 0, None) == m.KDA_OK
