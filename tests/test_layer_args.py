"""Refusals of the operators around the recurrence, on a machine without a GPU: the C entry
points reject bad arguments before any CUDA call is made, and the binding rejects tensors that
it cannot pass on."""
import ctypes

import pytest
import torch

FAKE = 1 << 32  # an aligned, never-dereferenced stand-in for a device pointer


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    import kda_delta_rule_fwd_gb300 as m
    from kda_delta_rule_fwd_gb300 import layer
    return m, layer, m.load()


def conv(layer, m, **kw):
    d = dict(B=2, T=10, D=64, W=4, num_seqs=0, dtype=m.KDA_BF16, silu=1, ldx=0)
    return layer.ConvShape(**{**d, **kw})


def scan(layer, m, **kw):
    d = dict(B=2, T=10, H=4, G=2, ds=128, dx=64, num_seqs=0, in_dtype=m.KDA_BF16,
             out_dtype=m.KDA_F32, dt_softplus=1, ldx=0, lddt=0, ldb=0, ldc=0)
    return layer.ScanShape(**{**d, **kw})


def norm(layer, m, **kw):
    d = dict(tokens=8, heads=1, d=64, dtype=m.KDA_BF16, res_dtype=m.KDA_BF16, gate=1, gate_first=0,
             scale=1.0, eps=1e-6, ldx=0, ldgate=0)
    return layer.NormShape(**{**d, **kw})


def call(f, shape, n, size=1 << 30, ws=FAKE, **at):
    """f(shape, n pointers, [workspace,] bytes, stream) with FAKE pointers, ``at`` by position."""
    ptrs = [at.get(f"p{i}", FAKE) for i in range(n)]
    return f(shape, *ptrs, ws, size, None)


def test_conv_arguments(lib):
    m, layer, L = lib
    bad, odd, ws = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE
    fwd = lambda s, **k: call(L.kda_conv_fwd, s, 7, p3=None, **k)
    for s, want in ((dict(T=-1), bad), (dict(B=-1), bad), (dict(D=0), bad), (dict(dtype=5), bad),
                    (dict(W=1), odd), (dict(W=5), odd), (dict(ldx=63), bad),
                    (dict(T=2 ** 31 - 1, B=2 ** 31 - 1, D=4096), bad)):
        assert fwd(conv(layer, m, **s)) == want, s
    assert call(L.kda_conv_fwd, None, 7) == bad
    s = conv(layer, m)
    assert fwd(s, p0=None) == bad and fwd(s, p1=None) == bad and fwd(s, p5=None) == bad
    assert fwd(s, p0=FAKE + 1) == bad and fwd(s, p1=FAKE + 2) == bad
    assert fwd(s, ws=FAKE + 16) == ws and fwd(s, size=255) == ws
    packed = conv(layer, m, B=2, num_seqs=3)
    assert call(L.kda_conv_fwd, packed, 7) == bad  # packed batches have B = 1
    assert call(L.kda_conv_fwd, conv(layer, m, B=1, num_seqs=0), 7) == bad  # tokens of no sequence
    step = lambda s, **k: call(L.kda_conv_step, s, 6, **k)
    assert step(conv(layer, m, T=0)) == odd and step(conv(layer, m, T=9)) == odd
    assert step(conv(layer, m, T=2), p4=None) == bad and step(conv(layer, m, T=2), p3=FAKE + 2) == bad
    assert step(conv(layer, m, T=2), p3=None, p5=None) == bad  # no outputs only with counts
    bwd = lambda s, **k: call(L.kda_conv_bwd, s, 11, p3=None, **k)
    assert bwd(s, p8=None) == bad and bwd(s, p5=None) == bad and bwd(s, ws=None) == ws
    assert bwd(s, size=L.kda_conv_bwd_workspace_size(s) - 1) == ws
    assert L.kda_conv_bwd_workspace_size(None) == 0


def test_scan_arguments(lib):
    m, layer, L = lib
    bad, odd, ws = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE
    fwd = lambda s, **k: call(L.kda_scan_fwd, s, 11, p7=None, **k)
    for s, want in ((dict(T=-1), bad), (dict(H=0), bad), (dict(H=3, G=2), bad), (dict(G=0), bad),
                    (dict(in_dtype=9), bad), (dict(ds=96), odd), (dict(dx=32), odd),
                    (dict(ldx=255), bad), (dict(lddt=3), bad), (dict(ldb=8), bad)):
        assert fwd(scan(layer, m, **s)) == want, s
    s = scan(layer, m)
    for i in (0, 1, 2, 3, 4, 9):
        assert fwd(s, **{f"p{i}": None}) == bad, i
    assert fwd(s, p8=FAKE + 4) == bad and fwd(s, p10=FAKE + 8) == bad  # states: 16 bytes
    assert fwd(scan(layer, m, dt_softplus=0)) == bad  # a bias without softplus
    assert fwd(s, ws=None) == ws and fwd(s, ws=FAKE + 128) == ws
    assert fwd(s, size=L.kda_scan_workspace_size(s) - 1) == ws
    step = lambda s, **k: call(L.kda_scan_step, s, 10, **k)
    assert step(scan(layer, m, T=0)) == odd and step(scan(layer, m, T=9)) == odd
    assert step(scan(layer, m, T=1), p8=None) == bad and step(scan(layer, m, T=1), p8=FAKE + 8) == bad
    assert step(scan(layer, m, T=1), p7=None, p9=None) == bad
    assert L.kda_scan_workspace_size(None) == 0 and L.kda_scan_workspace_size(scan(layer, m, ds=3)) == 0


def test_scan_workspace_covers_the_segments(lib):
    """Long sequences with few heads keep a state per segment; short ones only the header."""
    m, layer, L = lib
    size = lambda **k: L.kda_scan_workspace_size(scan(layer, m, dx=128, **k))
    assert size(B=4, T=4096, H=32, G=4) == 256
    long = size(B=1, T=131072, H=4, G=1)
    assert long > 256 and (long - 256) % 256 == 0
    assert size(B=1, T=131072, H=4, G=1, in_dtype=m.KDA_F32) == 256
    packed = size(B=1, T=131072, H=4, G=1, num_seqs=3)
    assert packed > 256


def test_norm_arguments(lib):
    m, layer, L = lib
    bad, odd, ws = m.KDA_ERR_INVALID_ARG, m.KDA_ERR_UNSUPPORTED, m.KDA_ERR_WORKSPACE

    def fwd(s, **k):
        return L.kda_norm_fwd(s, *[k.get(f"p{i}", FAKE) for i in range(8)], None)
    for s, want in ((dict(tokens=-1), bad), (dict(heads=0), bad), (dict(d=0), bad),
                    (dict(d=8193), odd), (dict(gate=3), bad), (dict(scale=float("nan")), bad),
                    (dict(eps=-1.0), bad), (dict(dtype=m.KDA_F32), bad), (dict(ldx=63), bad),
                    (dict(gate=0), bad)):  # a gate tensor without a gate
        assert fwd(norm(layer, m, **s)) == want, s
    s = norm(layer, m)
    assert fwd(s, p0=None) == bad and fwd(s, p2=None) == bad
    assert fwd(s, p5=None) == bad and fwd(s, p7=None) == bad  # y goes with out_weight
    assert fwd(s, p5=None, p6=None, p7=None) == bad           # nothing to write
    assert fwd(s, p1=FAKE + 2) == bad and fwd(s, p3=FAKE + 1) == bad
    bwd = lambda s, **k: call(L.kda_norm_bwd, s, 14, **k)
    assert bwd(s, p5=None) == bad                              # dy without out_weight
    assert bwd(s, p6=None, p7=None) == bad                     # no cotangent
    assert bwd(s, p3=None) == bad and bwd(s, p1=None) == bad   # a gradient without its operand
    assert bwd(s, p8=None) == bad and bwd(s, ws=None) == ws
    assert bwd(s, size=L.kda_norm_bwd_workspace_size(s) - 1) == ws


def test_binding_refuses(lib):
    m, layer, L = lib
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        m.conv_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        m.norm_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        m.scan_step(torch.zeros(1, 1, 2, 64), None, None, None, None, None)
    if torch.cuda.is_available():
        return
    # the checks themselves need no device
    with pytest.raises(TypeError, match="weight"):
        layer._conv_shape(x, w.double(), None, None, None)
    with pytest.raises(ValueError, match="shape"):
        layer._conv_shape(x, torch.zeros(7, 4), None, None, None)
    with pytest.raises(ValueError, match="activation"):
        layer._conv_shape(x, w, None, "relu", None)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        layer._conv_shape(x.half(), w, None, None, None)
    with pytest.raises(ValueError, match="one stride"):
        layer._conv_shape(torch.zeros(2, 8, 5).transpose(1, 2), w, None, None, None)
    with pytest.raises(ValueError, match="B = 1"):
        layer._conv_shape(x, w, None, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="num_commit"):
        layer._counts(torch.zeros(2), 2, x)
    with pytest.raises(ValueError, match="gate_act"):
        layer._norm_shape(x, None, x, "tanh", False, None, 1, None, None, 1e-6, None)
    with pytest.raises(TypeError, match="residual"):
        layer._norm_shape(x, None, None, "silu", False, x.bfloat16(), 1, None, None, 1e-6, None)
    s = layer._scan_shape
    X, dt, B, A = torch.zeros(1, 3, 4, 64), torch.zeros(1, 3, 4), torch.zeros(1, 3, 2, 64), torch.zeros(4)
    with pytest.raises(ValueError, match="dt"):
        s(X, dt[:, :2], A, B, B, None, None, False, None, torch.float32)
    with pytest.raises(TypeError, match="A must be"):
        s(X, dt, A.double(), B, B, None, None, False, None, torch.float32)
    with pytest.raises(TypeError, match="output"):
        s(X, dt, A, B, B, None, None, False, None, torch.float16)


def test_strides_of_slices(lib):
    """Token strides: a column slice's own, 0 where dense or empty, refused where rows overlap."""
    m, layer, L = lib
    p = torch.zeros(2, 5, 24)
    assert layer._token_stride(p, "x") == 0
    assert layer._token_stride(p[..., 3:11], "x") == 24
    assert layer._token_stride(p[..., 8:].unflatten(-1, (2, 8)), "x") == 24
    assert layer._token_stride(p[:, :0, 3:11], "x") == 0
    assert layer._token_stride(p[:1, :1, 3:11], "x") in (0, 8)
    with pytest.raises(ValueError):
        layer._token_stride(p[:, ::2], "x")  # the batch stride is not 3 tokens
    with pytest.raises(ValueError):
        layer._token_stride(p[..., :1].expand(2, 5, 8), "x")
    assert layer._row_strides(p[..., :8], None) == (1, 24, 0)
    assert layer._row_strides(p[..., :16].unflatten(-1, (2, 8)), None) == (2, 24, 0)
