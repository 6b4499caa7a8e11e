"""Further refusals of the operators around the recurrence, on a machine without a GPU."""
import pytest
import torch
import pytest
import torch

from test_layer_args import FAKE, call, conv, lib, norm, scan  # noqa: F401


def test_scan_workspace_of_fixed_lengths_ignores_num_seqs(lib):
    """A fixed-length call never gets less than it needs, whatever is in the field that it ignores."""
    m, layer, L = lib
    shape = dict(B=8, T=8192, H=2, G=1, ds=128, dx=128)
    fixed = lambda s, size: call(L.kda_scan_fwd, s, 11, p7=None, size=size)  # p7: cu_seqlens
    for few in (shape, dict(shape, B=1), dict(shape, B=1, T=2200)):
        need = L.kda_scan_workspace_size(scan(layer, m, **few))
        assert need > 256
        for n in (-1, -2 ** 31, 1, 3, 2 ** 31 - 1):
            s = scan(layer, m, num_seqs=n, **few)
            assert fixed(s, need - 1) == m.KDA_ERR_WORKSPACE, n
            if n <= 3:
                assert L.kda_scan_workspace_size(s) >= need, n
    # a packed call still gets what it needs
    packed = scan(layer, m, B=1, T=131072, H=4, G=1, ds=128, dx=128, num_seqs=3)
    size = L.kda_scan_workspace_size(packed)
    assert size > 256
    assert call(L.kda_scan_fwd, packed, 11, size=255) == m.KDA_ERR_WORKSPACE


def test_workspace_of_another_device_or_layout(lib):
    """The bytes passed on are bytes that the tensor has, on the device that writes them."""
    m, layer, L = lib
    x = torch.zeros(2, 5, 8)
    assert layer._ws(None, x) == (None, 0)
    ws = torch.zeros(512, dtype=torch.float32)
    assert layer._ws(ws, x) == (ws.data_ptr(), 2048)
    with pytest.raises(ValueError, match="workspace"):
        layer._ws(torch.zeros(1, dtype=torch.uint8).expand(1 << 20), x)
    with pytest.raises(ValueError, match="workspace"):
        layer._ws(ws[::2], x)

    class Elsewhere:  # stands for a tensor on a GPU
        get_device = staticmethod(lambda: 0)
    with pytest.raises(ValueError, match="workspace"):
        layer._ws(ws, Elsewhere)


def test_sizes_past_32_bits_are_refused(lib):
    """Not cut to their low bits: 2^32 + 10 tokens are not 10."""
    m, layer, L = lib
    big = 2 ** 32 + 10
    x = torch.empty(1, big, 1, dtype=torch.bfloat16, device="meta")
    w = torch.empty(1, 4, device="meta")
    with pytest.raises(ValueError, match="T = 4294967306"):
        layer._conv_shape(x, w, None, None, None)
    b = torch.empty(1, big, 1, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="T = 4294967306"):
        layer._scan_shape(b, x, torch.empty(1, device="meta"), b, b, None, None, False, None, torch.float32)
    with pytest.raises(ValueError, match="B = 4294967306"):
        layer._conv_shape(x.transpose(0, 1), w, None, None, None)
    rows = layer._norm_shape(x, None, None, "silu", False, None, 1, None, None, 1e-6, None)[0]
    assert rows.tokens == big and rows.d == 1  # 64 bits


@pytest.mark.parametrize("D", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 1023])
def test_channels_near_31_bits_are_refused(lib, D):
    """Before a block's last channel, or the number of blocks, passes 31 bits."""
    m, layer, L = lib
    s = conv(layer, m, B=1, T=1, D=D)
    assert call(L.kda_conv_fwd, s, 7, p3=None) == m.KDA_ERR_INVALID_ARG
    assert call(L.kda_conv_step, s, 6) == m.KDA_ERR_INVALID_ARG
    assert call(L.kda_conv_bwd, s, 11, p3=None, size=1 << 60) == m.KDA_ERR_INVALID_ARG
