"""Attention of new tokens with a window over tables whose pages behind it were given back."""
import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("bf16", "int8"), ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("T,rep", [(1, 4), (2, 8), (8, 8)])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_pages_behind_a_window(kda, page, T, rep, dtype, kind):
    """Pages of which no token sees a place may name anything: nothing is reported and every bit stays; the page
    of the first place that a token sees is reported where it is not in the pool.  Short tables and long ones."""
    g = torch.Generator().manual_seed(1)
    lens, w = [200, 470, 141, 9], 8
    for cap in (512, 1024):
        n, mp = len(lens), cap // page
        pool = n * mp
        pages = torch.randperm(pool, generator=g).reshape(n, mp).to(torch.int32)
        q = torch.randn(n, T, 2 * rep, 64, generator=g).to(KINDS[dtype]).cuda()
        made = []
        for _ in range(2):
            x = torch.randn(pool, 2, page, 64, generator=g)
            if kind in ("f32", "bf16"):
                made.append((x.to(KINDS[kind]), None))
            else:
                value, byte = ref.encode(x.double(), kind)
                made.append(((value * torch.exp2(127 - byte.double())[..., None]).float().to(KINDS[kind]), byte.to(torch.uint8)))
        cache = kda.KVCache(*(None if t is None else t.cuda() for t in (made[0][0], made[1][0], made[0][1], made[1][1])))
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = kda.attn._attn_shape(q, cache, pages.cuda(), ln, None, w)
        ws = torch.empty(kda.attn.attn_workspace_size(shape) // 4, dtype=torch.int32, device="cuda")

        def attend(table):
            out = kda.attn_step(q, cache, table.cuda(), ln, window=w, workspace=ws)
            return out, kda.read_device_status(ws)
        want, status = attend(pages)
        assert status == 0
        free, bad = pages.clone(), pages.clone()
        for b, m in enumerate(lens):
            first = max(0, m - T + 1 - w)
            free[b, :first // page] = -1 if b % 2 else 2 ** 30
            free[b, -(-m // page):] = -7
        got, status = attend(free)
        assert status == 0 and torch.equal(got, want)
        bad[1, (lens[1] - T + 1 - w) // page] = pool
        assert attend(bad)[1] == kda.KDA_ERR_INVALID_ARG
