"""The example block: a prompt in one call gives what a shorter prompt and single tokens after it
give, with KDA and with the scan as the mixer, and packed sequences what each gives alone."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mixer", ["kda", "scan"])
def test_prompt_and_steps_agree(kda, mixer):
    """Two paths of bf16 stages: each of the block's four bf16 roundings may fall differently
    (2^-9 of values up to about 5 rms, summed): 5e-2 of the rms."""
    import recurrent_block
    whole, parts = recurrent_block.run(mixer)
    for w, p in zip(whole, parts):
        w, p = w.float(), p.float()
        assert w.shape == p.shape and torch.isfinite(w).all()
        assert ((w - p).abs().max() / w.square().mean().sqrt()).item() <= 5e-2


@pytest.mark.parametrize("mixer", ["kda", "scan"])
def test_packed_sequences_are_independent(kda, mixer):
    import recurrent_block
    block = recurrent_block.Block(mixer=mixer)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [70, 1, 129]
    h = torch.randn(1, sum(lens), 512, device="cuda", generator=g).bfloat16()
    _, y = kda.norm_fwd(h, out_weight=block.block_norm)
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    r, z, state = block.prompt(h, y, cu)
    at = 0
    for i, n in enumerate(lens):
        r1, z1, one = block.prompt(h[:, at:at + n].contiguous(), y[:, at:at + n].contiguous())
        for a, b in ((r[:, at:at + n], r1), (z[:, at:at + n], z1)):
            assert ((a.float() - b.float()).abs().max() / b.float().square().mean().sqrt()).item() <= 5e-2
        assert torch.equal(state["conv"][i], one["conv"][0])
        at += n
