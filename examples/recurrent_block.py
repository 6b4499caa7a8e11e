"""One block of a model with recurrent token mixing, built from the library's entry points.

    pre-norm -> projections -> short convolution -> KDA or state-space scan
             -> gated head norm -> output projection -> scaled residual + next pre-norm

``Block`` runs whole prompts (packed or fixed length) and then single or drafted tokens from the
states that the prompt leaves; ``main`` checks that both ways give the same outputs and times a
step.  Projections are plain torch products; everything else is a library call.

    python examples/recurrent_block.py [--mixer kda|scan]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kda_delta_rule_fwd_gb300 as kda  # noqa: E402


class Block:
    """Weights and calls of one block: ``H`` heads of ``d`` channels, ``mixer`` "kda" (keys,
    queries and values of d channels per head) or "scan" (x of d channels per head, B and C of
    ``ds`` channels per group)."""

    def __init__(self, d_model=512, H=4, d=128, G=2, ds=128, W=4, mixer="kda", seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: torch.randn(*s, device=device, generator=g) * std
        self.H, self.d, self.G, self.ds, self.mixer = H, d, G, ds, mixer
        # channels that pass through the convolution, then the mixer's gates and the output gate
        self.conv_channels = 3 * H * d if mixer == "kda" else H * d + 2 * G * ds
        gates = H * d + H if mixer == "kda" else H
        cols = self.conv_channels + gates + H * d
        self.cols = (cols + 7) // 8 * 8  # 16-byte rows: slices of one projection stay wide
        self.w_in = r(d_model, self.cols, std=d_model ** -0.5).bfloat16()
        self.w_out = r(H * d, d_model, std=(H * d) ** -0.5).bfloat16()
        self.taps = r(self.conv_channels, W, std=W ** -0.5)
        self.conv_bias = r(self.conv_channels, std=0.1)
        self.head_norm = 1 + r(d, std=0.1)
        self.block_norm = 1 + r(d_model, std=0.1)
        self.res_scale = 0.5 + r(d_model, std=0.1)
        self.A = -torch.exp(r(H, std=0.5))
        self.D, self.dt_bias = 1 + r(H, std=0.1), -2 + r(H, std=0.5)

    def state(self, n):
        """Zero states of n sequences: the convolution's last inputs and the mixer's matrices."""
        rows = self.d if self.mixer == "kda" else self.ds
        dev = self.w_in.device
        return {"conv": torch.zeros(n, self.taps.shape[1] - 1, self.conv_channels,
                                    dtype=torch.bfloat16, device=dev),
                "mix": torch.zeros(n, self.H, rows, self.d, device=dev)}

    def _split(self, p, u):
        """The mixer's inputs from the projection p and the convolved channels u, and the gate."""
        B, T = p.shape[:2]
        H, d, c = self.H, self.d, self.conv_channels
        if self.mixer == "kda":
            q, k, v = (t.reshape(B, T, H, d) for t in u.split(H * d, -1))
            g = p[..., c:c + H * d].reshape(B, T, H, d)
            beta = p[..., c + H * d:c + H * d + H].contiguous()
            return (q, k, v, g, beta), p[..., c + H * d + H:c + 2 * H * d + H]
        x, b, cc = u.split([H * d, self.G * self.ds, self.G * self.ds], -1)
        heads = lambda t, n: t.unflatten(-1, (n, t.shape[-1] // n))  # views of u
        return ((heads(x, H), p[..., c:c + H], heads(b, self.G), heads(cc, self.G)),
                p[..., c + H:c + H + H * d])

    def _finish(self, o, gate, h):
        """Gated head norm, output projection, and the residual with the next block's norm."""
        B, T = o.shape[:2]
        o, _ = kda.norm_fwd(o.bfloat16(), weight=self.head_norm,
                            gate=gate.unflatten(-1, (self.H, self.d)))
        out = o.reshape(B, T, -1) @ self.w_out
        return kda.norm_fwd(out, residual=h, res_scale=self.res_scale, out_weight=self.block_norm)

    def prompt(self, h, y, cu_seqlens=None):
        """h: residual stream [B,T,d_model]; y: its normed value.  Returns the next pair and the
        states after the last tokens."""
        p = y @ self.w_in
        u, conv = kda.conv_fwd(p[..., :self.conv_channels], self.taps, self.conv_bias,
                               activation="silu", cu_seqlens=cu_seqlens)
        inputs, gate = self._split(p, u)
        if self.mixer == "kda":
            o, mix = kda.fwd_preproc(*(t.contiguous() for t in inputs), cu_seqlens=cu_seqlens)
        else:
            x, dt, b, c = inputs
            o, mix = kda.scan_fwd(x, dt, self.A, b, c, D=self.D, dt_bias=self.dt_bias,
                                  dt_softplus=True, cu_seqlens=cu_seqlens,
                                  out_dtype=torch.bfloat16)
        return *self._finish(o, gate, h), {"conv": conv, "mix": mix}

    def step(self, h, y, state):
        """1 to 8 tokens of each sequence; ``state`` is updated in place."""
        p = y @ self.w_in
        u = kda.conv_step(p[..., :self.conv_channels], self.taps, state["conv"], self.conv_bias,
                          activation="silu")
        inputs, gate = self._split(p, u)
        if self.mixer == "kda":
            o = kda.decode_preproc(*(t.contiguous() for t in inputs), state["mix"])
        else:
            x, dt, b, c = inputs
            o = kda.scan_step(x, dt, self.A, b, c, state["mix"], D=self.D, dt_bias=self.dt_bias,
                              dt_softplus=True, out_dtype=torch.bfloat16)
        return self._finish(o, gate, h)


def run(mixer, B=2, T=150, split=130, d_model=512, device="cuda", seed=0):
    """Outputs of whole prompts, and of prompts up to ``split`` followed by single tokens."""
    block = Block(d_model, mixer=mixer, device=device, seed=seed)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    h = torch.randn(B, T, d_model, device=device, generator=g).bfloat16()
    _, y = kda.norm_fwd(h, out_weight=block.block_norm)  # the first block's own norm
    whole = block.prompt(h, y)[:2]
    *first, state = block.prompt(h[:, :split].contiguous(), y[:, :split].contiguous())
    parts = [first]
    for t in range(split, T):
        parts.append(block.step(h[:, t:t + 1].contiguous(), y[:, t:t + 1].contiguous(), state))
    return whole, tuple(torch.cat([p[i] for p in parts], 1) for i in range(2))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--mixer", choices=("kda", "scan"), default="scan")
    a = ap.parse_args()
    whole, parts = run(a.mixer)
    worst = max(float((w.float() - p.float()).abs().max() / w.float().square().mean().sqrt())
                for w, p in zip(whole, parts))
    print(f"{a.mixer}: prompt against prompt + single tokens: max difference {worst:.1e} of the rms")
    block = Block(mixer=a.mixer)
    state = block.state(64)
    h = torch.randn(64, 1, 512, device="cuda").bfloat16()
    _, y = kda.norm_fwd(h, out_weight=block.block_norm)
    for _ in range(10):
        block.step(h, y, state)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(100):
        block.step(h, y, state)
    torch.cuda.synchronize()
    print(f"one token of 64 sequences: {(time.perf_counter() - t0) * 1e4:.0f} us")


if __name__ == "__main__":
    main()
