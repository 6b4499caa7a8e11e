"""Speculative decoding of a small hybrid stack, built from the library's entry points.

One recurrent layer (KDA) and one attention layer share a residual stream:

    KDA:        projections -> decode over the state pool -> residual
    attention:  projections -> query and key norms with rotation -> 8-bit paged cache
                -> attention of the new tokens over it -> residual

A round takes the last known token and K drafted ones of every sequence through the stack in one
step (``verify``), compares the drafts with the resulting probabilities (``draft_verify``) and keeps
the state after ``num_commit`` tokens: the recurrent layer by replay (``decode_commit``), the cache by
its length alone.  Sequences move on by different numbers of tokens.  ``main`` checks that the states
and outputs are those of the kept tokens taken one at a time, and times a round.

    python examples/hybrid_decode.py
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kda_delta_rule_fwd_gb300 as kda  # noqa: E402


class Stack:
    """Random weights; ``n`` sequences of up to ``places`` tokens each."""

    def __init__(self, n=4, vocab=1000, d_model=256, H=2, d=128, kv_heads=1, places=256, page=16, seed=0,
                 cache_dtype=torch.float8_e4m3fn, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: torch.randn(*s, device=device, generator=g) * std
        w = lambda i, o: r(i, o, std=i ** -0.5).bfloat16()
        self.n, self.H, self.d, self.G = n, H, d, kv_heads
        self.embed, self.head = r(vocab, d_model, std=1.0).bfloat16(), w(d_model, vocab)
        self.mix_in, self.mix_out = w(d_model, 4 * H * d + H), w(H * d, d_model)
        self.att_in, self.att_out = w(d_model, (H + 2 * kv_heads) * d), w(H * d, d_model)
        self.norms = [1 + r(d_model, std=0.1) for _ in range(2)]
        self.q_norm, self.k_norm = 1 + r(d, std=0.1), 1 + r(d, std=0.1)
        self.freqs = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=device) / d)
        per = -(-places // page)
        self.cache = kda.kv_cache(n * per, page, kv_heads, d, dtype=cache_dtype, device=device)
        self.pages = torch.randperm(n * per, device=device, generator=g).to(torch.int32).reshape(n, per)
        self.state = torch.zeros(n, H, d, d, device=device)
        self.lens = torch.zeros(n, dtype=torch.int32, device=device)  # tokens kept so far

    def _mixer(self, h):
        """The recurrent layer's inputs."""
        _, y = kda.norm_fwd(h, out_weight=self.norms[0])
        B, T, _ = h.shape
        q, k, v, g, beta = (y @ self.mix_in).split([self.H * self.d] * 4 + [self.H], -1)
        heads = lambda t: t.reshape(B, T, self.H, self.d).contiguous()
        return heads(q), heads(k), heads(v), heads(g), beta.contiguous()

    def verify(self, tokens):
        """All ``tokens [n, T]`` through the stack: float32 logits, and the recurrent layer's inputs
        for the replay.  The state stays; the cache holds the new rows, which count only once
        ``lens`` covers them."""
        n, T = tokens.shape
        h = self.embed[tokens.long()]
        raw = self._mixer(h)
        o = kda.decode_preproc(*raw, self.state.clone())
        h, y = kda.norm_fwd(o.bfloat16().reshape(n, T, -1) @ self.mix_out, residual=h, out_weight=self.norms[1])
        q, k, v = (t.unflatten(-1, (-1, self.d))
                   for t in (y @ self.att_in).split([self.H * self.d, self.G * self.d, self.G * self.d], -1))
        after = self.lens + T
        places = self.lens[:, None] + torch.arange(T, dtype=torch.int32, device=h.device)
        q, k = kda.qknorm_fwd(q, k, places, self.freqs, q_weight=self.q_norm, k_weight=self.k_norm)
        kda.cache_write(k, v, self.cache, self.pages, after)
        o = kda.attn_step(q, self.cache, self.pages, after)
        h = h + o.reshape(n, T, -1) @ self.att_out
        return (h @ self.head).float(), raw

    def commit(self, raw, counts):
        """Keep the first ``counts[i]`` tokens of each sequence's last step."""
        q, k, v, g, beta = raw
        # the preprocessing of the step's inputs, as its kernel makes it
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype)
        gate = -torch.nn.functional.softplus(g.float()).to(g.dtype)
        kda.decode_commit(unit(q), unit(k), v, gate, torch.sigmoid(beta), self.state, counts, want_out=False)
        self.lens += counts


def round_of(stack, last, drafts, q, u):
    """One round: the step over [last token, drafts], the decision, the kept states.  Returns the
    kept drafts and the drawn token (then -1), the counts and the logits."""
    logits, raw = stack.verify(torch.cat([last[:, None], drafts], 1))
    tokens, counts = kda.draft_verify(torch.softmax(logits, -1), q, drafts, u)
    stack.commit(raw, counts)
    return tokens, counts, logits


def run(rounds=6, K=3, n=4, vocab=1000, seed=0, **kw):
    """The same kept tokens in rounds of K drafts and one at a time; returns both stacks, the logits
    at the kept places of both, and how many drafts were kept."""
    a, b = (Stack(n, vocab, seed=seed, **kw) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    last = torch.randint(0, vocab, (n,), device="cuda", generator=g, dtype=torch.int32)
    pairs, kept = [], 0
    for _ in range(rounds):
        # drafts from a flat distribution, of which few would be kept: every second one is made certain
        q = torch.full((n, K, vocab), 1.0 / vocab, device="cuda")
        drafts = torch.randint(0, vocab, (n, K), device="cuda", generator=g, dtype=torch.int32)
        u = torch.rand(n, K + 1, device="cuda", generator=g)
        u[::2, :K] = 0  # these sequences keep every draft
        tokens, counts, logits = round_of(a, last, drafts, q, u)
        # the same tokens singly: column t of those sequences that kept it
        line = torch.cat([last[:, None], drafts], 1)
        for t in range(K + 1):
            on = counts > t
            one, raw = b.verify(line[:, t:t + 1].contiguous())
            b.commit(raw, on.to(torch.int32))
            pairs.append((logits[on, t], one[on, 0]))
        kept += int(counts.sum()) - n
        last = tokens.gather(1, (counts - 1).long()[:, None])[:, 0]
    return a, b, pairs, kept


def main():
    a, b, pairs, kept = run()
    worst = max(float((x - y).abs().max() / y.square().mean().sqrt()) for x, y in pairs if y.numel())
    print(f"rounds of drafts against single tokens: {kept} drafts kept, logits within {worst:.1e} of the rms")
    n, K, vocab = 64, 3, 32000
    s = Stack(n, vocab, places=1024)
    last = torch.zeros(n, dtype=torch.int32, device="cuda")
    q = torch.full((n, K, vocab), 1.0 / vocab, device="cuda")
    drafts = torch.zeros(n, K, dtype=torch.int32, device="cuda")
    u = torch.rand(n, K + 1, device="cuda")
    for _ in range(5):
        round_of(s, last, drafts, q, u)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        round_of(s, last, drafts, q, u)
    torch.cuda.synchronize()
    print(f"a round of {K} drafts for {n} sequences: {(time.perf_counter() - t0) * 5e4:.0f} us")


if __name__ == "__main__":
    main()
