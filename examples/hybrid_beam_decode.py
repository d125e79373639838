"""Beam search over a small hybrid decoder: KDA layers and window-attention layers, random weights.

    python examples/hybrid_beam_decode.py [--batch 2] [--beams 4] [--steps 8]

Every layer of the model and every part of a decode step runs through the library: kda_fwd for the prompt and
kda_fwd_recurrent for single tokens in the KDA layers, kda_kv_append and kda_window_attn over a paged cache in the
attention layers, kda_beam_select on the logits, kda_state_reorder for the KDA states and the cache pages of the beams.
The projections are plain matrix products.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_23_gb300 as kda  # noqa: E402

D = 128


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class KDALayer:
    """q, k, v, gate and beta projections, the delta rule, output projection; one state row a sequence."""

    def __init__(self, width, heads, gen):
        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device="cuda").mul(rows ** -0.5).to(torch.bfloat16)
        self.heads = heads
        self.proj = weight(width, heads * D * 4 + heads)
        self.out = weight(heads * D, width)
        self.A_log = torch.rand(heads, generator=gen, device="cuda")
        self.dt_bias = torch.randn((heads, D), generator=gen, device="cuda") * 0.1

    def start(self, rows, pages):
        self.state = torch.zeros((rows, self.heads, D, D), device="cuda")

    def __call__(self, x, lens, first):
        b, t, _ = x.shape
        y = x @ self.proj
        q, k, v, g = (z.unflatten(-1, (self.heads, D)).contiguous() for z in y[..., :4 * self.heads * D].chunk(4, -1))
        beta = y[..., 4 * self.heads * D:].contiguous()
        o = torch.empty_like(q)
        step = kda.kda_fwd if t > 1 else kda.kda_fwd_recurrent
        step(q, k, v, g, beta, D ** -0.5, o, self.A_log, self.dt_bias, -5.0,
             initial_state=None if first else self.state, final_state=self.state)
        return norm(o).flatten(2) @ self.out

    def follow(self, parents, beams):
        return [self.state]


class WindowLayer:
    """Grouped-query attention with rotary positions, a sliding window and sinks, over pages of its own a sequence."""
    page = 16

    def __init__(self, width, heads, kv_heads, window, sinks, most, gen):
        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device="cuda").mul(rows ** -0.5).to(torch.bfloat16)
        self.heads, self.kv_heads, self.window, self.sinks = heads, kv_heads, window, sinks
        self.proj = weight(width, (heads + 2 * kv_heads) * D)
        self.out = weight(heads * D, width)
        angle = torch.arange(most, device="cuda")[:, None] * 10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
        self.cos, self.sin = angle.cos(), angle.sin()

    def start(self, rows, pages):
        shape = (rows * pages, self.kv_heads, self.page, D)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = torch.arange(rows * pages, dtype=torch.int32, device="cuda").view(rows, pages)
        self.pages = pages

    def __call__(self, x, lens, first):
        b, t, _ = x.shape
        y = (x @ self.proj).unflatten(-1, (-1, D))
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 2)      # strided rows of one product
        turned = torch.empty((b, t, self.heads, D), dtype=torch.bfloat16, device="cuda")
        kda.kda_kv_append(k, v, self.k, self.v, self.table, lens, self.cos, self.sin, q=q, q_out=turned)
        o = torch.empty_like(turned)
        kda.kda_window_attn(turned, self.k, self.v, self.table, lens, o, self.window, sinks=self.sinks)
        return o.flatten(2) @ self.out

    def follow(self, parents, beams):
        return [c.view(-1, self.pages, *c.shape[1:]) for c in (self.k, self.v)]


class Decoder:
    def __init__(self, vocab=1000, width=512, heads=4, window=40, sinks=3, most=4096, layers="kwk", seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((vocab, width), generator=gen, device="cuda").to(torch.bfloat16)
        self.head = torch.randn((width, vocab), generator=gen, device="cuda").mul(2 * width ** -0.5).to(torch.bfloat16)
        self.layers = [KDALayer(width, heads, gen) if c == "k" else
                       WindowLayer(width, heads, 2, window, sinks, most, gen) for c in layers]

    def start(self, rows, tokens):
        for layer in self.layers:
            layer.start(rows, -(-tokens // WindowLayer.page))

    def forward(self, tokens, lens, first=False):
        """Logits of the last token of every row; tokens [rows, t], lens the rows' tokens with these."""
        x = self.embed[tokens.long()]
        for layer in self.layers:
            x = x + layer(norm(x), lens, first)
        return (norm(x[:, -1]) @ self.head).float()


def beam_search(model, prompts, beams, steps):
    """The beams' scores [batch, beams] and tokens [batch, beams, steps], best first."""
    b, t = prompts.shape
    rows = b * beams
    model.start(rows, t + steps)
    tokens = prompts.repeat_interleave(beams, 0)
    lens = torch.full((rows,), t, dtype=torch.int32, device="cuda")
    logits = model.forward(tokens, lens, first=True)
    scores = torch.full((b, beams), -math.inf, device="cuda")
    scores[:, 0] = 0.0                                           # the beams are equal before the first choice
    chosen = torch.empty((rows, 0), dtype=torch.int32, device="cuda")
    for step in range(steps):
        best = torch.empty((b, beams), device="cuda")
        token = torch.empty((b, beams), dtype=torch.int32, device="cuda")
        parents = torch.empty_like(token)
        kda.kda_beam_select(logits.view(b, beams, -1), scores, best, token, parents)
        scores = best
        chosen = torch.cat((chosen[parents.view(-1).long()], token.view(-1, 1)), 1)
        if step + 1 == steps:
            break
        # states and cache pages follow their beams, in place
        kda.kda_state_reorder([x for layer in model.layers for x in layer.follow(parents, beams)], parents.view(-1), beams)
        lens += 1
        logits = model.forward(token.view(-1, 1), lens)
    kda.device_status()
    return scores, chosen.view(b, beams, steps)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=100)
    a = ap.parse_args()
    model = Decoder()
    prompts = torch.randint(0, 1000, (a.batch, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    scores, tokens = beam_search(model, prompts, a.beams, a.steps)
    for i in range(a.batch):
        for w in range(a.beams):
            print(f"prompt {i} beam {w}: {scores[i, w].item():8.3f}  {tokens[i, w].tolist()}")


if __name__ == "__main__":
    main()
