"""Speculative decoding over a small decoder of linear-attention layers, random weights.

    python examples/speculative_decode.py [--batch 4] [--drafts 4] [--steps 32] [--temperature 0.8]

A round drafts tokens with a cheaper head on copies of the states, runs the model once over the last token and the drafts
(kda_linear_attn without a final state), lets kda_verify_drafts decide how many of them stand, and takes its counts as `lens` to
advance the states by exactly the tokens that were kept.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_23_gb300 as kda  # noqa: E402


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Model:
    """Embedding, linear-attention layers with a gate for each head and token, a head, and a noisy copy of it for drafts."""

    def __init__(self, vocab, heads, kv_heads, dim, layers, state=torch.float32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        width = heads * dim
        self.vocab, self.heads, self.kv_heads, self.dim, self.layers, self.kind = vocab, heads, kv_heads, dim, layers, state

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device="cuda").mul(rows ** -0.5)

        self.embed = weight(vocab, width).mul(vocab ** 0.5).to(torch.bfloat16)
        self.proj = [weight(width, (heads + 2 * kv_heads) * dim).to(torch.bfloat16) for _ in range(layers)]
        self.gates = [weight(width, heads) for _ in range(layers)]
        self.out = [weight(width, width).to(torch.bfloat16) for _ in range(layers)]
        self.head = weight(width, vocab)
        self.draft_head = self.head + 0.15 * weight(width, vocab)
        self.log_decay = -torch.exp2(-5.0 - torch.arange(heads, device="cuda"))

    def new_states(self, batch):
        return [torch.zeros((batch, self.heads, self.dim, self.dim), dtype=self.kind, device="cuda") for _ in range(self.layers)]

    def run(self, tokens, states, final=None):
        """The last layer's output for tokens [B, T] from these states, and what each layer read; the states after them into `final`."""
        x, read = self.embed[tokens], []
        for i in range(self.layers):
            y = norm(x)
            h, hk, d = self.heads, self.kv_heads, self.dim
            z = y @ self.proj[i]
            q, k, v = (p.unflatten(-1, (-1, d)) for p in z.split([h * d, hk * d, hk * d], -1))
            gate = -0.1 * torch.nn.functional.softplus(y.float() @ self.gates[i])
            o = torch.empty((*tokens.shape, h, d), dtype=torch.bfloat16, device="cuda")
            kda.kda_linear_attn(q, k, v, o, log_decay=self.log_decay, gate=gate, initial_state=states[i],
                                final_state=None if final is None else final[i])
            read.append((q, k, v, gate, o))
            x = x + norm(o.flatten(2)) @ self.out[i]
        return norm(x).float(), read

    def advance(self, read, states, counts):
        """The states after the first counts[b] tokens of a run."""
        for (q, k, v, gate, o), s in zip(read, states):
            kda.kda_linear_attn(q, k, v, o, log_decay=self.log_decay, gate=gate, initial_state=s, final_state=s, lens=counts)

    def states_of(self, tokens):
        states = self.new_states(tokens.shape[0])
        self.run(tokens, states, final=states)
        return states

    def margin(self, prompt, tokens):
        """How far apart the two largest logits are after these tokens."""
        whole = torch.cat((prompt, tokens))[None]
        top = (self.run(whole, self.new_states(1))[0][:, -1] @ self.head).topk(2).values[0]
        return float(top[0] - top[1])


def pick(logits, drafts, probs, temperature, gen):
    """kda_verify_drafts with random numbers of its own: tokens [B, K + 1] and counts [B]."""
    b, rows, vocab = logits.shape
    tokens = torch.empty((b, rows), dtype=torch.int32, device="cuda")
    counts = torch.empty((b,), dtype=torch.int32, device="cuda")
    noise = torch.empty((b, vocab), device="cuda").exponential_(generator=gen).clamp_(min=1e-20)
    kda.kda_verify_drafts(logits, drafts, torch.rand((b, rows - 1), generator=gen, device="cuda"), noise, tokens, counts,
                          draft_probs=probs, temperature=torch.full((b,), temperature, device="cuda"), first_largest=True)
    return tokens, counts


def speculative(model, prompt, steps, drafts, temperature, seed=0, whole=False):
    """Tokens [B, steps] after the prompt and the rounds it took; `whole`: all tokens kept, the states, and how many tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, n = prompt.shape
    states = model.states_of(prompt[:, :-1])
    last = prompt[:, -1:]
    kept = torch.full((b, steps + drafts + 1), -1, dtype=torch.long, device="cuda")
    length = torch.zeros((b,), dtype=torch.long, device="cuda")
    rounds = 0
    while int(length.min()) < steps:
        guess, inputs, probs, x = [s.clone() for s in states], [last], [], last
        for _ in range(drafts):
            logits = model.run(x, guess, final=guess)[0] @ model.draft_head
            if temperature > 0:
                p = torch.softmax(logits[:, 0] / temperature, -1)
                probs.append(p)
                x = torch.multinomial(p, 1, generator=gen)
            else:
                x = logits[:, 0].argmax(-1, keepdim=True)
            inputs.append(x)
        inputs = torch.cat(inputs, 1)
        y, read = model.run(inputs, states)
        tokens, counts = pick(y @ model.head, inputs[:, 1:].to(torch.int32), torch.stack(probs, 1) if probs else None, temperature, gen)
        # a request that has all its tokens stays where it is
        counts = torch.where(length < steps, counts, 0).to(torch.int32)
        model.advance(read, states, counts)
        at = torch.arange(drafts + 1, device="cuda")
        new = at < counts[:, None]
        kept[new.nonzero()[:, 0], (length[:, None] + at)[new]] = tokens[new].long()
        length += counts
        last = torch.where(counts[:, None] > 0, tokens.long().gather(1, (counts.long() - 1).clamp(min=0)[:, None]), last)
        rounds += 1
    kda.device_status()
    return (kept, states, length) if whole else (kept[:, :steps], rounds)


def single(model, prompt, steps):
    """The same tokens one at a time, greedily."""
    states = model.states_of(prompt[:, :-1])
    x, got = prompt[:, -1:], []
    nothing = torch.empty((prompt.shape[0], 0), dtype=torch.int32, device="cuda")
    for _ in range(steps):
        logits = model.run(x, states, final=states)[0] @ model.head
        x = pick(logits, nothing, None, 0.0, torch.Generator(device="cuda"))[0].long()
        got.append(x)
    return torch.cat(got, 1)


def main():
    parser = argparse.ArgumentParser(description=__doc__)
    parser.add_argument("--batch", type=int, default=4)
    parser.add_argument("--drafts", type=int, default=4)
    parser.add_argument("--steps", type=int, default=32)
    parser.add_argument("--temperature", type=float, default=0.8)
    args = parser.parse_args()
    model = Model(vocab=1000, heads=4, kv_heads=2, dim=128, layers=3)
    prompt = torch.randint(0, 1000, (args.batch, 50), device="cuda")
    tokens, rounds = speculative(model, prompt, args.steps, args.drafts, args.temperature)
    print(f"{args.steps} tokens of {args.batch} requests in {rounds} runs of the model")
    for row in tokens.tolist():
        print(" ".join(map(str, row)))


if __name__ == "__main__":
    main()
