"""The example that runs the decoder-step operators together: its beams' scores, which the decode path built up token by
token through appended caches, moved states and reordered pages, against the prompt path on the whole sequences.

Tolerance: the two paths round the same bf16 activations differently.  A logit is a sum over hidden values of which each
carries a few bf16 roundings (three layers, two each: under 8 x 2^-9 of its size), so at logits of size 2 to 8 a step's
log-probability is off by less than 0.1; the steps add up.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_beam_decode", os.path.join(ROOT, "examples", "hybrid_beam_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("beams, prompt, steps", [(4, 70, 6), (1, 33, 4), (3, 5, 5)])
def test_beams_score_as_their_sequences(example, beams, prompt, steps):
    model = example.Decoder(vocab=300, width=256, heads=4, window=24, sinks=2)
    prompts = torch.randint(0, 300, (2, prompt), generator=torch.Generator().manual_seed(prompt)).cuda()
    scores, tokens = example.beam_search(model, prompts, beams, steps)
    assert bool((scores[:, 1:] <= scores[:, :-1]).all())
    seen = [tuple(x) for x in tokens.view(-1, steps).tolist()]
    assert all(len(set(seen[i * beams:(i + 1) * beams])) == beams for i in range(2))
    # every beam's sequence again, one prompt of all its tokens a step
    whole = torch.cat((prompts.repeat_interleave(beams, 0), tokens.view(-1, steps).long()), 1)
    total = torch.zeros(2 * beams, dtype=torch.float64, device="cuda")
    for s in range(steps):
        t = prompt + s
        model.start(2 * beams, t)
        logits = model.forward(whole[:, :t], torch.full((2 * beams,), t, dtype=torch.int32, device="cuda"), first=True)
        logp = torch.log_softmax(logits.double(), -1)
        total += logp.gather(1, whole[:, t:t + 1])[:, 0]
    assert bool(((total - scores.view(-1).double()).abs() <= 0.1 * steps).all()), (total, scores)
