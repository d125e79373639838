"""Linear attention and draft verification together: a speculative decoder's loop, against the same model token by token."""
import pytest
import torch

from examples import speculative_decode as ex

pytestmark = pytest.mark.gpu


def test_the_loop_gives_the_tokens_of_single_steps():
    """Greedy requests: whatever the drafts, the tokens are those of decoding one at a time.  A request may part from them where
    two logits are nearer than the products' roundings (activations in bf16: 2^-8 of logits of about 4)."""
    model = ex.Model(vocab=500, heads=4, kv_heads=2, dim=64, layers=2, seed=1)
    prompt = torch.randint(0, 500, (6, 70), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    fast, rounds = ex.speculative(model, prompt, steps=24, drafts=4, temperature=0.0, seed=3)
    slow = ex.single(model, prompt, steps=24)
    same = fast == slow
    # a request may part from the single steps at a near tie; up to there it has to be the same
    for b in range(6):
        part = int(same[b].long().cumprod(0).sum())
        assert part == 24 or model.margin(prompt[b], slow[b, :part]) < 2.0 ** -5, (b, part)
    assert int(same.all(1).sum()) >= 4
    assert rounds < 24                                      # drafts were accepted


def test_the_loops_states_are_those_of_the_tokens_it_kept():
    """After any run the states are what the kept tokens alone make of the prompt's."""
    model = ex.Model(vocab=300, heads=4, kv_heads=4, dim=128, layers=1, state=torch.float32, seed=4)
    prompt = torch.randint(0, 300, (4, 33), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    tokens, states, lengths = ex.speculative(model, prompt, steps=16, drafts=5, temperature=0.9, seed=6, whole=True)
    for b in range(4):
        kept = torch.cat((prompt[b], tokens[b, :lengths[b] - 1]))      # the last token has not been read yet
        again = model.states_of(kept[None])
        for s, t in zip(states, again):
            assert float((s[b] - t[0]).norm() / t.norm()) <= 2.0 ** -14   # fp32, in other pieces
