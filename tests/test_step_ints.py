"""CPU checks of integers that the decoder-step binding hands to C: what does not fit is refused or clamped, never cut off."""
import pytest
import torch

from gated_delta_rule_23_gb300 import _native, step


@pytest.fixture
def calls(monkeypatch):
    """The checked way without a GPU: the compiled binding declines, and what would be called is kept."""
    class Declines:
        def __getattr__(self, name):
            return lambda *a: None
    kept = []

    def call(fn, dev, stream, *args):
        step._fit(fn, args)
        kept.append((fn.__name__, args))
    monkeypatch.setattr(_native, "_binding", Declines())
    monkeypatch.setattr(step, "_device", lambda t, name: t.device)
    monkeypatch.setattr(step, "_call", call)
    return kept


def _attn(**kw):
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 3, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    step.kda_window_attn(q, cache, cache.clone(), table, lens, torch.empty_like(q), **kw)


def _select(eos=0, v=5):
    logits = torch.zeros(1, 2, 5).as_strided((1, 2, v), (2 * v, v, 1)) if v == 5 else torch.empty(1, 2, v, device="meta")
    dev = logits.device
    out = [torch.zeros(1, 2, device=dev, dtype=t) for t in (torch.float32, torch.int32, torch.int32)]
    step.kda_beam_select(logits, torch.zeros(1, 2, device=dev), *out, eos=eos)


WIDE = [2 ** 31, 2 ** 32, 2 ** 32 + 3, -2 ** 31 - 1, -2 ** 32]


@pytest.mark.parametrize("value", WIDE)
def test_attention_window_and_sinks(calls, value):
    for kw in (dict(window=value), dict(window=7, sinks=value)):
        if value < 0:
            with pytest.raises(ValueError):
                _attn(**kw)
            continue
        _attn(**kw)
        window, sinks = calls.pop()[1][9:11]
        assert (window, sinks) == (2 ** 31 - 1 if kw["window"] > 7 else 7, 2 ** 31 - 1 if "sinks" in kw else 0)
    assert not calls
    _attn(window=3, sinks=2 ** 31 - 1)
    assert calls.pop()[1][9:11] == (3, 2 ** 31 - 1)


@pytest.mark.parametrize("value", WIDE)
def test_selection_and_reorder(calls, value):
    with pytest.raises(ValueError):
        _select(eos=value)
    with pytest.raises(ValueError):
        step.kda_state_reorder(torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32), value)
    if value > 0:
        with pytest.raises(ValueError):
            _select(v=value)                          # a vocabulary, on no device: only its shape is read
    assert not calls
    _select(eos=4)
    assert calls.pop()[1][5] == 4


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("name", ["N", "Hq", "Hkv", "page", "max_pages"])
def test_workspace_sizes(name, value):
    sizes = dict(N=2, T=3, Hq=8, Hkv=2, D=128, page=16, max_pages=4)
    with pytest.raises(ValueError):
        step.window_attn_workspace_size(8, 0, **dict(sizes, **{name: value}))
    beam = dict(B=1, W=2, V=100, K=2)
    for n in beam:
        with pytest.raises(ValueError):
            step.beam_select_workspace_size(**dict(beam, **{n: value}))
    assert step.window_attn_workspace_size(2 ** 40, 2 ** 40, **sizes) == step.window_attn_workspace_size(2 ** 31 - 1, 2 ** 31 - 1, **sizes)
