"""64-bit restatements of linear attention with a decay for each head and of draft verification, straight from the definitions."""
import torch


def linear(q, k, v, a, scale, init, ranges):
    """q [tokens, H, D], k and v [tokens, Hkv, D], a [tokens, H] (logarithms of the decays), init [N, H, D, D] or None, ranges
    [(first token, tokens)].  Returns out [tokens, H, D] (NaN where no sequence has the token), states [N, H, D, D], and the same
    two for the magnitudes of all operands: what the results would be if nothing cancelled."""
    h, d = q.shape[1:]
    share = h // k.shape[1]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    mag = out.clone()
    states = torch.zeros((len(ranges), h, d, d), dtype=torch.float64, device=q.device)
    if init is not None:
        states += init.double()
    sizes = states.abs()
    q, k, v, a = q.double(), k.double().repeat_interleave(share, 1), v.double().repeat_interleave(share, 1), a.double()
    for n, (first, count) in enumerate(ranges):
        s, m = states[n], sizes[n]
        for t in range(first, first + count):
            g = a[t].exp()[:, None, None]
            s = g * s + v[t][:, :, None] * k[t][:, None, :]
            m = g * m + v[t].abs()[:, :, None] * k[t].abs()[:, None, :]
            out[t] = scale * torch.einsum("hvk,hk->hv", s, q[t])
            mag[t] = abs(scale) * torch.einsum("hvk,hk->hv", m, q[t].abs())
        states[n], sizes[n] = s, m
    return out, states, mag, sizes


def verify(logits, drafts, probs, uniform, noise, temperature, lens):
    """tokens [B, K + 1], counts [B] and how near each request came to deciding otherwise: the smallest relative distance of a draft's
    test from its border, and of the race's winner from the runner-up."""
    b, rows, v = logits.shape
    tokens = torch.full((b, rows), -1, dtype=torch.long)
    counts = torch.ones((b,), dtype=torch.long)
    near = torch.full((b,), float("inf"), dtype=torch.float64)
    logits = logits.double().cpu()
    logits = torch.where(logits.isnan(), float("-inf"), logits)
    for i in range(b):
        tau = float(temperature[i])
        n = int(lens[i])
        r = 0
        while True:
            row = logits[i, r]
            top = row.max()
            if not torch.isfinite(top):
                p = torch.zeros(v, dtype=torch.float64)
            elif tau == 0:
                p = (row == top).double()
            else:
                p = ((row - top) / tau).exp()
                p = p / p.sum()
            x = int(drafts[i, r]) if r < n else -1
            if r == n or not 0 <= x < v:
                break
            if tau == 0:
                if p[x] == 0:
                    break
            else:
                bar = float(uniform[i, r]) * (float(probs[i, r, x]) if probs is not None else 1.0)
                near[i] = min(near[i], abs(float(p[x]) - bar) / max(float(p[x]), 1e-30))
                if not bar < p[x]:
                    break
            tokens[i, r] = x
            r += 1
        counts[i] = r + 1
        if tau == 0:
            if p.max() > 0:
                tokens[i, r] = int(p.argmax())
            continue
        w = p.clone()
        if r < n:
            if probs is not None:
                w = (p - probs[i, r].double().cpu()).clamp(min=0)
                w = torch.where(w.isnan(), 0.0, w)
            elif 0 <= x < v:
                w[x] = 0.0
        if not w.max() > 0:
            w = p
        if not w.max() > 0:
            continue
        e = noise[i].double().cpu()
        race = torch.where((w > 0) & (e >= 0), w / e, 0.0)
        best = race.max()
        if not best > 0:
            continue
        tokens[i, r] = int((race == best).nonzero()[0])
        rest = torch.where(torch.arange(v) == tokens[i, r], 0.0, race).max()
        # how much smaller the winner's lead is than the probabilities it is a difference of
        at = tokens[i, r]
        lead = float((best - rest) / best) * float(w[at] / p[at])
        near[i] = min(near[i], lead)
    return tokens, counts, near
