"""64-bit restatements of the decoder-step operators, and the inputs of their tests."""
import math

import torch


def make_cache(lens, hkv, dim, page, gen, device, spare=3, max_pages=None, keep=None):
    """A paged cache of random values whose pages are shuffled among the sequences.  keep(n, p): whether page p of
    sequence n is mapped (the others are -1).  Pages of nobody, and rows past a sequence's end, are NaN."""
    need = [(n, p) for n, length in enumerate(lens) for p in range(-(-length // page)) if keep is None or keep(n, p)]
    width = max_pages or max(1, max(-(-length // page) for length in lens) + 1)
    total = len(need) + spare
    order = torch.randperm(total, generator=gen, device=device).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    k = torch.full((total, hkv, page, dim), math.nan, dtype=torch.bfloat16, device=device)
    v = torch.full((total, hkv, page, dim), math.nan, dtype=torch.bfloat16, device=device)
    for (n, p), at in zip(need, order):
        table[n, p] = at
        rows = min(page, lens[n] - p * page)
        for c in (k, v):
            c[at, :, :rows] = torch.randn((hkv, rows, dim), generator=gen, device=device).to(torch.bfloat16)
    return k, v, table.to(device)


def gather(cache, table, n, positions):
    """Rows of the cache at `positions` (a list) of sequence n, [len, hkv, dim] fp64."""
    page = cache.shape[2]
    j = torch.as_tensor(positions, dtype=torch.long, device=cache.device)
    return cache[table[n].long()[j // page], :, j % page].double()


def attention(q, k_cache, v_cache, table, lens, new, window, sinks, scale):
    """q: list of [Q_n, Hq, D] (any float type).  Returns, per sequence, out, lse, sum p |v| (the weight of rounding the
    probabilities) and scale * max_j sum |q k| (that of the scores), all fp64."""
    res = []
    for n, x in enumerate(q):
        qn, hq, d = x.shape
        hkv = k_cache.shape[1]
        out = torch.zeros((qn, hq, d), dtype=torch.float64, device=x.device)
        lse = torch.full((qn, hq), -math.inf, dtype=torch.float64, device=x.device)
        mag, big = torch.zeros_like(out), torch.zeros_like(lse)
        for i in range(qn):
            p = lens[n] - new[n] + i
            seen = [j for j in range(p + 1) if j > p - window or j < sinks]
            if not seen:
                continue
            k = gather(k_cache, table, n, seen).repeat_interleave(hq // hkv, 1)
            v = gather(v_cache, table, n, seen).repeat_interleave(hq // hkv, 1)
            y = x[i].double()
            s = scale * torch.einsum("hd,jhd->hj", y, k)
            lse[i] = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[i][:, None])
            out[i] = torch.einsum("hj,jhd->hd", w, v)
            mag[i] = torch.einsum("hj,jhd->hd", w, v.abs())
            big[i] = scale * torch.einsum("hd,jhd->hj", y.abs(), k.abs()).amax(-1)
        res.append((out, lse, mag, big))
    return res


def rotate(x, cos, sin, interleaved):
    """x [heads, dim] fp64, cos / sin [rotary / 2] fp64."""
    r, y = cos.numel(), x.clone()
    for i in range(r):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        y[:, a] = x[:, a] * cos[i] - x[:, b] * sin[i]
        y[:, b] = x[:, b] * cos[i] + x[:, a] * sin[i]
    return y


def beam_scores(logits, scores, finished, eos):
    """fp64 scores [B, W, V] of every candidate."""
    x = logits.double()
    x = torch.where(x.isnan(), -math.inf, x)
    c = scores.double()[..., None] - torch.logsumexp(x, -1, keepdim=True)
    s = c + x
    dead = ~torch.isfinite(x.amax(-1)) | scores.isnan()
    s = torch.where(s.isnan() | dead[..., None], -math.inf, s)
    if finished is not None:
        only = torch.full_like(s, -math.inf)
        only[..., eos] = scores.double()
        s = torch.where(finished.bool()[..., None], only, s)
    return s
