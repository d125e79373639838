"""Workloads of the decoder-step operators: appending to a paged cache with rotary positions, attention with a sliding
window and sinks over that cache, beam selection over the vocabulary, and reordering of recurrent states.

Each workload runs in two forms on the same inputs: the operator in elementary torch operations in 32 bits
(``own = False``) or the library's entry points (``own = True``).  ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's decode step in a grouped-query layer: pure latency
        dict(name="append decode 1", op="append", batch=1, tokens=1, context=4096, heads=32, kv_heads=8, dim=128,
             rotary=128, page=16, interleaved=False, ragged=False, mix=1),
        # a full decode batch
        dict(name="append decode 256", op="append", batch=256, tokens=1, context=4096, heads=64, kv_heads=8, dim=128,
             rotary=64, page=64, interleaved=True, ragged=False, mix=2),
        # prompts of irregular lengths prefilled together
        dict(name="append ragged 8192", op="append", batch=12, tokens=8192, context=0, heads=96, kv_heads=8, dim=128,
             rotary=128, page=64, interleaved=False, ragged=True, mix=3),
        # one user's decode step, long context behind a window: latency
        dict(name="attn decode 1", op="attn", batch=1, tokens=1, context=32768, heads=32, kv_heads=8, dim=128,
             page=16, window=4096, sinks=4, ragged=False, mix=4),
        # a full decode batch: the cache's bytes
        dict(name="attn decode 256", op="attn", batch=256, tokens=1, context=32768, heads=64, kv_heads=8, dim=128,
             page=64, window=1024, sinks=16, ragged=False, mix=5),
        # a long prompt in a layer whose window covers all of it: the tensor cores
        dict(name="attn prefill 8192", op="attn", batch=1, tokens=8192, context=0, heads=96, kv_heads=8, dim=128,
             page=128, window=8192, sinks=0, ragged=False, mix=6),
        # prompts of irregular lengths behind a short window
        dict(name="attn ragged 8192", op="attn", batch=12, tokens=8192, context=0, heads=64, kv_heads=8, dim=128,
             page=32, window=512, sinks=4, ragged=True, mix=7),
        # the next piece of two long prompts, odd sizes, the small head
        dict(name="attn chunk 509", op="attn", batch=2, tokens=509, context=20011, heads=14, kv_heads=2, dim=64,
             page=16, window=2049, sinks=37, ragged=False, mix=8),
        # one request's beams: latency
        dict(name="beam 1x4", op="beam", batch=1, beams=4, keep=8, vocab=32001, dtype="bfloat16", finished=0.0, mix=9),
        # a batch of requests with twice the beams kept, some beams finished
        dict(name="beam 32x8", op="beam", batch=32, beams=8, keep=16, vocab=131072, dtype="float32", finished=0.1,
             mix=10),
        # one request's states of four layers
        dict(name="reorder 1x4", op="reorder", batch=1, beams=4, heads=96, layers=4, dtype="bfloat16", mix=11),
        # a full batch's states of one layer
        dict(name="reorder 32x8", op="reorder", batch=32, beams=8, heads=96, layers=1, dtype="float32", mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "beam", "reorder"])
    mix = rng.randrange(1 << 20)
    if op in ("append", "attn"):
        dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
        page = rng.choice([16, 32, 64, 128])
        kind = rng.choice(["decode", "short", "prompt", "ragged"])
        ragged = kind == "ragged"
        if kind == "decode":
            batch, tokens, context = _log_int(rng, 1, 256), 1, _log_int(rng, 64, 32768)
        elif kind == "short":
            batch, tokens, context = _log_int(rng, 1, 32), _log_int(rng, 2, 65), _log_int(rng, 64, 16384)
        elif kind == "prompt":
            batch = _log_int(rng, 1, 4)
            tokens, context = _log_int(rng, 100, 8192 // batch), rng.choice([0, 0, _log_int(rng, 1, 8192)])
        else:
            batch, tokens, context = _log_int(rng, 2, 40), _log_int(rng, 200, 8192), rng.choice([0, 1000])
        case = dict(op=op, batch=batch, tokens=tokens, context=context, heads=heads, kv_heads=kv_heads, dim=dim,
                    page=page, ragged=ragged, mix=mix)
        if op == "append":
            case.update(rotary=rng.choice([32, 64, dim]), interleaved=rng.random() < 0.4)
        else:
            case.update(window=_log_int(rng, 16, 8192), sinks=rng.choice([0, 4, _log_int(rng, 1, 130)]))
            most = max(_queries(case))

            def too_large():
                keys = min(case["window"] + most + case["sinks"], most + context)
                return batch * most * heads * keys > 2 ** 31 or batch * keys * kv_heads > 2 ** 21

            while too_large():
                case["window"] = max(16, case["window"] // 2)
                if case["window"] == 16:
                    case["tokens"] = case["tokens"] // 2 + 1
                    most = max(_queries(case))
        return case
    beams = rng.choice([2, 3, 4, 5, 8])
    if op == "beam":
        return dict(op=op, batch=_log_int(rng, 1, 32), beams=beams, keep=rng.choice([beams, 2 * beams]),
                    vocab=_log_int(rng, 1000, 131072), dtype=rng.choice(["bfloat16", "float32"]),
                    finished=rng.choice([0.0, 0.2]), mix=mix)
    return dict(op=op, batch=_log_int(rng, 1, 10), beams=beams, heads=_log_int(rng, 1, 96), layers=rng.choice([1, 2, 3]),
                dtype=rng.choice(["bfloat16", "float32"]), mix=mix)


# ---------------------------------------------------------------------------------------------- lengths of a case
def _queries(case):
    """New tokens of each sequence."""
    n, t = case["batch"], case["tokens"]
    if not case["ragged"]:
        return [t] * n
    r = random.Random(case["mix"])
    raw = [math.exp(r.uniform(math.log(16), math.log(2048))) for _ in range(n)]
    lens = [max(1, int(t * x / sum(raw))) for x in raw]
    lens[lens.index(max(lens))] += max(0, t - sum(lens))
    return lens


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    q = _queries(case)
    r = random.Random(case["mix"] + 1)
    c = case["context"]
    return q, [x + (c if case["batch"] == 1 else r.randint(c // 2, c)) for x in q]


def _pairs(q, total, window, sinks):
    """Visible (query, key) pairs of one sequence, and the keys that some query sees."""
    pos = range(total - q, total)
    pairs = 0
    for p in pos:
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, total - q - window + 1)
    return pairs, total - lo + min(sinks, lo)


def work(case):
    if case["op"] == "append":
        q, _ = _lengths(case)
        t, d = sum(q), case["dim"]
        rows = t * (case["heads"] + 2 * case["kv_heads"])
        table = (t if case["batch"] == 1 else min(t, max(_lengths(case)[1]))) * case["rotary"] * 4
        return {"bytes": 2 * rows * d * 2 + table, "flops": 3 * case["rotary"] * t * (case["heads"] + case["kv_heads"])}
    if case["op"] == "attn":
        q, total = _lengths(case)
        d = case["dim"]
        got = [_pairs(a, b, case["window"], case["sinks"]) for a, b in zip(q, total)]
        rows = sum(q) * case["heads"]
        return {"bytes": rows * (2 * d * 2 + 4) + sum(k for _, k in got) * case["kv_heads"] * d * 2 * 2,
                "flops": 4 * d * case["heads"] * sum(p for p, _ in got)}
    if case["op"] == "beam":
        rows, size = case["batch"] * case["beams"], 2 if case["dtype"] == "bfloat16" else 4
        n = rows * case["vocab"]
        return {"bytes": n * size + rows * 5 + case["batch"] * case["keep"] * 12, "flops": 4 * n}
    rows, w = case["batch"] * case["beams"], case["beams"]
    size = case["heads"] * 128 * 128 * (2 if case["dtype"] == "bfloat16" else 4) * case["layers"]
    distinct = w * (1 - (1 - 1 / w) ** w) / w       # expected share of rows that are somebody's parent
    return {"bytes": rows * size * (1 + distinct) + rows * 4, "flops": 0}


# ---------------------------------------------------------------------------------------------- inputs
def _pool(case, q, total, lowest, gen):
    """A pool of pages, shuffled among the sequences; pages before `lowest` and past the sinks are given back (-1)."""
    dev, page = _dev(), case["page"]
    most = max(-(-t // page) for t in total) + 1
    table = torch.full((len(q), most), -1, dtype=torch.int32)
    sink_pages = -(-case.get("sinks", 0) // page)
    need = []
    for n, t in enumerate(total):
        live = [i for i in range(-(-t // page)) if i < sink_pages or (i + 1) * page > lowest[n]]
        need += [(n, i) for i in live]
    order = torch.randperm(len(need) + 3, generator=torch.Generator().manual_seed(case["mix"]))
    at = torch.tensor(need, dtype=torch.long).reshape(-1, 2)
    table[at[:, 0], at[:, 1]] = order[:len(need)].to(torch.int32)
    shape = (len(need) + 3, case["kv_heads"], page, case["dim"])
    k = torch.randn(shape, device=dev, dtype=torch.bfloat16, generator=gen)
    v = torch.randn(shape, device=dev, dtype=torch.bfloat16, generator=gen)
    return k, v, table.to(dev)


def prepare(case, seed):
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, device=dev, dtype=dtype, generator=gen)

    if case["op"] in ("append", "attn"):
        q, total = _lengths(case)
        b, t = (1, sum(q)) if case["ragged"] else (len(q), case["tokens"])
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        if case["op"] == "append":
            lowest = [a - b_ for a, b_ in zip(total, q)]
        else:
            lowest = [max(0, a - b_ - case["window"] + 1) for a, b_ in zip(total, q)]
        k_cache, v_cache, table = _pool(case, q, total, lowest, gen)
        cu = None
        if case["ragged"]:
            cu = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int64, device=dev)
        state = dict(op=case["op"], k_cache=k_cache, v_cache=v_cache, table=table, cu=cu, most=max(q),
                     lens=torch.tensor(total, dtype=torch.int32, device=dev))
        if case["op"] == "append":
            # q, k and v lie side by side in the rows of one projection's output
            x = normal(b, t, (hq + 2 * hk) * d)
            state.update(q=x[..., :hq * d].unflatten(-1, (hq, d)), k=x[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d)),
                         v=x[..., (hq + hk) * d:].unflatten(-1, (hk, d)), interleaved=case["interleaved"])
            half = case["rotary"] // 2
            freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
            angle = torch.arange(max(total), dtype=torch.float64)[:, None] * freq
            state.update(cos=angle.cos().float().to(dev), sin=angle.sin().float().to(dev),
                         q_out=torch.empty((b, t, hq, d), device=dev, dtype=torch.bfloat16))
        else:
            state.update(q=normal(b, t, hq, d), window=case["window"], sinks=case["sinks"], scale=d ** -0.5)
            state.update(out=torch.empty_like(state["q"]), lse=torch.empty((b, t, hq), device=dev))
        return state
    if case["op"] == "beam":
        b, w, v = case["batch"], case["beams"], case["vocab"]
        logits = normal(b, w, v, dtype=torch.float32)
        # a language model's logits: a wide body and a few likely tokens
        logits = logits * 2.5 + torch.relu(normal(b, w, v, dtype=torch.float32) - 3.0) * 4.0
        scores = -20.0 * torch.rand((b, w), device=dev, generator=gen)
        done = torch.rand((b, w), device=dev, generator=gen) < case["finished"]
        k = case["keep"]
        return dict(op="beam", logits=logits.to(getattr(torch, case["dtype"])), beam_scores=scores,
                    finished=done.to(torch.uint8), eos=2, keep=k,
                    scores=torch.empty((b, k), device=dev), tokens=torch.empty((b, k), device=dev, dtype=torch.int32),
                    parents=torch.empty((b, k), device=dev, dtype=torch.int32))
    b, w = case["batch"], case["beams"]
    parents = torch.randint(0, w, (b, w), device=dev, generator=gen) + w * torch.arange(b, device=dev)[:, None]
    src = [normal(b * w, case["heads"], 128, 128, dtype=getattr(torch, case["dtype"])) for _ in range(case["layers"])]
    return dict(op="reorder", src=src, dst=[torch.empty_like(s) for s in src], beams=w,
                parents=parents.reshape(-1).to(torch.int32))


# ---------------------------------------------------------------------------------------------- plain forms
def _tokens(state, b, t):
    """Sequence and position of every token [b * t], and its index within the sequence."""
    dev, lens = state["lens"].device, state["lens"].long()
    if state["cu"] is None:
        seq = torch.arange(b, device=dev).repeat_interleave(t)
        at = torch.arange(t, device=dev).repeat(b)
        new = torch.full_like(lens, t)
    else:
        i = torch.arange(t, device=dev)
        seq = torch.searchsorted(state["cu"], i, right=True) - 1
        at = i - state["cu"][seq]
        new = state["cu"].diff()
    return seq, at, (lens - new)[seq] + at, new


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim] fp32, cos and sin [tokens, rotary / 2]."""
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _append(state):
    b, t = state["q"].shape[:2]
    seq, _, pos, _ = _tokens(state, b, t)
    cos, sin = state["cos"][pos], state["sin"][pos]
    page = state["k_cache"].shape[2]
    where = state["table"].long()[seq, pos // page]
    q = _rotate(state["q"].flatten(0, 1).float(), cos, sin, state["interleaved"])
    k = _rotate(state["k"].flatten(0, 1).float(), cos, sin, state["interleaved"])
    state["q_out"].copy_(q.unflatten(0, (b, t)))
    state["k_cache"][where, :, pos % page] = k.to(torch.bfloat16)
    state["v_cache"][where, :, pos % page] = state["v"].flatten(0, 1)
    return state["q_out"], state["k_cache"], state["v_cache"]


def _attn(state):
    q, table, lens = state["q"], state["table"].long(), state["lens"].long()
    b, t, hq, d = q.shape
    hk, page = state["k_cache"].shape[1:3]
    dev, n, most = q.device, table.shape[0], state["most"]
    window, sinks = state["window"], state["sinks"]
    seq, at, pos, new = _tokens(state, b, t)
    # queries [n, most, heads, dim], padded
    row = torch.zeros((n, most), dtype=torch.long, device=dev)
    row[seq, at] = torch.arange(b * t, device=dev)
    qs = q.flatten(0, 1)[row].float().unflatten(2, (hk, hq // hk))
    qpos = (lens - new)[:, None] + torch.arange(most, device=dev)
    # keys: the sinks, then everything from the first query's window on
    span = min(most + window - 1, table.shape[1] * page)
    first = torch.clamp(lens - span, min=0)
    j = torch.cat((torch.arange(sinks, device=dev).expand(n, sinks), first[:, None] + torch.arange(span, device=dev)), 1)
    live = j < lens[:, None]
    live[:, sinks:] &= j[:, sinks:] >= sinks
    pages = torch.gather(table, 1, torch.clamp(j // page, max=table.shape[1] - 1)).clamp(min=0)
    k = state["k_cache"][pages, :, j % page].float()
    v = state["v_cache"][pages, :, j % page].float()
    kp, qp = j[:, None, :], qpos[:, :, None]
    seen = live[:, None, :] & (kp <= qp) & ((kp > qp - window) | (kp < sinks))
    seen = seen[:, None, None]
    v = torch.where(live[:, :, None, None], v, torch.zeros((), device=dev))
    s = torch.einsum("nqhgd,njhd->nhgqj", qs, k).mul_(state["scale"])
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("nhgqj,njhd->nhgqd", p, v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)
    state["out"].copy_(o[seq, at].unflatten(0, (b, t)))
    state["lse"].copy_(lse[seq, at].unflatten(0, (b, t)))
    return state["out"], state["lse"]


def _beam(state):
    logits, scores, done = state["logits"].float(), state["beam_scores"], state["finished"].bool()
    b, w, v = logits.shape
    logits = torch.where(logits.isnan(), -math.inf, logits)
    m = logits.amax(-1)
    total = (logits - m[..., None]).exp().sum(-1)
    c = (scores - m) - total.log()
    cand = c[..., None] + logits
    eos = torch.arange(v, device=logits.device) == state["eos"]
    ended = torch.where(eos, scores[..., None], -math.inf)
    cand = torch.where(done[..., None], ended, cand)
    cand = torch.where(cand.isnan(), -math.inf, cand)
    best, at = torch.sort(cand.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :state["keep"]], at[:, :state["keep"]]
    state["scores"].copy_(best)
    state["tokens"].copy_(at % v)
    state["parents"].copy_(at // v + w * torch.arange(b, device=at.device)[:, None])
    return state["scores"], state["tokens"], state["parents"]


def _reorder(state):
    at = state["parents"].long()
    return [d.copy_(s[at]) for s, d in zip(state["src"], state["dst"])]


def run(state):
    op = state["op"]
    if not own:
        return {"append": _append, "attn": _attn, "beam": _beam, "reorder": _reorder}[op](state)
    import gated_delta_rule_23_gb300 as kda
    if op == "append":
        kda.kda_kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["table"], state["lens"],
                          cos=state["cos"], sin=state["sin"], interleaved=state["interleaved"], q=state["q"],
                          q_out=state["q_out"], cu_seqlens=state["cu"])
        return state["q_out"], state["k_cache"], state["v_cache"]
    if op == "attn":
        kda.kda_window_attn(state["q"], state["k_cache"], state["v_cache"], state["table"], state["lens"], state["out"],
                            window=state["window"], sinks=state["sinks"], scale=state["scale"], lse=state["lse"],
                            cu_seqlens=state["cu"])
        return state["out"], state["lse"]
    if op == "beam":
        kda.kda_beam_select(state["logits"], state["beam_scores"], state["scores"], state["tokens"], state["parents"],
                            finished=state["finished"], eos=state["eos"])
        return state["scores"], state["tokens"], state["parents"]
    kda.kda_state_reorder(state["src"], state["parents"], beams=state["beams"], dst=state["dst"])
    return state["dst"]


# ---------------------------------------------------------------------------------------------- 64-bit definitions
def _exact_append(case, state):
    q, total = _lengths(case)
    half, page = case["rotary"] // 2, case["page"]
    q_out = state["q"].double().clone()
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()
    table = state["table"].tolist()
    flat_q, flat_k, flat_v = q_out.flatten(0, 1), state["k"].double().flatten(0, 1), state["v"].double().flatten(0, 1)
    begin = 0
    for n, (new, length) in enumerate(zip(q, total)):
        pos = torch.arange(length - new, length, device=q_out.device)
        z = torch.complex(state["cos"][pos].double(), state["sin"][pos].double())[:, None]
        rows = slice(begin, begin + new)

        def turn(x):
            y = x.clone()
            r = x[..., :2 * half]
            pair = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
            out = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            y[..., :2 * half] = out.flatten(-2) if case["interleaved"] else out.transpose(-1, -2).flatten(-2)
            return y

        flat_q[rows] = turn(flat_q[rows])
        where = torch.tensor([table[n][p // page] for p in range(length - new, length)], device=q_out.device)
        k_cache[where, :, pos % page] = turn(flat_k[rows])
        v_cache[where, :, pos % page] = flat_v[rows]
        begin += new
    return q_out, k_cache, v_cache


def _exact_attn(case, state):
    q, total = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    window, sinks = case["window"], case["sinks"]
    if 4 * d * hq * sum(_pairs(a, b, window, sinks)[0] for a, b in zip(q, total)) > 4e12:
        return None
    dev = state["q"].device
    rows = state["q"].flatten(0, 1)
    out = torch.zeros(rows.shape, dtype=torch.float64, device=dev)
    lse = torch.full(rows.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    table = state["table"].long()
    begin = 0
    for n, (new, length) in enumerate(zip(q, total)):
        for lo in range(0, new, 512):
            hi = min(new, lo + 512)
            p = torch.arange(length - new + lo, length - new + hi, device=dev)
            left = max(sinks, length - new + lo - window + 1, 0)
            j = torch.cat((torch.arange(min(sinks, length), device=dev),
                           torch.arange(left, max(left, length - new + hi), device=dev)))
            at = table[n][j // page]
            k = state["k_cache"][at, :, j % page].double()        # [keys, kv heads, dim]
            v = state["v_cache"][at, :, j % page].double()
            x = rows[begin + lo:begin + hi].double().reshape(hi - lo, hk, hq // hk, d)
            s = torch.matmul(x.permute(1, 2, 0, 3), k.permute(1, 2, 0)[:, None]) * state["scale"]
            gap = p[:, None] - j[None]
            hidden = (gap < 0) | ((gap >= window) & (j >= sinks)[None])
            s = s.masked_fill(hidden, -math.inf)
            total_log = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(total_log.isinf(), 0.0, total_log)[..., None])
            o = torch.matmul(w, v.permute(1, 0, 2)[:, None])
            out[begin + lo:begin + hi] = o.permute(2, 0, 1, 3).reshape(hi - lo, hq, d)
            lse[begin + lo:begin + hi] = total_log.permute(2, 0, 1).reshape(hi - lo, hq)
        begin += new
    return out.reshape(state["q"].shape), lse.reshape(state["q"].shape[:3])


def _exact_beam(case, state):
    b, w, v = state["logits"].shape
    best = []
    for i in range(b):
        x = torch.log_softmax(state["logits"][i].double(), -1) + state["beam_scores"][i].double()[:, None]
        done = state["finished"][i].bool()
        x[done] = -math.inf
        x[done, state["eos"]] = state["beam_scores"][i].double()[done]
        best.append(torch.topk(x.flatten(), state["keep"]).values)
    return torch.stack(best), None, None


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, state)
    if case["op"] == "attn":
        return _exact_attn(case, state)
    if case["op"] == "beam":
        return _exact_beam(case, state)
    parents = state["parents"].tolist()
    return [torch.stack([s[p].double() for p in parents]) for s in state["src"]]
