"""Workloads of linear attention with a decay for each head (prompts, ragged batches, single tokens, speculative runs) and of
the verification of drafted tokens.

Each workload runs in two forms on the same inputs: the operator in elementary torch operations in 32 bits, with decays,
probabilities and what lies next to a border in 64 (``own = False``), or the library's entry points (``own = True``).
``exact`` restates the definitions in 64 bits.
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
        # one user's decode step: pure latency
        dict(name="linear decode 1", op="linear", batch=1, tokens=1, heads=32, kv_heads=32, dim=128, decay="head",
             state="float32", ragged="", mix=1),
        # a full decode batch with fp32 states: the states' bytes
        dict(name="linear decode 256", op="linear", batch=256, tokens=1, heads=96, kv_heads=96, dim=128, decay="token",
             state="float32", ragged="", mix=2),
        # a speculative run of which each sequence keeps the tokens that were accepted, bf16 states, shared keys
        dict(name="linear run 64x5", op="linear", batch=64, tokens=5, heads=64, kv_heads=8, dim=128, decay="both",
             state="bfloat16", ragged="lens", mix=3),
        # a long prompt with fixed decays
        dict(name="linear prompt 8192", op="linear", batch=1, tokens=8192, heads=96, kv_heads=96, dim=128, decay="head",
             state="float32", ragged="", mix=4),
        # a long prompt with a gate for each token, bf16 states, shared keys
        dict(name="linear prompt 8192 gated", op="linear", batch=1, tokens=8192, heads=64, kv_heads=8, dim=128,
             decay="token", state="bfloat16", ragged="", mix=5),
        # prompts of irregular lengths prefilled together
        dict(name="linear ragged 8192", op="linear", batch=12, tokens=8192, heads=96, kv_heads=96, dim=128,
             decay="token", state="float32", ragged="cu", mix=6),
        # a very long prompt on few heads: parallel along the tokens or not at all
        dict(name="linear long 32768", op="linear", batch=1, tokens=32768, heads=8, kv_heads=8, dim=128, decay="both",
             state="float32", ragged="", mix=7),
        # the next piece of two prompts, odd sizes, the small head
        dict(name="linear chunk 509", op="linear", batch=2, tokens=509, heads=14, kv_heads=2, dim=64, decay="head",
             state="bfloat16", ragged="", mix=8),
        # one request's drafts: latency
        dict(name="verify 1x4", op="verify", batch=1, drafts=4, vocab=32001, dtype="bfloat16", probs=True, greedy=0.0,
             ragged=False, mix=9),
        # a batch of requests with a draft model's probabilities, some requests greedy
        dict(name="verify 64x4", op="verify", batch=64, drafts=4, vocab=131072, dtype="float32", probs=True, greedy=0.1,
             ragged=False, mix=10),
        # drafts that were looked up in the text (no probabilities), irregular counts, odd vocabulary
        dict(name="verify 128x3 looked up", op="verify", batch=128, drafts=3, vocab=50257, dtype="bfloat16", probs=False,
             greedy=0.3, ragged=True, mix=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    mix = rng.randrange(1 << 20)
    if rng.random() < 0.3:
        return dict(op="verify", batch=_log_int(rng, 1, 128), drafts=rng.choice([1, 2, 3, 4, 5, 7]) if rng.random() < 0.8 else 11,
                    vocab=_log_int(rng, 1000, 65536), dtype=rng.choice(["bfloat16", "float32"]), probs=rng.random() < 0.6,
                    greedy=rng.choice([0.0, 0.2]), ragged=rng.random() < 0.3, mix=mix)
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 6])
    kind = rng.choice(["decode", "run", "prompt", "prompt", "ragged", "ragged"])
    if kind == "decode":
        batch, tokens, ragged = _log_int(rng, 1, 256), 1, ""
    elif kind == "run":
        batch, tokens, ragged = _log_int(rng, 1, 64), _log_int(rng, 2, 40), rng.choice(["", "lens"])
    elif kind == "prompt":
        batch = _log_int(rng, 1, 6)
        tokens, ragged = _log_int(rng, 41, 8192 // batch), rng.choice(["", "", "lens"])
    else:
        batch, tokens, ragged = _log_int(rng, 2, 40), _log_int(rng, 200, 8192), "cu"
    return dict(op="linear", batch=batch, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                decay=rng.choice(["head", "token", "both"]), state=rng.choice(["bfloat16", "float32"]), ragged=ragged, mix=mix)


# ---------------------------------------------------------------------------------------------- lengths and work
def _lengths(case):
    """Tokens of each sequence."""
    n, t = case["batch"], case["tokens"]
    r = random.Random(case["mix"])
    if case["ragged"] == "lens":
        return [r.randint(1, t) for _ in range(n)]
    if case["ragged"] != "cu":
        return [t] * n
    raw = [math.exp(r.uniform(math.log(16), math.log(2048))) for _ in range(n)]
    lens = [max(1, int(t * x / sum(raw))) for x in raw]
    lens[lens.index(max(lens))] += max(0, t - sum(lens))
    return lens


def _draft_lens(case):
    if not case["ragged"]:
        return [case["drafts"]] * case["batch"]
    r = random.Random(case["mix"])
    return [r.randint(0, case["drafts"]) for _ in range(case["batch"])]


def work(case):
    if case["op"] == "verify":
        size = 2 if case["dtype"] == "bfloat16" else 4
        # the rows up to a request's last draft, one row of the noise, and one of the draft's probabilities
        rows = sum(n + 1 for n in _draft_lens(case))
        b, v = case["batch"], case["vocab"]
        return {"bytes": rows * v * size + b * v * 4 * (2 if case["probs"] else 1), "flops": 4 * rows * v}
    tokens, h, hk, d = sum(_lengths(case)), case["heads"], case["kv_heads"], case["dim"]
    states = 2 * case["batch"] * h * d * d * (2 if case["state"] == "bfloat16" else 4)
    gates = tokens * h * 4 if case["decay"] != "head" else 0
    # token by token: the decay, the outer product and the read-out
    return {"bytes": tokens * (2 * h + 2 * hk) * d * 2 + gates + states, "flops": 5 * tokens * h * d * d}


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, device=dev, dtype=dtype, generator=gen)

    if case["op"] == "verify":
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        # a language model's logits: a wide body and a few likely tokens; the draft model's are these with an error
        logits = normal(b, k + 1, v, dtype=torch.float32)
        logits = logits * 2.5 + torch.relu(normal(b, k + 1, v, dtype=torch.float32) - 3.0) * 6.0
        guess = torch.softmax(logits[:, :k] + 0.7 * normal(b, k, v, dtype=torch.float32), -1)
        drafts = (guess / torch.rand((b, k, v), device=dev, generator=gen).log_().neg_().clamp_(min=1e-20)).argmax(-1)
        if not case["probs"]:
            # looked-up drafts are mostly the target's own favourites
            drafts = torch.where(torch.rand((b, k), device=dev, generator=gen) < 0.6, logits[:, :k].argmax(-1), drafts)
        temperature = 0.6 + 0.6 * torch.rand((b,), device=dev, generator=gen)
        temperature[torch.rand((b,), device=dev, generator=gen) < case["greedy"]] = 0.0
        noise = torch.rand((b, v), device=dev, generator=gen, dtype=torch.float64)
        return dict(op="verify", logits=logits.to(getattr(torch, case["dtype"])), drafts=drafts.to(torch.int32),
                    probs=guess if case["probs"] else None, uniform=torch.rand((b, k), device=dev, generator=gen),
                    noise=noise.log_().neg_().float().clamp_(min=1e-20), temperature=temperature,
                    draft_lens=torch.tensor(_draft_lens(case), dtype=torch.int32, device=dev) if case["ragged"] else None,
                    tokens=torch.empty((b, k + 1), device=dev, dtype=torch.int32),
                    counts=torch.empty((b,), device=dev, dtype=torch.int32))
    lens = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    n = case["batch"]
    b, t = (1, sum(lens)) if case["ragged"] == "cu" else (n, case["tokens"])
    # q, k and v lie side by side in the rows of one projection's output
    x = normal(b, t, (h + 2 * hk) * d)
    state = dict(op="linear", most=max(lens), lens=None, cu=None, gate=None, log_decay=None, scale=d ** -0.5,
                 q=x[..., :h * d].unflatten(-1, (h, d)), k=x[..., h * d:(h + hk) * d].unflatten(-1, (hk, d)),
                 v=x[..., (h + hk) * d:].unflatten(-1, (hk, d)))
    if case["ragged"] == "cu":
        state["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int64, device=dev)
    if case["ragged"] == "lens":
        state["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["decay"] != "token":
        # from a state of a few tokens to one of hundreds
        state["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, h + 1, device=dev, dtype=torch.float32) / h)
    if case["decay"] != "head":
        state["gate"] = -0.2 * torch.nn.functional.softplus(2.0 * normal(b, t, h, dtype=torch.float32) - 2.0)
    kind = getattr(torch, case["state"])
    state["initial"] = (4.0 * normal(n, h, d, d, dtype=torch.float32)).to(kind)
    state["final"] = torch.empty_like(state["initial"])
    state["out"] = torch.zeros((b, t, h, d), device=dev, dtype=torch.bfloat16)
    return state


# ---------------------------------------------------------------------------------------------- plain forms
CHUNK = 64


def _places(state):
    """Padded places [n, length] of every sequence's tokens in the batch's rows, and whether there is one."""
    dev, n = state["q"].device, state["initial"].shape[0]
    b, t = state["q"].shape[:2]
    at = torch.arange(state["most"], device=dev)
    if state["cu"] is not None:
        first, count = state["cu"][:-1], state["cu"].diff()
    else:
        first = t * torch.arange(n, device=dev)
        count = state["lens"].long() if state["lens"] is not None else torch.full((n,), t, device=dev)
    live = at < count[:, None]
    return torch.where(live, first[:, None] + at, 0), live


def _log_decays(state, row, live):
    """The logarithms [n, length, heads] in 64 bits, 0 where there is no token."""
    h = state["q"].shape[2]
    a = torch.zeros((*row.shape, h), dtype=torch.float64, device=row.device)
    if state["log_decay"] is not None:
        a = a + state["log_decay"].double()
    if state["gate"] is not None:
        a = a + state["gate"].flatten(0, 1)[row].double()
    return torch.where(live[..., None], a, 0.0)


def _linear(state):
    h, d = state["q"].shape[2:]
    hk = state["k"].shape[2]
    row, live = _places(state)
    n, length = row.shape
    pad = -length % CHUNK if length > 1 else 0
    row, live = (torch.nn.functional.pad(x, (0, pad)) for x in (row, live))
    c = min(CHUNK, row.shape[1])

    def chunks(x):
        """[n, chunks, heads, c, ...]"""
        return x.unflatten(1, (-1, c)).transpose(2, 3)

    q = chunks(state["q"].flatten(0, 1)[row].float())
    k = chunks(torch.where(live[..., None, None], state["k"].flatten(0, 1)[row].float(), 0.0).repeat_interleave(h // hk, 2))
    v = chunks(torch.where(live[..., None, None], state["v"].flatten(0, 1)[row].float(), 0.0).repeat_interleave(h // hk, 2))
    a = chunks(_log_decays(state, row, live)).cumsum(-1)                # [n, chunks, heads, c], 64 bits
    gap = a[..., :, None] - a[..., None, :]
    below = torch.ones((c, c), dtype=torch.bool, device=row.device).tril()
    inside = torch.where(below, gap.clamp(max=0.0).exp().float(), 0.0)
    # a chunk's own state, and the decay from the end of one chunk to the start of another
    tail = (a[..., -1:] - a).exp().float()
    added = torch.matmul(v.transpose(-1, -2), k * tail[..., None])      # [n, chunks, heads, d (v), d (k)]
    total = a[..., -1].cumsum(1)                                         # after each chunk
    before = torch.cat((torch.zeros_like(total[:, :1]), total), 1)       # [n, chunks + 1, heads]
    m = total.shape[1]
    span = (before[:, :, None] - before[:, None, 1:]).permute(0, 3, 1, 2)
    earlier = torch.ones((m + 1, m), dtype=torch.bool, device=row.device).tril(-1)
    carry = torch.where(earlier, span.clamp(max=0.0).exp().float(), 0.0)  # [n, heads, m + 1, m]
    flat = added.permute(0, 2, 1, 3, 4).flatten(3)                        # [n, heads, m, d * d]
    states = torch.matmul(carry, flat)
    states += before.permute(0, 2, 1)[..., None].exp().float() * state["initial"].float().flatten(2)[:, :, None]
    states = states.unflatten(-1, (d, d))                                 # [n, heads, m + 1, d, d]
    state["final"].copy_(states[:, :, -1])
    s = torch.matmul(q, k.transpose(-1, -2)) * inside
    o = torch.matmul(s, v)
    o += a.exp().float()[..., None] * torch.matmul(q, states[:, :, :-1].transpose(1, 2).transpose(-1, -2))
    o = (o * state["scale"]).transpose(2, 3).flatten(1, 2)
    out = state["out"].flatten(0, 1)
    out[row[live]] = o[live].to(torch.bfloat16)
    return state["out"], state["final"]


def _verify(state):
    logits, drafts, probs = state["logits"].double(), state["drafts"].long(), state["probs"]
    b, rows, v = logits.shape
    k, dev = rows - 1, logits.device
    at, each = torch.arange(v, device=dev), torch.arange(b, device=dev)
    length = state["draft_lens"].long() if state["draft_lens"] is not None else torch.full((b,), k, device=dev)
    tau = state["temperature"].double()[:, None]
    greedy = tau == 0
    logits = torch.where(logits.isnan(), -math.inf, logits)
    top = logits.amax(-1)
    weight = ((logits - top[..., None]) / torch.where(greedy, 1.0, tau)[..., None]).exp()
    z = weight.sum(-1)
    there = drafts[..., None]
    p = weight[:, :k].gather(-1, there).squeeze(-1) / z[:, :k]
    q = probs.gather(-1, there).squeeze(-1).double() if probs is not None else torch.ones_like(p)
    ok = torch.where(greedy, logits[:, :k].gather(-1, there).squeeze(-1) == top[:, :k], state["uniform"].double() * q < p)
    ok &= torch.arange(k, device=dev) < length[:, None]
    good = ok.long().cumprod(-1).sum(-1)                                   # drafts taken
    here = weight[each, good] / z[each, good][:, None]
    cut = torch.zeros_like(here)
    if k:
        r = good.clamp(max=k - 1)
        cut = probs[each, r].double() if probs is not None else (at == drafts[each, r][:, None]) * here
    left = torch.where((good < length)[:, None], (here - cut).clamp(min=0.0), here)
    left = torch.where(left.amax(-1, keepdim=True) > 0, left, here)
    race = torch.where(left > 0, left / state["noise"].double(), 0.0)
    race = torch.where(greedy, torch.where(logits[each, good] == top[each, good][:, None], 1.0, 0.0), race)
    token = torch.where(race == race.amax(-1, keepdim=True), at, v).amin(-1)
    place = torch.arange(k + 1, device=dev)
    taken = torch.nn.functional.pad(drafts, (0, 1))
    taken = torch.where(place < good[:, None], taken, torch.where(place == good[:, None], token[:, None], -1))
    state["tokens"].copy_(taken)
    state["counts"].copy_(good + 1)
    return state["tokens"], state["counts"]


def run(state):
    if not own:
        return _linear(state) if state["op"] == "linear" else _verify(state)
    import gated_delta_rule_23_gb300 as kda
    if state["op"] == "linear":
        kda.kda_linear_attn(state["q"], state["k"], state["v"], state["out"], log_decay=state["log_decay"],
                            gate=state["gate"], scale=state["scale"], initial_state=state["initial"],
                            final_state=state["final"], lens=state["lens"], cu_seqlens=state["cu"])
        return state["out"], state["final"]
    kda.kda_verify_drafts(state["logits"], state["drafts"], state["uniform"], state["noise"], state["tokens"],
                          state["counts"], draft_probs=state["probs"], temperature=state["temperature"],
                          draft_lens=state["draft_lens"])
    return state["tokens"], state["counts"]


# ---------------------------------------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    if case["op"] == "verify":
        return None                                                        # whole numbers
    state = prepare(case, seed)
    lens = _lengths(case)
    h, d = case["heads"], case["dim"]
    share = h // case["kv_heads"]
    dev = state["q"].device
    first = [sum(lens[:i]) for i in range(len(lens))] if case["ragged"] == "cu" else [i * case["tokens"] for i in range(len(lens))]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])              # the longest first: those left are the first ones
    q, k, v = (state[x].flatten(0, 1) for x in "qkv")
    s = state["initial"].double()[order]
    out = state["out"].double().flatten(0, 1)
    a = torch.zeros((q.shape[0], h), dtype=torch.float64, device=dev)
    if state["log_decay"] is not None:
        a += state["log_decay"].double()
    if state["gate"] is not None:
        a += state["gate"].double().flatten(0, 1)
    start = torch.tensor([first[i] for i in order], device=dev)
    for t in range(max(lens)):
        m = sum(x > t for x in lens)
        at = start[:m] + t
        kt, vt = (x[at].double().repeat_interleave(share, 1) for x in (k, v))
        live = s[:m]
        live.mul_(a[at].exp()[..., None, None])
        live.addcmul_(vt[..., :, None], kt[..., None, :])
        out[at] = torch.matmul(live, q[at].double()[..., None]).squeeze(-1) * state["scale"]
    final = torch.empty_like(s)
    final[order] = s
    return out.view(state["out"].shape), final
