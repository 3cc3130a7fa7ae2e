"""Operators of prompt processing and scoring over the paged cache: their cases, their plain forms and the
calls a program makes of them.

A chunk of new tokens (a prompt's segment, a chat turn, drafted tokens to be checked) goes through an
attention layer of a hybrid stack and ends in logits:

    rope     queries and keys are rotated by their positions (or back: the gradient)
    place    the same, with the keys and values going straight into the cache's pages
    chunk    every new token attends to what the pages hold up to itself (optionally only a window of last
             tokens and the first few)
    score    log-probabilities of the tokens that follow, with entropy and the best alternatives
    grad     the gradient of those with respect to the logits

Layouts: pages [n_pages, H_kv, page_size, d]; page_table int32 [N, P], -1 for no page; new tokens packed
[T, H, d] with cu_seqlens int32 [N + 1]; logits [R, V].
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # drafted tokens of a serving batch, checked in one pass over contexts of 1K to 16K tokens
        dict(name="chunk_draft_tokens", op="chunk", dtype=BF16, n=16, hq=32, hkv=8, d=128, page=64, new_lo=5, new_hi=5,
             past_lo=1000, past_hi=16379, window=0, sinks=0),
        # prompts and follow-up turns of different lengths in one batch
        dict(name="chunk_batch", op="chunk", dtype=BF16, n=8, hq=32, hkv=8, d=128, page=64, new_lo=48, new_hi=2048,
             past_lo=1, past_hi=8000, window=0, sinks=0),
        # the last 8192 tokens of a 32K prompt
        dict(name="chunk_long_prompt", op="chunk", dtype=BF16, n=1, hq=32, hkv=8, d=128, page=64, new_lo=8192,
             new_hi=8192, past_lo=24576, past_hi=24576, window=0, sinks=0),
        # sliding-window layers of long streams in fp32
        dict(name="chunk_window_sinks_f32", op="chunk", dtype=F32, n=6, hq=20, hkv=4, d=64, page=32, new_lo=100,
             new_hi=2500, past_lo=300, past_hi=20000, window=1024, sinks=4),
        # one decode step of an interactive session (latency)
        dict(name="place_one_token", op="place", dtype=BF16, n=1, hq=32, hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             past_lo=4000, past_hi=4000, rotary=128, layout="half", scaling="none"),
        # prompt segments of 1K to 16K tokens with positions scaled for a long context
        dict(name="place_segments", op="place", dtype=BF16, n=8, hq=32, hkv=8, d=128, page=64, new_lo=1024,
             new_hi=16384, past_lo=10, past_hi=120000, rotary=128, layout="half", scaling="smooth"),
        # gradients of a short fp32 batch: rotated back, interleaved pairs, part of the head
        dict(name="rope_back_f32", op="rope", dtype=F32, t=257, hq=16, hkv=16, d=64, rotary=40, layout="interleaved",
             scaling="linear", inverse=True),
        # a training batch
        dict(name="rope_training", op="rope", dtype=BF16, t=65536, hq=32, hkv=32, d=128, rotary=128, layout="half",
             scaling="none", inverse=False),
        # one sequence's drafted tokens: their log-probabilities and alternatives (latency)
        dict(name="score_draft_tokens", op="score", dtype=F32, rows=5, v=32000, top=5, entropy=True, ignored=0.0),
        # a prompt's tokens under a large vocabulary
        dict(name="score_prompt", op="score", dtype=BF16, rows=4096, v=131072, top=4, entropy=True, ignored=0.1),
        # a small fp32 training step with an entropy bonus; a vocabulary whose rows are not aligned
        dict(name="grad_entropy_f32", op="grad", dtype=F32, rows=96, v=32003, entropy=True, ignored=0.1),
        # a training batch under a large vocabulary
        dict(name="grad_batch", op="grad", dtype=BF16, rows=4096, v=131072, entropy=False, ignored=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "place", "rope", "score", "grad"])
    dtype = rng.choice([BF16, BF16, F32])
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(hq=hkv * rng.choice([1, 2, 4, 5, 7, 8]), hkv=hkv, d=rng.choice([64, 128, 256]))
    if op == "chunk":
        c = dict(op=op, dtype=dtype, n=_log_int(rng, 1, 64), **heads, page=rng.choice([16, 32, 48, 64, 128, 256]),
                 new_lo=1, new_hi=_log_int(rng, 1, 8192), past_lo=1, past_hi=_log_int(rng, 1, 65536),
                 window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), sinks=0)
        if c["window"]:
            c["sinks"] = rng.choice([0, 1, 4, 21, 64])
        c["new_lo"] = max(1, c["new_hi"] // rng.choice([1, 3, 40]))
        c["past_lo"] = max(1, c["past_hi"] // rng.choice([1, 3, 20]))
        # (an fp32 product runs at a sixteenth of the rate or less)
        most = 4e11 if dtype == F32 else 3e12
        while (work(c)["flops"] > most or c["n"] * c["new_hi"] * (c["new_hi"] + c["past_hi"]) * c["hq"] // hkv > 1e9
               or c["n"] * (c["new_hi"] + c["past_hi"]) * c["hkv"] * c["d"] > 3e8):
            c["new_hi"], c["past_hi"] = max(1, c["new_hi"] // 2), max(1, c["past_hi"] // 2)
            c["new_lo"], c["past_lo"] = min(c["new_lo"], c["new_hi"]), min(c["past_lo"], c["past_hi"])
        return c
    turn = dict(rotary=heads["d"], layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "smooth"]))
    if rng.random() < 0.4:
        turn["rotary"] = 2 * rng.randint(1, heads["d"] // 2)
    if op == "place":
        c = dict(op=op, dtype=dtype, n=_log_int(rng, 1, 64), **heads, page=rng.choice([16, 32, 48, 64, 128]), new_lo=1,
                 new_hi=_log_int(rng, 1, 16384), past_lo=1, past_hi=_log_int(rng, 1, 20000), **turn)
        while work(c)["bytes"] > 8e8 or c["n"] * (c["new_hi"] + c["past_hi"]) * c["hkv"] * c["d"] > 4e8:
            c["new_hi"], c["past_hi"] = max(1, c["new_hi"] // 2), max(1, c["past_hi"] // 2)
        return c
    if op == "rope":
        c = dict(op=op, dtype=dtype, t=_log_int(rng, 1, 65536), **heads, **turn, inverse=rng.random() < 0.5)
        while work(c)["bytes"] > 2e9:
            c["t"] //= 2
        return c
    c = dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 8192), v=_log_int(rng, 500, 151000),
             entropy=rng.random() < 0.5, ignored=rng.choice([0.0, 0.1]))
    while c["rows"] * c["v"] > 5e8:
        c["rows"] = max(1, c["rows"] // 2)
    if op == "score":
        c["top"] = rng.choice([0, 1, 2, 5, 10, 20])
    return c


def _spread(n, lo, hi, at=0.37):
    """n lengths between lo and hi, the same for every seed, spread evenly over their logarithm."""
    return [int(round(lo * (hi / lo) ** ((at + 0.6180339887498949 * i) % 1.0))) for i in range(n)]


def _lengths(c):
    """New and earlier tokens of each sequence."""
    return _spread(c["n"], c["new_lo"], c["new_hi"]), _spread(c["n"], c["past_lo"], c["past_hi"], 0.81)


def _sum_to(a, b, cap):
    """sum of min(t, cap) for t = a + 1 .. b"""
    low = max(a, min(b, cap))
    return (low * (low + 1) - a * (a + 1)) // 2 + (b - low) * cap


def work(c):
    es = 2 if c["dtype"] == BF16 else 4
    if c["op"] == "chunk":
        pairs = keys = new = 0
        for m, past in zip(*_lengths(c)):
            total = past + m
            new += m
            if not c["window"]:
                pairs += _sum_to(past, total, total)
                keys += total
            else:  # the last `window` tokens, and what they leave of the sinks
                pairs += _sum_to(past, total, c["window"])
                pairs += sum(min(c["sinks"], max(0, t - c["window"])) for t in range(past + 1, total + 1))
                near = max(0, past + 1 - c["window"])
                keys += total - near + min(c["sinks"], near)
        # queries, outputs and log-sums, and each visible key and value
        return {"bytes": new * c["hq"] * (2 * c["d"] * es + 4) + 2 * keys * c["hkv"] * c["d"] * es,
                "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] == "place":  # queries, keys and values, read and written
        t, rows = sum(_lengths(c)[0]), c["hq"] + c["hkv"]
        return {"bytes": 2 * t * (rows + c["hkv"]) * c["d"] * es, "flops": 3 * t * rows * c["rotary"]}
    if c["op"] == "rope":
        rows = c["t"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * rows * c["d"] * es + 4 * c["t"], "flops": 3 * rows * c["rotary"]}
    if c["op"] == "score":
        return {"bytes": c["rows"] * (c["v"] * es + 12 + 4 * c["entropy"] + 8 * c["top"]),
                "flops": c["rows"] * c["v"] * (6 if c["entropy"] else 4)}
    return {"bytes": c["rows"] * (2 * c["v"] * es + 12 + 8 * c["entropy"]),
            "flops": c["rows"] * c["v"] * (7 if c["entropy"] else 4)}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Radians per token of each pair (64 bits), and the factor of the rotated channels."""
    r = c["rotary"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    amplitude = 1.0
    if c["scaling"] == "linear":
        f = f / 4.0
    elif c["scaling"] == "smooth":  # slow pairs by the factor, fast ones as they are, those between by parts
        keep = ((8192 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 16.0)
        amplitude = 0.1 * math.log(16.0) + 1.0
    return f.cuda(), amplitude


def _entropy_of(x, lse):
    return lse - (torch.exp(x - lse[:, None]) * x).sum(1)


def prepare(c, seed):
    dev, dt = "cuda", getattr(torch, c["dtype"])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=dt, scale=1.0):
        x = torch.randn(shape, generator=g, device=dev, dtype=dtype)
        return x if scale == 1.0 else x * scale

    # scratch that a serving program keeps for its calls
    s = {"case": dict(c), "workspace": torch.empty(256 << 20, dtype=torch.uint8, device=dev)}
    if c["op"] in ("chunk", "place"):
        new, past = _lengths(c)
        total = [a + b for a, b in zip(new, past)]
        n, page, t = c["n"], c["page"], sum(new)
        width = -(-max(total) // page)
        col = torch.arange(width, device=dev)[None, :]
        begin, end = _i32(past)[:, None], _i32(total)[:, None]
        used = col * page < end
        if c.get("window"):  # pages that hold only tokens behind every window are given back
            used &= ((col + 1) * page > begin + 1 - c["window"]) | (col * page < c["sinks"])
        pages = sum(-(-x // page) for x in total) + 3
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["table"] = torch.where(used, ids[(torch.cumsum(used.flatten(), 0) - 1).clamp(min=0)].view(n, width),
                                 torch.full_like(ids[:1], -1))
        s["k_pages"], s["v_pages"] = normal(pages, c["hkv"], page, c["d"]), normal(pages, c["hkv"], page, c["d"])
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        s["cu"], s["start"], s["lengths"] = _i32(cu), _i32(past), _i32(total)
        s["longest"], s["most"] = max(total), max(new)  # tokens of a sequence, new ones of a sequence
        s["q"] = normal(t, c["hq"], c["d"], scale=2.0 if c["op"] == "chunk" else 1.0)
        if c["op"] == "place":
            s["k"], s["v"] = normal(t, c["hkv"], c["d"]), normal(t, c["hkv"], c["d"])
            s["freqs"], s["amplitude"] = _frequencies(c)
    elif c["op"] == "rope":
        s["q"], s["k"] = normal(c["t"], c["hq"], c["d"]), normal(c["t"], c["hkv"], c["d"])
        s["positions"] = (torch.arange(c["t"], device=dev) % 8192 + torch.randint(
            0, 100000, (1,), generator=g, device=dev)).to(torch.int32)
        s["freqs"], s["amplitude"] = _frequencies(c)
    else:
        rows, v = c["rows"], c["v"]
        s["logits"] = normal(rows, v, scale=3.0)
        tokens = torch.randint(0, v, (rows,), generator=g, device=dev)
        skip = torch.rand(rows, generator=g, device=dev) < c["ignored"]  # padding: no token to score
        s["tokens"] = torch.where(skip, torch.full_like(tokens, -1), tokens).to(torch.int32)
        if c["op"] == "grad":
            x = s["logits"].double()
            lse = torch.logsumexp(x, 1)
            s["lse"] = lse.float()
            s["d_logprobs"] = normal(rows, dtype=torch.float32)
            s["entropy"] = s["d_entropy"] = None
            if c["entropy"]:
                s["entropy"], s["d_entropy"] = _entropy_of(x, lse).float(), normal(rows, dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _plain_rotate(x, positions, freqs, layout, amplitude, inverse=False):
    a = positions.double()[:, None] * freqs
    cos, sin = (torch.cos(a) * amplitude).float()[:, None], (torch.sin(a) * amplitude).float()[:, None]
    if inverse:
        sin = -sin
    r, y = 2 * freqs.numel(), x.float()
    if layout == "half":
        lo, hi = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], 2)
    else:
        lo, hi = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([lo * cos - hi * sin, lo * sin + hi * cos], 3).flatten(2)
    return torch.cat([turned, y[..., r:]], 2).to(x.dtype)


def _plain_place(s):
    c, page = s["case"], s["case"]["page"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    at = s["start"].long()[seq] + t - s["cu"].long()[seq]
    q = _plain_rotate(s["q"], at, s["freqs"], c["layout"], s["amplitude"])
    ids, slot = s["table"][seq, at // page].long(), at % page
    s["k_pages"][ids, :, slot] = _plain_rotate(s["k"], at, s["freqs"], c["layout"], s["amplitude"])
    s["v_pages"][ids, :, slot] = s["v"]
    return q


def _plain_chunk(q, k_pages, v_pages, table, lengths, cu, most, window, sinks):
    hkv, page, d = k_pages.shape[1:]
    n, width = table.shape
    t, hq = q.shape[:2]
    group = hq // hkv
    lengths, cu = lengths.long(), cu.long()
    new = cu[1:] - cu[:-1]
    seq = torch.searchsorted(cu[1:], torch.arange(t, device=q.device), right=True)
    row = torch.arange(t, device=q.device) - cu[seq]
    at = (lengths - new)[:, None] + torch.arange(most, device=q.device)  # positions of the padded queries
    pos = torch.arange(width * page, device=q.device)
    seen = (pos <= at[..., None]) & (table >= 0).repeat_interleave(page, 1)[:, None]
    if window:
        seen &= (pos > at[..., None] - window) | (pos < sinks)
    ids = table.clamp(min=0).long()
    none = torch.full((1,), -math.inf, device=q.device)
    out, lse = torch.empty_like(q), torch.empty(t, hq, device=q.device)
    for h in range(hkv):  # one key head at a time: the scores of all of them take too much memory
        key, val = (x[:, h][ids].view(n, width * page, d).float() for x in (k_pages, v_pages))
        mine = slice(h * group, (h + 1) * group)
        rows = torch.zeros(n, most, group, d, device=q.device)
        rows[seq, row] = q[:, mine].float()
        x = torch.matmul(rows.view(n, most * group, d), key.transpose(1, 2)) / math.sqrt(d)
        x = torch.where(seen[:, :, None], x.view(n, most, group, -1), none).view(n, most * group, -1)
        top = x.amax(2, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        e = x.sub_(top).exp_()
        total = e.sum(2, keepdim=True)
        o = torch.matmul(e, val) / torch.where(total > 0, total, torch.ones_like(total))
        out[:, mine] = o.view(n, most, group, d)[seq, row].to(q.dtype)
        lse[:, mine] = (torch.log(total) + top).view(n, most, group)[seq, row]
    return out, lse


def _plain_score(logits, tokens, top, entropy):
    x = logits.float()
    v = x.shape[1]
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1, dtype=torch.float64)
    lse = torch.log(total) + most[:, 0]
    valid = (tokens >= 0) & (tokens < v)
    given = x.gather(1, tokens.clamp(0, v - 1).long()[:, None])[:, 0]
    logprobs = torch.where(valid, given - lse, torch.zeros_like(lse)).float()
    spread = best = which = None
    if entropy:
        spread = (torch.log(total) - (e * (x - most)).sum(1, dtype=torch.float64) / total).float()
    if top:
        col = torch.arange(v, device=x.device)
        bits = (x + 0.0).view(torch.int32).long()
        order = (torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) << 32) + (0xFFFFFFFF - col)  # ties: the lowest token
        which = 0xFFFFFFFF - (torch.topk(order, top, dim=1).values & 0xFFFFFFFF)
        best = (x.gather(1, which) - lse[:, None]).float()
        which = which.to(torch.int32)
    return logprobs, lse.float(), spread, best, which


def _plain_grad(s):
    x, v = s["logits"].float(), s["logits"].shape[1]
    lp = x - s["lse"][:, None]
    tokens = s["tokens"]
    valid = (tokens >= 0) & (tokens < v)
    d = torch.where(valid, s["d_logprobs"], torch.zeros_like(s["lse"]))[:, None]
    weight = -d
    if s["entropy"] is not None:
        weight = weight - s["d_entropy"][:, None] * (lp + s["entropy"][:, None])
    out = torch.exp(lp) * weight
    out.scatter_add_(1, tokens.clamp(0, v - 1).long()[:, None], d)
    return out.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import gated_delta_rule_75_amd as kda
    if c["op"] == "chunk":
        if own:
            out, lse = kda.paged_prefill(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["cu"],
                                         window=c["window"], sinks=c["sinks"], max_length=s["longest"], lse=True,
                                         workspace=s["workspace"])
        else:
            out, lse = _plain_chunk(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["cu"], s["most"],
                                    c["window"], c["sinks"])
        return {"out": out, "lse": lse}
    if c["op"] == "place":
        if own:
            q = kda.rotary_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["start"],
                                  s["freqs"], cu_seqlens=s["cu"], layout=c["layout"], amplitude=s["amplitude"])
        else:
            q = _plain_place(s)
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "rope":
        if own:
            q, k = kda.rotary(s["q"], s["k"], s["positions"], s["freqs"], layout=c["layout"],
                              amplitude=s["amplitude"], inverse=c["inverse"])
        else:
            q, k = (_plain_rotate(x, s["positions"], s["freqs"], c["layout"], s["amplitude"], c["inverse"])
                    for x in (s["q"], s["k"]))
        return {"q": q, "k": k}
    if c["op"] == "score":
        if own:
            got = kda.token_logprobs(s["logits"], s["tokens"], top=c["top"], entropy=c["entropy"],
                                     workspace=s["workspace"])
        else:
            got = _plain_score(s["logits"], s["tokens"], c["top"], c["entropy"])
        return dict(zip(("logprobs", "lse", "entropy", "top_logprobs", "top_tokens"), got))
    if own:
        d = kda.token_logprobs_grad(s["logits"], s["tokens"], s["lse"], s["d_logprobs"], entropy=s["entropy"],
                                    d_entropy=s["d_entropy"])
    else:
        d = _plain_grad(s)
    return {"d_logits": d}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_turned(x, position, freqs, c, amplitude):
    """One rotation per pair as a complex product."""
    r, y = c["rotary"], x.double().clone()
    sign = -1.0 if c.get("inverse") else 1.0
    angle = sign * position.double()[:, None, None] * freqs
    first = slice(0, r // 2) if c["layout"] == "half" else slice(0, r, 2)
    second = slice(r // 2, r) if c["layout"] == "half" else slice(1, r, 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.full_like(angle, amplitude), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return {x: _exact_turned(s[x], s["positions"], s["freqs"], c, s["amplitude"]) for x in ("q", "k")}
    if c["op"] in ("chunk", "place"):
        cu, past, page = s["cu"].tolist(), s["start"].tolist(), c["page"]
    if c["op"] == "place":
        q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        pools = {x: s[x].double() for x in ("k_pages", "v_pages")}
        for n in range(c["n"]):
            at = torch.arange(past[n], past[n] + cu[n + 1] - cu[n], device="cuda")
            mine = slice(cu[n], cu[n + 1])
            q[mine] = _exact_turned(s["q"][mine], at, s["freqs"], c, s["amplitude"])
            where = s["table"][n].long()[at // page]
            pools["k_pages"][where, :, at % page] = _exact_turned(s["k"][mine], at, s["freqs"], c, s["amplitude"])
            pools["v_pages"][where, :, at % page] = s["v"][mine].double()
        return {"q": q, **pools}
    if c["op"] == "chunk":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        group = c["hq"] // c["hkv"]
        for n in range(c["n"]):
            for a in range(cu[n], cu[n + 1], 512):  # some queries at a time: positions p0 .. of the sequence
                b = min(a + 512, cu[n + 1])
                p0, p1 = past[n] + a - cu[n], past[n] + b - cu[n]
                near = max(0, p0 + 1 - c["window"]) if c["window"] else 0
                keys = torch.cat([torch.arange(0, min(c["sinks"], near)), torch.arange(near, p1)]).cuda()
                where = s["table"][n].long()[keys // page]
                p = torch.arange(p0, p1, device="cuda")[:, None]
                hidden = keys > p
                if c["window"]:
                    hidden |= (keys <= p - c["window"]) & (keys >= c["sinks"])
                for h in range(c["hkv"]):
                    key, val = (s[x][where, h, keys % page].double() for x in ("k_pages", "v_pages"))
                    for e in range(h * group, (h + 1) * group):
                        x = s["q"][a:b, e].double() @ key.T / math.sqrt(c["d"])
                        x.masked_fill_(hidden, -math.inf)
                        lse[a:b, e] = torch.logsumexp(x, 1)
                        out[a:b, e] = torch.softmax(x, 1) @ val
        return {"out": out, "lse": lse}
    d = torch.float64
    got = {x: torch.empty(c["rows"], dtype=d, device="cuda") for x in ("logprobs", "lse", "entropy")}
    if c["op"] == "grad":
        grads = torch.empty(c["rows"], c["v"], dtype=d, device="cuda")
    best = torch.empty(c["rows"], c.get("top") or 1, dtype=d, device="cuda")
    which = torch.empty(best.shape, dtype=torch.int32, device="cuda")
    for a in range(0, c["rows"], 256):
        x = s["logits"][a:a + 256].double()
        token = s["tokens"][a:a + 256].long()
        pick = torch.arange(c["v"], device="cuda") == token[:, None]
        if c["op"] == "grad":
            lp = x - s["lse"][a:a + 256].double()[:, None]
            dl = s["d_logprobs"][a:a + 256].double() * (token >= 0)
            y = dl[:, None] * (pick.double() - torch.exp(lp))
            if c["entropy"]:
                h, dh = s["entropy"][a:a + 256].double(), s["d_entropy"][a:a + 256].double()
                y -= dh[:, None] * torch.exp(lp) * (lp + h[:, None])
            grads[a:a + 256] = y
            continue
        lse = torch.logsumexp(x, 1)
        got["lse"][a:a + 256] = lse
        got["logprobs"][a:a + 256] = torch.where(pick, x - lse[:, None], torch.zeros_like(x)).sum(1)
        got["entropy"][a:a + 256] = _entropy_of(x, lse)
        if c["top"]:
            y, at = torch.sort(x, dim=1, descending=True, stable=True)
            best[a:a + 256] = y[:, :c["top"]] - lse[:, None]
            which[a:a + 256] = at[:, :c["top"]]
    if c["op"] == "grad":
        return {"d_logits": grads}
    return {"logprobs": got["logprobs"], "lse": got["lse"], "entropy": got["entropy"] if c["entropy"] else None,
            "top_logprobs": best if c["top"] else None, "top_tokens": which if c["top"] else None}
