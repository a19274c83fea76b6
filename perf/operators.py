"""The attention operators of a hybrid stack and the acceptance of drafted
tokens: what is measured of them, and their plain forms.

Four operators: head_norm_rope (norms of queries and keys per head with the
position rotation, K and V written to their cache rows), attn_prefill (causal
attention of packed prompts), attn_shared_prefix (decode and verify rows that
share a long prefix) and accept_draft (drafted tokens tested against the
target's probabilities). ``own`` false: elementary torch operations in 32 bits
(64 for angles and for the sums a draw is made from); true: the library's
calls."""
import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decode step of 64 rows: latency; a quarter of each head rotates
        dict(name="norm_rope decode 64", op="norm_rope", tokens=64, hq=16, hk=4, d=256, rot=64, axes=1, pairing=0),
        # a long prompt in one call
        dict(name="norm_rope prompt 8192", op="norm_rope", tokens=8192, hq=16, hk=4, d=256, rot=64, axes=1, pairing=0),
        # image / video tokens with time, height and width positions; adjacent pairs, whole heads rotate
        dict(name="norm_rope video 4095", op="norm_rope", tokens=4095, hq=32, hk=8, d=128, rot=128, axes=3, pairing=1),
        # one 512-token call of a prompt that continues 7680 cached tokens
        dict(name="prefill chunk 512 of 8192", op="prefill", rows=1, lo=512, hi=512, past=7680, hq=32, hk=8, d=128,
             lens=0),
        # 32 prompts of 16 to 2048 tokens packed into one call
        dict(name="prefill packed 32", op="prefill", rows=32, lo=16, hi=2048, past=0, hq=16, hk=4, d=256, lens=4),
        # one whole long prompt
        dict(name="prefill prompt 8192", op="prefill", rows=1, lo=8192, hi=8192, past=0, hq=32, hk=8, d=128, lens=0),
        # speculative verify: 8 candidate paths of 8 tokens over one cached prompt
        dict(name="shared verify 8x8", op="shared", groups=1, rows=8, t=8, prefix_lo=8192, prefix_hi=8192, suffix_hi=8,
             hq=16, hk=4, d=256, lens=1),
        # a decode step of 64 rows that share a long system prompt, each with its own continuation
        dict(name="shared decode 64 of 32768", op="shared", groups=1, rows=64, t=1, prefix_lo=32768, prefix_hi=32768,
             suffix_hi=1024, hq=32, hk=8, d=128, lens=2),
        # a decode step over several prompts with few rows each, ragged lengths, an odd number of query heads per key head
        dict(name="shared decode 7 groups", op="shared", groups=7, rows=45, t=1, prefix_lo=100, prefix_hi=4001,
             suffix_hi=700, hq=15, hk=3, d=64, lens=3),
        # verify 8 paths of 8 tokens of a drafter that proposes its best token (no draft probabilities)
        dict(name="accept 8x8 certain", op="accept", rows=8, t=8, vocab=32000, draft=False),
        # 64 rows of 8 tokens sampled from a draft model
        dict(name="accept 64x8 sampled", op="accept", rows=64, t=8, vocab=131072, draft=True),
        # odd rows, tokens and vocabulary
        dict(name="accept 33x5 odd", op="accept", rows=33, t=5, vocab=99991, draft=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "prefill", "shared", "accept"))
    d = rng.choice((64, 128, 256))
    hk = rng.choice((1, 2, 3, 4, 8) if d < 256 else (1, 2, 3, 4))
    hq = hk * rng.randint(1, (32 if d < 256 else 16) // hk if hk > 3 else 8 if d < 256 else 5)
    if op == "norm_rope":
        return dict(op=op, tokens=_spread(rng, 1, 8192), hq=hq, hk=min(hk, 4) if hq % min(hk, 4) == 0 else 1, d=d,
                    rot=rng.choice((d, d // 2, d // 4)), axes=rng.choice((1, 1, 3)), pairing=rng.choice((0, 1)))
    if op == "prefill":
        rows = _spread(rng, 1, 32)
        hi = _spread(rng, 1, 8192 if rows == 1 else 2048 if rows <= 16 else 1024)
        lo = hi if rows == 1 else _spread(rng, 1, hi)
        past = rng.choice((0, 0, _spread(rng, 1, 2048))) if hi <= 2048 else 0
        return dict(op=op, rows=rows, lo=lo, hi=hi, past=past, hq=hq, hk=hk, d=d, lens=rng.randrange(1 << 20))
    if op == "shared":
        groups = _spread(rng, 1, 8)
        rows = groups * _spread(rng, 1, max(1, 64 // groups))
        hi = _spread(rng, 16, 32768 // groups)
        return dict(op=op, groups=groups, rows=rows, t=rng.choice((1, 1, 2, 5, 8)) if rows <= 16 else 1,
                    prefix_lo=_spread(rng, 1, hi), prefix_hi=hi, suffix_hi=_spread(rng, 8, 1024), hq=hq, hk=hk, d=d,
                    lens=rng.randrange(1 << 20))
    return dict(op=op, rows=_spread(rng, 1, 64), t=rng.randrange(1, 9), vocab=_spread(rng, 1000, 131072),
                draft=rng.random() < 0.7)


# ------------------------------------------------------------------- lengths

def _prefill_lens(case):
    r = random.Random(case["lens"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["rows"])]
    past = [case["past"] if case["rows"] == 1 else r.randint(0, case["past"]) for _ in n]
    return n, past


def _shared_lens(case):
    """(first rows of the groups, prefix lengths, suffix lengths); each group has a row at least, suffixes hold the T tokens."""
    r = random.Random(case["lens"])
    g, b = case["groups"], case["rows"]
    first = [0] + sorted(r.sample(range(1, b), g - 1)) + [b]
    return (first, [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(g)],
            [r.randint(case["t"], max(case["t"], case["suffix_hi"])) for _ in range(b)])


# ------------------------------------------------------------------- inputs

def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm_rope":
        n, hq, hk, d, rot, axes = (case[k] for k in ("tokens", "hq", "hk", "d", "rot", "axes"))
        qkv = _randn(g, n, (hq + 2 * hk) * d, std=2.0)  # the rows of one fused projection
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(n, hk, d)
        s["q_w"], s["k_w"] = ((1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2))
        if axes == 1:  # text: rows anywhere up to 128 Ki tokens
            s["pos"] = torch.randint(0, 1 << 17, (1, n), generator=g, device=DEV, dtype=torch.int32)
        else:  # patches: a clock and a 64 x 64 grid
            s["pos"] = torch.stack([torch.randint(0, m, (n,), generator=g, device=DEV) for m in (4096, 64, 64)]).int()
        s["inv_freq"] = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        s["axis"] = None if axes == 1 else (torch.arange(rot // 2, device=DEV) % 3).to(torch.uint8)
        s["kv_index"] = torch.randperm(2 * n, generator=g, device=DEV)[:n].int()
        s["q_out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
        s["k_cache"], s["v_cache"] = _randn(g, 2 * n, hk, d), _randn(g, 2 * n, hk, d)
    elif case["op"] == "prefill":
        lens, past = _prefill_lens(case)
        hq, hk, d = case["hq"], case["hk"], case["d"]
        n, total = sum(lens), [a + b for a, b in zip(lens, past)]
        s["q"] = _randn(g, n, hq, d, std=1.5)
        s["k"], s["v"] = _randn(g, sum(total), hk, d), _randn(g, sum(total), hk, d)
        s["cu"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["kv_start"], s["kv_len"] = _ints([sum(total[:i]) for i in range(len(total))]), _ints(total)
        s["out"] = torch.empty_like(s["q"])
        s["max_q"], s["max_kv"] = max(lens), max(total)
    elif case["op"] == "shared":
        first, prefix, suffix = _shared_lens(case)
        hq, hk, d, t, b = (case[k] for k in ("hq", "hk", "d", "t", "rows"))
        room = max(suffix) + 5  # the rows' slots, each with room to grow
        start = [sum(prefix[:i]) for i in range(len(prefix))]
        rows = sum(prefix) + b * room
        s["q"] = _randn(g, b, t, hq, d, std=1.5)
        s["k"], s["v"] = _randn(g, rows, hk, d), _randn(g, rows, hk, d)
        s["group_rows"], s["prefix_start"], s["prefix_len"] = _ints(first), _ints(start), _ints(prefix)
        slot = torch.randperm(b, generator=g, device=DEV)
        s["suffix_start"], s["suffix_len"] = (sum(prefix) + slot * room).int(), _ints(suffix)
        s["out"] = torch.empty_like(s["q"])
        s["max_rows"] = max(first[i + 1] - first[i] for i in range(len(prefix)))
        s["max_prefix"], s["max_suffix"] = max(prefix), max(suffix)
    else:
        b, t, v = case["rows"], case["t"], case["vocab"]
        logits = 2.5 * torch.randn((b, t, v), generator=g, device=DEV)
        s["target"] = torch.softmax(logits, -1)
        s["tokens"] = torch.randint(0, v, (b, t), generator=g, device=DEV, dtype=torch.int32)
        noise = logits[:, :t - 1] + 0.5 * torch.randn((b, t - 1, v), generator=g, device=DEV)
        s["draft"] = torch.softmax(noise, -1) if case["draft"] else None
        if t > 1:  # drafts as the drafter makes them: sampled from its rows, or its best token
            if case["draft"]:
                noise = noise - torch.log(-torch.log(torch.rand(noise.shape, generator=g, device=DEV) * 0.999999 + 5e-7))
            s["tokens"][:, 1:] = noise.argmax(-1)
        s["uniform"] = torch.rand((b, t), generator=g, device=DEV)
        s["accept_len"], s["next"] = (torch.empty(b, dtype=torch.int32, device=DEV) for _ in range(2))
    return s


# -------------------------------------------------------------- plain forms

def _plain_norm_rope(s):
    rot, half = s["rot"], s["rot"] // 2
    axis = torch.zeros(half, dtype=torch.long, device=DEV) if s["axis"] is None else s["axis"].long()
    angle = s["pos"].double()[axis].T * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    lo, hi = (slice(0, half), slice(half, rot)) if s["pairing"] == 0 else (slice(0, rot, 2), slice(1, rot, 2))

    def turn(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        z = y.clone()
        z[..., lo] = y[..., lo] * cos - y[..., hi] * sin
        z[..., hi] = y[..., hi] * cos + y[..., lo] * sin
        return z.to(torch.bfloat16)

    s["q_out"].copy_(turn(s["q"], s["q_w"]))
    at = s["kv_index"].long()
    s["k_cache"][at] = turn(s["k"], s["k_w"])
    s["v_cache"][at] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_parts(scores):
    """exp(s - max) and its sum over the last axis; all zero where every score is -inf."""
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return p, p.sum(-1, keepdim=True)


def _plain_prefill(s):
    hq, hk, d = s["hq"], s["hk"], s["d"]
    n, m = s["cu"][1:] - s["cu"][:-1], s["kv_len"]
    i, j = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_kv"], device=DEV)
    qi = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()  # rows padded to the longest
    kj = (s["kv_start"][:, None] + j).clamp(max=s["k"].shape[0] - 1).long()
    q = s["q"][qi].float().view(-1, len(i), hk, hq // hk, d)
    k, v = s["k"][kj].float(), s["v"][kj].float()
    scores = torch.einsum("bihgd,bjhd->bhgij", q, k) * d ** -0.5
    seen = (j[None, None] <= (m - n)[:, None, None] + i[None, :, None]) & (j[None, None] < m[:, None, None])
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    p, total = _softmax_parts(scores)
    o = torch.einsum("bhgij,bjhd->bihgd", p / total.clamp(min=1e-30), v)
    real = i[None] < n[:, None]
    return {"out": o[real].reshape(-1, hq, d).to(torch.bfloat16)}


def _plain_shared(s):
    b, t, hq, hk, d = s["rows"], s["t"], s["hq"], s["hk"], s["d"]
    g = hq // hk
    rows = torch.arange(b, device=DEV)
    group = torch.searchsorted(s["group_rows"][1:].contiguous(), rows.int(), right=True)
    place = rows - s["group_rows"][group]
    padded = torch.zeros((s["groups"], s["max_rows"], t, hk, g, d), device=DEV)
    q = s["q"].float().view(b, t, hk, g, d)
    padded[group, place] = q
    jp, js = torch.arange(s["max_prefix"], device=DEV), torch.arange(s["max_suffix"], device=DEV)
    pj = (s["prefix_start"][:, None] + jp).clamp(max=s["k"].shape[0] - 1).long()
    sj = (s["suffix_start"][:, None] + js).clamp(max=s["k"].shape[0] - 1).long()
    s1 = torch.einsum("nrthgd,njhd->nrthgj", padded, s["k"][pj].float())[group, place]
    s1 = s1.masked_fill((jp >= s["prefix_len"][group][:, None])[:, None, None, None], -math.inf)
    s2 = torch.einsum("bthgd,bjhd->bthgj", q, s["k"][sj].float())
    sees = s["suffix_len"][:, None] - t + torch.arange(t, device=DEV)  # the last suffix key of each token
    s2 = s2.masked_fill((js > sees[..., None])[:, :, None, None], -math.inf)
    p, total = _softmax_parts(torch.cat((s1, s2), -1) * d ** -0.5)
    p = p / total
    p1 = torch.zeros((s["groups"], s["max_rows"], t, hk, g, len(jp)), device=DEV)
    p1[group, place] = p[..., :len(jp)]
    o = torch.einsum("nrthgj,njhd->nrthgd", p1, s["v"][pj].float())[group, place]
    o = o + torch.einsum("bthgj,bjhd->bthgd", p[..., len(jp):], s["v"][sj].float())
    return {"out": o.reshape(b, t, hq, d).to(torch.bfloat16)}


def _plain_accept(s):
    b, t, v = s["target"].shape
    rows = torch.arange(b, device=DEV)
    x = s["tokens"][:, 1:].long()[..., None]
    p = s["target"][:, :-1].gather(-1, x)[..., 0].double()
    q = torch.ones_like(p) if s["draft"] is None else s["draft"].gather(-1, x)[..., 0].double()
    kept = (s["uniform"][:, :-1].double() * q < p).int().cumprod(1).sum(1)
    w = s["target"][rows, kept].double()
    refused = kept < t - 1
    if t > 1:
        at = kept.clamp(max=t - 2)
        if s["draft"] is None:
            taken = torch.zeros_like(w).scatter_(1, x[rows, at], 2.0)
        else:
            taken = s["draft"][rows, at].double()
        rest = (w - taken).clamp(min=0)
        w = torch.where((refused & (rest.sum(1) > 0))[:, None], rest, w)
    run = w.cumsum(1)
    spot = s["uniform"][:, -1:].double() * run[:, -1:]
    nxt = torch.searchsorted(run, spot, right=True)[:, 0].clamp(max=v - 1)
    return {"accept_len": (kept + 1).int(), "next": nxt.int()}


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"norm_rope": _plain_norm_rope, "prefill": _plain_prefill, "shared": _plain_shared,
                "accept": _plain_accept}[s["op"]](s)
    from gated_deltanet_recurrence_delta_gb300 import gdn
    if s["op"] == "norm_rope":
        dims = gdn.make_rope_dims(s["q"], s["k"], s["rot"], n_axes=s["axes"], kv_rows=s["k_cache"].shape[0],
                                  adjacent=s["pairing"] == 1)
        gdn.head_norm_rope(dims, s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["pos"], s["inv_freq"], s["q_out"],
                           s["k_cache"], s["v_cache"], axis=s["axis"], kv_index=s["kv_index"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "prefill":
        dims = gdn.make_attn_dims(s["q"], s["k"], B=s["rows"])
        gdn.attn_prefill(dims, s["q"], s["k"], s["v"], s["cu"], s["out"], kv_start=s["kv_start"], kv_len=s["kv_len"])
        return {"out": s["out"]}
    if s["op"] == "shared":
        dims = gdn.make_attn_dims(s["q"], s["k"], B=s["rows"], T=s["t"], n_groups=s["groups"])
        if "workspace" not in s:  # kept by a program from step to step
            s["workspace"] = gdn.attn_workspace(dims)
        gdn.attn_shared_prefix(dims, s["q"], s["k"], s["v"], s["group_rows"], s["prefix_start"], s["prefix_len"],
                               s["suffix_start"], s["suffix_len"], s["out"], s["workspace"])
        return {"out": s["out"]}
    gdn.accept_draft(s["tokens"], s["target"], s["draft"], s["uniform"], s["accept_len"], s["next"])
    return {"accept_len": s["accept_len"], "next": s["next"]}


def work(case):
    if case["op"] == "norm_rope":
        n, d, heads = case["tokens"], case["d"], case["hq"] + 2 * case["hk"]
        return {"bytes": n * (4 * d * heads + 4 * case["axes"] + 4), "flops": 8 * n * d * (case["hq"] + case["hk"])}
    hq, hk, d = case.get("hq"), case.get("hk"), case.get("d")
    if case["op"] == "prefill":
        lens, past = _prefill_lens(case)
        pairs = sum(n * (n + 1) // 2 + n * p for n, p in zip(lens, past))
        return {"bytes": 4 * d * (hq * sum(lens) + hk * (sum(lens) + sum(past))), "flops": 4 * d * hq * pairs}
    if case["op"] == "shared":
        first, prefix, suffix = _shared_lens(case)
        b, t = case["rows"], case["t"]
        pairs = sum((first[i + 1] - first[i]) * t * p for i, p in enumerate(prefix))
        pairs += sum(t * n - t * (t - 1) // 2 for n in suffix)
        return {"bytes": 4 * d * (hq * b * t + hk * (sum(prefix) + sum(suffix))), "flops": 4 * d * hq * pairs}
    rows = 2 if case["draft"] and case["t"] > 1 else 1
    return {"bytes": case["rows"] * (rows * case["vocab"] * 4 + case["t"] * 16 + 8), "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------ the definition in 64 bits

def _attend(q, k, v, seen):
    """q [n][G][d], k, v [m][d], seen [n][m], all 64 bits -> [n][G][d]."""
    a = torch.einsum("igd,jd->gij", q, k) / math.sqrt(q.shape[-1])
    a = torch.softmax(a.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
    return torch.einsum("gij,jd->igd", a, v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        half = case["rot"] // 2
        axis = [0] * half if s["axis"] is None else s["axis"].tolist()
        turns = torch.stack([s["pos"][a].double() * f for a, f in zip(axis, s["inv_freq"].tolist())], -1)
        spin = torch.polar(torch.ones_like(turns), turns)[:, None]

        def turned(x, w):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * w.double()
            a = y[..., :case["rot"]]
            if case["pairing"] == 0:
                z = torch.complex(a[..., :half].contiguous(), a[..., half:].contiguous()) * spin
                a = torch.cat((z.real, z.imag), -1)
            else:
                a = torch.view_as_real(torch.view_as_complex(a.unflatten(-1, (half, 2)).contiguous()) * spin).flatten(-2)
            return torch.cat((a, y[..., case["rot"]:]), -1)

        k, v, at = s["k_cache"].double(), s["v_cache"].double(), s["kv_index"].long()
        k[at], v[at] = turned(s["k"], s["k_w"]), s["v"].double()
        return {"q": turned(s["q"], s["q_w"]), "k_cache": k, "v_cache": v}
    if case["op"] == "accept":
        return None
    hq, hk, d = case["hq"], case["hk"], case["d"]
    g = hq // hk
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    if case["op"] == "prefill":
        lens, past = _prefill_lens(case)
        at, kv = 0, 0
        for n, p in zip(lens, past):
            seen = torch.ones((n, n + p), dtype=torch.bool, device=DEV).tril(p)
            for h in range(hk):
                out[at:at + n, h * g:(h + 1) * g] = _attend(s["q"][at:at + n, h * g:(h + 1) * g].double(),
                                                            s["k"][kv:kv + n + p, h].double(),
                                                            s["v"][kv:kv + n + p, h].double(), seen)
            at, kv = at + n, kv + n + p
        return {"out": out}
    first, prefix, suffix = _shared_lens(case)
    t, start, own_start = case["t"], s["prefix_start"].tolist(), s["suffix_start"].tolist()
    for i, p in enumerate(prefix):
        for b in range(first[i], first[i + 1]):
            n = suffix[b]
            rows = torch.cat((torch.arange(start[i], start[i] + p), torch.arange(own_start[b], own_start[b] + n))).to(DEV)
            seen = torch.ones((t, p + n), dtype=torch.bool, device=DEV).tril(p + n - t)
            for h in range(hk):
                out[b, :, h * g:(h + 1) * g] = _attend(s["q"][b, :, h * g:(h + 1) * g].double(), s["k"][rows, h].double(),
                                                       s["v"][rows, h].double(), seen)
    return {"out": out}
