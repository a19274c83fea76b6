"""Beam search over a paged cache held in 4 bits: what is measured of it, and
the operators' plain forms.

Five operators: kv4 (tokens' keys and values stored in 4-bit pages and loaded
back), attn_kv4 (decode and verify rows over their pages), beam_select (the
best continuations of each group's beams), cache_fork (rows that become copies
of other rows: page tables, new pages, state slots) and slots_copy (the state
slots or pages that a fork copies, in every layer). ``own`` false: elementary
torch operations in 32 bits (64 for the beams' scores); true: the library's
calls.

A page holds 64 tokens of every head. A head's block of 72 d bytes: the codes
of the keys, 64 rows of d/2 bytes, those of the values, the keys' scales
[64][d/16] and the values' scales [d/16][64]. Channel 2i of a token is the low
half of its byte i. In a block of codes the bits 4 to 6 of a byte's offset are
xored with its bits 7 to 9. A code u stands for (u - 8) times the e4m3 scale of
its 16 channels, times 2^exp of the pool."""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64


def listed():
    return [
        # one decode step of 64 rows: latency
        dict(name="kv4 decode 64", op="kv4", tokens=64, hk=8, d=128, k_exp=0, v_exp=-3),
        # a prompt's tokens go to the cache, and are read back by a later chunk of it
        dict(name="kv4 prompt 8192", op="kv4", tokens=8192, hk=4, d=256, k_exp=0, v_exp=0),
        # a small decode step: latency
        dict(name="attn decode 8 of 2048", op="attn", rows=8, t=1, lo=512, hi=2048, hq=16, hk=4, d=256, lens=1),
        # a large decode step over long rows
        dict(name="attn decode 64 of 8192", op="attn", rows=64, t=1, lo=8192, hi=8192, hq=32, hk=8, d=128, lens=2),
        # verify of 8 tokens a row, ragged rows
        dict(name="attn verify 16x8", op="attn", rows=16, t=8, lo=100, hi=4100, hq=16, hk=4, d=256, lens=3),
        # a decode step of many short and odd rows, five query heads per key head
        dict(name="attn decode 45 odd", op="attn", rows=45, t=1, lo=1, hi=1500, hq=15, hk=3, d=64, lens=4),
        # 4 prompts with 4 beams each
        dict(name="beam 4x4", op="beam", groups=4, beams=4, vocab=32000, half=False),
        # 16 prompts with 8 beams each, the logits in bf16
        dict(name="beam 16x8", op="beam", groups=16, beams=8, vocab=131072, half=True),
        # the bookkeeping of 64 rows (8 beams a prompt) of up to 8192 tokens
        dict(name="fork 64 rows", op="fork", groups=8, beams=8, t=1, lo=4000, hi=8192, lens=5),
        # short rows, verify tokens
        dict(name="fork 30 rows", op="fork", groups=10, beams=3, t=5, lo=1, hi=700, lens=6),
        # the recurrent states and conv tails that 32 rows' beams copy, in 8 layers
        dict(name="copy states 32", op="copy", kind="state", groups=4, beams=8, layers=8, slots=32, nk=16, nv=32, d=128,
             lens=7),
        # the last pages that 64 rows copy, in 4 layers of 8 key heads
        dict(name="copy pages 64", op="copy", kind="page", groups=8, beams=8, layers=4, slots=1000, nk=8, nv=8, d=128,
             lens=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("kv4", "attn", "attn", "beam", "fork", "copy"))
    d = rng.choice((64, 128, 256))
    hk = rng.choice((1, 2, 3, 4, 8) if d < 256 else (1, 2, 3, 4))
    seed = rng.randrange(1 << 20)
    if op == "kv4":
        return dict(op=op, tokens=_spread(rng, 1, 8192), hk=hk, d=d, k_exp=rng.randint(-3, 3), v_exp=rng.randint(-3, 3))
    if op == "attn":
        rows = _spread(rng, 1, 64)
        t, share = rng.choice((1, 1, 1, 2, 5, 8)) if rows <= 16 else 1, rng.randint(1, 8)
        hi = _spread(rng, 16, min(32768, 2000000000 // (rows * hk * d * max(4, t * share))))
        return dict(op=op, rows=rows, t=t, lo=_spread(rng, 1, hi), hi=hi, hq=hk * share, hk=hk, d=d, lens=seed)
    if op == "beam":
        groups = _spread(rng, 1, 32)
        beams = _spread(rng, 1, min(16, 128 // groups))
        half = rng.random() < 0.5
        most = 131072 if half or groups * beams <= 64 else 65536
        return dict(op=op, groups=groups, beams=beams, vocab=_spread(rng, 1000, most), half=half)
    beams = rng.randint(2, 8)
    groups = _spread(rng, 1, 64 // beams)
    if op == "fork":
        return dict(op=op, groups=groups, beams=beams, t=rng.choice((1, 1, 4, 8)), lo=_spread(rng, 1, 100),
                    hi=_spread(rng, 100, 8192), lens=seed)
    kind = rng.choice(("state", "page"))
    nk = rng.choice((2, 4, 8))
    return dict(op=op, kind=kind, groups=groups, beams=beams, layers=rng.randint(1, 4), slots=groups * beams + rng.randint(0, 9),
                nk=nk, nv=nk * rng.randint(1, 2) if kind == "state" else nk, d=rng.choice((64, 128)), lens=seed)


# ------------------------------------------------------------------- lengths

def _lens(case):
    r = random.Random(case["lens"])
    return [max(case["t"], r.randint(case["lo"], case["hi"])) for _ in range(case["rows"])]


def _parents(case):
    """Parents as beam search makes them: good beams have several children."""
    r = random.Random(case["lens"])
    w = case["beams"]
    return [g * w + min(r.randrange(w), r.randrange(w)) for g in range(case["groups"]) for _ in range(w)]


def _fork_rows(case):
    """(lengths, pages): a group's beams have one length, share all full pages of their prompt (half their tokens),
    and have own pages behind it."""
    r = random.Random(case["lens"] + 1)
    lens, table, n = [], [], 0
    for _ in range(case["groups"]):
        m = r.randint(case["lo"], case["hi"])
        shared = m // 2 // PAGE
        first = list(range(n, n + shared))
        n += shared
        for _ in range(case["beams"]):
            lens.append(m)
            mine = -(-m // PAGE) - shared
            table.append(first + list(range(n, n + mine)))
            n += mine
    return lens, table, n


# ------------------------------------------------------------------- inputs

def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _swizzle(d):
    """Where the bytes of a block of codes stand."""
    a = torch.arange(32 * d, device=DEV)
    return a ^ (((a >> 7) & 7) << 4)


def _to_blocks(codes_k, scale_k, codes_v, scale_v):
    """Codes uint8 [..., 64, d] and scale bytes uint8 [..., 64, d/16] of whole pages -> blocks uint8 [..., 72 d]."""
    lead, d = codes_k.shape[:-2], codes_k.shape[-1]
    at = _swizzle(d)
    parts = []
    for codes in (codes_k, codes_v):
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(*lead, 32 * d)
        parts.append(packed[..., at])  # the xor is its own inverse
    return torch.cat(parts + [scale_k.reshape(*lead, 4 * d), scale_v.transpose(-1, -2).reshape(*lead, 4 * d)], -1)


def _random_pool(g, n_pages, hk, d):
    """Pages of normal keys and values, quantised; a few at a time."""
    pool = torch.empty((n_pages, hk, 72 * d), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hk * PAGE * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        q = [_quantise(torch.randn((n, hk, PAGE, d), generator=g, device=DEV).to(torch.bfloat16), 0) for _ in range(2)]
        pool[i:i + n] = _to_blocks(q[0][0], q[0][1], q[1][0], q[1][1])
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "kv4":
        n, hk, d = case["tokens"], case["hk"], case["d"]
        pages = -(-n // PAGE) + 2
        kv = _randn(g, n, 2 * hk * d)  # the rows of one projection
        s["k"], s["v"] = kv[:, :hk * d].view(n, hk, d), kv[:, hk * d:].view(n, hk, d)
        s["v"].mul_(2.0 ** case["v_exp"])
        order = torch.randperm(pages, generator=g, device=DEV)  # pages in any order, the first token inside a page
        place = torch.arange(n, device=DEV) + 37
        s["kv_index"] = (order[place // PAGE] * PAGE + place % PAGE).int()
        s["pool"] = torch.zeros((pages, hk, 72 * d), dtype=torch.uint8, device=DEV)
        s["k_out"], s["v_out"] = (torch.empty((n, hk, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    elif op == "attn":
        lens = _lens(case)
        used = [-(-n // PAGE) for n in lens]
        s["max_pages"] = max(used) + 3
        pages = sum(used)
        s["pool"] = _random_pool(g, pages, case["hk"], case["d"])
        order = torch.randperm(pages, generator=g, device=DEV).int()
        s["table"] = torch.full((case["rows"], s["max_pages"]), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(used):
            s["table"][b, :n] = order[at:at + n]
            at += n
        s["kv_len"] = _ints(lens)
        s["q"] = _randn(g, case["rows"], case["t"], case["hq"], case["d"], std=1.5)
        s["out"] = torch.empty_like(s["q"])
    elif op == "beam":
        n, w, v = case["groups"], case["beams"], case["vocab"]
        s["logits"] = 2.5 * torch.randn((n, w, v), generator=g, device=DEV)
        if case["half"]:
            s["logits"] = s["logits"].to(torch.bfloat16)
        # beams whose scores lie together, the best first; some are finished
        s["scores"] = -20.0 - 1.5 * torch.rand((n, w), generator=g, device=DEV).sort(-1)[0]
        s["done"] = (torch.rand((n, w), generator=g, device=DEV) < 0.1).to(torch.uint8)
        s["eos"] = int(torch.randint(0, v, (1,), generator=g, device=DEV))
        s["parent"], s["token"] = (torch.empty((n, w), dtype=torch.int32, device=DEV) for _ in range(2))
        s["new_scores"], s["new_done"] = torch.empty_like(s["scores"]), torch.empty_like(s["done"])
    elif op == "fork":
        lens, table, used = _fork_rows(case)
        rows = len(lens)
        s["rows"], s["max_pages"] = rows, max(len(x) for x in table) + 3
        s["n_pages"] = used + 3 * rows + 5
        order = torch.randperm(s["n_pages"], generator=g, device=DEV).int()
        s["table"] = torch.full((rows, s["max_pages"]), -1, dtype=torch.int32, device=DEV)
        for b, x in enumerate(table):
            s["table"][b, :len(x)] = order[_ints(x).long()]
        s["kv_len"], s["parent"] = _ints(lens), _ints(_parents(case))
        s["pinned"] = (torch.rand(s["n_pages"], generator=g, device=DEV) < 0.01).to(torch.uint8)
        s["state_idx"] = torch.randperm(rows, generator=g, device=DEV).int()
        s["table_out"] = torch.full_like(s["table"], -1)
        s["kv_index"] = torch.empty((rows, case["t"]), dtype=torch.int32, device=DEV)
        for n in ("kv_len_out", "page_src", "page_dst", "state_idx_out", "state_src", "state_dst"):
            s[n] = torch.empty(rows, dtype=torch.int32, device=DEV)
    else:
        parent, rows = _parents(case), case["groups"] * case["beams"]
        src, dst, dead = [-1] * rows, [-1] * rows, sorted(set(range(rows)) - set(parent))
        for r, p in enumerate(parent):
            if p in parent[:r]:
                src[r], dst[r] = p, dead.pop(0)
        slot = torch.randperm(case["slots"], generator=g, device=DEV).tolist()
        s["src"], s["dst"] = (_ints([-1 if x < 0 else slot[x] for x in y]) for y in (src, dst))
        lead = (case["layers"], case["slots"])
        if case["kind"] == "state":
            c = (2 * case["nk"] + case["nv"]) * case["d"]
            s["pools"] = [torch.randn((*lead, case["nv"], case["d"], case["d"]), generator=g, device=DEV),
                          _randn(g, *lead, 3, c)]
        else:
            s["pools"] = [torch.randint(0, 256, (*lead, case["nk"], 72 * case["d"]), generator=g, device=DEV,
                                        dtype=torch.uint8)]
    return s


# -------------------------------------------------------------- plain forms

def _quantise(x, exp):
    """bf16 [..., d] -> codes uint8 [..., d], scale bytes uint8 [..., d/16]."""
    y = x.float().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    top = y.abs().amax(-1, keepdim=True)
    scale = (top.double() / 7).float().clamp(2.0 ** -9, 240.0).to(torch.float8_e4m3fn)  # ties have to stay ties
    codes = torch.round(y / scale.float()).clamp(-7, 7) + 8
    return codes.to(torch.uint8).flatten(-2), scale.view(torch.uint8)[..., 0]


def _from_blocks(blocks, d):
    """Blocks uint8 [..., 72 d] -> keys, values fp32 [..., 64, d], without the pool's exponents."""
    lead, at = blocks.shape[:-1], _swizzle(d)
    out = []
    for i in range(2):
        codes = blocks[..., 32 * d * i:32 * d * (i + 1)][..., at].view(*lead, PAGE, d // 2)
        scale = blocks[..., (64 + 4 * i) * d:(68 + 4 * i) * d].contiguous().view(torch.float8_e4m3fn).float()
        scale = scale.view(*lead, PAGE, d // 16) if i == 0 else scale.view(*lead, d // 16, PAGE).transpose(-1, -2)
        pair = torch.stack((codes & 15, codes >> 4), -1).view(*lead, PAGE, d // 16, 16)
        out.append(((pair.float() - 8) * scale[..., None]).flatten(-2))
    return out


def _plain_kv4(s):
    """Stores the tokens as bytes of their pages, and loads them from there."""
    d, hk = s["d"], s["hk"]
    row, page = s["kv_index"].long() % PAGE, s["kv_index"].long() // PAGE
    at = _swizzle(d)
    heads = torch.arange(hk, device=DEV)
    byte = torch.arange(d // 2, device=DEV)
    group = torch.arange(d // 16, device=DEV)
    out = []
    for i, (x, exp) in enumerate(((s["k"], s["k_exp"]), (s["v"], s["v_exp"]))):
        codes, scale = _quantise(x, exp)
        where = 32 * d * i + at[row[:, None] * (d // 2) + byte]  # [n, d/2]
        index = (page[:, None, None], heads[None, :, None], where[:, None])
        s["pool"][index] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        where = 64 * d + 4 * d * i + (row[:, None] * (d // 16) + group if i == 0 else group * PAGE + row[:, None])
        sindex = (page[:, None, None], heads[None, :, None], where[:, None])
        s["pool"][sindex] = scale
        got, sc = s["pool"][index], s["pool"][sindex].view(torch.float8_e4m3fn).float()
        pair = torch.stack((got & 15, got >> 4), -1).flatten(-2).unflatten(-1, (-1, 16))
        out.append((((pair.float() - 8) * sc[..., None]).flatten(-2) * 2.0 ** exp).to(torch.bfloat16))
    return {"k": out[0], "v": out[1]}


def _plain_attn(s):
    b, t, hq, hk, d = s["rows"], s["t"], s["hq"], s["hk"], s["d"]
    blocks = s["pool"][s["table"].clamp(min=0).long()]  # [b, pages, hk, 72 d]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in _from_blocks(blocks, d))  # [b, hk, keys, d]
    q = s["q"].float().view(b, t, hk, hq // hk, d)
    scores = torch.einsum("bthgd,bhjd->bhtgj", q, k) * d ** -0.5
    sees = s["kv_len"][:, None] - t + torch.arange(t, device=DEV)  # the last key of each token
    hidden = torch.arange(k.shape[2], device=DEV) > sees[..., None]
    scores = scores.masked_fill(hidden[:, None, :, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = torch.einsum("bhtgj,bhjd->bthgd", p / p.sum(-1, keepdim=True), v)
    return {"out": o.reshape(b, t, hq, d).to(torch.bfloat16)}


def _plain_beam(s):
    n, w, v = s["logits"].shape
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = torch.log(torch.exp(x - top).sum(-1, keepdim=True)) + top
    cand = s["scores"].double()[..., None] + (x - lse)
    over = s["done"].bool()
    carry = torch.full_like(cand, -math.inf)
    carry[..., s["eos"]] = s["scores"].double()
    cand = torch.where(over[..., None], carry, cand).view(n, w * v)
    best, at = torch.sort(cand, dim=-1, descending=True, stable=True)  # ties: the lowest place first
    best, at = best[:, :w], at[:, :w]
    beam, token = at // v, at % v
    done = over.gather(1, beam) | (token == s["eos"])
    return {"parent": (beam + w * torch.arange(n, device=DEV)[:, None]).int(), "token": token.int(),
            "scores": best.float(), "done": done.to(torch.uint8)}


def _plain_fork(s):
    rows, t, width, n_pages = s["rows"], s["t"], s["max_pages"], s["n_pages"]
    r = torch.arange(rows, device=DEV)
    parent = s["parent"].long()
    length = s["kv_len"].long()[parent]
    table = s["table"].long()[parent]
    used = (length + PAGE - 1) // PAGE
    held = torch.arange(width, device=DEV) < used[:, None]
    # the last page, where it is partial: who holds it, and who has the most tokens of it
    tail = (used - 1).clamp(min=0)
    part = length % PAGE != 0
    page = table.gather(1, tail[:, None])[:, 0]
    holds = (table[:, tail].T == page[:, None]) & (tail[:, None] < used)  # [row, other row]
    rank = length * rows + (rows - 1 - r)
    keeper = (torch.where(holds, rank, -1).amax(1) == rank) & (s["pinned"][page.clamp(min=0)] == 0)
    copies = part & ~keeper
    # free pages, lowest first
    taken = s["pinned"].bool()
    marks = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    marks.scatter_(0, torch.where(held, table, n_pages).flatten(), 1)
    taken = taken | marks[:n_pages].bool()
    free = torch.sort(taken.int(), stable=True)[1]
    used_out = (length + t + PAGE - 1) // PAGE
    need = copies.long() + used_out - used
    first = need.cumsum(0) - need
    out = torch.where(held, table, s["table_out"].long())
    fresh = free[(first[:, None] + torch.arange(width, device=DEV) - used[:, None] + copies.long()[:, None]).clamp(0, n_pages - 1)]
    new = (torch.arange(width, device=DEV) >= used[:, None]) & (torch.arange(width, device=DEV) < used_out[:, None])
    out = torch.where(new, fresh, out)
    copy_to = free[first.clamp(max=n_pages - 1)]
    out = torch.where(copies[:, None] & (torch.arange(width, device=DEV) == tail[:, None]), copy_to[:, None], out)
    place = length[:, None] + torch.arange(t, device=DEV)
    index = out.gather(1, place // PAGE) * PAGE + place % PAGE
    # state slots: a parent's first child keeps its slot, the others take the slots of rows without children, in order
    same = parent[:, None] == parent[None]
    again = (same & (r[None] < r[:, None])).any(1)
    childless = ~(parent[None] == r[:, None]).any(1)
    dead = torch.sort((~childless).int(), stable=True)[1]
    slot = s["state_idx"].long()
    spare = slot[dead[(again.long().cumsum(0) - again.long())]]
    none = torch.full_like(r, -1)
    return {"table": out.int(), "kv_len": (length + t).int(), "kv_index": index.int(),
            "page_src": torch.where(copies, page, none).int(), "page_dst": torch.where(copies, copy_to, none).int(),
            "state_idx": torch.where(again, spare, slot[parent]).int(),
            "state_src": torch.where(again, slot[parent], none).int(), "state_dst": torch.where(again, spare, none).int()}


def _plain_copy(s):
    real = s["src"] >= 0
    src, dst = s["src"][real].long(), s["dst"][real].long()
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]
    return {f"pool{i}": p for i, p in enumerate(s["pools"])}


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"kv4": _plain_kv4, "attn": _plain_attn, "beam": _plain_beam, "fork": _plain_fork, "copy": _plain_copy}[op](s)
    from gated_deltanet_recurrence_delta_gb300 import gdn
    if op == "kv4":
        dims = gdn.make_kv4_dims(s["k"], s["pool"], v=s["v"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        gdn.kv4_store(dims, s["k"], s["v"], s["kv_index"], s["pool"])
        dims = gdn.make_kv4_dims(s["k_out"], s["pool"], v=s["v_out"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        gdn.kv4_load(dims, s["pool"], s["kv_index"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attn":
        dims = gdn.make_attn_kv4_dims(s["q"], s["pool"], s["table"])
        if "workspace" not in s:  # kept by a program from step to step
            s["workspace"] = gdn.attn_kv4_workspace(dims)
        gdn.attn_kv4(dims, s["q"], s["pool"], s["table"], s["kv_len"], s["out"], s["workspace"])
        return {"out": s["out"]}
    if op == "beam":
        if "workspace" not in s:
            s["workspace"] = gdn.beam_workspace(s["logits"])
        gdn.beam_select(s["logits"], s["scores"], s["parent"], s["token"], s["new_scores"], s["workspace"], done=s["done"],
                        new_done=s["new_done"], eos=s["eos"])
        return {"parent": s["parent"], "token": s["token"], "scores": s["new_scores"], "done": s["new_done"]}
    if op == "fork":
        gdn.cache_fork(s["table"], s["kv_len"], s["table_out"], s["kv_len_out"], s["kv_index"], s["page_src"], s["page_dst"],
                       s["n_pages"], parent=s["parent"], pinned=s["pinned"], state_idx=s["state_idx"],
                       state_idx_out=s["state_idx_out"], state_src=s["state_src"], state_dst=s["state_dst"])
        return {"table": s["table_out"], "kv_len": s["kv_len_out"], "kv_index": s["kv_index"], "page_src": s["page_src"],
                "page_dst": s["page_dst"], "state_idx": s["state_idx_out"], "state_src": s["state_src"],
                "state_dst": s["state_dst"]}
    gdn.slots_copy([(p, s["src"], s["dst"]) for p in s["pools"]])
    return {f"pool{i}": p for i, p in enumerate(s["pools"])}


def work(case):
    op = case["op"]
    if op == "kv4":
        n = case["tokens"] * case["hk"] * case["d"]
        return {"bytes": n * 4 + n * 9 // 4 + n * 4 + 4 * case["tokens"], "flops": 8 * n}
    if op == "attn":
        lens, t = _lens(case), case["t"]
        pairs = sum(t * n - t * (t - 1) // 2 for n in lens)
        keys = sum(lens)
        return {"bytes": keys * case["hk"] * case["d"] * 9 // 8 + 4 * case["d"] * case["hq"] * case["rows"] * t,
                "flops": 4 * case["d"] * case["hq"] * pairs}
    if op == "beam":
        n = case["groups"] * case["beams"]
        return {"bytes": n * (case["vocab"] * (2 if case["half"] else 4) + 18), "flops": 4 * n * case["vocab"]}
    if op == "fork":
        lens = _fork_rows(case)[0]
        entries = sum(-(-n // PAGE) for n in lens)
        return {"bytes": 8 * entries + len(lens) * (36 + 4 * case["t"]), "flops": entries}
    pairs = sum(p in x[:r] for x in [_parents(case)] for r, p in enumerate(x))
    slot = (4 * case["nv"] * case["d"] ** 2 + 6 * (2 * case["nk"] + case["nv"]) * case["d"] if case["kind"] == "state"
            else 72 * case["nk"] * case["d"])
    return {"bytes": 2 * pairs * case["layers"] * slot, "flops": 0}


# ------------------------------------------------------ the definition in 64 bits

def _e4m3(x):
    """Positive 64-bit numbers rounded to the nearest of 4 significant bits, and no finer than 2^-9; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x)).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _value(block, d, token, channel, values):
    """The numbers at (token, channel) of heads' blocks [.., 72 d], element by element from the layout's description."""
    offset = token * (d // 2) + channel // 2
    offset = offset ^ ((offset // 128 % 8) * 16)
    byte = block[..., (32 * d if values else 0) + offset].long()
    code = torch.where(channel % 2 == 0, byte % 16, byte // 16) - 8
    place = (channel // 16) * PAGE + token if values else token * (d // 16) + channel // 16
    bits = block[..., (68 * d if values else 64 * d) + place].long()
    mantissa, exponent = bits % 8, bits // 8
    scale = torch.where(exponent == 0, mantissa.double() * 2.0 ** -9, (8 + mantissa).double() * torch.exp2(exponent.double() - 10))
    return code.double() * scale


def exact(case, seed):
    if case["op"] == "fork" or case.get("kind") == "page":  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "copy":
        out = {}
        for i, pool in enumerate(s["pools"]):
            out[f"pool{i}"] = pool.double()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                if a >= 0:
                    out[f"pool{i}"][:, b] = pool[:, a].double()
        return out
    if case["op"] == "kv4":
        out = {}
        for name, exp in (("k", case["k_exp"]), ("v", case["v_exp"])):
            y = s[name].double().unflatten(-1, (-1, 16)) / 2.0 ** exp
            scale = _e4m3((y.abs().max(-1, keepdim=True)[0] / 7).clamp(2.0 ** -9, 240.0))
            out[name] = (torch.round(y / scale).clamp(-7, 7) * scale * 2.0 ** exp).flatten(-2)
        return out
    if case["op"] == "beam":
        n, w, v = s["logits"].shape
        logp = torch.log_softmax(s["logits"].double(), -1)
        scores = torch.empty((n, w), dtype=torch.float64, device=DEV)
        for i in range(n):
            each = [s["scores"][i, j:j + 1].double() if int(s["done"][i, j]) else s["scores"][i, j].double() + logp[i, j]
                    for j in range(w)]
            scores[i] = torch.cat(each).topk(w)[0]
        return {"parent": None, "token": None, "scores": scores, "done": None}
    d, hk, t = case["d"], case["hk"], case["t"]
    g = case["hq"] // hk
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    token, channel = torch.arange(PAGE, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    for b, n in enumerate(_lens(case)):
        pages = s["table"][b, :-(-n // PAGE)].long()
        seen = torch.ones((t, n), dtype=torch.bool, device=DEV).tril(n - t)
        for h in range(hk):
            blocks = s["pool"][pages, h]
            k, v = (_value(blocks, d, token, channel, x).flatten(0, 1)[:n] for x in (False, True))
            a = torch.einsum("igd,jd->gij", s["q"][b, :, h * g:(h + 1) * g].double(), k) / math.sqrt(d)
            a = torch.softmax(a.masked_fill(~seen, -math.inf), -1)
            out[b, :, h * g:(h + 1) * g] = torch.einsum("gij,jd->igd", a, v)
    return {"out": out}
