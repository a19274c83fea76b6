"""Plain 64-bit forms of the paged 4-bit cache, its attention, beam selection and forking, for their tests: straight from
the definitions in include/gdn.h, on the host, element by element where order matters."""
import math

import torch

PAGE = 64


def e4m3(x):
    """Numbers >= 0 to the nearest of 4 significant bits (no finer than 2^-9), ties to even."""
    x = x.double()
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=1e-300))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def quantise(x, exp=0):
    """x [..., d] -> (codes u [..., d], scales [..., d/16]), float64; NaN scales where a group is not finite."""
    y = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    top = y.abs().amax(-1, keepdim=True)
    finite = torch.isfinite(y).all(-1, keepdim=True)
    s = e4m3((torch.where(finite, top, 1.0) / 7).clamp(2.0 ** -9, 240.0))
    u = torch.round(torch.where(finite, y, 0.0) / s).clamp(-7, 7) + 8
    return u.flatten(-2), torch.where(finite, s, math.nan)[..., 0]


def values(x, exp=0):
    """What stored numbers read back as."""
    u, s = quantise(x, exp)
    return ((u - 8).unflatten(-1, (-1, 16)) * s[..., None] * 2.0 ** exp).flatten(-2)


def scale_value(bits):
    bits = bits.long()
    m, e = bits % 8, bits // 8 % 16
    v = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * torch.exp2(e.double() - 10))
    return torch.where(bits % 128 == 127, math.nan, v)


def decode(pool, kv, exp=0):
    """A pool uint8 [pages, heads, 72 d] -> float64 [pages, heads, 64, d]; kv 0: keys, 1: values."""
    d = pool.shape[-1] // 72
    token, c = torch.arange(PAGE, device=pool.device)[:, None], torch.arange(d, device=pool.device)
    at = token * (d // 2) + c // 2
    at = at ^ ((at // 128 % 8) * 16)
    byte = pool[..., 32 * d * kv + at].long()
    u = torch.where(c % 2 == 0, byte % 16, byte // 16)
    where = token * (d // 16) + c // 16 if kv == 0 else c // 16 * PAGE + token
    return (u - 8).double() * scale_value(pool[..., 64 * d + 4 * d * kv + where]) * 2.0 ** exp


def encode(k, v, k_exp=0, v_exp=0):
    """Tokens [pages, 64, heads, d] -> a pool uint8 [pages, heads, 72 d]."""
    out = []
    d = k.shape[-1]
    scales = []
    for i, (x, exp) in enumerate(((k, k_exp), (v, v_exp))):
        u, s = quantise(x.transpose(1, 2), exp)  # [pages, heads, 64, .]
        u = u.long()
        at = torch.arange(32 * d, device=k.device)
        packed = (u[..., 0::2] + 16 * u[..., 1::2]).flatten(-2)[..., at ^ ((at // 128 % 8) * 16)]
        out.append(packed.to(torch.uint8))
        e = torch.floor(torch.log2(s)).clamp(min=-6)
        bits = torch.where(s < 2.0 ** -6, s * 2.0 ** 9, (s / torch.exp2(e) - 1) * 8 + 8 * (e + 7))
        bits = torch.where(torch.isnan(s), 127.0, bits).to(torch.uint8)
        scales.append((bits if i == 0 else bits.transpose(-1, -2)).flatten(-2))
    return torch.cat(out + scales, -1).contiguous()


def attend(q, k, v, sees, scale):
    """q [n, G, d] over k, v float64 [m, d]; query i sees the first sees[i] keys -> (out, bar) [n, G, d].

    bar is what the kernel may be off by: half a bf16 step of the output (2^-8); on the mass sum p |v|, half an fp16
    step of each probability (2^-11), twice the score's error delta, and m + 64 fp32 steps of accumulation; an fp16
    probability below 2^-14 of the row's largest is off by up to 2^-25 of it instead, so 2^-25 m max|v| more. delta: a
    d-term fp32 sum and its scaling, each step up to 2^-23, on sum |q| |k|; the query's channels in fp16 relative to
    the largest, 2^-25 max|q| sum |k|; 2^-21 for the exponential."""
    q = q.double()
    m, d = k.shape
    if m == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    s = torch.einsum("igd,jd->gij", q, k) * scale
    hidden = torch.arange(m, device=q.device)[None] >= torch.as_tensor(sees, device=q.device)[:, None]
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    size = torch.einsum("igd,jd->gij", q.abs(), k.abs()).masked_fill(hidden, 0.0).amax(-1) * abs(scale)
    small = q.abs().amax(-1).T * k.abs().sum(-1).amax() * abs(scale) * 2.0 ** -25
    delta = (d + 2) * 2.0 ** -23 * size + small + 2.0 ** -21
    out = torch.einsum("gij,jd->igd", p, v)
    mass = torch.einsum("gij,jd->igd", p, v.abs())
    bar = (2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * delta.T[..., None] + (m + 64) * 2.0 ** -23) * mass
           + 2.0 ** -25 * m * v.abs().amax(0))
    return out, bar + 1e-30


def beam(logits, scores, done, eos):
    """One group on the host: logits [W, V], scores [W], done [W] or None -> lists parent, token, score, done, and the
    score's bar: the logits' range R gives each exponential a relative error of (1.5 R + 4) 2^-24 (the product with
    log2(e), the function's two steps), a slice's sum of at most 2^13 such numbers one of (32 + 13) 2^-24."""
    W, V = logits.shape
    x = logits.double()
    cand = []
    bar = 0.0
    for w in range(W):
        s = float(scores[w].double())
        if done is not None and int(done[w]):
            if s > -math.inf:
                cand.append((-s, w, max(eos, 0), eos, 1))
            continue
        lse = float(torch.logsumexp(x[w], 0))
        if not s > -math.inf or not math.isfinite(lse):
            continue
        finite = x[w][torch.isfinite(x[w])]
        bar = max(bar, (1.5 * float(finite.max() - finite.min()) + 50) * 2.0 ** -24)
        top = torch.sort(x[w], descending=True, stable=True)
        for val, t in zip(top[0][:W].tolist(), top[1][:W].tolist()):
            if val > -math.inf:
                cand.append((-(s + (val - lse)), w, t, t, int(t == eos)))
    cand.sort(key=lambda c: c[:3])
    cand = cand[:W]
    parent = [c[1] for c in cand] + list(range(len(cand), W))
    token = [c[3] for c in cand] + [-1] * (W - len(cand))
    score = [-c[0] for c in cand] + [-math.inf] * (W - len(cand))
    over = [c[4] for c in cand] + [0] * (W - len(cand))
    return parent, token, score, over, bar


def fork(table, kv_len, n_pages, T, parent=None, n_new=None, pinned=None, state=None):
    """The bookkeeping on the host, lists in and out: dict of table (rows of used entries), kv_len, kv_index, page_src,
    page_dst, state_idx, state_src, state_dst, and whether a row found no pages."""
    R, width = len(kv_len), len(table[0]) if table else 0
    parent = list(range(R)) if parent is None else parent
    n_new = [T] * R if n_new is None else n_new
    L = [kv_len[p] if p >= 0 else 0 for p in parent]
    rows = [table[p][:-(-L[r] // PAGE)] if p >= 0 else [] for r, p in enumerate(parent)]
    used = {p for row in rows for p in row} | {i for i in range(n_pages) if pinned is not None and pinned[i]}
    free = [p for p in range(n_pages) if p not in used]
    copies = []
    for r in range(R):
        at = L[r] // PAGE
        copy = False
        if n_new[r] > 0 and L[r] % PAGE:
            page = rows[r][at]
            holders = [x for x in range(R) if len(rows[x]) > at and rows[x][at] == page]
            copy = min(holders, key=lambda x: (-L[x], x)) != r or (pinned is not None and bool(pinned[page]))
        copies.append(copy)
    out = dict(table=[], kv_len=[], kv_index=[], page_src=[-1] * R, page_dst=[-1] * R, full=False)
    start = 0
    for r in range(R):
        after = L[r] + n_new[r]
        need = int(copies[r]) + -(-after // PAGE) - len(rows[r]) if n_new[r] > 0 and -(-after // PAGE) <= width else 0
        row, n = list(rows[r]), n_new[r]
        if n > 0 and (-(-after // PAGE) > width or (need > 0 and start + need > len(free))):
            out["full"], n = True, 0
        else:
            mine = free[start:start + need]
            if copies[r]:
                out["page_src"][r], out["page_dst"][r] = row[-1], mine[0]
                row[-1], mine = mine[0], mine[1:]
            row += mine
        start += need
        out["table"].append(row)
        out["kv_len"].append(L[r] + n)
        out["kv_index"].append([row[(L[r] + t) // PAGE] * PAGE + (L[r] + t) % PAGE if t < n else -1 for t in range(T)])
    if state is not None:
        dead = [r for r in range(R) if r not in parent]
        out.update(state_idx=[], state_src=[-1] * R, state_dst=[-1] * R)
        for r, p in enumerate(parent):
            if p >= 0 and p not in parent[:r]:
                out["state_idx"].append(state[p])
                continue
            slot = state[dead.pop(0)]
            out["state_idx"].append(slot)
            if p >= 0:
                out["state_src"][r], out["state_dst"][r] = state[p], slot
    return out
