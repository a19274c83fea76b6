"""Plain 64-bit forms of the attention-layer operators, for their tests: straight from the formulas, one loop per
sequence and row, in torch float64 on whatever device the inputs are on."""
import math

import torch


def norm_rope(x, w, pos, inv_freq, axis, rot, adjacent, eps):
    """x [n, H, d]; pos int [axes, n]; -> float64 [n, H, d]."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    out = y.clone()
    for i in range(rot // 2):
        a = 0 if axis is None else int(axis[i])
        ang = pos[a].double() * inv_freq[i].double()
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        i0, i1 = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        out[..., i0] = y[..., i0] * c - y[..., i1] * s
        out[..., i1] = y[..., i1] * c + y[..., i0] * s
    return out


def attend(q, k, v, sees, scale):
    """q [n, G, d] over k, v [m, d]; query i sees the first sees[i] keys. -> (out [n, G, d], bar [n, G, d]).

    bar is what an fp32 pass that rounds the probabilities to bf16 may be off by: half a bf16 step of the output, half
    a bf16 step of each probability, and the scores' own error delta entering exp (a d-term fp32 sum whose every
    addition may be off by a whole fp32 step, one more step for the scaling, and 2^-21 for the exponential), on
    sum p |v|; plus m fp32 steps of the accumulation there."""
    q, k, v = q.double(), k.double(), v.double()
    n, G, d = q.shape
    m = k.shape[0]
    if m == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    s = torch.einsum("igd,jd->gij", q, k) * scale
    hidden = torch.arange(m, device=q.device)[None] >= torch.as_tensor(sees, device=q.device)[:, None]
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    size = torch.einsum("igd,jd->gij", q.abs(), k.abs()).masked_fill(hidden, 0.0).amax(-1) * abs(scale)
    delta = (d + 2) * 2.0 ** -23 * size + 2.0 ** -21
    out = torch.einsum("gij,jd->igd", p, v)
    mass = torch.einsum("gij,jd->igd", p, v.abs())
    bar = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * delta.T[..., None] + (m + 64) * 2.0 ** -23) * mass
    return out, bar + 1e-30


def accept(tokens, target, draft, uniform, n):
    """One row on the host: tokens [T], target [T][V], draft [T-1][V] or None, uniform [T] -> (accept_len, next)."""
    target = target.double()
    kept, weight = 0, None
    while kept < n - 1:
        x = int(tokens[kept + 1])
        q = 1.0 if draft is None else float(draft[kept, x].double())
        if not float(uniform[kept].double()) * q < float(target[kept, x]):
            other = torch.zeros_like(target[kept])
            if draft is None:
                other[x] = math.inf
            else:
                other = draft[kept].double()
            weight = target[kept] - other
            break
        kept += 1
    clean = lambda w: torch.where(w > 0, w, torch.zeros_like(w))  # noqa: E731  (NaN counts as zero)
    weight = clean(target[kept] if weight is None else weight)
    if not float(weight.sum()) > 0:
        weight = clean(target[kept])
    run = weight.cumsum(0)
    if not float(run[-1]) > 0:
        return kept + 1, -1
    over = (run > float(uniform[-1].double()) * float(run[-1])).nonzero()
    return kept + 1, int(over[0])
