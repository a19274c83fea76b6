"""gdn_attn_prefill and gdn_attn_shared_prefix where a visible key is not finite: a NaN or +inf score has to reach every
query that sees it and no other, wherever its block lies, and a score of -inf is a key that counts for nothing.

Bar where the result is finite: attn_plain.attend's, element for element."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from tests import attn_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _check(got, ref, bar, what):
    """NaN where the reference is, elsewhere within the bar."""
    bad = ref.isnan()
    assert torch.equal(got.isnan(), bad), f"{what}: {int((got.isnan() != bad).sum())} values are wrongly NaN or not"
    over = ((got.double() - ref).abs() - bar).nan_to_num(0.0).max() if ref.numel() else torch.tensor(0.0)
    assert float(over) <= 0, f"{what}: {float(over):.3e} beyond the bar"


def _without(x, at):
    return torch.cat((x[:at], x[at + 1:]))


def _reference(q, k, v, sees, at, value, scale):
    """attend with the key `at` holding a score that is not finite: -inf takes it out of every sum."""
    if value == float("-inf"):
        return attn_plain.attend(q, _without(k, at), _without(v, at), [n - (n > at) for n in sees], scale)
    ref, bar = attn_plain.attend(q, torch.cat((k[:at], torch.zeros_like(k[at:at + 1]), k[at + 1:])), v, sees, scale)
    ref[torch.as_tensor(sees, device=q.device) > at] = float("nan")
    return ref, bar


VALUES = [float("nan"), float("inf"), float("-inf")]


# 400 tokens are fewer tiles than SMs: one tile to a CTA, its blocks dealt to two groups (d 64, 128); 2500 tokens of 8 key
# heads are two tiles to a CTA. Keys 5, 130, 300 and 390 lie in blocks 0, 1, 2 and 3.
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,hq,hk", [(400, 4, 2), (2500, 16, 8)])
@pytest.mark.parametrize("at", [5, 130, 300, 390])
@pytest.mark.parametrize("value", VALUES)
def test_prompt_with_a_key_that_is_not_finite(d, n, hq, hk, at, value):
    g = torch.Generator(device="cuda").manual_seed(d + at)
    q, k, v = _bf16(g, n, hq, d, std=1.5), _bf16(g, n, hk, d), _bf16(g, n, hk, d)
    q[..., 3] = 1.0  # the score's sign is the key's
    k[at, 0, 3] = value
    out = torch.full_like(q, 7.0)
    gdn.attn_prefill(gdn.make_attn_dims(q, k, B=1), q, k, v, _ints([0, n]), out)
    gdn.check_status()
    G = hq // hk
    for h in range(2):  # the key head that holds it, and one that does not
        args = q[:, h * G:(h + 1) * G], k[:, h], v[:, h], list(range(1, n + 1))
        ref, bar = _reference(*args, at, value, d ** -0.5) if h == 0 else attn_plain.attend(*args, d ** -0.5)
        _check(out[:, h * G:(h + 1) * G], ref, bar, f"key head {h}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 2), (8, 4)])  # the rows' own keys in the join, or in lines of their own
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("value", VALUES)
def test_shared_rows_with_a_key_that_is_not_finite(d, T, G, where, value):
    g = torch.Generator(device="cuda").manual_seed(d + T)
    B, hk, prefix, own = 4, 2, 1500, [T, T + 200, T + 40, T + 300]
    hq, room = hk * G, 400
    k, v = (_bf16(g, prefix + B * room, hk, d) for _ in range(2))
    q = _bf16(g, B, T, hq, d, std=1.5)
    q[..., 3] = 1.0
    ss = [prefix + b * room for b in range(B)]
    k[700 if where == "prefix" else ss[1] + 150, 0, 3] = value
    out = torch.full_like(q, 7.0)
    dims = gdn.make_attn_dims(q, k, B=B, T=T, n_groups=1)
    gdn.attn_shared_prefix(dims, q, k, v, _ints([0, B]), _ints([0]), _ints([prefix]), _ints(ss), _ints(own), out,
                           gdn.attn_workspace(dims))
    gdn.check_status()
    for b in range(B):
        rows = torch.cat((torch.arange(prefix), torch.arange(ss[b], ss[b] + own[b]))).cuda()
        sees = [prefix + own[b] - T + t + 1 for t in range(T)]
        for h in range(hk):
            args = q[b, :, h * G:(h + 1) * G], k[rows, h], v[rows, h], sees
            if h == 0 and (where == "prefix" or b == 1):
                ref, bar = _reference(*args, 700 if where == "prefix" else prefix + 150, value, d ** -0.5)
            else:
                ref, bar = attn_plain.attend(*args, d ** -0.5)
            _check(out[b, :, h * G:(h + 1) * G], ref, bar, f"row {b}, key head {h}")
