"""The paths of the attention kernels that take many sequences, many rows or long extents of the rows' own: more than 32
packed prompts (a CTA looks at 32 at a time), more entries than a CTA has threads (384; 256 at d 256), own extents on
both sides of the 2048 keys that the join takes itself, and outputs that are 16- but not 32-byte aligned.

Bar: attn_plain.attend's, element for element (its docstring derives it)."""
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


def _check(got, q, k, v, sees, what):
    """got, q [n, Hq, d] over k, v [m, Hk, d]: query i sees the first sees[i] keys."""
    G = q.shape[1] // k.shape[1]
    for h in range(k.shape[1]):
        ref, bar = attn_plain.attend(q[:, h * G:(h + 1) * G], k[:, h], v[:, h], sees, q.shape[2] ** -0.5)
        over = float(((got[:, h * G:(h + 1) * G].double() - ref).abs() - bar).max()) if ref.numel() else 0.0
        assert over <= 0, f"{what}, key head {h}: {over:.3e} beyond the bar"


def _out(shape, aligned):
    """A buffer whose address is a multiple of 32 (aligned), or of 16 only."""
    n = 1
    for x in shape:
        n *= x
    whole = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    assert whole.data_ptr() % 32 == 0
    return whole[0 if aligned else 8:][:n].view(shape)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("n,hi", [(33, 40), (70, 9), (300, 3), (65, 200)])
def test_many_prompts_in_one_call(d, aligned, n, hi):
    """Among them empty ones; the first 32 all empty in the call of 70."""
    lens = [0 if (n == 70 and i < 32) or i % 7 == 3 else 1 + (i * 31) % hi for i in range(n)]
    g = torch.Generator(device="cuda").manual_seed(n + d)
    total, hq, hk = sum(lens), 4, 2
    q, k, v = _bf16(g, total, hq, d, std=1.5), _bf16(g, total, hk, d), _bf16(g, total, hk, d)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    out = _out((total, hq, d), aligned)
    gdn.attn_prefill(gdn.make_attn_dims(q, k, B=n), q, k, v, _ints(cu), out)
    gdn.check_status()
    for b, m in enumerate(lens):
        if m and (b % 5 == 0 or b in (31, 32, 33, 63, 64, n - 1)):
            a, z = cu[b], cu[b + 1]
            _check(out[a:z], q[a:z], k[a:z], v[a:z], list(range(1, m + 1)), f"prompt {b}")


def _shared(first, prefix, suffix, T, hq, hk, d, seed, look, aligned=True):
    """`look`: the rows that are compared."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, starts, at = len(suffix), [], 0
    for n in list(prefix) + list(suffix):
        starts.append(at)
        at += n + 1
    k, v, q = _bf16(g, at, hk, d), _bf16(g, at, hk, d), _bf16(g, B, T, hq, d, std=1.5)
    ng = len(prefix)
    ps, ss = starts[:ng], starts[ng:]
    dims = gdn.make_attn_dims(q, k, B=B, T=T, n_groups=ng)
    args = (_ints(first), _ints(ps), _ints(prefix)) if ng else (None, None, None)
    ws, out, again = gdn.attn_workspace(dims), _out(q.shape, aligned), _out(q.shape, True)
    ws.fill_(255)  # NaN wherever a partial result was not written
    for o in (out, again):
        gdn.attn_shared_prefix(dims, q, k, v, *args, _ints(ss), _ints(suffix), o, ws)
    gdn.check_status()
    assert torch.equal(out, again)
    for b in look:
        grp = [i for i in range(ng) if first[i] <= b < first[i + 1]]
        p0, p = (ps[grp[0]], prefix[grp[0]]) if grp else (0, 0)
        rows = torch.cat((torch.arange(p0, p0 + p), torch.arange(ss[b], ss[b] + suffix[b]))).cuda()
        _check(out[b], q[b], k[rows], v[rows], [p + max(0, suffix[b] - T + t + 1) for t in range(T)], f"row {b}")


@pytest.mark.parametrize("d,B", [(64, 900), (128, 400), (256, 600)])
@pytest.mark.parametrize("T,hq,hk", [(1, 2, 1), (1, 40, 2), (3, 12, 1)])  # T G of 2 (own keys in the join), 20 and 36
@pytest.mark.parametrize("groups", [0, 9])
def test_more_rows_than_a_cta_has_threads(d, B, T, hq, hk, groups):
    suffix = [T + (53 * b) % 97 for b in range(B)]
    first = [B * i // groups for i in range(groups)] + [B] if groups else []
    prefix = [(1 + 211 * i) % 700 for i in range(groups)]
    look = sorted({0, 1, B - 1, B // 2, 255, 256, 257, 383, 384, 385, *range(0, B, 61)} & set(range(B)))
    _shared(first, prefix, suffix, T, hq, hk, d, seed=B + T, look=look)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,hq,hk", [(1, 8, 2), (4, 4, 1), (5, 4, 1)])  # T G of 4, 16 and 20
@pytest.mark.parametrize("groups", [False, True])
@pytest.mark.parametrize("aligned", [False, True])
def test_own_extents_around_what_the_join_takes(d, T, hq, hk, groups, aligned):
    suffix = [2047, 2048, 2049, 5000, T, T + 1, 2176, 130]
    first, prefix = ([0, 3, 4, 8], [300, 0, 1000]) if groups else ([], [])
    _shared(first, prefix, suffix, T, hq, hk, d, seed=d + T, look=range(8), aligned=aligned)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,keys", [(1, 20001), (3, 9000)])
def test_few_rows_with_long_keys_of_their_own(d, B, keys):
    """Decode over long contexts and no shared prefix."""
    _shared([], [], [keys - 7 * b for b in range(B)], 1, 8, 2, d, seed=d + B, look=range(B))
