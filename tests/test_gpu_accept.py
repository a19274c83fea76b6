"""gdn_accept_draft against the 64-bit form, token for token, and the commit that it feeds.

Whole numbers have to be equal: the library's sums carry ~46 bits, so a draw can differ from exact arithmetic's only
where the random number lies within 2^-44 of one of V boundaries (1e-8 a draw at the sizes here)."""
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


def _case(B, T, V, sampled, seed, noise=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = 2.0 * torch.randn((B, T, V), generator=g, device="cuda")
    near = logits[:, :T - 1] + noise * torch.randn((B, T - 1, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    if T > 1:
        pick = near - torch.log(-torch.log(torch.rand(near.shape, generator=g, device="cuda") * 0.99 + 0.005)) if sampled else near
        tokens[:, 1:] = pick.argmax(-1)
    return dict(tokens=tokens, target=torch.softmax(logits, -1), draft=torch.softmax(near, -1) if sampled else None,
                uniform=torch.rand((B, T), generator=g, device="cuda"))


def _run(c, n=None, stream=None):
    B = c["tokens"].shape[0]
    a, x = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    gdn.accept_draft(c["tokens"], c["target"], c["draft"], c["uniform"], a, x, n, stream)
    return a, x


def _compare(c, a, x, n=None):
    h = {k: None if t is None else t.cpu() for k, t in c.items()}
    B, T = h["tokens"].shape
    for b in range(B):
        m = T if n is None else int(n[b])
        if m == 0:
            assert (int(a[b]), int(x[b])) == (0, -1)
            continue
        want = attn_plain.accept(h["tokens"][b], h["target"][b], None if h["draft"] is None else h["draft"][b],
                                 h["uniform"][b], m)
        assert (int(a[b]), int(x[b])) == want, f"row {b}"


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 2, 2), (5, 4, 31), (9, 8, 1000), (4, 32, 4097), (33, 5, 20011),
                                   (2, 8, 131072)])
@pytest.mark.parametrize("sampled", [False, True])
def test_tokens_match_exact_arithmetic(B, T, V, sampled):
    c = _case(B, T, V, sampled, seed=B + V)
    a, x = _run(c)
    gdn.check_status()
    _compare(c, a, x)


def test_real_lengths_and_every_refusal_place():
    """Rows that refuse at each place, rows that accept everything, real lengths from 0 to T."""
    c = _case(40, 6, 257, True, seed=3)
    c["uniform"][:, :-1] = 0.0  # accept all but ...
    for b in range(40):
        if b % 6 < 5:
            c["target"][b, b % 6, int(c["tokens"][b, b % 6 + 1])] = 0.0  # ... the one that the target rules out
    n = torch.arange(40, dtype=torch.int32, device="cuda") % 7
    for lens in (None, n):
        a, x = _run(c, lens)
        gdn.check_status()
        _compare(c, a, x, lens)
    a, _ = _run(c)
    assert a[:6].tolist() == [1, 2, 3, 4, 5, 6]


def test_edges_of_the_distribution():
    """One-hot targets, equal distributions (a residual without mass), no mass at all, NaN and negative weights, the
    least and the greatest random number."""
    V = 300
    c = _case(8, 2, V, True, seed=4)
    t, d = c["target"], c["draft"]
    t[0, 0] = 0.0
    t[0, 0, 17] = 1.0
    c["tokens"][0, 1] = 3
    d[1, 0] = t[1, 0]
    t[1, 0, 5] = d[1, 0, 5] = 0.0
    c["tokens"][1, 1] = 5  # refused (0 < 0 is false) with nothing left of target - draft
    t[2] = 0.0  # no mass anywhere
    t[3, 0, 7] = float("nan")
    t[3, 0, 8] = -1.0
    c["tokens"][3, 1] = 7  # NaN: refused, and never drawn
    c["uniform"][4] = 0.0
    c["uniform"][5] = 1 - 2.0 ** -24
    t[6, 0, :100] = 0.0
    t[6, 0, 200:] = 0.0
    c["tokens"][6, 1] = 250
    c["uniform"][6, 1] = 1 - 2.0 ** -24  # the last token with mass is not the last token
    a, x = _run(c)
    gdn.check_status()
    _compare(c, a, x)
    assert int(x[2]) == -1 and int(x[0]) == 17


def test_bad_tokens_and_lengths_are_reported():
    c = _case(6, 3, 50, True, seed=5)
    c["tokens"][1, 2] = 50
    c["tokens"][2, 1] = -1
    c["tokens"][0, 0] = -99  # token 0 is not read
    n = torch.tensor([3, 3, 3, 4, -1, 3], dtype=torch.int32, device="cuda")
    a, x = _run(c, n)
    with pytest.raises(gdn.GdnError) as e:
        gdn.check_status()
    assert e.value.name == "GDN_ERR_INDEX"
    assert a[1:5].tolist() == [0] * 4 and x[1:5].tolist() == [-1] * 4
    n[3:5] = 3
    keep = [0, 5]
    _compare({k: t[keep] for k, t in c.items()}, a[keep], x[keep])


def test_drawn_tokens_follow_the_target():
    """Accepted and redrawn tokens together have the target's distribution whatever the drafter's: 40000 rows over 8
    tokens; each count is binomial, five standard deviations."""
    N, V = 40000, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    p = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    drafts = torch.multinomial(q, N, replacement=True, generator=g).int()
    c = dict(tokens=torch.stack((torch.zeros_like(drafts), drafts), 1).contiguous(),
             target=p.expand(N, 2, V).contiguous(), draft=q.expand(N, 1, V).contiguous(),
             uniform=torch.rand((N, 2), generator=g, device="cuda"))
    a, x = _run(c)
    gdn.check_status()
    first = torch.where(a == 2, drafts, x)
    count = torch.bincount(first.long(), minlength=V).double()
    sd = torch.sqrt(N * p.double() * (1 - p.double()))
    assert float(((count - N * p.double()).abs() / sd).max()) < 5


def test_accept_lengths_feed_the_commit_in_one_graph():
    """accept_draft -> commit_accepted on the device, captured and replayed."""
    B, T, V, nk, nv, d = 4, 5, 700, 1, 2, 32
    c = _case(B, T, V, True, seed=8)
    dims = gdn.make_dims(B=B, T=T, nk=nk, nv=nv, dk=d, dv=d, n_slots=B)
    ckpt = torch.randn((1, B, T, nv, d, d), device="cuda")
    conv = torch.randn((1, B, T, 3, 2 * nk * d + nv * d), device="cuda").to(torch.bfloat16)
    pool, pconv = torch.zeros_like(ckpt[:, :, 0]).contiguous(), torch.zeros_like(conv[:, :, 0]).contiguous()
    slot = torch.arange(B, dtype=torch.int32, device="cuda")
    a, x = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        gdn.accept_draft(c["tokens"], c["target"], c["draft"], c["uniform"], a, x)
        gdn.commit_accepted(dims, 1, 1, ckpt, conv, pool, pconv, a, slot)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c["uniform"].copy_(torch.rand_like(c["uniform"]))
    graph.replay()
    gdn.check_status()
    _compare(c, a, x)
    for b in range(B):
        assert torch.equal(pool[0, b], ckpt[0, b, int(a[b]) - 1]) and torch.equal(pconv[0, b], conv[0, b, int(a[b]) - 1])
