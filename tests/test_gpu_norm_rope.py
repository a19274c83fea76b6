"""gdn_head_norm_rope against the 64-bit form: head sizes, pairings, partial rotation, several axes, far and negative
positions, strided inputs, pool rows, outputs in place.

Bar: half a bf16 step of the output (2^-8 relative), plus 2^-19 of the pair's size for the fp32 chain: the norm (d/32
additions, a square root and two products, ~2^-21) and the angle (2^-25 of a turn = 2^-22.3, sine and cosine to ~2^-22)."""
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


def _check(got, ref, what):
    size = ref.abs().amax(-1, keepdim=True)
    over = ((got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - 2.0 ** -19 * size).max()
    assert float(over) <= 0, f"{what}: {float(over):.3e} beyond the bar"


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _case(n, hq, hk, d, rot, axes, adjacent, seed=0, far=1 << 17, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(qkv=_bf16(g, n, hq + 2 * hk, d, std=2.0), rot=rot, axes=axes, adjacent=adjacent)
    c["q"], c["k"], c["v"] = c["qkv"][:, :hq], c["qkv"][:, hq:hq + hk], c["qkv"][:, hq + hk:]
    c["qw"], c["kw"] = (_bf16(g, d) for _ in range(2)) if weights else (None, None)
    c["pos"] = torch.randint(0, far, (axes, n), generator=g, device="cuda", dtype=torch.int32)
    c["freq"] = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    c["axis"] = None if axes == 1 else torch.randint(0, axes, (rot // 2,), generator=g, device="cuda").to(torch.uint8)
    return c


def _expect(c, eps=1e-6):
    return (attn_plain.norm_rope(c["q"], c["qw"], c["pos"], c["freq"], c["axis"], c["rot"], c["adjacent"], eps),
            attn_plain.norm_rope(c["k"], c["kw"], c["pos"], c["freq"], c["axis"], c["rot"], c["adjacent"], eps))


@pytest.mark.parametrize("n,hq,hk,d,rot,axes,adjacent", [
    (1, 1, 1, 64, 64, 1, False), (1, 16, 4, 256, 64, 1, False), (3, 5, 1, 64, 16, 1, True),
    (64, 16, 2, 128, 128, 1, False), (65, 7, 7, 128, 64, 3, True), (33, 3, 1, 256, 256, 3, False),
    (1000, 4, 2, 64, 32, 8, True), (6000, 6, 3, 128, 112, 1, False), (17, 8, 2, 256, 0, 1, False)])
def test_heads_match_the_formula(n, hq, hk, d, rot, axes, adjacent):
    c = _case(n, hq, hk, d, rot, axes, adjacent, seed=n)
    rows = n + 9
    at = torch.randperm(rows, generator=torch.Generator().manual_seed(n))[:n].int().cuda()
    qo = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = (torch.full((rows, hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dims = gdn.make_rope_dims(c["q"], c["k"], rot, axes, rows, adjacent)
    pos, freq = (c["pos"], c["freq"]) if rot else (None, None)
    gdn.head_norm_rope(dims, c["q"], c["k"], c["v"], c["qw"], c["kw"], pos, freq, qo, ko, vo, c["axis"], at)
    gdn.check_status()
    q, k = _expect(c)
    _check(qo, q, "q")
    _check(ko[at.long()], k, "k")
    assert torch.equal(vo[at.long()], c["v"])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at.long()] = False
    assert bool((ko[rest] == 7).all()) and bool((vo[rest] == 7).all())  # rows of others are untouched


@pytest.mark.parametrize("adjacent", [False, True])
def test_far_and_negative_positions(adjacent):
    """Positions over all of int32: the angle stays exact where pos * inv_freq in fp32 would be off by whole turns."""
    c = _case(64, 4, 2, 128, 128, 2, adjacent, seed=5)
    c["pos"] = torch.randint(-2 ** 31, 2 ** 31, (2, 64), generator=torch.Generator().manual_seed(1)).int().cuda()
    c["pos"][0, 0], c["pos"][1, 1] = -2 ** 31, 2 ** 31 - 1
    qo, ko = torch.empty_like(c["q"].contiguous()), torch.empty_like(c["k"].contiguous())
    dims = gdn.make_rope_dims(c["q"], c["k"], 128, 2, adjacent=adjacent)
    gdn.head_norm_rope(dims, c["q"], c["k"], None, c["qw"], c["kw"], c["pos"], c["freq"], qo, ko, None, c["axis"])
    gdn.check_status()
    # the reference's own angle is a double of up to 2^31: 2^-22 of a radian, so twice the bar's angle term
    q, k = _expect(c)
    for got, ref in ((qo, q), (ko, k)):
        size = ref.abs().amax(-1, keepdim=True)
        assert float(((got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - 2.0 ** -18 * size).max()) <= 0


def test_no_weights_in_place_and_skipped_rows():
    c = _case(40, 4, 2, 64, 64, 1, False, seed=9, weights=False)
    q, k, v = (c[n].contiguous() for n in "qkv")
    eq, ek = _expect(c)
    dims = gdn.make_rope_dims(q, k, 64)
    gdn.head_norm_rope(dims, q, k, v, None, None, c["pos"], c["freq"], q, k, v)
    gdn.check_status()
    _check(q, eq, "q in place")
    _check(k, ek, "k in place")
    assert torch.equal(v, c["v"])
    at = torch.arange(40, dtype=torch.int32, device="cuda")
    at[::3] = -1  # not kept
    ko = torch.full((40, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    dims = gdn.make_rope_dims(c["q"], c["k"], 64)
    gdn.head_norm_rope(dims, c["q"], c["k"], c["v"], None, None, c["pos"], c["freq"], q, ko, vo, None, at)
    gdn.check_status()
    assert bool((ko[::3] == 3).all()) and bool((vo[::3] == 3).all())
    _check(ko[1::3], ek[1::3], "k kept")


def test_zero_rows_eps_and_bad_rows_are_reported():
    c = _case(8, 2, 1, 64, 64, 1, False, seed=2)
    c["qkv"].zero_()  # a zero head stays zero
    qo = torch.empty((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((10, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    at = torch.tensor([0, 1, 2, 10, -2, 5, 6, 7], dtype=torch.int32, device="cuda")
    dims = gdn.make_rope_dims(c["q"], c["k"], 64, kv_rows=10)
    gdn.head_norm_rope(dims, c["q"], c["k"], c["v"], c["qw"], c["kw"], c["pos"], c["freq"], qo, ko, vo, None, at)
    with pytest.raises(gdn.GdnError) as e:
        gdn.check_status()
    assert e.value.name == "GDN_ERR_INDEX"
    assert bool((qo == 0).all()) and bool((ko[[3, 4, 8, 9]] == 3).all()) and bool((ko[[0, 5, 7]] == 0).all())


def test_empty_call_and_other_stream():
    c = _case(64, 4, 2, 128, 64, 1, False, seed=3)
    dims = gdn.make_rope_dims(c["q"][:0], c["k"][:0], 64)
    qo, ko = torch.empty_like(c["q"].contiguous()), torch.empty_like(c["k"].contiguous())
    gdn.head_norm_rope(dims, c["q"], c["k"], None, None, None, c["pos"], c["freq"], qo, ko, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dims = gdn.make_rope_dims(c["q"], c["k"], 64)
    with torch.cuda.stream(s):
        gdn.head_norm_rope(dims, c["q"], c["k"], None, c["qw"], c["kw"], c["pos"], c["freq"], qo, ko, None)
    gdn.check_status(s)
    _check(qo, _expect(c)[0], "q")
