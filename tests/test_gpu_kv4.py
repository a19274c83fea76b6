"""gdn_kv4_store / gdn_kv4_load against the definition, bit for bit, and gdn_attn_kv4 against the 64-bit form within
kv4_plain.attend's bar."""
import math

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from tests import kv4_plain

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _same(a, b):
    return torch.equal(a.double().nan_to_num(-1e30, 1e31, -1e31), b.double().nan_to_num(-1e30, 1e31, -1e31))


@pytest.mark.parametrize("n,hk,d,k_exp,v_exp", [(1, 1, 64, 0, 0), (3, 3, 64, 1, -2), (5, 1, 128, -5, 4), (67, 8, 128, 0, 0),
                                                (130, 5, 256, 0, -1), (1000, 4, 256, 2, 2)])
@pytest.mark.parametrize("fused", [False, True])
def test_store_and_load_match_the_definition(n, hk, d, k_exp, v_exp, fused):
    """Every byte of the pool: stored rows hold the definition's codes and scales, the others what they held."""
    g = _gen(n + d)
    pages = (n + PAGE - 1) // PAGE + 3
    if fused:  # views of one projection's rows
        rows = torch.randn((n, (2 * hk + 1) * d), generator=g, device="cuda").to(torch.bfloat16)
        k, v = rows[:, :hk * d].unflatten(1, (hk, d)), rows[:, hk * d:2 * hk * d].unflatten(1, (hk, d))
    else:
        k, v = (torch.randn((n, hk, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    at = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n].int()
    if n > 2:
        at[n // 2] = -1
    old = torch.randint(0, 256, (pages, hk, 72 * d), generator=g, device="cuda", dtype=torch.uint8)
    pool = old.clone()
    dims = gdn.make_kv4_dims(k, pool, v=v, k_exp=k_exp, v_exp=v_exp)
    gdn.kv4_store(dims, k, v, at, pool)
    kept = at >= 0
    page, row = at[kept].long() // PAGE, at[kept].long() % PAGE
    for i, (x, exp) in enumerate(((k, k_exp), (v, v_exp))):
        want = kv4_plain.decode(old, i, exp)
        want[page, :, row] = kv4_plain.values(x[kept], exp)
        assert _same(kv4_plain.decode(pool, i, exp), want)
    ko, vo = (torch.full((n, hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gdn.kv4_load(gdn.make_kv4_dims(ko, pool, v=vo, k_exp=k_exp, v_exp=v_exp), pool, at, ko, vo)
    gdn.check_status()
    for got, x, exp in ((ko, k, k_exp), (vo, v, v_exp)):
        assert _same(got[kept], kv4_plain.values(x[kept], exp))
        assert bool((got[~kept] == 7.0).all())


def test_every_bf16_number_beside_every_kind_of_scale():
    """All 65536 bf16 bit patterns as a group's first channel, beside a largest channel of many sizes: ties, saturation,
    tiny and huge numbers, infinities and NaN."""
    tops = [0.0, 2.0 ** -12, 7 * 2.0 ** -9, 0.11, 1.0, 3.5, 6.9375, 7.0, 100.0, 1680.0, 5000.0, 3e38]
    every = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for t in tops:
        x = torch.zeros((65536, 16), dtype=torch.bfloat16, device="cuda")
        x[:, 0], x[:, 1] = every, t
        x = x.view(-1, 8, 128)  # 1024 tokens... of 8 heads
        n = x.shape[0]
        pool = gdn.kv4_pool(n // PAGE, 8, 128)
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        dims = gdn.make_kv4_dims(x, pool)
        gdn.kv4_store(dims, x, x, at, pool)
        got = [torch.empty_like(x) for _ in range(2)]
        gdn.kv4_load(dims, pool, at, *got)
        want = kv4_plain.values(x)
        assert _same(got[0], want) and _same(got[1], want)
    gdn.check_status()


def test_bad_rows_are_reported_and_not_kept():
    k = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pool = gdn.kv4_pool(2, 2, 64)
    dims = gdn.make_kv4_dims(k, pool)
    for bad in (-2, 128, 2 ** 31 - 1, -2 ** 31):
        pool.zero_()
        gdn.kv4_store(dims, k, k, _ints([0, bad, 5, -1]), pool)
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
        assert int((kv4_plain.decode(pool, 0) != -8 * 0.0).any(-1).sum()) == 4  # two tokens of two heads
        out = torch.full_like(k, 3.0)
        gdn.kv4_load(dims, pool, _ints([0, bad, 5, -1]), out, out.clone())
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
        assert bool((out[0] != 3).all()) and bool((out[1] == 3).all()) and bool((out[3] == 3).all())


# ------------------------------------------------------------------ attention

def _case(lens, T, hq, hk, d, seed, extra=2, k_exp=0, v_exp=0, std=1.5, garbage=True):
    """Rows of the given lengths over random pages in random order; what no row's tokens fill is garbage."""
    g = _gen(seed)
    used = [-(-n // PAGE) for n in lens]
    pages, width = sum(used) + extra, max(used + [1]) + 1
    k, v = (torch.randn((pages, PAGE, hk, d), generator=g, device="cuda") * 2.0 ** e for e in (k_exp, v_exp))
    pool = kv4_plain.encode(k.to(torch.bfloat16), v.to(torch.bfloat16), k_exp, v_exp)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -7 if garbage else 0, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    if garbage:  # behind a row's tokens: NaN scales and any codes
        for b, n in enumerate(lens):
            if n % PAGE:
                page, r = int(table[b, n // PAGE]), n % PAGE
                pool[page, :, 64 * d:68 * d].unflatten(1, (PAGE, d // 16))[:, r:] = 0x7f
                pool[page, :, 68 * d:].unflatten(1, (d // 16, PAGE))[:, :, r:] = 0xff
    q = (torch.randn((len(lens), T, hq, d), generator=g, device="cuda") * std).to(torch.bfloat16)
    return dict(q=q, pool=pool, table=table, lens=lens, k_exp=k_exp, v_exp=v_exp)


def _run(c, q_len=None, scale=None, out=None, stream=None, workspace=None):
    dims = gdn.make_attn_kv4_dims(c["q"], c["pool"], c["table"], scale=scale, k_exp=c["k_exp"], v_exp=c["v_exp"])
    out = torch.full(c["q"].shape, 5.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    gdn.attn_kv4(dims, c["q"], c["pool"], c["table"], _ints(c["lens"]), out,
                 gdn.attn_kv4_workspace(dims) if workspace is None else workspace,
                 None if q_len is None else _ints(q_len), stream)
    return out


def _compare(c, out, q_len=None, scale=None):
    B, T, hq, d = c["q"].shape
    hk = c["pool"].shape[1]
    G = hq // hk
    worst = 0.0
    for b, n in enumerate(c["lens"]):
        ql = T if q_len is None else q_len[b]
        pages = c["table"][b, :-(-n // PAGE)].long()
        sees = [max(0, min(n, n - ql + t + 1)) if t < ql else 0 for t in range(T)]
        for h in range(hk):
            k, v = (kv4_plain.decode(c["pool"][pages][:, h:h + 1], i, e).flatten(0, 2)[:n]
                    for i, e in ((0, c["k_exp"]), (1, c["v_exp"])))
            ref, bar = kv4_plain.attend(c["q"][b, :, h * G:(h + 1) * G], k, v, sees, d ** -0.5 if scale is None else scale)
            err = (out[b, :, h * G:(h + 1) * G].double() - ref).abs()
            assert bool((err <= bar).all()), f"row {b} head {h}: {float((err / bar).max())}"
            worst = max(worst, float((err / bar).max()))
    return worst


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (15, 3), (16, 2), (12, 1), (40, 2)])
def test_decode_rows_of_many_lengths(d, hq, hk):
    """Lengths of zero and one, around a page's and a tile's ends, and long ones, ragged in one call."""
    c = _case([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 2049], 1, hq, hk, d, seed=d + hq)
    out = _run(c)
    gdn.check_status()
    _compare(c, out)


@pytest.mark.parametrize("d,hq,hk,T", [(64, 6, 2, 2), (128, 8, 2, 8), (256, 8, 2, 3), (128, 5, 1, 7), (256, 16, 4, 8),
                                       (64, 2, 2, 64), (128, 64, 1, 2), (256, 9, 1, 5), (128, 64, 1, 64)])
def test_verify_rows(d, hq, hk, T):
    """T tokens a row, causal among themselves; rows shorter than T, real lengths from 0 to T."""
    lens = [1, T - 1, T, T + 1, 64, 64 + T, 130, 700]
    c = _case(lens, T, hq, hk, d, seed=T + d)
    out = _run(c)
    gdn.check_status()
    _compare(c, out)
    q_len = [0, 1, T // 2, T, T - 1, 1, T, 0]
    out = _run(c, q_len)
    gdn.check_status()
    _compare(c, out, q_len)


def test_one_long_row_and_many_short_ones():
    for lens, hq, hk, d in (([40000], 8, 2, 128), ([20001], 4, 1, 256), ([3] * 700, 4, 2, 64),
                            ([9000] + [1] * 40 + [5000, 0, 0, 64], 8, 4, 128)):
        c = _case(lens, 1, hq, hk, d, seed=len(lens))
        out = _run(c)
        gdn.check_status()
        _compare(c, out)


def test_scales_exponents_and_sizes_of_queries():
    """Pools with exponents, negative and large scales, queries of any size, a query of zeros."""
    for k_exp, v_exp, scale, std in ((3, -4, None, 1.0), (-10, 12, None, 200.0), (0, 0, -0.3, 1.0), (0, 0, 3.0, 2.0),
                                     (0, 0, 0.0, 1.0), (0, 0, None, 1e-20), (-32, 0, 1e-3, 1e12)):
        c = _case([70, 400, 1], 2, 6, 2, 128, seed=11, k_exp=k_exp, v_exp=v_exp, std=std)
        c["q"][1, 0, 2] = 0
        c["q"][0, 0, 1, 7] *= 300  # one channel far above the others
        out = _run(c, scale=scale)
        gdn.check_status()
        _compare(c, out, scale=scale)


def test_scores_that_climb_along_the_row():
    """Keys ordered so that the running maximum rises (and falls) again and again over the row."""
    for order in (1, -1):
        c = _case([2500], 1, 4, 1, 128, seed=3, garbage=False)
        c["q"][:] = 1.0
        ramp = torch.linspace(0.02, 4.0, 2560, device="cuda")[::order] if order > 0 else torch.linspace(4.0, 0.02, 2560, device="cuda")
        n = c["pool"].shape[0]
        k = torch.randn((n * PAGE, 1, 128), generator=_gen(5), device="cuda") * 0.2
        place = torch.zeros(n * PAGE, device="cuda")
        for i, p in enumerate(c["table"][0, :40].tolist()):
            place[p * PAGE:(p + 1) * PAGE] = ramp[i * PAGE:(i + 1) * PAGE]
        k = (k + place[:, None, None]).to(torch.bfloat16).view(n, PAGE, 1, 128)
        v = torch.randn((n, PAGE, 1, 128), generator=_gen(6), device="cuda").to(torch.bfloat16)
        c["pool"] = kv4_plain.encode(k, v)
        for scale in (0.088, 1.0):
            out = _run(c, scale=scale)
            gdn.check_status()
            _compare(c, out, scale=scale)


def test_rows_share_pages_and_strided_queries():
    c = _case([200, 200, 330], 1, 6, 2, 128, seed=8)
    c["table"][1, :3] = c["table"][0, :3]
    c["table"][2, :2] = c["table"][0, :2]
    wide = torch.randn((3, 1, 10 * 128), generator=_gen(9), device="cuda").to(torch.bfloat16)
    c["q"] = wide[:, :, 128 * 2:128 * 8].unflatten(2, (6, 128))
    out = _run(c, out=torch.empty((3, 1, 6, 128), dtype=torch.bfloat16, device="cuda"))
    gdn.check_status()
    _compare(c, out)


def test_bad_rows_are_skipped_and_reported():
    """A length or page outside its range: that row's outputs stay, the others are right."""
    for what in ("long", "negative", "page", "low page", "q_len"):
        c = _case([100, 500, 70, 1000], 2, 4, 2, 128, seed=4, garbage=False)
        q_len = None
        lens = list(c["lens"])
        if what == "long":
            c["lens"][1] = c["table"].shape[1] * PAGE + 1
        elif what == "negative":
            c["lens"][1] = -1
        elif what == "q_len":
            q_len = [2, 3, 2, 2]
        else:
            c["table"][1, 3] = c["pool"].shape[0] if what == "page" else -1
        out = _run(c, q_len)
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
        assert bool((out[1] == 5.0).all())
        for b in (0, 2, 3):
            one = dict(c, q=c["q"][b:b + 1], table=c["table"][b:b + 1], lens=lens[b:b + 1])
            _compare(one, out[b:b + 1])


def test_nan_in_a_row_reaches_that_row_only():
    c = _case([130, 130, 64], 1, 4, 2, 64, seed=6, garbage=False)
    page = int(c["table"][1, 0])
    c["pool"][page, 0, 64 * 64] = 0x7f  # a key's scale of head 0
    out = _run(c)
    gdn.check_status()
    assert bool(out[1, :, :2].isnan().all()) and not bool(out[1, :, 2:].isnan().any())
    _compare(dict(c, q=c["q"][::2], table=c["table"][::2].contiguous(), lens=[130, 64]), out[::2])
    c["q"][2, 0, 3, 5] = math.nan
    out = _run(c)
    assert bool(out[2, :, 3].isnan().all()) and not bool(out[2, :, :3].isnan().any())


def test_results_repeat_on_streams_and_in_graphs():
    """The same bits again, on another stream, and from a replayed graph with other lengths in the same buffers."""
    c = _case([900, 64, 3000, 1], 1, 8, 2, 128, seed=12)
    ref = _run(c)
    dims = gdn.make_attn_kv4_dims(c["q"], c["pool"], c["table"])
    lens, out, ws = _ints(c["lens"]), torch.empty_like(ref), gdn.attn_kv4_workspace(dims)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        ws.random_(0, 256)  # a call expects nothing of it
        torch.cuda.synchronize()
        gdn.attn_kv4(dims, c["q"], c["pool"], c["table"], lens, out, ws, stream=side)
        side.synchronize()
        assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.attn_kv4(dims, c["q"], c["pool"], c["table"], lens, out, ws)
    for now in ([900, 64, 3000, 1], [5, 0, 2999, 1], [0, 0, 0, 0]):
        lens.copy_(_ints(now))
        ws.random_(0, 256)
        out.fill_(9.0)
        graph.replay()
        gdn.check_status()
        _compare(dict(c, lens=now), out)
