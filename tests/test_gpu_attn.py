"""gdn_attn_prefill and gdn_attn_shared_prefix against the 64-bit form: head sizes and groupings, ragged and empty
sequences, continued prompts, queries that see no key, whatever lies outside a sequence's keys, strides, streams, pools
past 32-bit offsets, bad extents.

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


def _check(got, ref, bar, what):
    over = ((got.double() - ref).abs() - bar).max() if ref.numel() else torch.tensor(0.0)
    assert float(over) <= 0, f"{what}: {float(over):.3e} beyond the bar"


def _pool(g, rows, hk, d, extents, stride=None, trap=float("nan")):
    """Two pools whose rows outside `extents` hold `trap`."""
    pools = []
    for _ in range(2):
        x = torch.full((rows, stride or hk * d), trap, dtype=torch.bfloat16, device="cuda")
        x = x[:, :hk * d].view(rows, hk, d) if stride is None else x.as_strided((rows, hk, d), (stride, d, 1))
        for s, n in extents:
            x[s:s + n] = _bf16(g, n, hk, d)
        pools.append(x)
    return pools


# ------------------------------------------------------------------ prompts

def _prefill(lens, kv, hq, hk, d, seed=0, gap=3, stride=None, std=1.5, trap=float("nan"), q_pad=0, scale=None,
             stream=None):
    """lens: queries of each sequence; kv: keys of each. Keys lie `gap` rows apart, the rows between hold `trap`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens)
    rows = torch.full((n, hq * d + q_pad), trap, dtype=torch.bfloat16, device="cuda")
    rows[:, :hq * d] = _bf16(g, n, hq * d, std=std)
    q = rows.as_strided((n, hq, d), (hq * d + q_pad, d, 1))
    start, at = [], gap
    for m in kv:
        start.append(at)
        at += m + gap
    k, v = _pool(g, at, hk, d, list(zip(start, kv)), stride, trap)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    out = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dims = gdn.make_attn_dims(q, k, B=len(lens), scale=scale)
    gdn.attn_prefill(dims, q, k, v, _ints(cu), out, _ints(start), _ints(kv), stream)
    gdn.check_status(stream)
    return q, k, v, cu, start, out


def _check_prefill(q, k, v, cu, start, kv, out, scale=None):
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    G = hq // hk
    for b, (s, m) in enumerate(zip(start, kv)):
        n = cu[b + 1] - cu[b]
        for h in range(hk):
            ref, bar = attn_plain.attend(q[cu[b]:cu[b + 1], h * G:(h + 1) * G], k[s:s + m, h], v[s:s + m, h],
                                         [max(0, m - n + i + 1) for i in range(n)], scale or d ** -0.5)
            _check(out[cu[b]:cu[b + 1], h * G:(h + 1) * G], ref, bar, f"sequence {b}, key head {h}")


@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (8, 2, 64), (15, 3, 64), (4, 4, 128), (8, 1, 128), (14, 2, 128),
                                     (4, 2, 256), (5, 1, 256), (16, 2, 256), (64, 1, 64), (33, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 5], [127, 128, 129], [300, 64, 17, 1, 511]])
def test_prompts(hq, hk, d, lens):
    q, k, v, cu, start, out = _prefill(lens, lens, hq, hk, d, seed=hq + len(lens))
    _check_prefill(q, k, v, cu, start, lens, out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,kv", [([1, 3, 200], [1000, 129, 712]), ([64, 0, 5], [64 + 256, 300, 5]),
                                     ([130, 7], [128, 3]), ([0, 0], [5, 0]), ([9, 4], [0, 4])])
def test_continued_empty_and_keyless(d, lens, kv):
    """Prompts that continue cached keys, empty sequences, and fewer keys than queries (the first queries see none)."""
    q, k, v, cu, start, out = _prefill(lens, kv, 6, 2, d, seed=d)
    _check_prefill(q, k, v, cu, start, kv, out)
    for b, (n, m) in enumerate(zip(lens, kv)):
        assert bool((out[cu[b]:cu[b] + max(0, n - m)] == 0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("trap", [float("nan"), float("inf"), -3.0e38])
def test_values_outside_a_sequence_do_not_matter(d, trap):
    q, k, v, cu, start, out = _prefill([100, 33], [100, 261], 4, 2, d, seed=1, trap=trap, gap=150)
    q2, *_, out2 = _prefill([100, 33], [100, 261], 4, 2, d, seed=1, trap=0.5, gap=150)
    assert torch.equal(q, q2) and torch.equal(out, out2)
    _check_prefill(q, k, v, cu, start, [100, 261], out)


@pytest.mark.parametrize("d,std", [(64, 8.0), (128, 6.0), (256, 20.0)])
def test_peaked_and_growing_scores(d, std):
    """Scores whose maximum keeps growing along the keys, over hundreds: the running maximum has to follow."""
    g = torch.Generator(device="cuda").manual_seed(d)
    n = 700
    q, v = _bf16(g, n, 2, d, std=std), _bf16(g, n, 1, d)
    k = (_bf16(g, n, 1, d).float() * torch.linspace(0.1, 3.0, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    k = (k.float() + 0.5 * q[:, :1].float() * torch.linspace(0, 1, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    out = torch.empty_like(q)
    gdn.attn_prefill(gdn.make_attn_dims(q, k, B=1), q, k, v, _ints([0, n]), out)
    gdn.check_status()
    _check_prefill(q, k, v, [0, n], [0], [n], out)


def test_packed_tokens_without_extents_strides_and_scale():
    """kv_start / kv_len absent: the pools hold the packed tokens; q, k, v are views of one projection's rows; the
    scale is negative, zero, or large."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, hq, hk, d = 333, 6, 2, 128
    qkv = _bf16(g, n, (hq + 2 * hk) * d + 8)
    st = qkv.stride(0)
    q, k, v = (qkv.as_strided((n, h, d), (st, d, 1), o * d) for h, o in ((hq, 0), (hk, hq), (hk, hq + hk)))
    cu = [0, 100, 101, 333]
    for scale in (-0.1, 0.0, 1.0):
        out = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
        gdn.attn_prefill(gdn.make_attn_dims(q, k, B=3, scale=scale), q, k, v, _ints(cu), out)
        gdn.check_status()
        for b in range(3):
            for h in range(hk):
                m = cu[b + 1] - cu[b]
                ref, bar = attn_plain.attend(q[cu[b]:cu[b + 1], 3 * h:3 * h + 3], k[cu[b]:cu[b + 1], h],
                                             v[cu[b]:cu[b + 1], h], list(range(1, m + 1)), scale)
                _check(out[cu[b]:cu[b + 1], 3 * h:3 * h + 3], ref, bar, f"scale {scale}, sequence {b}")


def test_pool_past_32_bit_offsets():
    """A pool whose last rows lie more than 2^31 elements in."""
    q, k, v, cu, start, out = _prefill([70], [300], 4, 2, 64, seed=2, gap=2 ** 15, stride=2 ** 16 + 8, trap=0.0)
    assert (start[0] + 300) * k.stride(0) > 2 ** 31
    _check_prefill(q, k, v, cu, start, [300], out)


def test_long_prompt_many_heads_other_stream_and_repeat():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q, k, v, cu, start, out = _prefill([2500], [2500], 16, 4, 128, seed=5, stream=s)
        again = torch.empty_like(out)
        gdn.attn_prefill(gdn.make_attn_dims(q, k, B=1), q, k, v, _ints(cu), again, _ints(start), _ints([2500]))
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    _check_prefill(q, k, v, cu, start, [2500], out)


def test_bad_extents_are_reported_and_skipped():
    g = torch.Generator(device="cuda").manual_seed(4)
    q, (k, v) = _bf16(g, 40, 4, 64), _pool(g, 50, 2, 64, [(0, 50)])
    out = torch.full_like(q, 7.0)
    dims = gdn.make_attn_dims(q, k, B=4)
    gdn.attn_prefill(dims, q, k, v, _ints([0, 10, 20, 30, 40]), out, _ints([0, 45, -1, 30]), _ints([10, 10, 10, -2]))
    with pytest.raises(gdn.GdnError) as e:
        gdn.check_status()
    assert e.value.name == "GDN_ERR_INDEX"
    assert bool((out[10:] == 7).all())
    _check_prefill(q, k, v, [0, 10], [0], [10], out)
    out.fill_(7.0)
    for cu in ([0, 10, 5, 30, 40], [0, 10, 20, 30, 41], [-3, 10, 20, 30, 40]):  # the ranges of queries
        gdn.attn_prefill(dims, q, k, v, _ints(cu), out, _ints([0, 10, 20, 30]), _ints([10, 10, 10, 10]))
        with pytest.raises(gdn.GdnError) as e:
            gdn.check_status()
        assert e.value.name == "GDN_ERR_INDEX"


# ------------------------------------------------------------ shared prefixes

def _shared(first, prefix, suffix, T, hq, hk, d, seed=0, q_len=None, gap=3, stride=None, trap=float("nan"), std=1.5,
            ws=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(suffix)
    extents, at = [], gap
    for n in list(prefix) + list(suffix):
        extents.append((at, n))
        at += n + gap
    k, v = _pool(g, at, hk, d, extents, stride, trap)
    q = _bf16(g, B, T, hq, d, std=std)
    out = torch.full_like(q, 7.0)
    ng = len(prefix)
    dims = gdn.make_attn_dims(q, k, B=B, T=T, n_groups=ng)
    ws = gdn.attn_workspace(dims) if ws is None else ws
    ps, ss = [s for s, _ in extents[:ng]], [s for s, _ in extents[ng:]]
    args = (_ints(first), _ints(ps), _ints(prefix)) if ng else (None, None, None)
    ql = None if q_len is None else _ints(q_len)
    gdn.attn_shared_prefix(dims, q, k, v, *args, _ints(ss), _ints(suffix), out, ws, ql)
    gdn.check_status()
    again = torch.full_like(q, 7.0)
    gdn.attn_shared_prefix(dims, q, k, v, *args, _ints(ss), _ints(suffix), again, ws, ql)
    assert torch.equal(out, again)
    G = hq // hk
    for b in range(B):
        grp = [i for i in range(ng) if first[i] <= b < first[i + 1]]
        p0, p = (ps[grp[0]], prefix[grp[0]]) if grp else (0, 0)
        real = T if q_len is None else q_len[b]
        rows = torch.cat((torch.arange(p0, p0 + p), torch.arange(ss[b], ss[b] + suffix[b]))).cuda()
        sees = [p + max(0, suffix[b] - real + t + 1) for t in range(real)]
        for h in range(hk):
            ref, bar = attn_plain.attend(q[b, :real, h * G:(h + 1) * G], k[rows, h], v[rows, h], sees, d ** -0.5)
            _check(out[b, :real, h * G:(h + 1) * G], ref, bar, f"row {b}, key head {h}")
        assert bool((out[b, real:] == 0).all())
    return out


@pytest.mark.parametrize("hq,hk,d", [(2, 2, 64), (15, 3, 64), (8, 2, 128), (7, 1, 128), (16, 4, 256), (40, 1, 256)])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_rows_over_one_prefix(hq, hk, d, T):
    _shared([0, 8], [777], [T, T + 1, T + 130, T, 40 + T, 300, T, 129], T, hq, hk, d, seed=T)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_ragged_groups(d):
    """Empty groups, empty prefixes, a group of one row, suffixes of one key, a long prefix with few rows."""
    _shared([0, 3, 3, 4, 9, 11], [1, 500, 0, 129, 3001], [1, 2, 3, 1, 260, 1, 7, 128, 129, 1, 5], 1, 6, 2, d, seed=d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_no_groups_and_padded_rows(d):
    """Rows without prefixes; rows with fewer real tokens than T, among them none; suffixes shorter than their tokens."""
    _shared([], [], [40, 1, 300, 3], 2, 4, 2, d, seed=1)
    _shared([0, 2, 6], [70, 0], [3, 9, 5, 2, 0, 1], 4, 4, 2, d, seed=2, q_len=[3, 0, 4, 4, 2, 1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_long_prefix(d):
    """Enough rows to fill several query tiles and enough keys to split them over the GPU."""
    _shared([0, 70], [5003], [1 + (37 * i) % 400 for i in range(70)], 1, 8, 1, d, seed=7)


def test_verify_of_64_tokens_and_peaked_scores():
    _shared([0, 3], [400], [64, 100, 65], 64, 12, 2, 128, seed=8, std=8.0)


@pytest.mark.parametrize("rows", [1, 300])
def test_one_row_and_many(rows):
    _shared([0, rows], [640], [1 + i % 90 for i in range(rows)], 1, 4, 2, 64, seed=9)


def test_shared_pool_past_32_bit_offsets():
    _shared([0, 2], [200], [5, 9], 1, 4, 2, 64, seed=10, gap=2 ** 14, stride=2 ** 16 + 8, trap=0.0)


def test_bad_groups_and_rows_are_reported_and_skipped():
    g = torch.Generator(device="cuda").manual_seed(11)
    q, (k, v) = _bf16(g, 4, 1, 4, 64), _pool(g, 60, 2, 64, [(0, 60)])
    dims = gdn.make_attn_dims(q, k, B=4, T=1, n_groups=2)
    ws = gdn.attn_workspace(dims)

    def run(first=(0, 2, 4), ps=(0, 10), pl=(10, 10), ss=(20, 30, 40, 50), sl=(5, 5, 5, 5), ql=(1, 1, 1, 1)):
        out = torch.full_like(q, 7.0)
        gdn.attn_shared_prefix(dims, q, k, v, _ints(first), _ints(ps), _ints(pl), _ints(ss), _ints(sl), out, ws,
                               _ints(ql))
        with pytest.raises(gdn.GdnError) as e:
            gdn.check_status()
        assert e.value.name == "GDN_ERR_INDEX"
        return [bool((out[b] == 7).all()) for b in range(4)]

    assert run(ps=(0, 51)) == [False, False, True, True]
    assert run(pl=(-1, 10)) == [True, True, False, False]
    assert run(ss=(20, 56, 40, 50)) == [False, True, False, False]
    assert run(sl=(5, 5, -1, 5)) == [False, False, True, False]
    assert run(ql=(1, 1, 1, 2)) == [False, False, False, True]
    assert run(first=(0, 2, 5)) == [True] * 4
    assert run(first=(1, 2, 4)) == [True] * 4


def test_captured_step_follows_its_device_lengths():
    """A captured step replayed with other lengths on the device."""
    g = torch.Generator(device="cuda").manual_seed(12)
    B, hq, hk, d = 3, 4, 2, 128
    q, (k, v) = _bf16(g, B, 1, hq, d), _pool(g, 2000, hk, d, [(0, 2000)])
    first, ps, pl = _ints([0, B]), _ints([0]), _ints([900])
    ss, sl = _ints([1000, 1300, 1600]), _ints([1, 2, 3])
    out = torch.empty_like(q)
    dims = gdn.make_attn_dims(q, k, B=B, T=1, n_groups=1)
    ws = gdn.attn_workspace(dims)
    step = lambda: gdn.attn_shared_prefix(dims, q, k, v, first, ps, pl, ss, sl, out, ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for p, own in ((900, [7, 250, 40]), (1, [300, 1, 200])):
        pl.fill_(p)
        sl.copy_(_ints(own))
        graph.replay()
        got = out.clone()
        step()
        gdn.check_status()
        assert torch.equal(got, out)
        ref, bar = attn_plain.attend(q[1, :, :2], torch.cat((k[:p, 0], k[1300:1300 + own[1], 0])),
                                     torch.cat((v[:p, 0], v[1300:1300 + own[1], 0])), [p + own[1]], d ** -0.5)
        _check(got[1, :, :2], ref, bar, "row 1")
