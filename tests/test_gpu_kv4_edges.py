"""The paged 4-bit cache, its attention, beam selection and forking where they may be called in ways the other tests do
not: pools beyond 4 GiB, lines of the page table that are full, thousands of rows, one workspace for calls of several
sizes, two streams at once, unaligned strides, the largest pools and vocabularies, candidates without end."""
import math

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from tests import kv4_plain
from tests.test_gpu_beam import _check, _check_fork, _fork, _logits, _select
from tests.test_gpu_kv4 import _case, _compare, _gen, _ints, _run, _same

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


def test_pools_beyond_4_gib():
    """Tokens in the last pages of a 5.3 GB pool: stored, read by attention, loaded, copied as slots."""
    pages, hk, d, n = 72000, 8, 128, 200
    pool = gdn.kv4_pool(pages, hk, d)
    g = _gen(1)
    k, v = (torch.randn((n, hk, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = _ints([[pages - 1, pages - 5, 3, pages - 2]])
    place = torch.arange(n, device="cuda")
    at = (table[0, place // PAGE] * PAGE + (place % PAGE).int()).contiguous()
    dims = gdn.make_kv4_dims(k, pool)
    gdn.kv4_store(dims, k, v, at, pool)
    q = torch.randn((1, 1, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    c = dict(q=q, pool=pool, table=table, lens=[n], k_exp=0, v_exp=0)
    out = _run(c)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.kv4_load(dims, pool, at, ko, vo)
    gdn.check_status()
    assert _same(ko, kv4_plain.values(k)) and _same(vo, kv4_plain.values(v))
    _compare(c, out)
    moved = _ints([[pages - 7, pages - 5, 3, pages - 2]])
    gdn.slots_copy([(pool[None], _ints([pages - 1]), _ints([pages - 7]))])
    gdn.check_status()
    assert torch.equal(_run(dict(c, table=moved)), out)


def test_a_full_line_of_the_page_table():
    for d, T in ((64, 1), (128, 4), (256, 1)):
        c = _case([256, 255, 193, 64], T, 4, 2, d, seed=2, garbage=False)
        c["table"] = c["table"][:, :4].contiguous()
        _compare(c, _run(c))
        gdn.check_status()


@pytest.mark.parametrize("rows,T", [(5000, 1), (1500, 3)])
def test_thousands_of_rows(rows, T):
    lens = [(7 * i) % 70 for i in range(rows)]
    c = _case(lens, T, 4, 2, 64, seed=5)
    out = _run(c)
    gdn.check_status()
    pick = list(range(0, 90)) + list(range(rows - 90, rows))
    _compare(dict(c, q=c["q"][pick], table=c["table"][pick].contiguous(), lens=[lens[i] for i in pick]), out[pick])
    assert bool((out[[i for i, n in enumerate(lens) if n == 0]] == 0).all())


def test_one_workspace_for_calls_of_several_sizes_and_streams():
    """Calls of other sizes follow one another in one workspace; two streams run at once, each with its own."""
    cases = [_case([3000, 5, 700], 1, 8, 2, 128, seed=1), _case([900, 64], 8, 16, 2, 256, seed=2),
             _case([5000], 1, 4, 1, 64, seed=3), _case([800, 800, 30, 0], 4, 6, 2, 128, seed=4)]
    size = max(gdn.attn_kv4_workspace(gdn.make_attn_kv4_dims(c["q"], c["pool"], c["table"])).numel() for c in cases)
    work = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [_run(c) for c in cases]
    for c, w in zip(cases, want):
        _compare(c, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(w) for w in want] for _ in streams]
    lens = [_ints(c["lens"]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(cases):
            for s, ws, o in zip(streams, work, outs):
                dims = gdn.make_attn_kv4_dims(c["q"], c["pool"], c["table"])
                gdn.attn_kv4(dims, c["q"], c["pool"], c["table"], lens[i], o[i], ws, stream=s)
    torch.cuda.synchronize()
    gdn.check_status()
    for o in outs:
        for a, b in zip(o, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("pad", [8, 24])
def test_strides_that_allow_no_wide_accesses(pad):
    for d in (64, 128, 256):
        rows = torch.randn((130, 4 * d + pad), generator=_gen(pad), device="cuda").to(torch.bfloat16)
        k, v = rows[:, 8:8 + 2 * d].unflatten(1, (2, d)), rows[:, 8 + 2 * d:8 + 4 * d].unflatten(1, (2, d)) if pad > 8 else None
        if v is None:
            v = rows[:, 8 + 2 * d:8 + 4 * d].unflatten(1, (2, d))
        pool = gdn.kv4_pool(4, 2, d)
        at = torch.randperm(256, generator=_gen(1), device="cuda")[:130].int()
        dims = gdn.make_kv4_dims(k, pool, v=v)
        gdn.kv4_store(dims, k, v, at, pool)
        back = torch.zeros_like(rows)
        ko, vo = back[:, 8:8 + 2 * d].unflatten(1, (2, d)), back[:, 8 + 2 * d:8 + 4 * d].unflatten(1, (2, d))
        gdn.kv4_load(gdn.make_kv4_dims(ko, pool, v=vo), pool, at, ko, vo)
        gdn.check_status()
        assert _same(ko, kv4_plain.values(k)) and _same(vo, kv4_plain.values(v))
        assert bool((back[:, :8] == 0).all()) and bool((back[:, 8 + 4 * d:] == 0).all())


def test_layers_share_nothing_and_other_heads_stay():
    """A store touches its own tokens of its own layer's pool only."""
    pool = torch.randint(0, 256, (3, 4, 2, 72 * 64), generator=_gen(4), device="cuda", dtype=torch.uint8)
    old = pool.clone()
    k = torch.randn((5, 2, 64), generator=_gen(5), device="cuda").to(torch.bfloat16)
    gdn.kv4_store(gdn.make_kv4_dims(k, pool[1]), k, k, _ints([0, 70, 71, 255, 130]), pool[1])
    gdn.check_status()
    assert torch.equal(pool[0], old[0]) and torch.equal(pool[2], old[2])
    keep = torch.ones(256, dtype=torch.bool, device="cuda")
    keep[[0, 70, 71, 255, 130]] = False
    for i in range(2):
        a, b = (kv4_plain.decode(x[1], i).transpose(1, 2).flatten(0, 1)[keep] for x in (pool, old))
        assert _same(a, b)


# ------------------------------------------------------------------ selection, forking

@pytest.mark.parametrize("G,W,V,half", [(16, 32, 30011, False), (60, 8, 40000, True), (1, 1, 1 << 24, False),
                                        (1, 3, 1 << 22, True), (300, 1, 999, False)])
def test_selection_of_many_rows_and_vocabularies(G, W, V, half):
    logits, scores, _ = _logits(G, W, V, half, seed=G + W)
    got = _select(logits, scores)
    if G > 4:  # the host's form of a few groups
        pick = [0, G // 2, G - 1]
        got = [None if t is None else t[pick] for t in got]
        got[0] = got[0] - torch.tensor([[(p - i) * W] for i, p in enumerate(pick)], device="cuda")
        logits, scores = logits[pick], scores[pick]
    _check(logits, scores, None, -1, got)


def test_candidates_without_end():
    """Rows of equal logits in 32 beams (more finalists than are ranked at once), all beams finished, one candidate each."""
    x = torch.zeros((2, 32, 9000), device="cuda")
    scores = torch.full((2, 32), -3.0, device="cuda")
    _check(x, scores, None, -1, _select(x, scores))
    x[:, 5, 8000] = 1e-3
    _check(x, scores, None, -1, _select(x, scores))
    done = torch.ones((2, 32), dtype=torch.uint8, device="cuda")
    scores = -torch.arange(64, device="cuda").view(2, 32).float()
    _check(x, scores, done, 17, _select(x, scores, done, 17))
    x = torch.full((1, 4, 50000), -math.inf, device="cuda")
    for w in range(4):
        x[0, w, 12345 * w + 7] = float(w)
    scores = torch.full((1, 4), -1.0, device="cuda")
    _check(x, scores, None, -1, _select(x, scores))
    low = torch.full((1, 2, 30000), -3e38, device="cuda")  # far logits whose differences overflow
    low[0, :, 29999] = 3e38
    _check(low, scores[:, :2], None, -1, _select(low, scores[:, :2].contiguous()))


def test_large_sums_between_beams():
    """Scores and logits whose sums cancel: what fp32 may be off by decides nothing."""
    g = _gen(9)
    x = 1e6 + torch.randn((3, 4, 5000), generator=g, device="cuda").double()
    logits = x.float()
    scores = torch.randn((3, 4), generator=g, device="cuda") * 1e-3 - 1e5
    parent, token, new, _ = _select(logits, scores)
    for b in range(3):
        p, t, s, _, bar = kv4_plain.beam(logits[b].cpu(), scores[b].cpu(), None, -1)
        lse = torch.logsumexp(logits[b].double(), -1)
        own = [float(scores[b, w].double() + (logits[b, w, c].double() - lse[w]))
               for w, c in zip((parent[b] - 4 * b).tolist(), token[b].tolist())]
        assert own == sorted(own, reverse=True) or max(abs(u - v) for u, v in zip(own, sorted(own, reverse=True))) <= 2 * bar
        for u, v in zip(own, s):  # each place's score is the exact one's but for the sums' error
            assert abs(u - v) <= 2 * bar


def test_fork_of_the_largest_pools_and_wide_tables():
    table, lens = [[5, (1 << 20) - 1], [7, 9]], [100, 64]
    kw = dict(parent=[0, 0], state=[1, 0])
    pinned = [1] * (1 << 20)
    pinned[(1 << 20) - 7] = pinned[12345] = pinned[600000] = 0
    want = kv4_plain.fork(table, lens, 1 << 20, 20, pinned=pinned, **kw)
    _check_fork(_fork(table, lens, 1 << 20, 20, pinned=pinned, **kw), want)
    assert not want["full"]
    gdn.check_status()
    # a prompt of many pages, beyond those that shared memory lists
    width = 3000
    table = [[-1] * width, [0] + [-1] * (width - 1)]
    want = kv4_plain.fork(table, [0, 10], 6000, 160000, n_new=[160000, 1000])
    _check_fork(_fork(table, [0, 10], 6000, 160000, n_new=[160000, 1000]), want)
    gdn.check_status()
