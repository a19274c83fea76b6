"""gdn_beam_select, gdn_cache_fork and gdn_slots_copy against their plain forms on the host."""
import math
import random

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


# ------------------------------------------------------------------ selection

def _select(logits, scores, done=None, eos=-1, stream=None, in_place=False):
    G, W, _ = logits.shape
    parent, token = (torch.full((G, W), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    new = scores if in_place else torch.full((G, W), 3.0, device="cuda")
    over = None if done is None else done if in_place else torch.full((G, W), 7, dtype=torch.uint8, device="cuda")
    gdn.beam_select(logits, scores, parent, token, new, gdn.beam_workspace(logits), done=done, new_done=over, eos=eos,
                    stream=stream)
    return parent, token, new, over


def _check(logits, scores, done, eos, got):
    G, W, _ = logits.shape
    parent, token, new, over = (None if t is None else t.cpu() for t in got)
    for g in range(G):
        p, t, s, o, bar = kv4_plain.beam(logits[g].cpu(), scores[g].cpu(), None if done is None else done[g].cpu(), eos)
        assert (parent[g] - g * W).tolist() == p, f"group {g}"
        assert token[g].tolist() == t, f"group {g}"
        for a, b in zip(new[g].tolist(), s):
            assert a == b or abs(a - b) <= 2.0 ** -24 * abs(b) + bar
        if over is not None:
            assert over[g].tolist() == o


def _logits(G, W, V, half, seed, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = std * torch.randn((G, W, V), generator=g, device="cuda")
    scores = -10 - 3 * torch.rand((G, W), generator=g, device="cuda")
    return (x.to(torch.bfloat16) if half else x), scores, g


@pytest.mark.parametrize("G,W,V", [(1, 1, 1), (2, 1, 7), (1, 4, 3), (3, 2, 100), (1, 5, 1000), (4, 4, 2047), (2, 8, 8193),
                                   (5, 3, 32001), (1, 32, 4099), (2, 16, 131072), (20, 8, 5000), (1, 1, 1000003)])
@pytest.mark.parametrize("half", [False, True])
def test_selection_matches_exact_arithmetic(G, W, V, half):
    logits, scores, g = _logits(G, W, V, half, seed=V + W)
    _check(logits, scores, None, -1, _select(logits, scores))
    eos = V // 2
    logits[:, :, eos] = logits.amax(-1)  # eos is likely
    done = (torch.rand((G, W), generator=g, device="cuda") < 0.3).to(torch.uint8)
    _check(logits, scores, done, eos, _select(logits, scores, done, eos))
    if W > 1:  # the first step: one beam
        scores[:, 1:] = -math.inf
        _check(logits, scores, None, eos, _select(logits, scores, None, eos))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_ties_go_to_the_lowest_place(V, half):
    """Equal logits in any number, equal beams, whole rows of one number."""
    dtype = torch.bfloat16 if half else torch.float32
    for kind in range(6):
        x = torch.zeros((2, 6, V), dtype=dtype, device="cuda")
        scores = torch.full((2, 6), -2.0, device="cuda")
        if kind == 1:
            x[:, :, V // 3:V // 2] = 1.0
        elif kind == 2:
            x[:, 3, V - 1] = 4.0
            x[:, 2, V - 2] = 4.0
        elif kind == 3:
            x[:, :, ::7] = -math.inf
            scores[:, 4] = -1.0
        elif kind == 4:  # a few values only
            x = torch.randint(0, 3, x.shape, generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").to(dtype)
        elif kind == 5:  # zeros of both signs are equal
            x[:, :, 1::2] = -0.0
            x[:, ::2, :V // 2] = -0.0
        _check(x, scores, None, -1, _select(x, scores))


def test_rows_without_candidates():
    """Masked, infinite and NaN logits, beams that are not there, fewer candidates than beams, all beams finished."""
    x, scores, _ = _logits(6, 4, 300, False, seed=2)
    x[0, 1] = -math.inf                      # a masked row
    x[1, 0, 5], x[1, 2, 7] = math.nan, math.inf
    x[2] = -math.inf
    x[2, 3, 9], x[2, 3, 4] = 0.5, 0.25       # two candidates in all
    scores[3] = -math.inf
    scores[4, :2] = math.nan
    x[5] = torch.finfo(torch.float32).min    # masks of the type's lowest value
    x[5, :, 17] = 0.0
    got = _select(x, scores)
    _check(x, scores, None, -1, got)
    assert got[1][2].tolist() == [9, 4, -1, -1] and got[0][2].tolist() == [11, 11, 10, 11]
    assert got[1][3].tolist() == [-1] * 4 and got[0][3].tolist() == [12, 13, 14, 15]
    done = torch.ones((6, 4), dtype=torch.uint8, device="cuda")
    done[0, 0] = 0
    got = _select(x, scores, done, 299)
    _check(x, scores, done, 299, got)
    low = torch.full((1, 2, 9000), -1000.0, device="cuda")  # slices far below zero, and one without anything
    low[0, :, :5000] = -math.inf
    sc = torch.tensor([[-1.0, -2.0]], device="cuda")
    _check(low, sc, None, -1, _select(low, sc))


def test_strided_rows_in_place_streams_and_graphs():
    G, W, V = 3, 4, 5003
    for half in (False, True):
        wide, scores, _ = _logits(G, W, V + 13, half, seed=9)
        for off in (0, 1, 5):  # rows at any address
            x = wide[..., off:off + V]
            _check(x, scores, None, -1, _select(x, scores))
        x = wide[..., :V]
        done = torch.zeros((G, W), dtype=torch.uint8, device="cuda")
        done[1, 2] = 1
        ref = _select(x, scores, done, 3)
        sc, dn = scores.clone(), done.clone()
        for a, b in zip(_select(x, sc, dn, 3, in_place=True), ref):
            assert torch.equal(a, b)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = _select(x, scores, done, 3, stream=side)
        side.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
        ws = gdn.beam_workspace(x)
        bufs = [torch.empty_like(t) for t in ref]
        live = scores.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.beam_select(x, live, bufs[0], bufs[1], bufs[2], ws, done=done, new_done=bufs[3], eos=3)
        for shift in (0.0, 1.5):
            live.copy_(scores + shift * torch.arange(W, device="cuda"))
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            _check(x, live, done, 3, bufs)


# ------------------------------------------------------------------ forking

def _fork(table, lens, n_pages, T, parent=None, n_new=None, pinned=None, state=None, stream=None):
    R = len(lens)
    t = _ints(table).view(R, -1)
    out = torch.full_like(t, -77)
    new = lambda: torch.full((R,), -55, dtype=torch.int32, device="cuda")  # noqa: E731
    ln, src, dst, idx = new(), new(), new(), torch.full((R, T), -55, dtype=torch.int32, device="cuda")
    opt = lambda x, dt=torch.int32: None if x is None else torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    st = {} if state is None else dict(state_idx=_ints(state), state_idx_out=new(), state_src=new(), state_dst=new())
    args = [opt(parent), opt(n_new), opt(pinned, torch.uint8), _ints(lens)]
    torch.cuda.synchronize()
    gdn.cache_fork(t, args[3], out, ln, idx if T else None, src, dst, n_pages, parent=args[0], n_new=args[1], pinned=args[2],
                   stream=stream, **st)
    torch.cuda.synchronize()
    got = dict(table=out.tolist(), kv_len=ln.tolist(), kv_index=idx.tolist(), page_src=src.tolist(), page_dst=dst.tolist())
    if state is not None:
        got.update({k: st[n].tolist() for k, n in (("state_idx", "state_idx_out"), ("state_src", "state_src"),
                                                   ("state_dst", "state_dst"))})
    return got


def _check_fork(got, want):
    for key, x in want.items():
        if key == "full":
            continue
        if key == "table":
            for a, b in zip(got["table"], x):
                assert a[:len(b)] == b and a[len(b):] == [-77] * (len(a) - len(b))
        else:
            assert got[key] == x, key


def _rows(rng, R, width, n_pages, room):
    """Rows over distinct pages, some of them copies of others."""
    order = list(range(n_pages))
    rng.shuffle(order)
    table, lens = [], []
    for r in range(R):
        if r and rng.random() < 0.4:
            p = rng.randrange(r)
            n = lens[p] if rng.random() < 0.5 else rng.randint(0, lens[p])
            table.append(list(table[p]))
        else:
            n = rng.choice((0, 1, 63, 64, 65, rng.randint(0, width * PAGE - room)))
            n = min(n, width * PAGE)
            used = -(-n // PAGE)
            table.append([order.pop() for _ in range(used)] + [-3] * (width - used))
        lens.append(n)
    return table, lens


@pytest.mark.parametrize("R,T,n_pages", [(1, 1, 20), (4, 1, 40), (7, 5, 70), (30, 1, 300), (33, 64, 400), (64, 8, 1000),
                                         (200, 1, 5001), (1024, 2, 9000), (5, 200, 200001), (3, 0, 30)])
def test_fork_matches_the_plain_form(R, T, n_pages):
    for seed in range(4):
        rng = random.Random(100 * R + seed)
        width = max(5, min(12, n_pages // R))
        table, lens = _rows(rng, R, width, n_pages, T if T < width * PAGE else 0)
        parent = [rng.randrange(-1, R) if rng.random() < 0.1 else rng.randrange(R) for _ in range(R)]
        state = rng.sample(range(3 * R), R)
        pinned = [int(rng.random() < 0.02) for _ in range(n_pages)]
        n_new = [rng.choice((0, T, rng.randint(0, T))) for _ in range(R)]
        for kw in (dict(), dict(parent=parent, state=state), dict(parent=parent, n_new=n_new, pinned=pinned, state=state)):
            want = kv4_plain.fork(table, lens, n_pages, T, **kw)
            got = _fork(table, lens, n_pages, T, **kw)
            _check_fork(got, want)
            if want["full"]:
                with pytest.raises(gdn.GdnError, match="GDN_ERR_FULL"):
                    gdn.check_status()
            else:
                gdn.check_status()


def test_fork_without_pages_left():
    """Rows that find no page take no tokens and are reported; the others are served in order."""
    table, lens = [[0, 1, 9], [2, 9, 9], [3, 9, 9], [9, 9, 9]], [128, 64, 30, 0]
    for n_pages in (4, 5, 6, 7):
        for parent in (None, [0, 2, 2, 1], [3, 3, 3, 3], [-1, 0, 0, 0]):
            want = kv4_plain.fork(table, lens, n_pages, 1, parent=parent)
            _check_fork(_fork(table, lens, n_pages, 1, parent=parent), want)
            if want["full"]:
                with pytest.raises(gdn.GdnError, match="GDN_ERR_FULL"):
                    gdn.check_status()
            gdn.check_status()
    table, lens = [[0, 1], [2, 3]], [128, 127]  # a line of the table is full
    want = kv4_plain.fork(table, lens, 50, 2)
    assert want["full"] and want["kv_len"] == [128, 127]
    _check_fork(_fork(table, lens, 50, 2), want)
    with pytest.raises(gdn.GdnError, match="GDN_ERR_FULL"):
        gdn.check_status()


def test_fork_bad_numbers_are_reported():
    table, lens = [[0, 1, 9], [2, 4, 9]], [100, 70]
    for kw, want in ((dict(parent=[0, 2]), dict(parent=[0, -1])), (dict(parent=[-5, 1]), dict(parent=[-1, 1])),
                     (dict(n_new=[1, 3]), dict(n_new=[1, 0])), (dict(n_new=[-1, 1]), dict(n_new=[0, 1]))):
        _check_fork(_fork(table, lens, 20, 2, **kw), kv4_plain.fork(table, lens, 20, 2, **want))
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
    for bad in (193, -1):
        _check_fork(_fork(table, [100, bad], 20, 2), kv4_plain.fork(table, [100, 0], 20, 2))
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
    got = _fork([[0, 1, 9], [2, 20, 9]], lens, 20, 2)  # row 1's last page does not exist: nothing is stored there
    assert got["kv_index"] == [[64 + 36, 64 + 37], [-1, -1]] and got["page_src"] == [-1, -1]
    with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
        gdn.check_status()


def test_slots_copy_all_layers_and_pools():
    g = torch.Generator(device="cuda").manual_seed(3)
    for shape, n in (((1, 2, 4), 1), ((3, 10, 2, 36), 5), ((2, 40, 16, 17, 4), 20), ((2, 5, 300000), 2)):
        a = torch.randn(shape, generator=g, device="cuda")
        b = torch.randint(0, 256, (4, shape[1], 48), generator=g, device="cuda", dtype=torch.uint8)
        order = torch.randperm(shape[1], generator=g, device="cuda").int()
        src, dst = order[:n].clone(), order[n:2 * n].clone()
        if n > 2:
            src[1] = src[0]  # a slot may go to several
            src[2], dst[2] = -1, 12345
        want = [a.clone(), b.clone()]
        for x in want:
            for i in range(n):
                if int(src[i]) >= 0:
                    x[:, int(dst[i])] = x[:, int(src[i])]
        gdn.slots_copy([(a, src, dst), (b, src, dst)])
        gdn.check_status()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_slots_copy_bad_slots_and_graphs():
    x = torch.arange(2 * 6 * 8, dtype=torch.float32, device="cuda").view(2, 6, 8)
    for src, dst in (([0, 6], [1, 2]), ([0, -2], [1, 2]), ([0, 3], [1, 6]), ([0, 3], [1, -1])):
        y = x.clone()
        gdn.slots_copy([(y, _ints(src), _ints(dst))])
        with pytest.raises(gdn.GdnError, match="GDN_ERR_INDEX"):
            gdn.check_status()
        want = x.clone()
        want[:, 1] = want[:, 0]
        assert torch.equal(y, want)
    src, dst, y = _ints([-1, -1]), _ints([0, 0]), x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.slots_copy([(y, src, dst)])
    src.copy_(_ints([4, 2]))
    dst.copy_(_ints([0, 5]))
    graph.replay()
    gdn.check_status()
    want = x.clone()
    want[:, 0], want[:, 5] = x[:, 4], x[:, 2]
    assert torch.equal(y, want)
