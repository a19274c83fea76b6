"""Calls of the paged 4-bit cache and of beam search in orders that no other test makes: a process's first call at sizes of
its own, steps captured before any ran, selections whose vocabulary changes, prompts without tokens."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from gated_deltanet_recurrence_delta_gb300.hybrid import Beams, PagedAttentionLayers
from tests.test_gpu_kv4 import _case, _compare, _run

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


def test_a_first_fork_at_any_number_of_pages():
    """The fork of 60000 pages as the only one of a process: its shared memory passes the default limit."""
    code = """
import torch
from gated_deltanet_recurrence_delta_gb300 import gdn
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
out, new, src, dst, index = ints([[-1, -1]]), ints([0]), ints([0]), ints([0]), ints([[0]])
pinned = torch.ones(60000, dtype=torch.uint8, device="cuda")
pinned[59999] = 0
gdn.cache_fork(ints([[7, -1]]), ints([64]), out, new, index, src, dst, 60000, pinned=pinned)
gdn.check_status()
assert (out.tolist(), new.tolist(), index.tolist()) == ([[7, 59999]], [65], [[59999 * 64]]), (out, new, index)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=Path(__file__).resolve().parents[1], timeout=300)


def _layers(rows=3, hq=4, hk=2, d=64):
    inv = 1e4 ** (-torch.arange(0, 32, 2, dtype=torch.float64, device="cuda") / 32)
    weights = [dict(q_norm=None, k_norm=None)]
    return PagedAttentionLayers(hq, hk, d, weights, inv, rows, 64, 16)


def _prompts(att, lens, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    index = att.take(max(lens), n_new=_ints(lens))
    kv_index = torch.cat([index[r, :n] for r, n in enumerate(lens)])
    n = sum(lens)
    qkv = torch.randn((n, (att.hq + 2 * att.hk) * att.d), generator=g, device="cuda").to(torch.bfloat16)
    q, out = (torch.empty((n, att.hq, att.d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    att.prefill(0, qkv, list(range(len(lens))), lens, [0] * len(lens), kv_index, q, out)
    gdn.check_status()
    return out


def test_graphs_that_share_a_workspace_replay_in_any_order():
    """Two graphs captured from one stream before anything ran on it: the second is replayed first, over a workspace
    full of ones."""
    lens = [700, 64, 5]
    eager, att = _layers(), _layers()
    for x in (eager, att):
        _prompts(x, lens)
    g = torch.Generator(device="cuda").manual_seed(6)
    qkv = torch.randn((2, 3, 1, (att.hq + 2 * att.hk) * att.d), generator=g, device="cuda").to(torch.bfloat16)
    new = lambda: torch.empty((2, 3, 1, att.hq, att.d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want, got, q = new(), new(), new()
    for i in (1, 0):
        eager.step(0, qkv[i], eager.take(1), q[i], want[i])
    torch.cuda.synchronize()
    graphs, side = [torch.cuda.CUDAGraph() for _ in range(2)], torch.cuda.Stream()
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph, stream=side):
            att.step(0, qkv[i], att.take(1), q[i], got[i])
    for key, x in att.buffers.items():
        if key[0] == "workspace" and key[2] == side.cuda_stream:
            x.fill_(1)
    for i in (1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    gdn.check_status()
    assert torch.equal(got, want) and torch.equal(att.kv_len, eager.kv_len)


def test_selections_over_vocabularies_of_several_sizes():
    g = torch.Generator(device="cuda").manual_seed(7)
    beams, single = Beams(2, 4), Beams(2, 4)
    for V in (50, 40000, 9000, 40000):
        logits = torch.randn((2, 4, V), generator=g, device="cuda")
        fresh = Beams(2, 4)
        fresh.scores.copy_(single.scores), fresh.done.copy_(single.done)
        for b in (beams, fresh):
            b.select(logits, eos=3)
        gdn.check_status()
        single = fresh
        for n in ("scores", "done", "parent", "token"):
            assert torch.equal(getattr(beams, n), getattr(fresh, n))
    with pytest.raises(ValueError):
        beams.select(logits[:, :3])


def test_prompts_without_tokens():
    """A chunk of which some rows, or all, have none: the others' outputs are as without them, nothing else is written."""
    a, b = _layers(), _layers()
    want = _prompts(a, [70, 0, 9])
    index = b.take(70, n_new=_ints([70, 0, 9]))
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn((79, (b.hq + 2 * b.hk) * b.d), generator=g, device="cuda").to(torch.bfloat16)
    q, out = (torch.empty((79, b.hq, b.d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b.prefill(0, qkv, [0, 2], [70, 9], [0, 0], torch.cat((index[0], index[2, :9])), q, out)
    gdn.check_status()
    assert torch.equal(out, want) and torch.equal(a.pool, b.pool)
    for x in (a, b):  # a second chunk, of the last row alone
        n = 66
        index = x.take(n, n_new=_ints([0, 0, n]))
        qkv = torch.randn((n, (b.hq + 2 * b.hk) * b.d), generator=g.manual_seed(8), device="cuda").to(torch.bfloat16)
        q, out = (torch.empty((n, b.hq, b.d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        rows, lens, past = ([0, 1, 2], [0, 0, n], [70, 0, 9]) if x is a else ([2], [n], [9])
        x.prefill(0, qkv, rows, lens, past, index[2, :n].contiguous(), q, out)
        gdn.check_status()
        want = out if x is a else want
    assert torch.equal(out, want) and torch.equal(a.pool, b.pool)
    before, none = a.pool.clone(), torch.empty((0, b.hq, b.d), dtype=torch.bfloat16, device="cuda")
    for rows, lens, past in (([], [], []), ([0, 1], [0, 0], [70, 0])):
        a.prefill(0, qkv[:0], rows, lens, past, a.take(0).flatten(), none, none)
    gdn.check_status()
    assert torch.equal(a.pool, before) and a.kv_len.tolist() == [70, 0, 75]


def test_selections_at_the_ends_of_fp32():
    """Scores and logits up to the largest numbers: sums that pass fp32's range in between rank as in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(9)
    G, W, V = 6, 4, 700
    sizes = torch.tensor([[1.0, 1e20, 1e37, 3e38, 1e38, 1e30], [3e38, 1e25, 1e37, 3e38, 1.0, 1e30]], device="cuda")
    logits = (2 * torch.rand((G, W, V), generator=g, device="cuda") - 1) * sizes[0, :, None, None]
    scores = (2 * torch.rand((G, W), generator=g, device="cuda") - 1) * sizes[1, :, None]
    assert bool(logits.isfinite().all() and scores.isfinite().all())
    ints = lambda: torch.zeros((G, W), dtype=torch.int32, device="cuda")  # noqa: E731
    parent, token, new = ints(), ints(), torch.empty_like(scores)
    gdn.beam_select(logits, scores, parent, token, new, gdn.beam_workspace(logits))
    gdn.check_status()
    x, s = logits.double(), scores.double()
    cand = (x + (s - torch.logsumexp(x, -1))[..., None]).flatten(1)
    for i in range(G):
        order = sorted(range(W * V), key=lambda j: (-float(cand[i, j]), j))[:W + 1]
        gap = min(float(cand[i, a] - cand[i, b]) for a, b in zip(order, order[1:]))
        top = float(s[i].abs().max() + x[i].abs().max())
        if gap > 2.0 ** -50 * top:  # apart in 64 bits
            assert (parent[i] - W * i).tolist() == [j // V for j in order[:W]]
            assert token[i].tolist() == [j % V for j in order[:W]]
        want = cand[i, order[:W]].float()
        assert bool(((new[i] == want) | ((new[i] - want).abs() <= 2.0 ** -22 * want.abs() + 1e-5)).all())


@pytest.mark.parametrize("d,hq,hk,T", [(64, 1, 1, 1), (128, 8, 1, 2), (256, 8, 2, 8)])
def test_attention_without_pages(d, hq, hk, T):
    """Tables without entries, or pools without pages: rows without tokens give zeros, others are refused on the device."""
    q = torch.ones((1, T, hq, d), dtype=torch.bfloat16, device="cuda")
    for n_pages, width in ((0, 0), (3, 0), (0, 2), (1, 1)):
        pool, table = gdn.kv4_pool(n_pages, hk, d), torch.zeros((1, width), dtype=torch.int32, device="cuda")
        dims = gdn.make_attn_kv4_dims(q, pool, table)
        out, work = torch.full_like(q, 7.0), gdn.attn_kv4_workspace(dims)
        gdn.attn_kv4(dims, q, pool, table, _ints([0]), out, work)
        gdn.check_status()
        assert not bool(out.any())
        if (n_pages, width) != (1, 1):
            out.fill_(7.0)
            gdn.attn_kv4(dims, q, pool, table, _ints([5]), out, work)
            with pytest.raises(gdn.GdnError, match="INDEX"):
                gdn.check_status()
            assert bool((out == 7.0).all())


@pytest.mark.parametrize("rows,T,hq,hk,d", [(31, 1, 4, 2, 128), (33, 2, 8, 2, 256), (64, 1, 4, 4, 64), (65, 8, 4, 1, 256),
                                            (1024, 1, 1, 1, 64), (1025, 1, 1, 1, 64), (1150, 1, 2, 1, 64), (1100, 1, 2, 2, 128)])
def test_long_rows_among_many(rows, T, hq, hk, d):
    """Rows whose pages many CTAs share, at the ends of every 32 and every 1024 rows, among short and empty ones."""
    lens = [(7 * i) % 90 if i % 5 else 0 for i in range(rows)]
    for i in {0, rows // 2, rows - 1, min(rows - 1, 31), min(rows - 1, 32), min(rows - 1, 1023)}:
        lens[i] = 1500 + 64 * (i % 3) + i % 64
    lens = [n if n == 0 else max(n, T) for n in lens]
    c = _case(lens, T, hq, hk, d, seed=rows)
    _compare(c, _run(c))
    gdn.check_status()
