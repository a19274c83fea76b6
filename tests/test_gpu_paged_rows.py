"""Rows of the paged 4-bit cache and beams where one depends on what others do: forks of rows whose last pages are pinned,
streams beside one another, places without a beam."""
import random

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from gated_deltanet_recurrence_delta_gb300.hybrid import Beams, beam_step
from tests import kv4_plain
from tests.test_gpu_beam import _check_fork, _fork
from tests.test_gpu_beam_search import _World

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


@pytest.mark.parametrize("R", [2, 33, 64, 200, 1024])
def test_fork_of_pinned_last_pages(R):
    """Last pages that are pinned, shared, both or neither, in rows of very different lengths (whose warps come to the
    look at the other rows at different times): who copies is decided the same way every time."""
    for seed in range(3):
        rng = random.Random(R + seed)
        n_pages, width = 40 * R + 64, 20
        order = list(range(n_pages))
        rng.shuffle(order)
        table, lens, pinned = [], [], [0] * n_pages
        for r in range(R):
            if r and rng.random() < 0.5:  # a copy of a row
                p = rng.randrange(r)
                table.append(list(table[p]))
                lens.append(lens[p])
                continue
            n = rng.choice((1, 5, 70, 18 * PAGE + 3, rng.randint(1, 18 * PAGE)))
            used = -(-n // PAGE)
            table.append([order.pop() for _ in range(used)] + [-3] * (width - used))
            lens.append(n)
            pinned[table[r][used - 1]] = int(rng.random() < 0.5)
        n_new = [rng.choice((0, 1, 1, 2)) for _ in range(R)]
        want = kv4_plain.fork(table, lens, n_pages, 2, n_new=n_new, pinned=pinned)
        assert not want["full"] and (R == 2 or any(p >= 0 for p in want["page_src"]))
        for _ in range(10):
            _check_fork(_fork(table, lens, n_pages, 2, n_new=n_new, pinned=pinned), want)
    gdn.check_status()


def test_a_first_selection_on_a_stream_beside_a_busy_one():
    """The current stream still writes to memory that torch has taken back: a selection's workspace on another stream is
    none of it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((16, 8, 50000), generator=g, device="cuda")
    want = Beams(16, 8)
    want.select(logits)
    gdn.check_status()
    n = gdn.beam_workspace(logits).numel()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = Beams(16, 8)
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000)  # 1 ms
        x = torch.empty(n, dtype=torch.uint8, device="cuda")
        for _ in range(200):
            x.fill_(255)
        del x
        got.select(logits, stream=side)
        torch.cuda.synchronize()
        gdn.check_status()
        for name in ("scores", "parent", "token", "done"):
            assert torch.equal(getattr(got, name), getattr(want, name))


def test_places_without_a_beam_leave_their_pages_to_the_others():
    """One allowed token a row and step: each group has one beam of four for 70 steps, in a pool of as many pages as the
    first step takes. The other rows would need a second page each after 64 steps."""
    w = _World(W=4, layers=1, n_pages=11)  # 4 pages of prompts, one for the second's next token, 6 rows' first ones
    att, W, R, V = w.att, w.W, w.R, 200
    beams, acts, s = Beams(2, W), w.stack.static_acts(R, 1), w.shape
    qkv = [w.rand(R, 1, (w.hq + 2 * w.hk) * w.d)]
    buf = dict(gdn_out=torch.empty((2, R, 1, s.nv, s.dv), dtype=torch.bfloat16, device="cuda"),
               q=torch.empty((R, 1, w.hq, w.d), dtype=torch.bfloat16, device="cuda"),
               attn_out=torch.empty((1, R, 1, w.hq, w.d), dtype=torch.bfloat16, device="cuda"))
    for i in range(70):
        logits = torch.full((2, W, V), -float("inf"), device="cuda")
        logits[:, :, (17 * i) % V] = 0.5
        beam_step(w.stack, att, beams, acts, qkv, logits, w.state_idx, buf)
        gdn.check_status()
        other = 1 if i == 0 else 0
        assert att.kv_len.tolist() == [131 + i, *[other] * 3, 65 + i, *[other] * 3]
        assert beams.token.tolist() == [[(17 * i) % V, -1, -1, -1]] * 2
        assert sorted(w.state_idx.tolist()) == list(range(R))
    assert bool((buf["attn_out"][0, [0, W]] != 0).any()) and not bool(buf["attn_out"][0, [1, 2, 3]].any())


def test_rows_wait_for_those_in_front_of_them():
    """Three free pages, of which row 1 needs five: it takes nothing, nor does row 2 behind it, which needs one; row 3 needs
    none and takes its tokens, as row 0 in front does. Without row 1's tokens row 2 is served."""
    table, lens = [[0, 1, -3, -3, -3, -3], [2, -3, -3, -3, -3, -3], [3, -3, -3, -3, -3, -3], [4, -3, -3, -3, -3, -3]], [
        128, 64, 64, 10]
    got = _fork(table, lens, 9, 300, n_new=[1, 300, 1, 2])
    with pytest.raises(gdn.GdnError, match="GDN_ERR_FULL"):
        gdn.check_status()
    assert got["kv_len"] == [129, 64, 64, 12]
    index = [[x for x in row if x >= 0] for row in got["kv_index"]]
    assert index == [[5 * PAGE], [], [], [4 * PAGE + 10, 4 * PAGE + 11]]
    assert got["page_src"] == got["page_dst"] == [-1] * 4
    assert [row[:2] for row in got["table"]] == [[0, 1], [2, -77], [3, -77], [4, -77]] and got["table"][0][2] == 5
    got = _fork(table, lens, 9, 300, n_new=[1, 0, 1, 2])
    gdn.check_status()
    assert got["kv_len"] == [129, 64, 65, 12] and got["table"][2][:2] == [3, 6] and got["kv_index"][2][0] == 6 * PAGE


def test_lengths_that_change_between_calls():
    """Lengths written anew by the kernel in front of every call, among calls of few CTAs (a part of the GPU's SMs): the
    parts of each call are joined by the lengths that it has, 300 calls on end without a wait, eager and as a graph."""
    g = torch.Generator(device="cuda").manual_seed(4)
    R, width = 5, 40
    pool = torch.randint(0, 256, (R * width, 2, 72 * 128), generator=g, device="cuda", dtype=torch.uint8)
    pool[:, :, 64 * 128:] = 0x38  # scales of one
    table = torch.randperm(R * width, generator=g, device="cuda").int().view(R, width)
    q = torch.randn((R, 1, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    dims = gdn.make_attn_kv4_dims(q, pool, table)
    work, lens = gdn.attn_kv4_workspace(dims), torch.zeros(R, dtype=torch.int32, device="cuda")
    sets = torch.randint(0, width * PAGE + 1, (300, R), generator=g, device="cuda").int()
    want, got = (torch.zeros((300, *q.shape), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run(out):
        for i in range(300):
            lens.copy_(sets[i])
            gdn.attn_kv4(dims, q, pool, table, lens, out[i], work)

    for i in range(300):
        lens.copy_(sets[i])
        torch.cuda.synchronize()
        gdn.attn_kv4(dims, q, pool, table, lens, want[i], work)
        torch.cuda.synchronize()
    assert bool(want.isfinite().all())
    run(got)
    gdn.check_status()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for _ in range(5):
        got.fill_(7.0)
        graph.replay()
        gdn.check_status()
        assert torch.equal(got, want)
