"""Beam search over a hybrid stack as a whole (hybrid.PagedAttentionLayers, Beams, beam_step): prompts into 4-bit pages,
then steps of forking, decoding, storing, attention and selection, eager and as one captured graph, against a plain
simulation that keeps every row's keys, values and states by itself.

Bars: attention kv4_plain.attend's on the very numbers that the pages stand for; the pages' numbers against the 64-bit
norm and rotation within half a step of their scale, amax / 14 (1 + 2^-4) and 0.4375 / 7 of it where the scale was rounded
down, at most 0.076 of the group's largest, and half a bf16 step 2^-8 of it before that: 0.08; all else is equal."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from gated_deltanet_recurrence_delta_gb300 import inputs as I
from gated_deltanet_recurrence_delta_gb300.hybrid import Beams, PagedAttentionLayers, beam_step
from gated_deltanet_recurrence_delta_gb300.stack import LayerStack
from tests import attn_plain, kv4_plain

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


def _within(got, ref, bar):
    assert float(((got.double() - ref).abs() - bar).max()) <= 0


class _World:
    """A hybrid stack's layers with two prompts in the pages of the first row of each of two groups."""

    def __init__(self, d=64, hq=6, hk=2, W=3, layers=2, lens=(130, 64), n_pages=60):
        self.g = torch.Generator(device="cuda").manual_seed(1)
        self.d, self.hq, self.hk, self.W, self.L, self.rot = d, hq, hk, W, layers, 32
        self.R = 2 * W
        inv = 1e4 ** (-torch.arange(0, self.rot, 2, dtype=torch.float64, device="cuda") / self.rot)
        weights = [dict(q_norm=self.rand(d), k_norm=self.rand(d)) for _ in range(layers)]
        self.att = PagedAttentionLayers(hq, hk, d, weights, inv, self.R, n_pages, 8, k_exp=1, v_exp=-2)
        shape = self.shape = I.TINY
        w = [{n: t.cuda() for n, t in I.decode_batch(seed=s, B=1, shape=shape).items()
              if n in ("A_log", "dt_bias", "conv_w", "norm_w")} for s in range(2)]
        self.stack = LayerStack(shape, w, n_slots=self.R)
        self.plain = LayerStack(shape, w, n_slots=self.R)
        self.stack.state_pool.copy_(0.1 * torch.randn(self.stack.state_pool.shape, generator=self.g, device="cuda"))
        self.state_idx = torch.randperm(self.R, generator=self.g, device="cuda").int()
        # the prompts, and what each row holds: keys, values [layers][len, hk, d], float64
        self.rows, self.lens = [0, W], list(lens)
        n_new = [0] * self.R
        for r, n in zip(self.rows, lens):
            n_new[r] = n
        index = self.att.take(max(lens), n_new=_ints(n_new))
        gdn.check_status()
        assert self.att.kv_len.tolist() == n_new
        self.hist = [[self._empty() for _ in range(layers)] for _ in range(self.R)]
        self.prefill(index, [0, 0])

    def rand(self, *s):
        return torch.randn(s, generator=self.g, device="cuda").to(torch.bfloat16)

    def _empty(self):
        return [torch.zeros((0, self.hk, self.d), dtype=torch.float64, device="cuda") for _ in range(2)]

    def stored(self, layer, row, a, b):
        """What the pages of a row hold of its tokens [a, b)."""
        place = torch.arange(a, b, device="cuda")
        page = self.att.table[row, place // PAGE].long()
        return [kv4_plain.decode(self.att.pool[layer], i, e)[page, :, place % PAGE]
                for i, e in ((0, self.att.k_exp), (1, self.att.v_exp))]

    def prefill(self, index, past):
        """A chunk of each prompt behind `past` tokens; looks at its outputs and at what the pages hold afterwards."""
        att, n = self.att, sum(self.lens)
        kv_index = torch.cat([index[r, :m] for r, m in zip(self.rows, self.lens)])
        pos = torch.cat([torch.arange(p, p + m) for m, p in zip(self.lens, past)]).int().cuda()[None]
        for layer in range(self.L):
            qkv = self.rand(n, (self.hq + 2 * self.hk) * self.d)
            q, out = (torch.empty((n, self.hq, self.d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            att.prefill(layer, qkv, self.rows, self.lens, past, kv_index, q, out)
            gdn.check_status()
            xq, xk, xv = att._split(qkv)
            ref_k = attn_plain.norm_rope(xk, att.weights[layer]["k_norm"], pos, att.inv_freq, None, self.rot, False, 1e-6)
            at = 0
            for r, m, p in zip(self.rows, self.lens, past):
                k, v = self.stored(layer, r, p, p + m)
                for got, x in ((k, ref_k[at:at + m]), (v, xv[at:at + m].double())):
                    top = x.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
                    _within(got, x, 0.08 * top)
                assert torch.equal(v, kv4_plain.values(xv[at:at + m], att.v_exp))
                old = self.hist[r][layer]
                kk = torch.cat((old[0], ref_k[at:at + m].to(torch.bfloat16).double()))
                vv = torch.cat((old[1], xv[at:at + m].double()))
                G = self.hq // self.hk
                for h in range(self.hk):  # ref_k may be a bf16 step off: twice half a step on each score
                    ref, bar = attn_plain.attend(q[at:at + m, G * h:G * h + G], kk[:, h], vv[:, h],
                                                 [p + i + 1 for i in range(m)], self.d ** -0.5)
                    s = torch.einsum("igd,jd->gij", q[at:at + m, G * h:G * h + G].double().abs(), kk[:, h].abs()).amax()
                    extra = 2.0 ** -7 * float(s) * self.d ** -0.5 * vv[:, h].abs().amax()
                    _within(out[at:at + m, G * h:G * h + G], ref, bar + extra)
                self.hist[r][layer] = [torch.cat((o, x)) for o, x in zip(old, (k, v))]
                at += m

    def expect(self, parent, done, kv_index):
        """The rows after a fork, before the step's tokens: who has which history; the states, one slot a row."""
        hist = [[[x.clone() for x in kv] for kv in self.hist[p]] for p in parent]
        slots = self.state_idx.tolist()
        state = self.stack.state_pool[:, [slots[p] for p in parent]].clone()
        conv = self.stack.conv_pool[:, [slots[p] for p in parent]].clone()
        return hist, state, conv


@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_beam_steps(captured):
    w = _World()
    att, stack, W, R, V, L = w.att, w.stack, w.W, w.R, 400, w.L
    beams = Beams(2, W)
    acts = stack.static_acts(R, 1)
    qkv = [torch.empty((R, 1, (w.hq + 2 * w.hk) * w.d), dtype=torch.bfloat16, device="cuda") for _ in range(L)]
    logits = torch.empty((2, W, V), device="cuda")
    s = w.shape
    buf = dict(gdn_out=torch.empty((2, R, 1, s.nv, s.dv), dtype=torch.bfloat16, device="cuda"),
               q=torch.empty((R, 1, w.hq, w.d), dtype=torch.bfloat16, device="cuda"),
               attn_out=torch.empty((L, R, 1, w.hq, w.d), dtype=torch.bfloat16, device="cuda"))
    eos = 7

    def step():
        beam_step(stack, att, beams, acts, qkv, logits, w.state_idx, buf, eos)

    def fill(i):
        for layer in acts:
            for t in layer.values():
                t.copy_(w.rand(*t.shape))
        for t in qkv:
            t.copy_(w.rand(*t.shape))
        logits.copy_(2.5 * torch.randn(logits.shape, generator=w.g, device="cuda"))
        if i % 5 == 3:
            logits[:, 0, eos] = 12.0  # a beam ends

    graph = None
    if captured:
        fill(0)
        things = [att.table, att.kv_len, att.pool, stack.state_pool, stack.conv_pool, w.state_idx, beams.scores, beams.done,
                  beams.parent, beams.token, att.taken]
        kept = [t.clone() for t in things]
        step()  # first use, outside the capture; put back afterwards
        torch.cuda.synchronize()
        for t, k in zip(things, kept):
            t.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    copied = 0
    for i in range(70):  # past the end of a page in both groups
        fill(i)
        parent, done = beams.parent.flatten().tolist(), beams.done.flatten().tolist()
        scores, was_done = beams.scores.clone(), beams.done.clone()
        hist, state, conv = w.expect(parent, done, None)
        graph.replay() if captured else step()
        gdn.check_status()
        copied += sum(p in parent[:r] for r, p in enumerate(parent))
        assert sorted(w.state_idx.tolist()) == list(range(R))
        # the recurrent layers: the same step on states gathered by hand
        w.plain.state_pool.copy_(state)
        w.plain.conv_pool.copy_(conv)
        ref = torch.empty_like(buf["gdn_out"])
        w.plain.decode(acts, torch.arange(R, dtype=torch.int32, device="cuda"), ref)
        assert torch.equal(buf["gdn_out"], ref)
        slots = w.state_idx.long()
        assert torch.equal(stack.state_pool[:, slots], w.plain.state_pool)
        assert torch.equal(stack.conv_pool[:, slots], w.plain.conv_pool)
        # the attention layers
        for layer in range(L):
            for r in range(R):
                n = len(hist[r][layer][0])
                assert int(att.kv_len[r]) == n + (0 if done[r] else 1)
                if not done[r]:
                    new = w.stored(layer, r, n, n + 1)
                    v = qkv[layer][r, 0, (w.hq + w.hk) * w.d:].view(1, w.hk, w.d)
                    assert torch.equal(new[1], kv4_plain.values(v, att.v_exp))
                    hist[r][layer] = [torch.cat((o, x)) for o, x in zip(hist[r][layer], new)]
        w.hist = hist
        G = w.hq // w.hk
        for r in range(R):
            k, v = w.hist[r][L - 1]
            for h in range(w.hk):
                ref, bar = kv4_plain.attend(buf["q"][r, :, G * h:G * h + G], k[:, h], v[:, h], [0 if done[r] else len(k)],
                                            w.d ** -0.5)
                _within(buf["attn_out"][L - 1][r, :, G * h:G * h + G], ref, bar)
        if i % 10 == 0:  # all that the rows hold, not only what was added
            for r in range(R):
                for a, b in zip(w.stored(0, r, 0, len(w.hist[r][0][0])), w.hist[r][0]):
                    assert torch.equal(a, b)
        for g in range(2):
            p, t, sc, o, bar = kv4_plain.beam(logits[g].cpu(), scores[g].cpu(), was_done[g].cpu(), eos)
            assert (beams.parent[g] - g * W).tolist() == p and beams.token[g].tolist() == t
            assert beams.done[g].tolist() == o
            for x, y in zip(beams.scores[g].tolist(), sc):
                assert x == y or abs(x - y) <= 2.0 ** -24 * abs(y) + bar
        if bool(beams.done.all()):
            break
    assert copied > 20 and i > 15


def test_a_prompt_in_chunks_over_its_pages():
    """Further chunks of the prompts behind what the pages hold, and a row emptied and filled anew."""
    w = _World(d=128, hq=4, hk=2, W=1, layers=1, lens=(100, 70))
    for more in ((50, 1), (64, 30)):
        past = [int(n) for n in w.att.kv_len]
        w.lens = list(more)
        index = w.att.take(max(more), n_new=_ints(list(more)))
        w.prefill(index, past)
        assert w.att.kv_len.tolist() == [a + b for a, b in zip(past, more)]
    used = set(w.att.table[0, :4].tolist()) | set(w.att.table[1, :2].tolist())
    assert len(used) == 6
    w.att.take(0, parent=_ints([-1, 1]))
    assert w.att.kv_len.tolist() == [0, 101]
    w.hist[0] = [w._empty()]
    w.lens, w.rows = [90], [0]
    index = w.att.take(90, n_new=_ints([90, 0]))
    w.prefill(index, [0])
    gdn.check_status()
    assert set(w.att.table[1, :2].tolist()).isdisjoint(w.att.table[0, :2].tolist())


def test_pinned_pages_are_kept_and_full_pools_reported():
    w = _World(W=2, layers=1, lens=(70, 10), n_pages=4)
    pages = w.att.table[0, :2].tolist()
    w.att.pinned[pages] = 1
    before = w.att.pool[:, pages].clone()
    index = w.att.take(1, parent=_ints([0, 0, 2, 3]), n_new=_ints([1, 1, 1, 0]))  # three copies or pages, one left
    with pytest.raises(gdn.GdnError, match="GDN_ERR_FULL"):
        gdn.check_status()
    assert w.att.kv_len.tolist() == [71, 70, 11, 0] and w.att.taken.tolist() == [1, 0, 1, 0]
    assert index[:, 0].tolist()[1] == -1 and index[:, 0].tolist()[3] == -1
    w.att.step(0, w.rand(4, 1, (w.hq + 2 * w.hk) * w.d), index, *(torch.empty((4, 1, w.hq, w.d), dtype=torch.bfloat16,
                                                                              device="cuda") for _ in range(2)))
    gdn.check_status()
    assert torch.equal(w.att.pool[:, pages], before) and w.att.table[0, 1] != pages[1]
