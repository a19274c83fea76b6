"""What the paged layers of hybrid.py and its beams keep and hand to the library, without a GPU: the library's calls are
replaced by recorders."""
import types

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn, hybrid

HQ, HK, D, ROWS = 4, 2, 64, 3


@pytest.fixture
def calls(monkeypatch):
    """The recorded calls: (name, arguments by name)."""
    seen = []

    def fork(page_table, kv_len, page_table_out, kv_len_out, kv_index, page_src, page_dst, n_pages, parent=None, n_new=None,
             **kw):
        T = 0 if kv_index is None else kv_index.shape[1]
        new = torch.full_like(kv_len, T) if n_new is None else n_new
        copy = lambda x: None if x is None else x.clone()  # noqa: E731
        seen.append(("fork", types.SimpleNamespace(T=T, parent=copy(parent), n_new=copy(n_new), **kw)))
        page_table_out.copy_(page_table)
        kv_len_out.copy_(kv_len + new)
        if T:
            kv_index.copy_(torch.where(torch.arange(T) < new[:, None], len(seen), -1))

    monkeypatch.setattr(gdn, "cache_fork", fork)
    monkeypatch.setattr(gdn, "slots_copy", lambda pools, stream=None: seen.append(("copy", len(pools))))
    monkeypatch.setattr(gdn, "_stream", lambda s: 0 if s is None else s if isinstance(s, int) else s.cuda_stream)
    return seen


def _layers():
    weights = [dict(q_norm=None, k_norm=None)]
    return hybrid.PagedAttentionLayers(HQ, HK, D, weights, torch.ones(16, dtype=torch.float64), ROWS, 20, 300, device="cpu")


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_prompts_of_any_length_leave_nothing_behind(calls):
    """The rows of a prompt's tokens are the caller's: no later take() writes them, none is kept."""
    att = _layers()
    first = att.take(1000)
    for T in (1, 64, *range(65, 400, 7), 1000):
        att.take(T)
    assert bool((first == 1).all())
    assert sum(x.nbytes for x in att.buffers.values()) == 4 * ROWS * (1 + 64)
    step = att.take(8)
    assert att.take(8) is step and att.take(0).shape == (ROWS, 0)


def test_a_selection_takes_its_workspace_from_its_stream(calls, monkeypatch):
    """One for each shape and stream, made while that stream is torch's own."""
    on, used = [None], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            on.append(self.stream)

        def __exit__(self, *_):
            on.pop()

    def select(logits, scores, parent, token, new_scores, workspace, done=None, new_done=None, eos=-1, stream=None):
        used.append((workspace, stream))

    monkeypatch.setattr(hybrid, "_on", On)
    monkeypatch.setattr(gdn, "beam_workspace", lambda logits: (tuple(logits.shape), on[-1]))
    monkeypatch.setattr(gdn, "beam_select", select)
    beams, shape = hybrid.Beams(2, 3, device="cpu"), (2, 3, 50)
    for stream in (None, 7, 9, None, 7):
        beams.select(torch.zeros(shape), stream=stream)
    assert used == [((shape, s), s) for s in (None, 7, 9, None, 7)] and len(beams.workspaces) == 3
    with pytest.raises(ValueError):
        beams.select(torch.zeros((2, 4, 50)))


def test_places_without_a_beam_take_nothing(calls):
    """At the start every row takes a token; what a selection left without a beam (token -1) is emptied and takes none, and
    a finished beam keeps its row as it is, whatever its token."""
    att, beams = _layers(), hybrid.Beams(1, ROWS, device="cpu")
    att.step = lambda *a, **k: None
    select = types.SimpleNamespace(next=None)
    beams.select = lambda logits, eos: [getattr(beams, n).copy_(torch.tensor([x])) for n, x in select.next.items()]
    stack = types.SimpleNamespace(decode=lambda *a: None, state_pool=None, conv_pool=None)
    buf = dict(gdn_out=None, q=None, attn_out=[None])
    inf = float("inf")
    chosen = [dict(parent=[0, 1, 2], token=[7, -1, -1], scores=[-1.0, -inf, -inf], done=[0, 0, 0]),
              dict(parent=[0, 0, 2], token=[5, -1, -1], scores=[-1.0, -2.0, -inf], done=[0, 1, 0]),
              dict(parent=[1, 0, 0], token=[3, 9, 5], scores=[-2.0, -3.0, -4.0], done=[1, 0, 0]),
              dict(parent=[0, 1, 2], token=[-1, -1, -1], scores=[0.0, -inf, -inf], done=[0, 0, 0]), {}]  # set back by hand
    want = [([0, 1, 2], [1, 1, 1]), ([0, -1, -1], [1, 0, 0]), ([0, 0, -1], [1, 0, 0]), ([1, 0, 0], [0, 1, 1]),
            ([0, -1, -1], [1, 0, 0])]
    for select.next, (parent, n_new) in zip(chosen, want):
        hybrid.beam_step(stack, att, beams, None, [None], None, None, buf)
        got = [x for kind, x in calls if kind == "fork"][-1]
        assert (got.parent.tolist(), got.n_new.tolist()) == (parent, n_new) and got.parent.dtype == torch.int32


def test_steps_and_prompts_refuse_another_number_of_tokens(calls):
    """The pool rows of another take(), or all rows' where one prompt's are meant: tokens would go to others' places."""
    att, new = _layers(), lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    qkv, q = new(ROWS, 2, (HQ + 2 * HK) * D), new(ROWS, 2, HQ, D)
    for index, x in ((att.take(4), qkv), (att.take(1), qkv), (att.take(2), qkv[:, :1]), (att.take(2), qkv[:2])):
        with pytest.raises(ValueError, match="kv_index"):
            att.step(0, x, index, q, q.clone())
    index = att.take(100, n_new=_ints(0, 100, 0))
    qkv, q = new(100, (HQ + 2 * HK) * D), new(100, HQ, D)
    for at, x in ((index, qkv), (index[1, :99], qkv), (index[1], qkv[:99])):
        with pytest.raises(ValueError, match="kv_index"):
            att.prefill(0, x, [1], [100], [0], at, q, q.clone())
