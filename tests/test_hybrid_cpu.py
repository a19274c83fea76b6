"""What hybrid.py hands to the library, without a GPU: the library's calls are replaced by recorders, so every index,
length and stream that a step derives is seen as it is."""
import types

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn, hybrid

HQ, HK, D = 4, 2, 64


@pytest.fixture
def calls(monkeypatch):
    """The recorded calls: (name, arguments by name)."""
    seen = []

    def rope(dims, q, k, v, qw, kw, positions, inv_freq, q_out, k_out, v_out, axis=None, kv_index=None, stream=None):
        seen.append(("rope", types.SimpleNamespace(positions=positions.clone(), kv_index=kv_index.clone(), dims=dims)))

    def attn(dims, q, k, v, group_rows, prefix_start, prefix_len, suffix_start, suffix_len, out, workspace, q_len=None,
             stream=None):
        B, T = dims.B, dims.T
        real = torch.full((B,), T, dtype=torch.int32) if q_len is None else q_len.clone()
        seen.append(("attn", types.SimpleNamespace(start=suffix_start.clone(), len=suffix_len.clone(), real=real,
                                                   n_groups=dims.n_groups, prefix_len=prefix_len)))

    def accept(tokens, target, draft, uniform, accept_len, next_token, n_tokens=None, stream=None):
        seen.append(("accept", types.SimpleNamespace(n_tokens=None if n_tokens is None else n_tokens.clone())))
        accept_len.copy_(torch.full_like(accept_len, tokens.shape[1]) if n_tokens is None else n_tokens)

    monkeypatch.setattr(gdn, "head_norm_rope", rope)
    monkeypatch.setattr(gdn, "attn_shared_prefix", attn)
    monkeypatch.setattr(gdn, "accept_draft", accept)
    monkeypatch.setattr(gdn, "attn_workspace", lambda dims, device: torch.zeros(1))
    monkeypatch.setattr(gdn, "_stream", lambda s: 0 if s is None else s if isinstance(s, int) else s.cuda_stream)
    return seen


def _layers(n_rows, room, prompt_rows=100, n_layers=1):
    return hybrid.AttentionLayers(HQ, HK, D, [dict(q_norm=None, k_norm=None)] * n_layers, torch.ones(16, dtype=torch.float64),
                                  prompt_rows, n_rows, room, device="cpu")


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def _step(att, B, T, prompts, **kw):
    qkv = torch.zeros((B, T, (HQ + 2 * HK) * D), dtype=torch.bfloat16)
    q = torch.zeros((B, T, HQ, D), dtype=torch.bfloat16)
    att.step(0, qkv, *prompts, q, torch.zeros_like(q), **kw)


def _stack(log):
    return types.SimpleNamespace(verify=lambda *a, **k: log.append("verify"), commit=lambda *a, **k: log.append("commit"))


# ------------------------------------------------------------- rows and rooms

def test_a_rows_extent_never_leaves_its_room(calls):
    """Room 10, four tokens a step: behind 3 keys all fit, behind 8 two do, behind 10 or more none."""
    att = _layers(n_rows=5, room=10)
    att.own_len.copy_(_ints(3, 8, 10, 6, 13))
    _step(att, 5, 4, (_ints(0, 5), _ints(0), _ints(100)))
    rope, attn = calls[0][1], calls[1][1]
    start = [100 + 10 * b for b in range(5)]
    assert attn.start.tolist() == start
    assert bool((attn.len <= 10).all()), f"extents {attn.len.tolist()} leave rooms of 10"
    assert attn.real.tolist() == [4, 2, 0, 4, 0]
    assert attn.len[:4].tolist() == [7, 10, 10, 10]
    at = rope.kv_index.view(5, 4).tolist()
    assert at[0] == [103, 104, 105, 106] and at[1] == [118, 119, -1, -1] and at[3] == [136, 137, 138, 139]
    # a row without room for one token is reported: the library takes an index past the pool for a device error
    assert att.kv_rows in at[2] and att.kv_rows in at[4]
    assert all(x in (-1, att.kv_rows) for x in at[2] + at[4])


def test_a_speculative_step_accepts_no_more_than_the_room_holds(calls):
    att = _layers(n_rows=3, room=10, n_layers=2)
    att.own_len.copy_(_ints(0, 7, 10))
    B, T = 3, 4
    log = []
    buf = dict(gdn_out=None, ckpt_state=None, ckpt_conv=None, q=torch.zeros((B, T, HQ, D), dtype=torch.bfloat16),
               attn_out=torch.zeros((2, B, T, HQ, D), dtype=torch.bfloat16), accept_len=_ints(0, 0, 0),
               next_token=_ints(0, 0, 0))
    qkv = [torch.zeros((B, T, (HQ + 2 * HK) * D), dtype=torch.bfloat16)] * 2
    step = lambda: hybrid.speculative_step(_stack(log), att, None, qkv, None, (_ints(0, 3), _ints(0), _ints(100)),  # noqa: E731
                                           torch.zeros((B, T), dtype=torch.int32), None, None, None, buf)
    step()
    (accept,) = [c for n, c in calls if n == "accept"]
    assert accept.n_tokens is not None and accept.n_tokens.tolist() == [4, 3, 0]
    assert att.own_len.tolist() == [4, 10, 10] and log == ["verify", "commit"]
    step()
    step()
    assert att.own_len.tolist() == [10, 10, 10]
    for name, c in calls:
        if name == "attn":
            assert bool((c.len <= 10).all())


# -------------------------------------------------------------------- streams

class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("as_handle", [False, True])
def test_everything_a_step_does_is_on_its_stream(calls, monkeypatch, as_handle):
    """The index arithmetic, the workspace and the library's calls of a step given a stream: nothing on another one, and
    no workspace shared between streams."""
    import contextlib

    from torch.utils._python_dispatch import TorchDispatchMode
    current, stray = [0], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    held = []
    monkeypatch.setattr(gdn, "attn_shared_prefix",
                        lambda *a, q_len=None, stream=None: held.append((a[10], gdn._stream(a[12] if len(a) > 12 else stream))))

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            views = ("select", "slice", "view", "unsqueeze", "split", "expand", "reshape", "alias", "detach", "t.")
            name = func.name().split("::")[1]
            if current[-1] != 77 and not name.startswith(views):
                stray.append(name)
            return func(*args, **(kwargs or {}))

    att = _layers(n_rows=3, room=20)
    prompts = (_ints(0, 3), _ints(0), _ints(100))
    qkv = torch.zeros((3, 2, (HQ + 2 * HK) * D), dtype=torch.bfloat16)
    q, out, got = torch.zeros((3, 2, HQ, D), dtype=torch.bfloat16), torch.zeros((3, 2, HQ, D)), _ints(1, 2, 1)
    side = 77 if as_handle else _Stream(77)
    with Watch():
        att.step(0, qkv, *prompts, q, out, stream=side)
        assert stray == [], f"on another stream than the step's: {stray}"
        att.advance(got, stream=side)
        assert stray == [], f"on another stream than the step's: {stray}"
    assert att.own_len.tolist() == [1, 2, 1]
    att.step(0, qkv, *prompts, q, out)
    att.step(0, qkv, *prompts, q, out, stream=side)
    assert [h for _, h in held] == [77, 0, 77]
    assert held[0][0] is held[2][0] and held[0][0] is not held[1][0]


# ---------------------------------------------------- rows without a prompt

@pytest.mark.parametrize("prompts", [(None, None, None), (_ints(0), _ints(), _ints())])
def test_rows_without_a_shared_prompt(calls, prompts):
    """Ordinary decode: positions count from the row's own first key, and the call has no groups."""
    att = _layers(n_rows=3, room=20, prompt_rows=0)
    att.own_len.copy_(_ints(0, 5, 18))
    _step(att, 3, 2, prompts)
    rope, attn = calls[0][1], calls[1][1]
    assert rope.positions.tolist() == [[0, 1, 5, 6, 18, 19]]
    assert rope.kv_index.tolist() == [0, 1, 25, 26, 58, 59]
    assert attn.n_groups == 0 and attn.start.tolist() == [0, 20, 40] and attn.len.tolist() == [2, 7, 20]
