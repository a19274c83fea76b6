"""What gdn.py refuses before an address reaches the library: arrays of another type, too short, with gaps, tensors that
are not on the device. No GPU: a call that got through would raise the library's error, not ValueError."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import build, gdn

R, T, PAGES, WIDTH = 4, 2, 5, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    gdn.load_library()


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _kv4():
    a = dict(k=_bf16(R, 2, 64), v=_bf16(R, 2, 64), kv_index=_ints(R), pool=torch.zeros((PAGES, 2, 72 * 64), dtype=torch.uint8))
    dims = gdn.make_kv4_dims(a["k"], a["pool"])
    return a, lambda **x: gdn.kv4_store(dims, **{**a, **x}), ("kv_index",)


def _load():
    a, _, names = _kv4()
    dims = gdn.make_kv4_dims(a["k"], a["pool"])
    return a, lambda **x: gdn.kv4_load(dims, **{**a, **x}), names


def _attn():
    a = dict(q=_bf16(R, T, 4, 64), pool=torch.zeros((PAGES, 2, 72 * 64), dtype=torch.uint8), page_table=_ints(R, WIDTH),
             kv_len=_ints(R), q_len=_ints(R), out=_bf16(R, T, 4, 64), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    dims = gdn.make_attn_kv4_dims(a["q"], a["pool"], a["page_table"])
    return a, lambda **x: gdn.attn_kv4(dims, **{**a, **x}), ("page_table", "kv_len", "q_len")


def _beam():
    flags = lambda: torch.zeros((R, T), dtype=torch.uint8)  # noqa: E731
    a = dict(logits=torch.zeros((R, T, 50)), scores=torch.zeros((R, T)), parent=_ints(R, T), token=_ints(R, T),
             new_scores=torch.zeros((R, T)), workspace=torch.zeros(1 << 20, dtype=torch.uint8), done=flags(), new_done=flags())
    return a, lambda **x: gdn.beam_select(**{**a, **x}), ("scores", "parent", "token", "new_scores", "done", "new_done")


def _fork():
    one = ("kv_len", "kv_len_out", "page_src", "page_dst", "parent", "n_new", "state_idx", "state_idx_out", "state_src",
           "state_dst")
    a = dict(page_table=_ints(R, WIDTH), page_table_out=_ints(R, WIDTH), kv_index=_ints(R, T), n_pages=PAGES,
             pinned=torch.zeros(PAGES, dtype=torch.uint8), **{n: _ints(R) for n in one})
    return a, lambda **x: gdn.cache_fork(**{**a, **x}), ("page_table", "page_table_out", "kv_index", "pinned") + one


def _copy():
    a = dict(src=_ints(R), dst=_ints(R))
    pool = torch.zeros((2, PAGES, 16))
    return a, lambda **x: gdn.slots_copy([(pool, *{**a, **x}.values())]), ("src", "dst")


CALLS = dict(kv4_store=_kv4, kv4_load=_load, attn_kv4=_attn, beam_select=_beam, cache_fork=_fork, slots_copy=_copy)


@pytest.mark.parametrize("call", CALLS)
def test_arrays_that_a_kernel_would_misread(call, monkeypatch):
    a, run, names = CALLS[call]()
    monkeypatch.setattr(gdn, "_here", lambda x, name: None)
    for n in names:  # every other array passes
        x = a[n]
        bad = [x.long(), x.float() if x.dtype != torch.float32 else x.double(),
               torch.zeros((*x.shape, 2), dtype=x.dtype)[..., 0], x[:-1].contiguous(), x[:1].expand(x.shape)]
        for b in bad:
            with pytest.raises(ValueError):
                run(**{n: b})


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_another_device(call):
    with pytest.raises(ValueError, match="current device"):
        CALLS[call]()[1]()


def _others(x):
    """What is not x's layout: other types, fewer tokens, heads or channels, other strides."""
    wide = torch.zeros((*x.shape[:-1], 2 * x.shape[-1]), dtype=x.dtype)
    return [x.float(), x[:-1], x[..., :-1, :].contiguous(), x[..., : x.shape[-1] // 2].contiguous(),
            wide[..., :x.shape[-1]], wide[..., ::2], x[:1].expand(x.shape)]


@pytest.mark.parametrize("call,names", [("kv4_store", "kv"), ("kv4_load", "kv"), ("attn_kv4", ("q", "out"))])
def test_tokens_that_are_not_as_the_sizes_say(call, names, monkeypatch):
    a, run, _ = CALLS[call]()
    monkeypatch.setattr(gdn, "_here", lambda x, name: None)
    for n in names:
        for b in _others(a[n]):
            with pytest.raises(ValueError):
                run(**{n: b})


@pytest.mark.parametrize("call", ["kv4_store", "kv4_load", "attn_kv4"])
def test_pools_that_are_not_as_the_sizes_say(call, monkeypatch):
    a, run, _ = CALLS[call]()
    monkeypatch.setattr(gdn, "_here", lambda x, name: None)
    pool = a["pool"]
    for b in (pool.int(), pool[:-1], pool[:, :1], pool[..., ::2], pool[:1].expand(pool.shape)):
        with pytest.raises(ValueError):
            run(pool=b)


@pytest.mark.parametrize("call", ["attn_kv4", "beam_select"])
def test_workspaces_with_gaps(call, monkeypatch):
    a, run, _ = CALLS[call]()
    monkeypatch.setattr(gdn, "_here", lambda x, name: None)
    with pytest.raises(ValueError):
        run(workspace=torch.zeros((1 << 20, 2), dtype=torch.uint8)[:, 0])


def test_arrays_that_pass(monkeypatch):
    x = _ints(2, 3)
    assert gdn._arrays(torch.int32, 20, "abc", None, 1 << 20, x) == [None, 1 << 20, x.data_ptr()]
    with pytest.raises(ValueError, match="b must be a dense torch.int32 tensor of 7 elements"):
        gdn._arrays(torch.int32, 28, "ab", None, x)
    assert gdn._flags(None) is None and gdn._flags(torch.ones(3, dtype=torch.bool)).dtype is torch.uint8
    assert gdn._flags(x) is x
    gdn._here(1 << 20, "an address")
    gdn._here(None, "nothing")
