"""The refusals of the attention-layer entry points: every invalid call returns its status on the host and launches
nothing (fake pointers; nothing here reaches a CUDA call)."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import build, gdn

P = 1 << 30  # a fake aligned device pointer


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


def _rope(lib, ptrs=None, **kw):
    d = dict(n_tokens=4, n_q_heads=4, n_kv_heads=2, head_dim=64, rot_dim=64, n_axes=1, adjacent=0, eps=1e-6,
             q_stride=256, k_stride=128, v_stride=128, kv_rows=4)
    d.update(kw)
    names = ("q", "k", "v", "q_weight", "k_weight", "positions", "inv_freq", "axis", "kv_index", "q_out", "k_out", "v_out")
    p = dict.fromkeys(names, P)
    p.update(axis=None, kv_index=None)
    p.update(ptrs or {})
    return gdn.STATUS[lib.gdn_head_norm_rope(ctypes.byref(gdn.RopeDims(**d)), *(p[n] for n in names), None)]


@pytest.mark.parametrize("kw", [dict(n_tokens=-1), dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=96),
                                dict(rot_dim=8), dict(rot_dim=80), dict(rot_dim=-16), dict(n_axes=0), dict(n_axes=9),
                                dict(q_stride=255), dict(q_stride=248), dict(k_stride=120), dict(v_stride=64),
                                dict(kv_rows=3), dict(kv_rows=-1)])
def test_rope_refuses_bad_sizes(lib, kw):
    assert _rope(lib, **kw) == "GDN_ERR_SHAPE"


@pytest.mark.parametrize("ptrs", [dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(v=None),
                                  dict(v_out=None), dict(positions=None), dict(inv_freq=None), dict(q=P + 8),
                                  dict(k_out=P + 2), dict(q_weight=P + 2), dict(positions=P + 2), dict(inv_freq=P + 4),
                                  dict(kv_index=P + 1)])
def test_rope_refuses_bad_pointers(lib, ptrs):
    assert _rope(lib, ptrs) == "GDN_ERR_ARG"


def test_rope_refuses_nan_eps_and_null_dims_and_takes_no_tokens(lib):
    assert _rope(lib, eps=float("nan")) == "GDN_ERR_ARG"
    assert _rope(lib, eps=-1.0) == "GDN_ERR_ARG"
    assert gdn.STATUS[lib.gdn_head_norm_rope(None, *[P] * 12, None)] == "GDN_ERR_ARG"
    assert _rope(lib, n_tokens=0) == "GDN_OK"


ATTN = dict(B=2, T=3, n_tokens=6, n_groups=1, n_q_heads=4, n_kv_heads=2, head_dim=64, scale=0.125, q_stride=256,
            kv_stride=128, kv_rows=10)


def _prefill(lib, ptrs=None, **kw):
    names = ("q", "k", "v", "cu_seqlens", "kv_start", "kv_len", "out")
    p = {**dict.fromkeys(names, P), **(ptrs or {})}
    return gdn.STATUS[lib.gdn_attn_prefill(ctypes.byref(gdn.AttnDims(**{**ATTN, **kw})), *(p[n] for n in names), None)]


def _shared(lib, ptrs=None, **kw):
    names = ("q", "k", "v", "group_rows", "prefix_start", "prefix_len", "suffix_start", "suffix_len", "q_len", "out",
             "workspace")
    p = {**dict.fromkeys(names, P), **(ptrs or {})}
    size = p.pop("size", 1 << 40)
    return gdn.STATUS[lib.gdn_attn_shared_prefix(ctypes.byref(gdn.AttnDims(**{**ATTN, **kw})), *(p[n] for n in names),
                                                 size, None)]


BAD_SIZES = [dict(B=-1), dict(n_tokens=-1), dict(n_groups=-1), dict(n_groups=3), dict(n_q_heads=0), dict(n_q_heads=3),
             dict(n_q_heads=130, q_stride=130 * 64), dict(head_dim=32), dict(head_dim=96), dict(q_stride=252),
             dict(q_stride=128), dict(kv_stride=64), dict(kv_stride=129), dict(kv_rows=-1), dict(kv_rows=1 << 31),
             dict(kv_stride=1 << 33)]


@pytest.mark.parametrize("kw", BAD_SIZES)
def test_attention_refuses_bad_sizes(lib, kw):
    assert _prefill(lib, **kw) == "GDN_ERR_SHAPE"
    assert _shared(lib, **kw) == "GDN_ERR_SHAPE"
    assert lib.gdn_attn_workspace_size(ctypes.byref(gdn.AttnDims(**{**ATTN, **kw}))) == 0


@pytest.mark.parametrize("ptrs", [{n: x} for n in ("q", "k", "v", "out") for x in (None, P + 8)]
                         + [dict(cu_seqlens=None), dict(kv_start=None), dict(kv_len=None), dict(kv_len=P + 2)])
def test_prefill_refuses_bad_pointers(lib, ptrs):
    assert _prefill(lib, ptrs) == "GDN_ERR_ARG"


@pytest.mark.parametrize("ptrs", [{n: x} for n in ("q", "k", "v", "out") for x in (None, P + 8)]
                         + [{n: x} for n in ("group_rows", "prefix_start", "prefix_len", "suffix_start", "suffix_len")
                            for x in (None, P + 2)] + [dict(q_len=P + 1)])
def test_shared_refuses_bad_pointers(lib, ptrs):
    assert _shared(lib, ptrs) == "GDN_ERR_ARG"


def test_shared_refuses_bad_tokens_and_workspaces(lib):
    assert _shared(lib, T=0, n_tokens=0) == "GDN_ERR_SHAPE"
    assert _shared(lib, T=65, n_tokens=130) == "GDN_ERR_SHAPE"
    assert _shared(lib, n_tokens=5) == "GDN_ERR_SHAPE"
    need = lib.gdn_attn_workspace_size(ctypes.byref(gdn.AttnDims(**ATTN)))
    assert need > 0
    assert _shared(lib, dict(workspace=None)) == "GDN_ERR_WORKSPACE"
    assert _shared(lib, dict(workspace=P + 16)) == "GDN_ERR_WORKSPACE"
    assert _shared(lib, dict(size=need - 1)) == "GDN_ERR_WORKSPACE"
    assert _shared(lib, B=0, n_tokens=0, n_groups=0) == "GDN_OK"
    assert _prefill(lib, B=0, n_groups=0) == "GDN_OK" and _prefill(lib, n_tokens=0) == "GDN_OK"
    for scale in ("nan", "inf", "-inf"):
        assert _prefill(lib, scale=float(scale)) == "GDN_ERR_ARG" and _shared(lib, scale=float(scale)) == "GDN_ERR_ARG"
    huge = dict(B=1 << 24, T=64, n_tokens=1 << 30, n_q_heads=64, n_kv_heads=1, q_stride=4096)
    assert _shared(lib, **huge) == "GDN_ERR_SHAPE"  # more than a grid holds


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=(1 << 20) + 1), dict(T=0), dict(T=33), dict(V=0), dict(V=(1 << 30) + 1)])
def test_accept_refuses_bad_sizes(lib, kw):
    d = {**dict(B=2, T=3, V=10), **kw}
    assert gdn.STATUS[lib.gdn_accept_draft(d["B"], d["T"], d["V"], *[P] * 7, None)] == "GDN_ERR_SHAPE"


@pytest.mark.parametrize("at", range(7))
def test_accept_refuses_bad_pointers(lib, at):
    ptrs = [P] * 7
    ptrs[at] = P + 2
    assert gdn.STATUS[lib.gdn_accept_draft(2, 3, 10, *ptrs, None)] == "GDN_ERR_ARG"
    ptrs[at] = None
    if at not in (2, 4):  # draft_probs and n_tokens may be absent
        assert gdn.STATUS[lib.gdn_accept_draft(2, 3, 10, *ptrs, None)] == "GDN_ERR_ARG"
    assert gdn.STATUS[lib.gdn_accept_draft(0, 3, 10, *[P] * 7, None)] == "GDN_OK"


def test_binding_refuses_layouts_it_cannot_describe():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    assert gdn.make_attn_dims(x, x, B=1).q_stride == 128
    fused = torch.zeros((4, 6 * 64), dtype=torch.bfloat16)
    assert gdn.make_attn_dims(fused[:, :256].view(4, 4, 64), fused[:, 256:].view(4, 2, 64), B=1).kv_stride == 384
    for bad in (x.float(), x[..., ::2], x.transpose(0, 1), x[0]):
        with pytest.raises(ValueError):
            gdn.make_attn_dims(bad, x, B=1)
    rows = torch.zeros((3, 5, 2, 64), dtype=torch.bfloat16)
    assert gdn.make_attn_dims(rows, x, B=3, T=5).n_tokens == 15
    with pytest.raises(ValueError):
        gdn.make_attn_dims(rows[:, :4], x, B=3, T=4)
