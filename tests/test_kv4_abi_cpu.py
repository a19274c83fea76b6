"""The refusals of the paged 4-bit cache's and the beam search's entry points: every invalid call returns its status on
the host and launches nothing (fake pointers; nothing here reaches a CUDA call). And the plain forms against themselves."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import build, gdn
from tests import kv4_plain

P = 1 << 30  # a fake aligned device pointer


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


KV4 = dict(n_tokens=4, n_kv_heads=2, head_dim=64, n_pages=3, k_exp=0, v_exp=0, k_stride=128, v_stride=128)


def _kv4(lib, ptrs=None, **kw):
    p = {**dict.fromkeys(("k", "v", "kv_index", "pool"), P), **(ptrs or {})}
    d = gdn.Kv4Dims(**{**KV4, **kw})
    a = lib.gdn_kv4_store(ctypes.byref(d), p["k"], p["v"], p["kv_index"], p["pool"], None)
    b = lib.gdn_kv4_load(ctypes.byref(d), p["pool"], p["kv_index"], p["k"], p["v"], None)
    assert a == b
    return gdn.STATUS[a]


@pytest.mark.parametrize("kw", [dict(n_tokens=-1), dict(n_kv_heads=0), dict(n_kv_heads=4097), dict(head_dim=32),
                                dict(head_dim=96), dict(n_pages=-1), dict(n_pages=1 << 25), dict(k_exp=33),
                                dict(v_exp=-33), dict(k_stride=120), dict(v_stride=129), dict(k_stride=1 << 32)])
def test_kv4_refuses_bad_sizes(lib, kw):
    assert _kv4(lib, **kw) == "GDN_ERR_SHAPE"


@pytest.mark.parametrize("ptrs", [{n: x} for n in ("k", "v", "pool") for x in (None, P + 8)]
                         + [dict(kv_index=None), dict(kv_index=P + 2)])
def test_kv4_refuses_bad_pointers(lib, ptrs):
    assert _kv4(lib, ptrs) == "GDN_ERR_ARG"
    assert _kv4(lib, n_tokens=0) == "GDN_OK"
    assert gdn.STATUS[lib.gdn_kv4_store(None, P, P, P, P, None)] == "GDN_ERR_ARG"


ATTN = dict(B=2, T=3, n_q_heads=4, n_kv_heads=2, head_dim=64, n_pages=5, max_pages=4, k_exp=0, v_exp=0, scale=0.125,
            q_stride=256)


def _attn(lib, ptrs=None, **kw):
    names = ("q", "pool", "page_table", "kv_len", "q_len", "out", "workspace")
    p = {**dict.fromkeys(names, P), **(ptrs or {})}
    size = p.pop("size", 1 << 40)
    return gdn.STATUS[lib.gdn_attn_kv4(ctypes.byref(gdn.AttnKv4Dims(**{**ATTN, **kw})), *(p[n] for n in names), size, None)]


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=(1 << 20) + 1), dict(T=0), dict(T=65), dict(n_q_heads=0),
                                dict(n_kv_heads=0), dict(n_q_heads=3), dict(n_q_heads=130, q_stride=130 * 64),
                                dict(head_dim=32), dict(head_dim=96), dict(n_pages=-1), dict(n_pages=1 << 25),
                                dict(max_pages=-1), dict(max_pages=1 << 25), dict(k_exp=-33), dict(v_exp=33),
                                dict(q_stride=252), dict(q_stride=128), dict(q_stride=1 << 32)])
def test_attention_refuses_bad_sizes(lib, kw):
    assert _attn(lib, **kw) == "GDN_ERR_SHAPE"
    assert lib.gdn_attn_kv4_workspace_size(ctypes.byref(gdn.AttnKv4Dims(**{**ATTN, **kw}))) == 0


@pytest.mark.parametrize("ptrs", [{n: x} for n in ("q", "pool", "out") for x in (None, P + 8)]
                         + [{n: x} for n in ("page_table", "kv_len") for x in (None, P + 2)] + [dict(q_len=P + 1)])
def test_attention_refuses_bad_pointers(lib, ptrs):
    assert _attn(lib, ptrs) == "GDN_ERR_ARG"


def test_attention_refuses_bad_scales_and_workspaces(lib):
    for scale in ("nan", "inf", "-inf"):
        assert _attn(lib, scale=float(scale)) == "GDN_ERR_ARG"
    assert _attn(lib, scale=1e38, k_exp=32) == "GDN_ERR_ARG"
    assert _attn(lib, dict(workspace=None)) == "GDN_ERR_WORKSPACE"
    assert _attn(lib, dict(workspace=P + 16)) == "GDN_ERR_WORKSPACE"
    assert _attn(lib, dict(size=0)) == "GDN_ERR_WORKSPACE"
    assert _attn(lib, B=0) == "GDN_OK"


BEAM = dict(n_groups=2, beams=3, vocab=50, half=0, eos=-1, row_stride=50)


def _beam(lib, ptrs=None, **kw):
    names = ("logits", "scores", "done", "parent", "token", "new_scores", "new_done", "workspace")
    p = {**dict.fromkeys(names, P), **(ptrs or {})}
    size = p.pop("size", 1 << 40)
    return gdn.STATUS[lib.gdn_beam_select(ctypes.byref(gdn.BeamDims(**{**BEAM, **kw})), *(p[n] for n in names), size, None)]


@pytest.mark.parametrize("kw", [dict(n_groups=-1), dict(beams=0), dict(beams=33), dict(n_groups=1 << 16), dict(vocab=0),
                                dict(vocab=(1 << 24) + 1, row_stride=1 << 25), dict(eos=-2), dict(eos=50),
                                dict(row_stride=49), dict(row_stride=1 << 40)])
def test_beam_refuses_bad_sizes(lib, kw):
    assert _beam(lib, **kw) == "GDN_ERR_SHAPE"
    assert lib.gdn_beam_workspace_size(ctypes.byref(gdn.BeamDims(**{**BEAM, **kw}))) == 0


@pytest.mark.parametrize("ptrs", [dict(logits=None), dict(logits=P + 2), dict(scores=None), dict(parent=None),
                                  dict(token=P + 2), dict(new_scores=None), dict(done=None), dict(new_done=None)])
def test_beam_refuses_bad_pointers(lib, ptrs):
    assert _beam(lib, ptrs) == "GDN_ERR_ARG"
    need = lib.gdn_beam_workspace_size(ctypes.byref(gdn.BeamDims(**BEAM)))
    assert need > 0
    for bad in (dict(workspace=None), dict(workspace=P + 8), dict(size=need - 1)):
        assert _beam(lib, bad) == "GDN_ERR_WORKSPACE"
    assert _beam(lib, n_groups=0) == "GDN_OK"


FORK = dict(n_rows=4, T=2, max_pages=3, n_pages=20)
FORK_PTRS = ("parent", "n_new", "page_table", "kv_len", "pinned", "page_table_out", "kv_len_out", "kv_index", "page_src",
             "page_dst", "state_idx", "state_idx_out", "state_src", "state_dst")


def _fork(lib, ptrs=None, **kw):
    p = {n: P + 64 * i for i, n in enumerate(FORK_PTRS)}
    p.update(ptrs or {})
    return gdn.STATUS[lib.gdn_cache_fork(ctypes.byref(gdn.ForkDims(**{**FORK, **kw})), *(p[n] for n in FORK_PTRS), None)]


@pytest.mark.parametrize("kw", [dict(n_rows=-1), dict(n_rows=1025), dict(T=-1), dict(T=(1 << 20) + 1), dict(n_pages=-1),
                                dict(n_pages=(1 << 20) + 1), dict(max_pages=-1), dict(max_pages=(1 << 20) + 1)])
def test_fork_refuses_bad_sizes(lib, kw):
    assert _fork(lib, **kw) == "GDN_ERR_SHAPE"


@pytest.mark.parametrize("ptrs", [{n: P + 2} for n in FORK_PTRS if n != "pinned"]
                         + [{n: None} for n in FORK_PTRS if n not in ("parent", "n_new", "pinned")]
                         + [dict(page_table=P, page_table_out=P), dict(kv_len=P, kv_len_out=P),
                            dict(state_idx=P, state_idx_out=P)])
def test_fork_refuses_bad_pointers(lib, ptrs):
    assert _fork(lib, ptrs) == "GDN_ERR_ARG"
    assert _fork(lib, n_rows=0) == "GDN_OK"


def _copy(lib, n_pools=1, **kw):
    d = dict(base=P, src=P, dst=P, slot_bytes=64, n=2, n_layers=3, n_slots=4)
    arr = (gdn.SlotPool * 8)(*[gdn.SlotPool(**{**d, **kw}) for _ in range(8)])
    return gdn.STATUS[lib.gdn_slots_copy(arr, n_pools, None)]


def test_slots_copy_refuses(lib):
    for kw in (dict(slot_bytes=24), dict(slot_bytes=-16), dict(n=-1), dict(n_layers=-1), dict(n_slots=-1),
               dict(n=1 << 12, n_layers=1 << 9), dict(n_pools=5), dict(n_pools=-1), dict(slot_bytes=1 << 40, n=1 << 20, n_layers=1)):
        assert _copy(lib, **kw) == "GDN_ERR_SHAPE"
    for kw in (dict(base=None), dict(base=P + 8), dict(src=None), dict(dst=P + 2)):
        assert _copy(lib, **kw) == "GDN_ERR_ARG"
    for kw in (dict(n=0), dict(n_layers=0), dict(slot_bytes=0), dict(n_pools=0)):
        assert _copy(lib, **kw) == "GDN_OK"
    assert gdn.STATUS[lib.gdn_slots_copy(None, 1, None)] == "GDN_ERR_ARG"


def test_binding_refuses_layouts_it_cannot_describe():
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pool = torch.zeros((3, 2, 72 * 64), dtype=torch.uint8)
    assert gdn.make_kv4_dims(k, pool).n_pages == 3
    table = torch.zeros((4, 5), dtype=torch.int32)
    q = torch.zeros((4, 1, 6, 64), dtype=torch.bfloat16)
    d = gdn.make_attn_kv4_dims(q, pool, table)
    assert (d.B, d.T, d.n_q_heads, d.n_kv_heads, d.max_pages, d.q_stride) == (4, 1, 6, 2, 5, 384)
    for bad in (lambda: gdn.make_kv4_dims(k, pool[:, :1]), lambda: gdn.make_kv4_dims(k, pool[..., ::2]),
                lambda: gdn.make_kv4_dims(k, pool.int()), lambda: gdn.make_attn_kv4_dims(q[:, 0], pool, table),
                lambda: gdn.make_attn_kv4_dims(q, pool, table[:2]), lambda: gdn.make_attn_kv4_dims(q, pool, table.long()),
                lambda: gdn.make_attn_kv4_dims(q, pool, table.T), lambda: gdn.make_beam_dims(torch.zeros(4, 5)),
                lambda: gdn.make_beam_dims(torch.zeros(2, 4, 5).double()),
                lambda: gdn.make_beam_dims(torch.zeros(2, 5, 4).transpose(1, 2)),
                lambda: gdn.make_beam_dims(torch.zeros(2, 8, 5)[:, :4]),
                lambda: gdn.slots_copy([(pool.transpose(0, 1), table[0], table[0])]),
                lambda: gdn.slots_copy([(pool, table[0], table[0, :2])]),
                lambda: gdn.cache_fork(table, None, table[:, :3].contiguous(), None, None, None, None, 3)):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros((2, 4, 7))[..., :5]
    assert gdn.make_beam_dims(wide).row_stride == 7


def test_plain_pages_hold_what_quantise_says():
    g = torch.Generator().manual_seed(1)
    k = torch.randn((2, 64, 3, 64), generator=g).to(torch.bfloat16)
    v = 0.01 * torch.randn((2, 64, 3, 64), generator=g)
    v[0, 5, 1, 20], v[1, 63, 2, 63] = math.nan, math.inf
    pool = kv4_plain.encode(k, v, 0, -3)
    assert pool.shape == (2, 3, 72 * 64)
    for i, (x, exp) in enumerate(((k, 0), (v, -3))):
        assert torch.equal(kv4_plain.decode(pool, i, exp).nan_to_num(-1e9),
                           kv4_plain.values(x.transpose(1, 2), exp).nan_to_num(-1e9))
    bf = torch.arange(256, dtype=torch.uint8)
    scales = kv4_plain.scale_value(bf[:127])
    assert torch.equal(scales.float(), bf[:127].view(torch.float8_e4m3fn).float())
    assert torch.equal(kv4_plain.e4m3(scales), scales)


def test_plain_fork_by_hand():
    """Three rows of a table of 3: row 0 (70 tokens, pages 4, 1), row 1 (64, page 0), row 2 (3, page 2)."""
    table, lens = [[4, 1, -1], [0, -1, -1], [2, -1, -1]], [70, 64, 3]
    r = kv4_plain.fork(table, lens, 8, 1, parent=[0, 0, 1], state=[5, 6, 7])
    # page 1 stays with row 0, row 1 copies it to the first free page (2: row 2's old page); row 2 needs a new page (3)
    assert r["table"] == [[4, 1], [4, 2], [0, 3]] and r["kv_len"] == [71, 71, 65]
    assert r["page_src"] == [-1, 1, -1] and r["page_dst"] == [-1, 2, -1]
    assert r["kv_index"] == [[64 + 6], [128 + 6], [192]]
    assert r["state_idx"] == [5, 7, 6] and r["state_src"] == [-1, 5, -1] and r["state_dst"] == [-1, 7, -1]
    r = kv4_plain.fork(table, lens, 5, 60, parent=[0, 1, 2], pinned=[0, 0, 0, 1, 0])
    assert r["full"] and r["kv_len"] == [130 - 60, 64, 63]  # both rows that need a page find none


def test_binding_looks_at_strides_in_every_call():
    """Also where the sizes were made from that very tensor, which has been laid out anew since."""
    pool = torch.zeros((2, 2, 72 * 64), dtype=torch.uint8)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    v, index = k.clone(), torch.zeros(4, dtype=torch.int32)
    dims = gdn.make_kv4_dims(k, pool)
    k.as_strided_((3, 2, 64), (144, 64, 1))
    for call in (lambda: gdn.kv4_store(dims, k, v, index, pool), lambda: gdn.kv4_load(dims, pool, index, v, k)):
        with pytest.raises(ValueError):
            call()


def test_binding_reads_sizes_of_any_strides():
    q = torch.zeros((3, 1, 6, 64), dtype=torch.bfloat16)
    pool, table = torch.zeros((2, 2, 72 * 64), dtype=torch.uint8), torch.zeros((3, 5), dtype=torch.int32)
    wide = torch.zeros((3, 1, 10, 64), dtype=torch.bfloat16)[:, :, 2:8]
    for x, stride in ((q, 384), (wide, 640), (q.transpose(0, 1).contiguous().transpose(0, 1), 384)):
        dims = gdn.make_attn_kv4_dims(x, pool, table)
        assert (dims.B, dims.T, dims.n_q_heads, dims.n_kv_heads, dims.head_dim, dims.max_pages, dims.q_stride) == (
            3, 1, 6, 2, 64, 5, stride)
    rows = torch.zeros((3, 4, 10, 64), dtype=torch.bfloat16)
    assert gdn.make_attn_kv4_dims(rows[:, :, :6], pool, table).q_stride == 640
    for bad in (rows[:, :2], rows.transpose(2, 3), rows.float(), rows[0]):
        with pytest.raises(ValueError):
            gdn.make_attn_kv4_dims(bad, pool, table)
    k = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    dims = gdn.make_kv4_dims(k[:, :2], pool, v=torch.zeros((4, 2, 64), dtype=torch.bfloat16))
    assert (dims.k_stride, dims.v_stride) == (256, 128)
    assert gdn.make_kv4_dims(k[:, :2], pool, v=k[:, 2:]).v_stride == 256
    with pytest.raises(ValueError):
        gdn.make_kv4_dims(k[:, :2], pool, v=k[:, ::2])
