"""Scales and layouts at the edge of what the attention entry points take, refused or taken on the host (fake pointers;
nothing here reaches a CUDA call)."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import build, gdn

P = 1 << 30  # a fake aligned device pointer


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


# the kernels multiply by scale log2(e), 1.4427 times the scale: 3.4028e38 / 1.4427 = 2.3587e38 is the most that stays finite
@pytest.mark.parametrize("scale,ok", [(2.3586e38, True), (2.3588e38, False), (3.0e38, False), (3.4e38, False)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scales_whose_product_with_log2e_is_not_finite_are_refused(lib, scale, ok, sign):
    d = dict(B=2, T=3, n_tokens=6, n_groups=1, n_q_heads=4, n_kv_heads=2, head_dim=64, scale=sign * scale, q_stride=256,
             kv_stride=128, kv_rows=10)
    # NULL workspace and no queries: what follows the check of the sizes, without a CUDA call
    shared = lib.gdn_attn_shared_prefix(ctypes.byref(gdn.AttnDims(**d)), *[P] * 10, None, 0, None)
    assert gdn.STATUS[shared] == ("GDN_ERR_WORKSPACE" if ok else "GDN_ERR_ARG")
    assert (lib.gdn_attn_workspace_size(ctypes.byref(gdn.AttnDims(**d))) > 0) == ok
    empty = {**d, "n_tokens": 0}
    prefill = lib.gdn_attn_prefill(ctypes.byref(gdn.AttnDims(**empty)), *[P] * 7, None)
    assert gdn.STATUS[prefill] == ("GDN_OK" if ok else "GDN_ERR_ARG")


def _fake(monkeypatch):
    names = ("gdn_head_norm_rope", "gdn_attn_prefill", "gdn_attn_shared_prefix")
    calls = []
    fake = type("Lib", (), {n: staticmethod(lambda *a, n=n: calls.append(n) or 0) for n in names})
    monkeypatch.setattr(gdn, "load_library", lambda *a: fake)
    monkeypatch.setattr(gdn, "_stream", lambda s: 0)
    return calls


def test_values_spaced_otherwise_than_the_sizes_say_are_refused(monkeypatch):
    """The sizes hold one spacing for k and v (attention), or v's as it was given or k's (norms): values of another
    spacing would be read at the wrong places, past their end too."""
    calls = _fake(monkeypatch)
    fused = torch.zeros((8, (4 + 2 + 2) * 64), dtype=torch.bfloat16)
    q, k, v = (fused[:, a * 64:z * 64].unflatten(1, (z - a, 64)) for a, z in ((0, 4), (4, 6), (6, 8)))
    dense = v.contiguous()
    ints = torch.zeros(9, dtype=torch.int32)

    dims = gdn.make_attn_dims(q, k, B=1)
    gdn.attn_prefill(dims, q, k, v, ints, q)
    with pytest.raises(ValueError):
        gdn.attn_prefill(dims, q, k, dense, ints, q)
    with pytest.raises(ValueError):  # sizes of another pool than the one that is read
        gdn.attn_prefill(dims, q, k.contiguous(), v, ints, q)
    gdn.attn_prefill(gdn.make_attn_dims(q, dense, B=1), q, dense, dense, ints, q)

    dims, ws = gdn.make_attn_dims(q, k, B=8), torch.zeros(1)
    gdn.attn_shared_prefix(dims, q, k, v, ints, ints, ints, ints, ints, q, ws)
    with pytest.raises(ValueError):
        gdn.attn_shared_prefix(dims, q, k, dense, ints, ints, ints, ints, ints, q, ws)

    def rope(v, sized=None):
        gdn.head_norm_rope(gdn.make_rope_dims(q, k, 0, v=sized), q, k, v, None, None, None, None, q, dense, dense)

    rope(v)
    rope(dense, sized=dense)
    rope(None)
    with pytest.raises(ValueError):
        rope(dense)
    # one token has no spacing; raw addresses and flat tensors are taken as they are
    one = gdn.make_attn_dims(q[:1], k[:1], B=1)
    gdn.attn_prefill(one, q[:1], k[:1], dense[:1], ints, q)
    gdn.attn_prefill(dims, P, P, P, P, P)
    gdn.attn_prefill(dims, q, k.flatten(1), dense.flatten(), ints, q)
    assert calls == ["gdn_attn_prefill"] * 2 + ["gdn_attn_shared_prefix"] + ["gdn_head_norm_rope"] * 3 + ["gdn_attn_prefill"] * 3
