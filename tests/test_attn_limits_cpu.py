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
