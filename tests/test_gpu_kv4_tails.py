"""Attention over 4-bit pages where one key outweighs every other by so much that single probabilities are near the end of
fp16's range, and their sum still matters: an early key of the highest score whose value is zero, and tens of thousands
behind it.

Bar: kv4_plain.attend's, with 2^-32 m max|v| as its last term: probabilities are fp16 numbers relative to 2^-7 of the
largest, whose smallest step is 2^-24, so that one is off by at most 2^-25 2^-7 of the largest (attend's 2^-25 is for
probabilities relative to the largest itself)."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from tests import kv4_plain

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


@pytest.mark.parametrize("nats", [15.0, 16.0, 17.0])
@pytest.mark.parametrize("at", [0, 20000])
@pytest.mark.parametrize("rows,T,G,d", [(1024, 1, 1, 64), (800, 2, 5, 128), (400, 8, 4, 256)])
def test_many_small_probabilities_behind_a_large_one(rows, T, G, d, at, nats):
    """As many rows (all over the same pages) as leave each its pages to one CTA or two, where one reference serves them."""
    hk, n = 2, 40000
    g = torch.Generator(device="cuda").manual_seed(d + at)
    pages = n // PAGE
    u = torch.randint(0, 2, (hk, d), generator=g, device="cuda") * 2.0 - 1.0
    k = 0.02 * torch.randn((n, hk, d), generator=g, device="cuda")
    v = 1.0 + 0.1 * torch.randn((n, hk, d), generator=g, device="cuda")
    k[at], v[at] = u, 0.0
    pool = gdn.kv4_pool(pages, hk, d)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    index = torch.arange(n, dtype=torch.int32, device="cuda")
    gdn.kv4_store(gdn.make_kv4_dims(k, pool), k, v, index, pool)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(rows, -1).contiguous()
    q = u[:, None].expand(rows, T, hk, G, d).reshape(rows, T, hk * G, d).to(torch.bfloat16).contiguous()
    scale = nats / d  # q.k of the large one is d, of the others about 0
    dims = gdn.make_attn_kv4_dims(q, pool, table, scale=scale)
    out = torch.empty_like(q)
    lens = torch.full((rows,), n, dtype=torch.int32, device="cuda")
    gdn.attn_kv4(dims, q, pool, table, lens, out, gdn.attn_kv4_workspace(dims))
    gdn.check_status()
    kd, vd = (kv4_plain.decode(pool, i).transpose(1, 2).flatten(0, 1) for i in range(2))
    for h in range(hk):
        ref, bar = kv4_plain.attend(q[0, :, G * h:G * h + G], kd[:, h], vd[:, h], [n - T + t + 1 for t in range(T)], scale)
        bar = bar - (2.0 ** -25 - 2.0 ** -32) * n * vd[:, h].abs().amax(0)
        assert bool((bar < 0.03 * ref.abs()).all())  # it is the small ones that are looked at
        assert float(((out[:, :, G * h:G * h + G].double() - ref).abs() - bar).max()) <= 0
