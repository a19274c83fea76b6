"""The attention operators together, as a hybrid stack uses them (hybrid.py): a prompt's prefill into the pools, then
speculative steps over it -- the GDN layers' verify, the attention layers' verify, acceptance, commit -- eager and as
one captured graph.

Bar of the attention outputs: attn_plain.attend's on the queries, keys and values that the pools and buffers hold
(bit for bit what the kernels read); the pools themselves against the 64-bit norm and rotation within half a bf16 step
and 2^-19 of the head's size; whole numbers and copied states are equal."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from gated_deltanet_recurrence_delta_gb300 import inputs as I
from gated_deltanet_recurrence_delta_gb300.hybrid import AttentionLayers, speculative_step
from gated_deltanet_recurrence_delta_gb300.stack import LayerStack
from tests import attn_plain

pytestmark = pytest.mark.gpu


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


def _check_step(att, layer, q, out, prompts, own_len, T):
    """The step's attention against the pools: own_len keys were there before it."""
    first, start, length = (t.tolist() for t in prompts)
    G = att.hq // att.hk
    for b in range(q.shape[0]):
        g = max(i for i in range(len(start)) if first[i] <= b)
        s = int(att.own_start[b])
        rows = torch.cat((torch.arange(start[g], start[g] + length[g]), torch.arange(s, s + own_len[b] + T))).cuda()
        sees = [length[g] + own_len[b] + t + 1 for t in range(T)]
        for h in range(att.hk):
            ref, bar = attn_plain.attend(q[b, :, h * G:(h + 1) * G], att.k_pool[layer][rows, h],
                                         att.v_pool[layer][rows, h], sees, att.d ** -0.5)
            _within(out[b, :, h * G:(h + 1) * G], ref, bar)


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_then_speculative_steps(captured):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    shape = I.TINY
    B, T, V, L, hq, hk, d, rot = 4, 4, 500, 2, 6, 2, 64, 32
    inv_freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    att = AttentionLayers(hq, hk, d, [dict(q_norm=rand(d), k_norm=rand(d)) for _ in range(L)], inv_freq, 500, B, 40)
    weights = [{n: t.cuda() for n, t in I.decode_batch(seed=s, B=1, shape=shape).items()
                if n in ("A_log", "dt_bias", "conv_w", "norm_w")} for s in range(2)]
    stack = LayerStack(shape, weights, n_slots=B)
    stack.state_pool.copy_(0.1 * torch.randn(stack.state_pool.shape, generator=g, device="cuda"))

    # two prompts, 300 and 170 tokens, packed in the pool rows 0..469
    lens, cu = [300, 170], _ints([0, 300, 470])
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()[None]
    q, out = (torch.empty((470, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for layer in range(L):
        qkv = rand(470, (hq + 2 * hk) * d)
        att.prefill(layer, qkv, cu, pos, torch.arange(470, dtype=torch.int32, device="cuda"), _ints([0, 300]), _ints(lens),
                    q, out)
        gdn.check_status()
        xq, xk, xv = att._split(qkv)
        for got, x, w in ((q, xq, "q_norm"), (att.k_pool[layer][:470], xk, "k_norm")):
            ref = attn_plain.norm_rope(x, att.weights[layer][w], pos, inv_freq, None, rot, False, 1e-6)
            _within(got, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True))
        assert torch.equal(att.v_pool[layer][:470], xv)
        for b, n in enumerate(lens):
            a = 300 * b
            for h in range(hk):
                ref, bar = attn_plain.attend(q[a:a + n, 3 * h:3 * h + 3], att.k_pool[layer][a:a + n, h],
                                             att.v_pool[layer][a:a + n, h], list(range(1, n + 1)), d ** -0.5)
                _within(out[a:a + n, 3 * h:3 * h + 3], ref, bar)

    # speculative steps: rows 0-2 continue the first prompt, row 3 the second
    prompts = (_ints([0, 3, 4]), _ints([0, 300]), _ints(lens))
    state_idx = torch.arange(B, dtype=torch.int32, device="cuda")
    acts = stack.static_acts(B, T)
    qkv = [torch.empty((B, T, (hq + 2 * hk) * d), dtype=torch.bfloat16, device="cuda") for _ in range(L)]
    tokens = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    target, draft = torch.zeros((B, T, V), device="cuda"), torch.zeros((B, T - 1, V), device="cuda")
    uniform = torch.zeros((B, T), device="cuda")
    s = shape
    buf = dict(gdn_out=torch.empty((2, B, T, s.nv, s.dv), dtype=torch.bfloat16, device="cuda"),
               ckpt_state=torch.empty((2, B, T, s.nv, s.dk, s.dv), device="cuda"),
               ckpt_conv=torch.empty((2, B, T, s.Kc, s.C), dtype=torch.bfloat16, device="cuda"),
               q=torch.empty((B, T, hq, d), dtype=torch.bfloat16, device="cuda"),
               attn_out=torch.empty((L, B, T, hq, d), dtype=torch.bfloat16, device="cuda"),
               accept_len=_ints([0] * B), next_token=_ints([0] * B))

    def step():
        speculative_step(stack, att, acts, qkv, state_idx, prompts, tokens, target, draft, uniform, buf)

    def fill():
        for layer in acts:
            for t in layer.values():
                t.copy_(rand(*t.shape))
        for t in qkv:
            t.copy_(rand(*t.shape))
        target.copy_(torch.softmax(2 * torch.randn(target.shape, generator=g, device="cuda"), -1))
        draft.copy_(torch.softmax(torch.log(target[:, :-1]) + 0.3 * torch.randn(draft.shape, generator=g, device="cuda"), -1))
        tokens[:, 1:].copy_(torch.multinomial(draft.flatten(0, 1), 1, generator=g).view(B, T - 1))
        uniform.copy_(torch.rand(uniform.shape, generator=g, device="cuda"))

    graph = None
    if captured:
        fill()
        kept = stack.state_pool.clone(), stack.conv_pool.clone()
        step()  # first use, outside the capture; put back afterwards
        torch.cuda.synchronize()
        stack.state_pool.copy_(kept[0])
        stack.conv_pool.copy_(kept[1])
        att.own_len.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    own = [0] * B
    for _ in range(3):
        fill()
        before = stack.state_pool.clone()
        graph.replay() if captured else step()
        gdn.check_status()
        _check_step(att, L - 1, buf["q"], buf["attn_out"][L - 1], prompts, own, T)
        for b in range(B):
            want = attn_plain.accept(tokens[b].cpu(), target[b].cpu(), draft[b].cpu(), uniform[b].cpu(), T)
            got = int(buf["accept_len"][b]), int(buf["next_token"][b])
            assert got == want
            assert torch.equal(stack.state_pool[:, b], buf["ckpt_state"][:, b, got[0] - 1])
            own[b] += got[0]
        assert att.own_len.tolist() == own and not torch.equal(before, stack.state_pool)
