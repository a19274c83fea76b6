"""AttentionLayers and speculative_step on the GPU where a row's room ends, on a stream of their own, without shared
prompts, and in every layer of a stack.

Bar of the attention outputs: attn_plain.attend's on the queries, keys and values that the pools and buffers hold (bit
for bit what the kernels read); whole numbers, copied states and repeated calls are equal."""
import pytest
import torch

from gated_deltanet_recurrence_delta_gb300 import gdn
from gated_deltanet_recurrence_delta_gb300 import inputs as I
from gated_deltanet_recurrence_delta_gb300.hybrid import AttentionLayers, speculative_step
from gated_deltanet_recurrence_delta_gb300.stack import LayerStack
from tests import attn_plain

pytestmark = pytest.mark.gpu

HQ, HK, D, ROT = 6, 2, 64, 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gated_deltanet_recurrence_delta_gb300 import build
    build.build()
    gdn.load_library()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _layers(g, n_rows, room, prompt_rows, n_layers=1):
    inv_freq = 1e4 ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device="cuda") / ROT)
    att = AttentionLayers(HQ, HK, D, [dict(q_norm=_rand(g, D), k_norm=_rand(g, D)) for _ in range(n_layers)], inv_freq,
                          prompt_rows, n_rows, room)
    att.k_pool.copy_(_rand(g, *att.k_pool.shape))
    att.v_pool.copy_(_rand(g, *att.v_pool.shape))
    return att


def _check_rows(att, layer, q, out, prompt, own, real):
    """Row b: `own[b]` keys were there before the step, real[b] tokens are new; prompt: (start, length) of every row."""
    G = HQ // HK
    for b in range(q.shape[0]):
        s, (p0, p), n = int(att.own_start[b]), prompt[b], real[b]
        assert bool((out[b, n:] == 0).all()), f"row {b}: outputs of tokens that are not there"
        rows = torch.cat((torch.arange(p0, p0 + p), torch.arange(s, s + own[b] + n))).cuda()
        for h in range(HK):
            ref, bar = attn_plain.attend(q[b, :n, h * G:(h + 1) * G], att.k_pool[layer][rows, h],
                                         att.v_pool[layer][rows, h], [p + own[b] + t + 1 for t in range(n)], D ** -0.5)
            over = (out[b, :n, h * G:(h + 1) * G].double() - ref).abs() - bar
            assert n == 0 or float(over.max()) <= 0, f"row {b}, key head {h}: {float(over.max()):.3e} beyond the bar"


# ------------------------------------------------------------- rows and rooms

@pytest.mark.parametrize("T", [1, 4])
def test_a_row_at_the_end_of_its_room_sees_its_own_keys_only(T):
    """Rows with place for all, some and none of the step's tokens; the rows behind them hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(T)
    att = _layers(g, 6, 10, 50)
    own = [10 - T, 0, 10 - max(1, T // 2), 0, 10, 0]  # rows 1, 3 and 5 follow the ones that end
    for b in (1, 3, 5):
        for pool in (att.k_pool, att.v_pool):
            pool[:, 50 + 10 * b:60 + 10 * b] = float("nan")
    att.own_len.copy_(_ints(own))
    real = [T, T, max(1, T // 2), T, 0, T]
    prompts = (_ints([0, 6]), _ints([0]), _ints([50]))
    qkv, q = _rand(g, 6, T, (HQ + 2 * HK) * D), torch.empty((6, T, HQ, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    pools = att.k_pool.clone(), att.v_pool.clone()
    att.step(0, qkv, *prompts, q, out)
    with pytest.raises(gdn.GdnError) as e:  # row 4 is full
        gdn.check_status()
    assert e.value.name == "GDN_ERR_INDEX"
    _check_rows(att, 0, q, out, [(0, 50)] * 6, own, real)
    written = torch.zeros(att.kv_rows, dtype=torch.bool, device="cuda")
    for b in range(6):
        written[50 + 10 * b + own[b]:50 + 10 * b + own[b] + real[b]] = True
    for pool, was in zip((att.k_pool, att.v_pool), pools):
        assert torch.equal(pool[0][~written].view(torch.int16), was[0][~written].view(torch.int16))
    att.own_len[4] = 0  # without the full row nothing is reported
    att.step(0, qkv, *prompts, q, out)
    gdn.check_status()


def test_speculative_steps_until_the_room_is_full():
    """Every draft is accepted, so three rows of 10 places fill up at different steps; then they stay as they are."""
    g = torch.Generator(device="cuda").manual_seed(7)
    B, T, V, L, s = 3, 4, 50, 2, I.TINY
    att = _layers(g, B, 10, 30, L)
    weights = [{n: t.cuda() for n, t in I.decode_batch(seed=x, B=1, shape=s).items()
                if n in ("A_log", "dt_bias", "conv_w", "norm_w")} for x in range(2)]
    stack = LayerStack(s, weights, n_slots=B)
    acts = stack.static_acts(B, T)
    for layer in acts:
        for t in layer.values():
            t.copy_(_rand(g, *t.shape))
    att.own_len.copy_(_ints([0, 5, 9]))
    target = torch.softmax(torch.randn((B, T, V), generator=g, device="cuda"), -1)
    tokens = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    uniform = torch.zeros((B, T), device="cuda")  # 0 < target: everything stands
    buf = dict(gdn_out=torch.empty((2, B, T, s.nv, s.dv), dtype=torch.bfloat16, device="cuda"),
               ckpt_state=torch.empty((2, B, T, s.nv, s.dk, s.dv), device="cuda"),
               ckpt_conv=torch.empty((2, B, T, s.Kc, s.C), dtype=torch.bfloat16, device="cuda"),
               q=torch.empty((B, T, HQ, D), dtype=torch.bfloat16, device="cuda"),
               attn_out=torch.empty((L, B, T, HQ, D), dtype=torch.bfloat16, device="cuda"),
               accept_len=_ints([0] * B), next_token=_ints([0] * B))
    own = [0, 5, 9]
    for i, want in enumerate([(4, 4, 1), (4, 1, 0), (2, 0, 0), (0, 0, 0)]):
        before = stack.state_pool.clone()
        qkv = [_rand(g, B, T, (HQ + 2 * HK) * D) for _ in range(L)]
        speculative_step(stack, att, acts, qkv, torch.arange(B, dtype=torch.int32, device="cuda"),
                         (_ints([0, B]), _ints([0]), _ints([30])), tokens, target, None, uniform, buf)
        if 0 in want:
            with pytest.raises(gdn.GdnError) as e:
                gdn.check_status()
            assert e.value.name == "GDN_ERR_INDEX"
        else:
            gdn.check_status()
        assert tuple(buf["accept_len"].tolist()) == want, f"step {i}"
        _check_rows(att, L - 1, buf["q"], buf["attn_out"][L - 1], [(0, 30)] * B, own, want)
        for b, n in enumerate(want):
            own[b] += n
            assert torch.equal(stack.state_pool[:, b], buf["ckpt_state"][:, b, n - 1] if n else before[:, b])
            assert n > 0 or int(buf["next_token"][b]) == -1
        assert att.own_len.tolist() == own
    assert own == [10, 10, 10]


# -------------------------------------------------------------------- streams

@pytest.mark.parametrize("held", ["side", "current"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_steps_on_a_stream_of_their_own(held, as_handle):
    """The stream's work, or the current stream's, lies milliseconds behind; memory that a step gave back is reused at
    once. Both steps give what they give on the current stream."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T, prompts = 5, 3, (_ints([0, 2, 5]), _ints([0, 20]), _ints([20, 30]))
    qkv = [_rand(g, B, T, (HQ + 2 * HK) * D) for _ in range(2)]
    accept = _ints([1, 3, 2, 1, 2])
    start = [2, 0, 7, 1, 4]
    results = []
    for stream in (None, torch.cuda.Stream()):
        g.manual_seed(4)
        att = _layers(g, B, 20, 50)
        att.own_len.copy_(_ints(start))
        q = torch.empty((B, T, HQ, D), dtype=torch.bfloat16, device="cuda")
        outs = [torch.full_like(q, 7.0) for _ in range(2)]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream if held == "side" else torch.cuda.current_stream()):
                torch.cuda._sleep(10_000_000)
        on = stream if stream is None or not as_handle else stream.cuda_stream
        for x, out in zip(qkv, outs):
            att.step(0, x, *prompts, q, out, stream=on)
            if stream is not None:  # small blocks that the step freed, if they are the current stream's
                for n in (1, B, B * T, 4 * B * T):
                    torch.full((n,), 1 << 20, dtype=torch.int32, device="cuda")
            att.advance(accept, stream=on)
        gdn.check_status(stream)
        torch.cuda.synchronize()
        results.append((*outs, att.k_pool, att.v_pool, att.own_len))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[1][-1].tolist() == [x + 2 * y for x, y in zip(start, accept.tolist())]


# ---------------------------------------------------- rows without a prompt

@pytest.mark.parametrize("T", [1, 3])
def test_rows_without_a_shared_prompt(T):
    g = torch.Generator(device="cuda").manual_seed(5)
    att = _layers(g, 4, 300, 0)
    own = [0, 130, 7, 300 - T]
    att.own_len.copy_(_ints(own))
    qkv, q = _rand(g, 4, T, (HQ + 2 * HK) * D), torch.empty((4, T, HQ, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    att.step(0, qkv, None, None, None, q, out)
    gdn.check_status()
    _check_rows(att, 0, q, out, [(0, 0)] * 4, own, [T] * 4)
    xq, xk, xv = att._split(qkv.flatten(0, 1))
    pos = torch.cat([o + torch.arange(T) for o in own]).int().cuda()[None]
    at = torch.cat([300 * b + own[b] + torch.arange(T) for b in range(4)]).cuda()
    for got, x, w in ((q.flatten(0, 1), xq, "q_norm"), (att.k_pool[0][at], xk, "k_norm")):
        ref = attn_plain.norm_rope(x, att.weights[0][w], pos, att.inv_freq, None, ROT, False, 1e-6)
        bar = 2.0 ** -8 * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True)
        assert float(((got.double() - ref).abs() - bar).max()) <= 0
    assert torch.equal(att.v_pool[0][at], xv)


# --------------------------------------------------------------- every layer

def test_every_layer_of_a_speculative_step():
    """Each layer's output in speculative_step is that layer's own step, bit for bit, and that one is right."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, T, V, L, s = 4, 3, 40, 3, I.TINY
    att = _layers(g, B, 60, 200, L)
    weights = [{n: t.cuda() for n, t in I.decode_batch(seed=x, B=1, shape=s).items()
                if n in ("A_log", "dt_bias", "conv_w", "norm_w")} for x in range(2)]
    stack = LayerStack(s, weights, n_slots=B)
    own = [0, 17, 40, 57]
    att.own_len.copy_(_ints(own))
    prompts, prompt = (_ints([0, 1, 4]), _ints([0, 90]), _ints([90, 110])), [(0, 90)] + [(90, 110)] * 3
    qkv = [_rand(g, B, T, (HQ + 2 * HK) * D) for _ in range(L)]
    q = torch.empty((B, T, HQ, D), dtype=torch.bfloat16, device="cuda")
    alone = [torch.full_like(q, 7.0) for _ in range(L)]
    for layer in range(L):
        att.step(layer, qkv[layer], *prompts, q, alone[layer])
        gdn.check_status()
        _check_rows(att, layer, q, alone[layer], prompt, own, [T] * B)
    target = torch.softmax(torch.randn((B, T, V), generator=g, device="cuda"), -1)
    buf = dict(gdn_out=torch.empty((2, B, T, s.nv, s.dv), dtype=torch.bfloat16, device="cuda"),
               ckpt_state=torch.empty((2, B, T, s.nv, s.dk, s.dv), device="cuda"),
               ckpt_conv=torch.empty((2, B, T, s.Kc, s.C), dtype=torch.bfloat16, device="cuda"), q=q,
               attn_out=torch.full((L, *q.shape), 7.0, dtype=torch.bfloat16, device="cuda"),
               accept_len=_ints([0] * B), next_token=_ints([0] * B))
    speculative_step(stack, att, stack.static_acts(B, T), qkv, torch.arange(B, dtype=torch.int32, device="cuda"), prompts,
                     torch.zeros((B, T), dtype=torch.int32, device="cuda"), target, None,
                     torch.rand((B, T), generator=g, device="cuda"), buf)
    gdn.check_status()
    for layer in range(L):
        assert torch.equal(buf["attn_out"][layer], alone[layer]), f"layer {layer}"
