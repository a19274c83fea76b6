"""The full-attention layers of a hybrid stack beside its GDN layers, and the
speculative step of both.

statecache.py (squad-0.8b, qev_fast): a hybrid model's layers are GDN layers,
whose cache is a state slot, and full-attention layers, whose cache is the keys
and values of every token; a prompt's cache is kept and later rows continue from
it. generate.py (sparkle, mlx_streaming/mtp): a verify forward runs the drafted
tokens of every row through all layers, the accepted prefix is committed in the
recurrent caches and the key/value caches are trimmed to it.

Here the attention layers keep their keys and values in token pools,
[n_layers][kv_rows][n_kv_heads][head_dim]. A prompt that several rows continue is
one extent of pool rows; every row has an extent of its own behind it, with room
for its continuation. Lengths live on the device, so a step can be captured: the
class marshals buffers and issues the library's calls, as LayerStack does for the
GDN layers.
"""
from __future__ import annotations

import contextlib

import torch

from . import gdn


def _on(stream):
    """The context in which torch's own operations and allocations belong to `stream` (a stream or its handle; None: the
    current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class AttentionLayers:
    """n_layers full-attention layers of one head layout over a pool of kv_rows tokens each.

    weights: one dict per layer with the bf16 norms q_norm, k_norm [head_dim] (or None). inv_freq: fp64 [rot_dim/2]
    (device). prompt_rows: the pool rows [0, prompt_rows) hold shared prompts, packed; row b's own extent starts at
    prompt_rows + b * room, whose room holds its continuation and a step's T tokens. Of a step's tokens a row takes as
    many as its room still holds (room_for); the others are no tokens of it: no key is kept, their outputs are zeros. A
    row without room for one token is a device error (GDN_ERR_INDEX, gdn.check_status) and stays as it is.

    A call given a stream does all its work on it, its index arithmetic too; calls on several streams are ordered by the
    caller (the pools and the rows' lengths are one set; each stream has workspaces of its own)."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, weights, inv_freq, prompt_rows, n_rows, room, device="cuda"):
        self.hq, self.hk, self.d = n_q_heads, n_kv_heads, head_dim
        self.weights, self.inv_freq, self.device = weights, inv_freq, device
        self.n_layers, self.n_rows, self.room, self.prompt_rows = len(weights), n_rows, room, prompt_rows
        self.kv_rows = prompt_rows + n_rows * room
        shape = (self.n_layers, self.kv_rows, n_kv_heads, head_dim)
        self.k_pool = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v_pool = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        ints = lambda n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        self.own_start = (prompt_rows + room * torch.arange(n_rows, device=device)).to(torch.int32)
        self.own_len = ints(n_rows)
        self.workspace = {}

    def _split(self, qkv):
        """q, k, v heads of a projection's rows [n, (hq + 2 hk) d]: views, nothing is copied."""
        hq, hk, d = self.hq, self.hk, self.d
        return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                qkv[:, (hq + hk) * d:].unflatten(1, (hk, d)))

    def _norm_rope(self, layer, qkv, positions, kv_index, q_out, stream):
        q, k, v = self._split(qkv)
        dims = gdn.make_rope_dims(q, k, 2 * self.inv_freq.numel(), kv_rows=self.kv_rows)
        w = self.weights[layer]
        gdn.head_norm_rope(dims, q, k, v, w["q_norm"], w["k_norm"], positions, self.inv_freq, q_out, self.k_pool[layer],
                           self.v_pool[layer], kv_index=kv_index, stream=stream)

    def prefill(self, layer, qkv, cu_seqlens, positions, kv_index, kv_start, kv_len, q_buf, out, stream=None):
        """A layer's prompts: qkv bf16 [n, (hq + 2 hk) d], the tokens of cu_seqlens' sequences; each token's keys and
        values go to pool row kv_index[t], and sequence b attends over pool rows [kv_start[b], + kv_len[b]).
        q_buf, out: bf16 [n, hq, d], the rotated queries and the layer's output."""
        self._norm_rope(layer, qkv, positions, kv_index, q_buf, stream)
        dims = gdn.make_attn_dims(q_buf, self.k_pool[layer], B=cu_seqlens.numel() - 1)
        gdn.attn_prefill(dims, q_buf, self.k_pool[layer], self.v_pool[layer], cu_seqlens, out, kv_start, kv_len, stream)

    def room_for(self, B, T):
        """int32 [B]: how many of a step's T tokens fit each row's room, gdn.accept_draft's n_tokens."""
        return (self.room - self.own_len[:B]).clamp(0, T)

    def step(self, layer, qkv, group_rows, prompt_start, prompt_len, q_buf, out, stream=None):
        """A layer's decode (T = 1) or verify (T drafted tokens) of the rows [B][T]: qkv bf16 [B, T, (hq + 2 hk) d].
        The tokens stand behind the row's own keys (own_len, which advance() moves afterwards) at position
        prompt_len of the row's group + place in its own extent. Rows without shared prompts: group_rows, prompt_start
        and prompt_len None (or empty)."""
        with _on(stream):
            self._step(layer, qkv, group_rows, prompt_start, prompt_len, q_buf, out, stream)

    def _step(self, layer, qkv, group_rows, prompt_start, prompt_len, q_buf, out, stream):
        B, T = q_buf.shape[0], q_buf.shape[1]
        place = self.own_len[:B, None] + torch.arange(T, dtype=torch.int32, device=self.device)
        real = self.room_for(B, T)
        past = (real == 0)[:, None] * (self.kv_rows + 1) - 1  # -1: not kept; a full row: past the pool, and so reported
        at = torch.where(place < self.room, self.own_start[:B, None] + place, past).to(torch.int32).flatten()
        own_len = (self.own_len[:B] + T).clamp(max=self.room)
        n_groups = 0 if prompt_start is None else prompt_start.numel()
        positions = place
        if n_groups > 0:
            group = torch.bucketize(torch.arange(B, dtype=torch.int32, device=self.device), group_rows[1:], right=True)
            positions = (prompt_len[group][:, None] + place).to(torch.int32)
        positions = positions.reshape(1, -1)
        self._norm_rope(layer, qkv.flatten(0, 1), positions, at, q_buf, stream)
        dims = gdn.make_attn_dims(q_buf, self.k_pool[layer], B=B, T=T, n_groups=n_groups)
        key = (B, T, n_groups, gdn._stream(stream))
        if key not in self.workspace:
            self.workspace[key] = gdn.attn_workspace(dims, self.device)
        gdn.attn_shared_prefix(dims, q_buf, self.k_pool[layer], self.v_pool[layer], group_rows, prompt_start, prompt_len,
                               self.own_start[:B], own_len, out, self.workspace[key], real, stream)

    def advance(self, accept_len, stream=None):
        """Every layer's caches keep the accepted tokens of the step: the next step overwrites the others."""
        with _on(stream):
            self.own_len[:accept_len.numel()] += accept_len


def speculative_step(stack, attention, acts, qkv, state_idx, prompts, tokens, target_probs, draft_probs, uniform, buffers):
    """One speculative step of a hybrid stack, entirely on the device (and so capturable): every layer's verify of
    the rows' T tokens, the acceptance of the drafts, and the commit of the accepted prefix in the recurrent pools
    and the key/value pools.

    stack: LayerStack; attention: AttentionLayers; acts / qkv: the layers' inputs (LayerStack.verify;
    AttentionLayers.step), prompts: (group_rows, prompt_start, prompt_len); tokens, target_probs, draft_probs,
    uniform: gdn.accept_draft's; buffers: dict with gdn_out, ckpt_state, ckpt_conv (LayerStack.verify), q, attn_out
    [n_layers][B][T][hq][d], accept_len, next_token int32 [B].
    A row whose room holds fewer than T tokens takes part with those (AttentionLayers.room_for); a full row accepts 0,
    draws -1, keeps its states and is reported.
    The target's probabilities come from the layers' outputs; here they are given."""
    b = buffers
    stack.verify(acts, state_idx, b["gdn_out"], b["ckpt_state"], b["ckpt_conv"])
    for layer in range(attention.n_layers):
        attention.step(layer, qkv[layer], *prompts, b["q"], b["attn_out"][layer])
    gdn.accept_draft(tokens, target_probs, draft_probs, uniform, b["accept_len"], b["next_token"],
                     attention.room_for(*tokens.shape))
    stack.commit(1, b["accept_len"], state_idx, b["ckpt_state"], b["ckpt_conv"])
    attention.advance(b["accept_len"])
