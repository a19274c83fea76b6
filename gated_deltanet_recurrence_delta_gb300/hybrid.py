"""The full-attention layers of a hybrid stack beside its GDN layers, the
speculative step of both, and beam search over both.

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

PagedAttentionLayers keeps them in 4-bit pages instead, in which a row grows page by
page and rows that part later share what they have in common: what beam search
needs, whose rows become copies of one another after every selection.
"""
from __future__ import annotations

import contextlib

import torch

from . import gdn

_STEP = 64  # the most tokens of a row that a step over pages takes (gdn.attn_kv4)


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


class PagedAttentionLayers:
    """n_layers full-attention layers of one head layout over n_pages pages of 64 tokens each, held in 4 bits (gdn.kv4_pool);
    n_rows rows of at most max_pages pages each, all layers sharing the page table and the rows' lengths.

    weights, inv_freq: as in AttentionLayers. k_exp, v_exp: the pools' exponents. pinned: uint8 [n_pages], the pages that
    others hold (set by the caller; never taken or written). A step is take() -- rows become copies of other rows, get
    pages for the tokens that they take now, and the copies of pages and states are made -- and then each layer's step().
    Everything stays on the device, so that a step can be captured; what take() cannot give a page for takes no tokens and
    is reported (GDN_ERR_FULL, gdn.check_status). A call given a stream does all its work on it."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, weights, inv_freq, n_rows, n_pages, max_pages, k_exp=0, v_exp=0,
                 device="cuda"):
        self.hq, self.hk, self.d = n_q_heads, n_kv_heads, head_dim
        self.weights, self.inv_freq, self.device = weights, inv_freq, device
        self.n_layers, self.n_rows, self.n_pages, self.max_pages = len(weights), n_rows, n_pages, max_pages
        self.k_exp, self.v_exp = k_exp, v_exp
        self.pool = torch.zeros((self.n_layers, n_pages, n_kv_heads, 72 * head_dim), dtype=torch.uint8, device=device)
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        self.table, self.kv_len, self.taken = ints(n_rows, max_pages), ints(n_rows), ints(n_rows)
        self._table, self._kv_len = ints(n_rows, max_pages), ints(n_rows)
        self.page_src, self.page_dst = ints(n_rows), ints(n_rows)
        self.pinned = torch.zeros(n_pages, dtype=torch.uint8, device=device)
        self.buffers = {}

    def _buffer(self, name, shape, dtype, stream):
        key = (name, shape, gdn._stream(stream))
        if key not in self.buffers:
            self.buffers[key] = torch.empty(shape, dtype=dtype, device=self.device)
        return self.buffers[key]

    def take(self, T, parent=None, n_new=None, state_idx=None, stack=None, stream=None):
        """Row r becomes a copy of row parent[r] (int32 [n_rows], -1: emptied; None: itself) and takes n_new[r] tokens
        (int32 [n_rows] in [0, T]; None: T). With state_idx int32 [n_rows], the rows' slots of `stack` (a LayerStack), it
        is brought along in place and the states and conv tails are copied too (an emptied row's slot, state_idx[r], holds
        what its last row left there: set it to zeros before a new sequence starts in it). Returns kv_index int32 [n_rows, T], the
        tokens' pool rows (up to the 64 tokens of a step it is the same tensor every time, which the stream's next take()
        of T tokens writes anew; a prompt's is the caller's); kv_len holds the rows' lengths with them."""
        with _on(stream):
            if T <= _STEP:
                index = self._buffer("index", (self.n_rows, T), torch.int32, stream)
            else:  # prompts are of any length: one kept for each would be without end
                index = torch.empty((self.n_rows, T), dtype=torch.int32, device=self.device)
            states = {}
            if state_idx is not None:
                names = ("state_idx_out", "state_src", "state_dst")
                states = {n: self._buffer(n, (self.n_rows,), torch.int32, stream) for n in names}
                states["state_idx"] = state_idx
            gdn.cache_fork(self.table, self.kv_len, self._table, self._kv_len, index if T else None, self.page_src,
                           self.page_dst, self.n_pages, parent=parent, n_new=n_new, pinned=self.pinned, stream=stream,
                           **states)
            pools = [(self.pool, self.page_src, self.page_dst)]
            if state_idx is not None:
                pools += [(p, states["state_src"], states["state_dst"]) for p in (stack.state_pool, stack.conv_pool)]
            gdn.slots_copy(pools, stream)
            if state_idx is not None:
                state_idx.copy_(states["state_idx_out"])
            self.table.copy_(self._table)
            self.kv_len.copy_(self._kv_len)
            if T:
                torch.sum(index >= 0, 1, out=self.taken)
            else:
                self.taken.zero_()
            return index

    def _split(self, qkv):
        hq, hk, d = self.hq, self.hk, self.d
        return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                qkv[:, (hq + hk) * d:].unflatten(1, (hk, d)))

    def _norm_rope(self, layer, qkv, positions, q_out, k_out, v_out, kv_index, stream):
        q, k, v = self._split(qkv)
        dims = gdn.make_rope_dims(q, k, 2 * self.inv_freq.numel(), kv_rows=k_out.shape[0])
        w = self.weights[layer]
        gdn.head_norm_rope(dims, q, k, v, w["q_norm"], w["k_norm"], positions, self.inv_freq, q_out, k_out, v_out,
                           kv_index=kv_index, stream=stream)

    def step(self, layer, qkv, kv_index, q_buf, out, stream=None):
        """A layer's decode (T = 1) or verify (T tokens) of all rows: qkv bf16 [n_rows, T, (hq + 2 hk) d], kv_index
        take()'s; q_buf, out: bf16 [n_rows, T, hq, d]. A row's tokens behind the ones it took are none of it: their
        outputs are zeros."""
        R, T = q_buf.shape[:2]
        if qkv.shape[:2] != (R, T) or kv_index.numel() != R * T:
            raise ValueError(f"qkv and kv_index must be of q_buf's {R} rows of {T} tokens, they are {list(qkv.shape)} and "
                             f"{list(kv_index.shape)}")
        with _on(stream):
            first = self.kv_len - self.taken
            positions = (first[:, None] + torch.arange(T, dtype=torch.int32, device=self.device)).reshape(1, -1)
            k, v = (self._buffer(n, (R * T, self.hk, self.d), torch.bfloat16, stream) for n in ("k", "v"))
            self._norm_rope(layer, qkv.flatten(0, 1), positions, q_buf, k, v, None, stream)
            pool = self.pool[layer]
            dims = gdn.make_kv4_dims(k, pool, k_exp=self.k_exp, v_exp=self.v_exp)
            gdn.kv4_store(dims, k, v, kv_index, pool, stream)
            dims = gdn.make_attn_kv4_dims(q_buf, pool, self.table, k_exp=self.k_exp, v_exp=self.v_exp)
            workspace = self._buffer("workspace", (gdn.attn_kv4_workspace_size(dims),), torch.uint8, stream)
            gdn.attn_kv4(dims, q_buf, pool, self.table, self.kv_len, out, workspace, self.taken, stream)

    def prefill(self, layer, qkv, rows, lens, past, kv_index, q_buf, out, stream=None):
        """A layer's prompts, or further chunks of them: sequence i is lens[i] tokens of row rows[i], behind past[i] tokens
        that its pages hold already (host lists); take() has given the rows their pages and kv_index is the tokens' of
        it, int32 [n]. qkv bf16 [n, (hq + 2 hk) d]; q_buf, out bf16 [n, hq, d]. The new tokens attend in bf16; the past
        ones as the pages hold them."""
        if qkv.shape[0] != sum(lens) or kv_index.numel() != sum(lens):
            raise ValueError(f"qkv and kv_index must be of {sum(lens)} tokens, they are {list(qkv.shape)} and "
                             f"{list(kv_index.shape)}")
        if not sum(lens):
            return
        with _on(stream):
            dev, total = self.device, [a + b for a, b in zip(lens, past)]
            ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
            places = torch.cat([torch.arange(p, p + n) for n, p in zip(lens, past)])
            starts = [sum(total[:i]) for i in range(len(total))]
            at = torch.cat([torch.arange(s + p, s + p + n) for s, n, p in zip(starts, lens, past)])
            k, v = (torch.empty((sum(total), self.hk, self.d), dtype=torch.bfloat16, device=dev) for _ in range(2))
            self._norm_rope(layer, qkv, places.int().to(dev)[None], q_buf, k, v, at.int().to(dev), stream)
            pool = self.pool[layer]
            new_k, new_v = (k, v) if not any(past) else (x[at.to(dev)] for x in (k, v))
            gdn.kv4_store(gdn.make_kv4_dims(new_k, pool, k_exp=self.k_exp, v_exp=self.v_exp), new_k, new_v, kv_index, pool,
                          stream)
            if any(past):  # the cached tokens in front of them; -1: not loaded
                old = torch.full((sum(total),), -1, dtype=torch.int32, device=dev)
                for r, s, p in zip(rows, starts, past):
                    j = torch.arange(p, device=dev)
                    old[s:s + p] = self.table[r, j // gdn.PAGE_TOKENS] * gdn.PAGE_TOKENS + (j % gdn.PAGE_TOKENS).int()
                gdn.kv4_load(gdn.make_kv4_dims(k, pool, k_exp=self.k_exp, v_exp=self.v_exp), pool, old, k, v, stream)
            cu = ints([sum(lens[:i]) for i in range(len(lens) + 1)])
            dims = gdn.make_attn_dims(q_buf, k, B=len(lens))
            gdn.attn_prefill(dims, q_buf, k, v, cu, out, ints(starts), ints(total), stream)


class Beams:
    """What a beam search carries from step to step, [groups, beams] each: the scores (fp32, -inf: no beam), done (uint8),
    and the last selection's parent (row numbers) and token (-1: a place that it left without a beam; -2: none was made
    yet). At the start each group has one beam, its first row."""

    def __init__(self, groups, beams, device="cuda"):
        new = lambda dtype, fill: torch.full((groups, beams), fill, dtype=dtype, device=device)  # noqa: E731
        self.scores, self.done = new(torch.float32, float("-inf")), new(torch.uint8, 0)
        self.scores[:, 0] = 0.0
        self.parent = torch.arange(groups * beams, dtype=torch.int32, device=device).view(groups, beams)
        self.token = new(torch.int32, -2)
        self.workspaces = {}  # for each shape of logits and stream: a captured step keeps its own

    def select(self, logits, eos=-1, stream=None):
        """The best continuations, from the rows' logits [groups, beams, V] (fp32 or bf16). A call given a stream does all
        its work on it."""
        if logits.shape[:2] != self.scores.shape:
            raise ValueError(f"logits must be {list(self.scores.shape)} rows, they are {list(logits.shape[:2])}")
        key = (logits.shape, gdn._stream(stream))
        if key not in self.workspaces:
            with _on(stream):  # of that stream's memory: a block of another one's may still be in use there
                self.workspaces[key] = gdn.beam_workspace(logits)
        gdn.beam_select(logits, self.scores, self.parent, self.token, self.scores, self.workspaces[key],
                        done=self.done, new_done=self.done, eos=eos, stream=stream)


def beam_step(stack, attention, beams, acts, qkv, logits, state_idx, buffers, eos=-1):
    """One step of beam search over a hybrid stack, entirely on the device (and so capturable): the rows become what the
    last selection made of them (pages shared, partly filled ones and the recurrent states copied), every layer decodes
    one token a row, and the next selection is made.

    stack: LayerStack; attention: PagedAttentionLayers; beams: Beams; acts / qkv: the layers' inputs (LayerStack.decode;
    PagedAttentionLayers.step with T = 1); logits: [groups, beams, V]; state_idx int32 [n_rows], the rows' state slots;
    buffers: dict with gdn_out (LayerStack.decode), q and attn_out [n_layers][n_rows][1][hq][d]. A finished beam takes no
    tokens. The row of a place that the last selection left without a beam is emptied and takes none: nobody reads it, and
    its pages are the others'. The logits come from the layers' outputs; here they are given."""
    none = (beams.token == -1) & (beams.scores == float("-inf"))
    n_new = ((beams.done == 0) > none).flatten().to(torch.int32)
    index = attention.take(1, beams.parent.masked_fill(none, -1).flatten(), n_new, state_idx, stack)
    stack.decode(acts, state_idx, buffers["gdn_out"])
    for layer in range(attention.n_layers):
        attention.step(layer, qkv[layer], index, buffers["q"], buffers["attn_out"][layer])
    beams.select(logits, eos)


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
