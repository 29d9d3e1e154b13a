"""Attention-layer dispatch over the library's calls.

One call per layer and step, following "从零实现 vLLM (1.3)：如何加速 Attention
计算", section "Attention 源码分析": the step's new K/V are first written into the
paged cache (store_kvcache at slot_mapping), then

  * prefill: varlen attention over the packed new tokens; when the step carries
    block tables (prefix cache), K/V are read from the caches instead of the
    step's own k/v;
  * decode: one query token per sequence against the cache (context_lens =
    cache_seqlens, which include the token just stored).  A decode step that
    carries the same number of new tokens for every sequence (speculative
    verification; the page shows one) goes through the kv-cache entry with
    bottom-right causality among the new tokens.

With a Rotary the rotation of q and k and the store are one call
(rope_store_kvcache).  LinearAttention and DeltaAttention are the layers of models
that mix attention with linear attention: the same step metadata, a state cache
instead of a paged one.  PagePool keeps the page tables on the GPU and builds each
step's metadata there from request lengths; Beams runs a beam search over its
requests.

Everything runs in the library's kernels; this module only routes tensors.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (StepTables, attn_decode_paged, attn_varlen_fwd, attn_with_kvcache, beam_rows, beam_select,
               copy_kvcache, copy_states, delta_attn_decode, delta_attn_varlen_fwd, linear_attn_decode,
               linear_attn_varlen_fwd, rope_store_kvcache, step_tables, store_kvcache, trim_pages)


@dataclass
class AttentionContext:
    """Per-step metadata shared by all attention layers of a forward pass."""
    is_prefill: bool
    slot_mapping: torch.Tensor | None = None     # int64 [N]: flat cache slot of each new token (< 0: skip)
    cu_seqlens_q: torch.Tensor | None = None     # int32 [B+1] (prefill; linear attention: any step)
    cu_seqlens_k: torch.Tensor | None = None     # int32 [B+1] (prefill)
    max_seqlen_q: int = 0
    max_seqlen_k: int = 0
    context_lens: torch.Tensor | None = None     # int32 [B] (decode): cached keys incl. the new tokens
    block_tables: torch.Tensor | None = None     # int32 [B, max_blocks] (prefix prefill, decode)
    positions: torch.Tensor | None = None        # int32 [N] or [axes, N]: rotary positions of the new tokens
    state_slots: torch.Tensor | None = None      # int32 [B]: state slot of each sequence (linear attention; < 0: none)
    past_lens: torch.Tensor | None = None        # int32 [B]: tokens before this step (linear attention; 0: from zero)
    cache_seqlens: torch.Tensor | None = None    # int32 [B]: and after it (linear attention; no more: refused, state kept)


@dataclass
class Rotary:
    """Rotary positions of an attention layer (see rope_store_kvcache)."""
    inv_freq: torch.Tensor                       # float32 [rot_dim / 2]
    pair_axis: bytes | None = None               # position axis of each pair, for positions with several axes
    interleaved: bool = False
    scale: float = 1.0


class Attention:
    """Causal attention of one layer with a paged KV cache.

    k_cache / v_cache ([num_blocks, block_size, num_kv_heads, head_dim] bf16)
    are bound by the owner (for instance after sizing the pool); until then the
    layer runs without a cache (prefill only).  An optional v16_cache (float16,
    same shape) keeps V / 16 next to the bf16 V: the store fills it and the
    prefix prefill reads it instead of converting the cached V every step.  With
    `rotary` the layer takes unrotated q and k, and ctx.positions."""

    def __init__(self, num_heads: int, head_dim: int, scale: float, num_kv_heads: int, rotary: Rotary | None = None):
        if num_heads % num_kv_heads:
            raise ValueError("num_heads must be a multiple of num_kv_heads")
        self.num_heads = num_heads
        self.head_dim = head_dim
        self.scale = float(scale)
        self.num_kv_heads = num_kv_heads
        self.rotary = rotary
        self.k_cache: torch.Tensor | None = None
        self.v_cache: torch.Tensor | None = None
        self.v16_cache: torch.Tensor | None = None

    def forward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ctx: AttentionContext) -> torch.Tensor:
        """q [N, Hq*D] or [N, Hq, D]; k, v [N, Hkv*D] or [N, Hkv, D].  Returns o
        with q's shape."""
        shape = q.shape
        q = q.view(-1, self.num_heads, self.head_dim)
        k = k.view(-1, self.num_kv_heads, self.head_dim)
        v = v.view(-1, self.num_kv_heads, self.head_dim)
        cached = self.k_cache is not None and self.v_cache is not None and self.k_cache.numel() > 0
        stored = cached and ctx.slot_mapping is not None and ctx.slot_mapping.numel() > 0
        if self.rotary is not None:
            q, k = self._rotate_and_store(q, k, v, ctx, stored)
        elif stored:
            store_kvcache(k, v, self.k_cache, self.v_cache, ctx.slot_mapping, v16_cache=self.v16_cache)
        if ctx.is_prefill:
            if ctx.block_tables is not None:
                if not cached:
                    raise ValueError("prefix prefill needs the KV cache")
                o = attn_varlen_fwd(q, self.k_cache, self.v_cache, ctx.cu_seqlens_q, ctx.cu_seqlens_k,
                                    ctx.max_seqlen_q, ctx.max_seqlen_k, self.scale, causal=True,
                                    block_table=ctx.block_tables, v16_cache=self.v16_cache)
            else:
                o = attn_varlen_fwd(q, k, v, ctx.cu_seqlens_q, ctx.cu_seqlens_k, ctx.max_seqlen_q,
                                    ctx.max_seqlen_k, self.scale, causal=True)
        else:
            if not cached:
                raise ValueError("decode needs the KV cache")
            if ctx.context_lens is None or ctx.block_tables is None:
                raise ValueError("decode needs context_lens and block_tables")
            batch, n = ctx.context_lens.numel(), q.shape[0]
            if n == batch:
                o = attn_decode_paged(q, self.k_cache, self.v_cache, ctx.context_lens, ctx.block_tables, self.scale,
                                      max_cache_seqlen=ctx.max_seqlen_k or None)
            else:
                if batch == 0 or n % batch:
                    raise ValueError("a decode step carries the same number of new tokens for every sequence")
                sq = n // batch
                o = attn_with_kvcache(q.reshape(batch, sq, self.num_heads, self.head_dim), self.k_cache,
                                      self.v_cache, ctx.context_lens, ctx.block_tables, self.scale, causal=True,
                                      max_cache_seqlen=ctx.max_seqlen_k or None, v16_cache=self.v16_cache)
        return o.view(shape)

    def _rotate_and_store(self, q, k, v, ctx: AttentionContext, stored: bool):
        if ctx.positions is None:
            raise ValueError("a layer with rotary positions needs ctx.positions")
        r = self.rotary
        how = dict(pair_axis=r.pair_axis, interleaved=r.interleaved, scale=r.scale)
        if not stored:
            return rope_store_kvcache(q, k, None, ctx.positions, r.inv_freq, return_k=True, **how)
        # only a prefill without block tables reads the step's own k again
        own_k = ctx.is_prefill and ctx.block_tables is None
        got = rope_store_kvcache(q, k, v, ctx.positions, r.inv_freq, self.k_cache, self.v_cache, ctx.slot_mapping,
                                 v16_cache=self.v16_cache, return_k=own_k, **how)
        return got if own_k else (got, k)

    __call__ = forward


def _state_step(state_cache, ctx: AttentionContext, rows: int):
    """How a layer with a state cache runs a step of `rows` rows: (slots, offsets,
    lengths before it, most tokens of a sequence).  No offsets in a decode step: one
    row for each sequence."""
    slots = ctx.state_slots if state_cache is not None else None
    if state_cache is not None and slots is None:
        raise ValueError("a layer with a state cache needs ctx.state_slots")
    if not ctx.is_prefill and slots is None:
        raise ValueError("decode needs the state cache")
    offsets, past, most = ctx.cu_seqlens_q, ctx.past_lens, ctx.max_seqlen_q or rows
    # offsets that are not of these sequences say nothing about them
    if not ctx.is_prefill and (offsets is None or offsets.numel() != slots.numel() + 1):
        if rows != slots.numel():
            raise ValueError("a decode step of several tokens needs the sequences' offsets (ctx.cu_seqlens_q)")
        return slots, None, past, 1
    if not ctx.is_prefill and past is None:
        if most > 1:
            raise ValueError("a decode step of several tokens needs ctx.past_lens")
        past = torch.ones_like(slots)            # as without offsets: every slot continues
    return slots, offsets, past, most


class LinearAttention:
    """Linear attention of one layer with a decay per head and a cache of fp32
    states: S_t = exp(log_decay) S_{t-1} + v_t k_t^T, o_t = scale * S_t q_t.

    state_cache ([num_slots, num_kv_heads, head_dim, head_dim] float32) is bound
    by the owner; ctx.state_slots names each sequence's slot.  Without it every
    step starts from zero states and keeps none (prefill only)."""

    def __init__(self, num_heads: int, head_dim: int, scale: float, num_kv_heads: int, log_decay: torch.Tensor):
        if num_heads % num_kv_heads:
            raise ValueError("num_heads must be a multiple of num_kv_heads")
        self.num_heads = num_heads
        self.head_dim = head_dim
        self.scale = float(scale)
        self.num_kv_heads = num_kv_heads
        self.log_decay = log_decay
        self.state_cache: torch.Tensor | None = None

    def forward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ctx: AttentionContext) -> torch.Tensor:
        """q [N, Hq*D] or [N, Hq, D]; k, v [N, Hkv*D] or [N, Hkv, D].  Returns o
        with q's shape.  A step of at most one token per sequence
        (ctx.max_seqlen_q 1) takes the recurrent form, any other runs in chunks,
        both over ctx.cu_seqlens_q: sequences may have no token, and rows behind
        the last one are not computed.  A decode step without offsets has one row
        for each sequence."""
        shape = q.shape
        q = q.view(-1, self.num_heads, self.head_dim)
        k = k.view(-1, self.num_kv_heads, self.head_dim)
        v = v.view(-1, self.num_kv_heads, self.head_dim)
        slots, offsets, past, most = _state_step(self.state_cache, ctx, q.shape[0])
        if offsets is None and not ctx.is_prefill:
            o = linear_attn_decode(q, k, v, self.log_decay, self.state_cache, slots, self.scale, context_lens=past)
        else:
            o = linear_attn_varlen_fwd(q, k, v, self.log_decay, offsets, most, self.scale,
                                       state_cache=self.state_cache, state_slots=slots, context_lens=past,
                                       cache_seqlens=ctx.cache_seqlens)
        return o.view(shape)

    __call__ = forward


class DeltaAttention:
    """Linear attention of one layer by the gated delta rule (see
    delta_attn_varlen_fwd), with a cache of fp32 states.

    state_cache ([num_slots, num_v_heads, head_dim, head_dim] float32) is bound by
    the owner, as LinearAttention's.  qk_norm_eps: q and k are normalised on the way
    (None: the caller has done it)."""

    def __init__(self, num_k_heads: int, num_v_heads: int, head_dim: int, scale: float,
                 qk_norm_eps: float | None = 1e-6):
        if num_v_heads % num_k_heads:
            raise ValueError("num_v_heads must be a multiple of num_k_heads")
        self.num_k_heads = num_k_heads
        self.num_v_heads = num_v_heads
        self.head_dim = head_dim
        self.scale = float(scale)
        self.qk_norm_eps = qk_norm_eps
        self.state_cache: torch.Tensor | None = None

    def forward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, beta: torch.Tensor,
                ctx: AttentionContext) -> torch.Tensor:
        """q, k [N, Hk*D] or [N, Hk, D]; v [N, Hv*D] or [N, Hv, D]; log_decay, beta
        float32 [N, Hv].  Returns o with v's shape.  Steps as for LinearAttention; up
        to 16 tokens per sequence run in one pass over the states, more in chunks.

        The states then hold all of the step's tokens.  Guessed tokens that are accepted in
        part: copy_states(state_cache, rows, spares) before the step, and after it
        copy_states(state_cache, spares, rows) and another step over the accepted ones
        (a source of -1 leaves out the sequences that keep all of theirs)."""
        shape = v.shape
        q = q.view(-1, self.num_k_heads, self.head_dim)
        k = k.view(-1, self.num_k_heads, self.head_dim)
        v = v.view(-1, self.num_v_heads, self.head_dim)
        slots, offsets, past, most = _state_step(self.state_cache, ctx, q.shape[0])
        if offsets is None and not ctx.is_prefill:
            o = delta_attn_decode(q, k, v, log_decay, beta, self.state_cache, slots, self.scale, context_lens=past,
                                  qk_norm_eps=self.qk_norm_eps)
        else:
            o = delta_attn_varlen_fwd(q, k, v, log_decay, beta, offsets, most, self.scale,
                                      state_cache=self.state_cache, state_slots=slots, context_lens=past,
                                      cache_seqlens=ctx.cache_seqlens, qk_norm_eps=self.qk_norm_eps)
        return o.view(shape)

    __call__ = forward


class PagePool:
    """The pages of a paged cache and the requests that hold them, on the GPU.

    A request is a row 0 .. max_requests - 1 that the caller assigns.  grow()
    adds a step's new tokens and returns its tables, trim() cuts requests (0
    ends one); neither waits for the GPU.  Pages that cannot be served are
    reported by get_last_device_error (status 9) and leave their request as it
    was here, in the paged caches and in the state caches.  The step's layers
    still run over its tokens (attention sees the old context only): drop their
    output.  A page belongs to one request: requests cannot share a prefix's
    pages."""

    def __init__(self, num_blocks: int, block_size: int, max_requests: int, max_blocks: int, device=None):
        i32 = torch.int32
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.block_size = block_size
        self.seq_lens = torch.zeros(max_requests, dtype=i32, device=device)
        self.page_table = torch.full((max_requests, max_blocks), -1, dtype=i32, device=device)
        self.free_pages = torch.arange(num_blocks - 1, -1, -1, dtype=i32, device=device)
        self.num_free = torch.full((1,), num_blocks, dtype=i32, device=device)

    def grow(self, new_lens: torch.Tensor, max_tokens: int, request_rows: torch.Tensor | None = None,
             out: StepTables | None = None, stream=None) -> StepTables:
        """Tables of a step in which request request_rows[b] (None: row b) gets
        new_lens[b] tokens; max_tokens bounds their sum."""
        return step_tables(request_rows, new_lens, self.seq_lens, self.page_table, self.free_pages, self.num_free,
                           self.block_size, max_tokens, out=out, stream=stream)

    def trim(self, keep_lens: torch.Tensor, request_rows: torch.Tensor | None = None, stream=None) -> None:
        """Cut request request_rows[b] to its first keep_lens[b] tokens."""
        trim_pages(request_rows, keep_lens, self.seq_lens, self.page_table, self.free_pages, self.num_free,
                   self.block_size, stream=stream)

    @staticmethod
    def context(tables: StepTables, is_prefill: bool, max_seqlen_q: int, max_seqlen_k: int, paged: bool = True,
                state_slots: torch.Tensor | None = None, positions: torch.Tensor | None = None) -> AttentionContext:
        """The step's AttentionContext.  paged=False: a prefill of fresh prompts,
        whose attention reads the step's own k and v.  positions: instead of the
        tables' (for instance several axes).  A decode step (is_prefill False)
        gives every entry the same number of tokens where it meets an Attention
        layer; entries of unequal counts go through a paged prefill."""
        # the step's own k has a row for every new token, also of an entry that was not served and so
        # counts as empty in cu_seqlens_k
        cu_k, most_k = (tables.cu_seqlens_k, max_seqlen_k) if paged else (tables.cu_seqlens_q, max_seqlen_q)
        return AttentionContext(
            is_prefill, slot_mapping=tables.slot_mapping, cu_seqlens_q=tables.cu_seqlens_q,
            cu_seqlens_k=cu_k, max_seqlen_q=max_seqlen_q, max_seqlen_k=most_k,
            context_lens=tables.cache_seqlens, block_tables=tables.block_table if paged else None,
            positions=tables.positions if positions is None else positions, state_slots=state_slots,
            past_lens=tables.context_lens, cache_seqlens=tables.cache_seqlens)


class Beams:
    """A beam search over requests of a PagePool: `rows` int32 [R, W] are the request
    rows of R searches with W beams each, all different.  A row is also its beam's state
    slot in the caches of LinearAttention and DeltaAttention layers.  Nothing here waits
    for the GPU.

    All beams of a search hold the same number of tokens.  A prompt is stored in its
    search's first beam, after every beam's row has grown by it; start() hands it to the
    others.  A step then is: select() on the step's logits (a row per beam, in the
    order of `rows`), advance() to the chosen parents, and the next step with the
    tokens and the new `rows`."""

    def __init__(self, pool: PagePool, rows: torch.Tensor):
        self.pool = pool
        self.rows = rows
        self.first_tokens: torch.Tensor | None = None
        self.scores = self._first_scores()

    def _first_scores(self) -> torch.Tensor:
        # the search starts from its first beam alone: the others hold the same prompt
        scores = torch.full(self.rows.shape, float("-inf"), device=self.rows.device)
        scores[:, 0] = 0
        return scores

    def select(self, logits: torch.Tensor, num_out: int | None = None):
        """(tokens, parents, scores) of the best continuations, [R, num_out] each
        (None: as many as there are beams), best first; see beam_select."""
        beams = self.rows.shape[1]
        return beam_select(logits, self.scores.view(-1), beams, beams if num_out is None else num_out)

    def advance(self, parents: torch.Tensor, scores: torch.Tensor, layers=()) -> None:
        """Beam w of each search becomes a continuation of beam parents[:, w] with
        scores[:, w] (both [R, W], for instance the first W of what select() returned; -1
        and -inf: none): the beams' rows, and in the
        caches of `layers` (Attention, LinearAttention, DeltaAttention) what beams that go on
        more than once have cached."""
        self.rows, source = beam_rows(parents.contiguous(), self.rows)
        self.scores = scores.contiguous()
        for layer in layers:
            if isinstance(layer, Attention):
                copy_kvcache(layer.k_cache, layer.v_cache, source, self.rows, self.pool.page_table, self.pool.seq_lens,
                             first_tokens=self.first_tokens, v16_cache=layer.v16_cache)
            else:
                copy_states(layer.state_cache, source, self.rows)

    def start(self, layers=()) -> None:
        """Copy the prompts from the first beams to the others; what is copied later
        begins behind them.  Called again, with new prompts in the first beams (and the
        old tokens trimmed from every row), it starts the next search over the same rows."""
        if self.first_tokens is not None:
            self.first_tokens, self.scores = None, self._first_scores()
        self.advance(torch.zeros_like(self.rows), self.scores, layers)
        self.first_tokens = self.pool.seq_lens.clone()
