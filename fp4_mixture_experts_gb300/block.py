"""A decoder layer's two blocks, as a serving loop runs them:

    residual, normed = attention_forward(residual, normed, attention_weights, cache, block_table, pages, prompt)
    residual, normed = block_forward(residual, normed, weights, k)

The MoE block (block_forward) takes the residual stream and its norm before the block, and returns the
residual stream after the block and its norm before the next one.  Per token

    logits = normed . w_gate^T                                   (router)
    routed = the routed experts' outputs, weighted
    shared = W2s (silu(W1s normed) * W3s normed)                 (mxfp4_linear or fp8_linear, twice)
    residual' = residual + scale * gate * norm(routed + shared)  (block_residual)
    normed' = norm(residual')

The routed experts run as the layer (`forward`: bf16 activations), or, with
mxfp4_experts, as MXFP4 x MXFP4 products grouped by expert (`mxfp4_linear` with
the offsets and sorted slots of `route`): W13 with SwiGLU from the tokens, W2
from its rows, and the weighted sum of each token's k rows (that sum in PyTorch's
own operations, several passes over the rows in fp32; the layer has its own).

The attention block (attention_forward) writes the new tokens' latent vectors to
the paged cache and attends, every projection an FP8 product:

    q', c, kr = W_down normed;  q', c = norm(q'), norm(c);  kr = rotary(kr)
    q = W_q q', its rotary part turned;  cache[slots] = (c, kr)
    prompt:  kv = W_kv c of all the sequences' tokens;  o = latent_attention(q, kv, kr)
    decode:  ql = W_k[h] q of each head;  o = W_v[h] latent_decode((ql, qr), cache)  (products grouped by head)
    residual' = residual + W_o o;  normed' = norm(residual')     (block_residual)

(the rotary turn, the concatenations and the cache's scatter and gather in
PyTorch's own operations; indices that point nowhere are kept from those).

prepare() lays the scales out once, when the weights are loaded.  Everything
runs on the current stream.
"""
from __future__ import annotations

from dataclasses import dataclass

from ._binding import forward, route, router
from ._ops import (PageSlots, block_residual, fp8_linear, fp8_tile_scales, latent_attention, latent_decode, mxfp4_linear,
                   mxfp4_tile_scales, rms_norm)

NOPE, ROPE, VALUE, LATENT = 128, 64, 128, 512   # of a head: without and with positions, values; of a token: the latent vector


@dataclass
class BlockWeights:
    """Weights of one block (GPU tensors).  Codes and row-major scales as in the layer; the *_tiled scales are
    prepare()'s.  Shared expert and gates may be missing.  The shared expert may be in FP8 instead: float8_e4m3fn
    [2Is, d] and [d, Is] with scales [rows / 128, columns / 128] (rounded up)."""
    w_gate: object                    # bf16 [E, d]
    w13: object                       # uint8 [E, 2I, d/2]
    w13_scale: object                 # uint8 [E, 2I, d/32]
    w2: object                        # uint8 [E, d, I/2]
    w2_scale: object                  # uint8 [E, d, I/32]
    norm: object                      # [d], of the norm before the block
    next_norm: object                 # [d], of the norm before the next block
    shared_w13: object = None         # uint8 [2Is, d/2]
    shared_w13_scale: object = None   # uint8 [2Is, d/32]
    shared_w2: object = None          # uint8 [d, Is/2]
    shared_w2_scale: object = None    # uint8 [d, Is/32]
    post_norm: object = None          # [d], of the norm after the block
    gate: object = None               # [d] or None: a channel gate of the block's output
    scale: float = 1.0                # of the block's output
    w13_tiled: object = None
    w2_tiled: object = None
    shared_w13_tiled: object = None
    shared_w2_tiled: object = None

    @property
    def shared_fp8(self) -> bool:
        import torch
        return self.shared_w13.dtype == torch.float8_e4m3fn

    def prepare(self, mxfp4_experts: bool = False) -> "BlockWeights":
        """The scales of the products' operands in their layout, once."""
        if self.shared_w13 is not None and self.shared_fp8:
            self.shared_w13_tiled = fp8_tile_scales(self.shared_w13_scale, *self.shared_w13.shape, swiglu=True)
            self.shared_w2_tiled = fp8_tile_scales(self.shared_w2_scale, *self.shared_w2.shape)
        elif self.shared_w13 is not None:
            self.shared_w13_tiled = mxfp4_tile_scales(self.shared_w13_scale, swiglu=True)
            self.shared_w2_tiled = mxfp4_tile_scales(self.shared_w2_scale)
        if mxfp4_experts:
            self.w13_tiled = mxfp4_tile_scales(self.w13_scale, swiglu=True)
            self.w2_tiled = mxfp4_tile_scales(self.w2_scale)
        return self


def first_norm(residual, weights: BlockWeights, eps: float = 1e-6):
    """The norm before the first block of a stack (later ones come from block_forward)."""
    return rms_norm(residual, weights.norm, eps=eps)


def routed_mxfp4(x, logits, weights: BlockWeights, k: int):
    """The routed experts as grouped MXFP4 products, fp32 [T, d]; deterministic."""
    import torch
    T, d = x.shape
    _, topk_weights, offsets, sorted_slot = route(logits, k)
    h = mxfp4_linear(x, weights.w13, weights.w13_tiled, offsets=offsets, row_index=sorted_slot, index_div=k, swiglu=True)
    y = mxfp4_linear(h, weights.w2, weights.w2_tiled, offsets=offsets, dtype=torch.float32)
    at = torch.empty_like(sorted_slot).scatter_(0, sorted_slot.long(),
                                                torch.arange(T * k, dtype=torch.int32, device=x.device))
    return (y[at.long()].view(T, k, d) * topk_weights[:, :, None]).sum(dim=1)


def block_forward(residual, normed, weights: BlockWeights, k: int, mxfp4_experts: bool = False, eps: float = 1e-6,
                  flags: int = 0, workspace=None):
    """One block on residual [T, d] (bf16 or fp32) and its norm normed (bf16 [T, d]); returns (residual', normed')."""
    logits = router(normed, weights.w_gate)
    if mxfp4_experts:
        routed = routed_mxfp4(normed, logits, weights, k)
    else:
        routed = forward(normed, logits, weights.w13, weights.w13_scale, weights.w2, weights.w2_scale, k, flags=flags,
                         workspace=workspace)
    shared = None
    if weights.shared_w13 is not None:
        linear = fp8_linear if weights.shared_fp8 else mxfp4_linear
        h = linear(normed, weights.shared_w13, weights.shared_w13_tiled, swiglu=True)
        shared = linear(h, weights.shared_w2, weights.shared_w2_tiled)
    return block_residual(residual, routed, y2=shared, post_norm=weights.post_norm is not None,
                          post_weight=weights.post_norm, gate=None if weights.gate is None else weights.gate[None],
                          scale=weights.scale, next_weight=weights.next_norm, eps=eps)


@dataclass
class AttentionWeights:
    """Weights of one attention block of H heads (GPU tensors): matrices float8_e4m3fn, scales uint8 (E8M0) for each 128
    x 128 of a matrix; r is the width of the queries' latent vector.  The *_tiled scales are prepare()'s."""
    w_down: object        # [r + 576, d]: the queries' latent vector, the tokens' and their rotary key
    w_down_scale: object
    q_norm: object        # [r]
    kv_norm: object       # [512]
    w_q: object           # [192 H, r]: a head's 128 and 64
    w_q_scale: object
    w_kv: object          # [256 H, 512]: a head's keys and values of a latent vector (prompts)
    w_kv_scale: object
    w_k: object           # [H, 512, 128]: a head's query into the latent space (its keys' matrix, transposed)
    w_k_scale: object
    w_v: object           # [H, 128, 512]: a head's values of a latent vector
    w_v_scale: object
    w_o: object           # [d, 128 H]
    w_o_scale: object
    next_norm: object     # [d], of the norm before the next block
    rope_base: float = 10000.0
    w_down_tiled: object = None
    w_q_tiled: object = None
    w_kv_tiled: object = None
    w_k_tiled: object = None
    w_v_tiled: object = None
    w_o_tiled: object = None

    @property
    def heads(self) -> int:
        return self.w_k.shape[0]

    def prepare(self) -> "AttentionWeights":
        """The scales of the products' operands in their layout, once."""
        for name in ("w_down", "w_q", "w_kv", "w_k", "w_v", "w_o"):
            w = getattr(self, name)
            setattr(self, name + "_tiled", fp8_tile_scales(getattr(self, name + "_scale"), w.shape[-2], w.shape[-1]))
        return self


def rotary(x, positions, base: float = 10000.0):
    """bf16 x [T, 64] or [T, H, 64] turned by the tokens' positions (int32 [T]): elements 2 i and 2 i + 1 are a pair, turned
    by position base^(-i / 32).  Angles in 64 bits: at position 10^6 those in 32 are 1/16 apart."""
    return turned(x, *turns(positions, base))


def turns(positions, base: float):
    """cosines and sines of the positions' angles, fp32 [T, 32] each"""
    import torch
    i = torch.arange(ROPE // 2, dtype=torch.float64, device=positions.device)
    angle = positions.double()[:, None] * base ** (-i / (ROPE // 2))
    return angle.cos().float(), angle.sin().float()


def turned(x, cos, sin):
    """rotary's x turned by these"""
    import torch
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(x.dtype)


def write_rows(cache, slots, rows):
    """The tokens' latent vectors, bf16 [T, 576], to their places in cache (slots int64 [T], no two the same place); a token
    without a place (slot -1, or one beyond the cache) writes nothing.

    PyTorch's copies by index end the process's CUDA context on such an index.  So the difference to the bits that a place
    holds is added to them, as integers: for a token without a place 0, anywhere, which changes nothing, whatever is there
    and whoever writes it meanwhile."""
    import torch
    if cache.dtype != torch.bfloat16 or cache.dim() != 3 or cache.shape[2] != LATENT + ROPE or not cache.is_contiguous():
        raise ValueError("cache must be contiguous bf16 [pages, page, 576]")
    if rows.dtype != cache.dtype or rows.shape != (slots.numel(), LATENT + ROPE):
        raise ValueError("rows must be bf16 [T, 576] with a slot each")
    if cache.numel() == 0:
        return
    words = cache.view(-1, LATENT + ROPE).view(torch.int64)
    at = slots.clamp(0, words.shape[0] - 1)
    words.index_add_(0, at, (rows.contiguous().view(torch.int64) - words.index_select(0, at)) * (at == slots)[:, None])


def cached_rows(cache, block_table, pages: PageSlots, tokens: int):
    """The latent vectors of all tokens of a batch's sequences, side by side in the requests' order: [tokens, 576];
    tokens: their number (pages.k_offsets' last) or more, whose rows then hold anything.  Pages outside the cache read as
    zeros, as in latent_decode (PyTorch's own reads there would end the process's CUDA context)."""
    import torch
    i = torch.arange(tokens, dtype=torch.int32, device=cache.device)
    b = torch.searchsorted(pages.k_offsets[1:], i, right=True).clamp_(max=block_table.shape[0] - 1)
    at = (i - pages.k_offsets[b]).long()
    page = block_table[b, (at // cache.shape[1]).clamp_(max=block_table.shape[1] - 1)].long()
    inside = page.clamp(0, cache.shape[0] - 1)
    return cache[inside, at % cache.shape[1]].masked_fill_((inside != page)[:, None], 0)


def attention_forward(residual, normed, weights: AttentionWeights, cache, block_table, pages: PageSlots, prompt: bool,
                      cached_tokens: int | None = None, eps: float = 1e-6, workspace=None):
    """One attention block on residual [T, d] (bf16 or fp32) and its norm normed (bf16 [T, d]); returns (residual',
    normed').  pages is page_slots' result for these T tokens, whose latent vectors are written to cache (bf16 [pages,
    page, 576]; those of tokens without a slot are not).  prompt: any number of new tokens a sequence, the expanded form;
    cached_tokens, for sequences with tokens in the cache already, is the number of all their tokens (pages.k_offsets'
    last) or more; None: all tokens are new (if they are not, or cached_tokens is too small, ops_check reports it).  Otherwise
    one new token a sequence, the absorbed form, for T requests (those without a new token, which fill the batch up, behind
    the others: ops_check reports it if they are not); workspace is latent_decode's."""
    import torch
    W, T, H = weights, normed.shape[0], weights.heads
    if not prompt and pages.lengths.shape[0] != T:
        raise ValueError("the absorbed form takes a row for each request")
    scale = (NOPE + ROPE) ** -0.5
    down = fp8_linear(normed, W.w_down, W.w_down_tiled)
    r = down.shape[1] - LATENT - ROPE
    c = rms_norm(down[:, r:r + LATENT], W.kv_norm, eps=eps)
    angles = turns(pages.positions, W.rope_base)
    new = torch.cat([c, turned(down[:, r + LATENT:], *angles)], 1)
    write_rows(cache, pages.slots, new)
    q = fp8_linear(rms_norm(down[:, :r], W.q_norm, eps=eps), W.w_q, W.w_q_tiled).view(T, H, NOPE + ROPE)
    q_rope = turned(q[..., NOPE:], *angles)
    if prompt:
        if cached_tokens is None:  # the new tokens' rows; an offset that latent_attention reports where a request has others
            rows, k_offsets = new, pages.q_offsets.clone()
            k_offsets[1:].masked_fill_(pages.lengths > k_offsets[1:] - k_offsets[:-1], 2 ** 31 - 2)
        else:
            rows, k_offsets = cached_rows(cache, block_table, pages, cached_tokens), pages.k_offsets
        kv = fp8_linear(rows[:, :LATENT], W.w_kv, W.w_kv_tiled).view(-1, H, NOPE + VALUE)
        q = torch.cat([q[..., :NOPE], q_rope], 2)
        o = latent_attention(q, kv, rows[:, LATENT:], pages.q_offsets, k_offsets, scale)
    else:
        by_head = torch.arange(H + 1, dtype=torch.int32, device=q.device) * T
        ql = fp8_linear(q[..., :NOPE].transpose(0, 1).reshape(H * T, NOPE), W.w_k, W.w_k_tiled, offsets=by_head)
        q = torch.cat([ql.view(H, T, LATENT), q_rope.transpose(0, 1)], 2).transpose(0, 1)
        # token b is request b's; where it is not (one without a token is ahead), a length that latent_decode reports
        own = torch.arange(1, T + 1, dtype=torch.int32, device=q.device).minimum(pages.q_offsets[-1:])
        lengths = torch.where(pages.q_offsets[1:] == own, pages.lengths, -1)
        ol = latent_decode(q, cache, block_table, lengths, scale, workspace=workspace)
        o = fp8_linear(ol.transpose(0, 1).reshape(H * T, LATENT), W.w_v, W.w_v_tiled, offsets=by_head)
        o = o.view(H, T, VALUE).transpose(0, 1)
    y = fp8_linear(o.reshape(T, H * VALUE), W.w_o, W.w_o_tiled)
    return block_residual(residual, y, post_norm=False, next_weight=W.next_norm, eps=eps)
