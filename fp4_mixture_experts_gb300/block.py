"""A whole MoE block around the layer, as a serving loop runs it:

    residual, normed = block_forward(residual, normed, weights, k)

takes the residual stream and its norm before the block, and returns the
residual stream after the block and its norm before the next one.  Per token

    logits = normed . w_gate^T                                   (router)
    routed = the routed experts' outputs, weighted
    shared = W2s (silu(W1s normed) * W3s normed)                 (mxfp4_linear, twice)
    residual' = residual + scale * gate * norm(routed + shared)  (block_residual)
    normed' = norm(residual')

The routed experts run as the layer (`forward`: bf16 activations), or, with
mxfp4_experts, as MXFP4 x MXFP4 products grouped by expert (`mxfp4_linear` with
the offsets and sorted slots of `route`): W13 with SwiGLU from the tokens, W2
from its rows, and the weighted sum of each token's k rows (that sum in PyTorch's
own operations, several passes over the rows in fp32; the layer has its own).

prepare() lays the scales out once, when the weights are loaded.  Everything
runs on the current stream.
"""
from __future__ import annotations

from dataclasses import dataclass

from ._binding import forward, route, router
from ._ops import block_residual, mxfp4_linear, mxfp4_tile_scales, rms_norm


@dataclass
class BlockWeights:
    """Weights of one block (GPU tensors).  Codes and row-major scales as in the layer; the *_tiled scales are
    prepare()'s.  Shared expert and gates may be missing."""
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

    def prepare(self, mxfp4_experts: bool = False) -> "BlockWeights":
        """The scales of the products' operands in their layout, once."""
        if self.shared_w13 is not None:
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
        h = mxfp4_linear(normed, weights.shared_w13, weights.shared_w13_tiled, swiglu=True)
        shared = mxfp4_linear(h, weights.shared_w2, weights.shared_w2_tiled)
    return block_residual(residual, routed, y2=shared, post_norm=weights.post_norm is not None,
                          post_weight=weights.post_norm, gate=None if weights.gate is None else weights.gate[None],
                          scale=weights.scale, next_weight=weights.next_norm, eps=eps)
