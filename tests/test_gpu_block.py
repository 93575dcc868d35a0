"""The whole block (norm, router, routed experts, shared expert, block end)
against the fp64 definitions, stage by stage on the GPU's own intermediate
values, so that each stage's bound is its own (a rounding boundary crossed in
one stage is an input of the next, not an error of it)."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
import oracle
from fp4_mixture_experts_gb300 import block
from oracle import mxfp4 as O
from tests.test_gpu_block_norm import close, reference, rms
from tests.test_gpu_mxfp4_ops import check_product, f64, gpu, rows, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(rng, d, I, E, Is, shared=True):
    w13, w13s = weights(rng, E, 2 * I, d)
    w2, w2s = weights(rng, E, d, I)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV).to(torch.bfloat16)  # noqa: E731
    W = block.BlockWeights(w_gate=bf(E, d), w13=gpu(w13), w13_scale=gpu(w13s), w2=gpu(w2), w2_scale=gpu(w2s), norm=1 + 0.1 * bf(d),
                           next_norm=1 + 0.1 * bf(d), post_norm=bf(d), gate=bf(d), scale=0.5)
    if shared:
        s13, s13s = weights(rng, 1, 2 * Is, d)
        s2, s2s = weights(rng, 1, d, Is)
        W.shared_w13, W.shared_w13_scale, W.shared_w2, W.shared_w2_scale = (gpu(a[0]) for a in (s13, s13s, s2, s2s))
    return W


@pytest.mark.parametrize("T", [1, 33, 300])
def test_block_stage_by_stage(T, monkeypatch):
    rng = np.random.default_rng(T)
    d, I, E, Is, k = 256, 128, 8, 192, 2
    W = make(rng, d, I, E, Is).prepare(mxfp4_experts=True)
    residual = rows(rng, T, d)
    seen = {}
    for name in ("router", "forward", "mxfp4_linear", "block_residual"):
        def keep(*a, _f=getattr(block, name), _n=name, **kw):
            seen.setdefault(_n, []).append((a, kw, _f(*a, **kw)))
            return seen[_n][-1][2]
        monkeypatch.setattr(block, name, keep)
    normed = block.first_norm(residual, W)
    n = f64(residual) * rms(f64(residual), 1e-6) * f64(W.norm)
    close(normed, n, 2.0 ** -17 * np.abs(n), "first norm")
    out, nxt = block.block_forward(residual, normed, W, k)
    # routed experts: the layer, whose own tests hold it to this tolerance
    logits = seen["router"][0][2]
    ref = oracle.forward(normed.view(torch.int16).cpu().numpy().view(np.uint16), logits.cpu().numpy(), W.w13.cpu().numpy(),
                         W.w13_scale.cpu().numpy(), W.w2.cpu().numpy(), W.w2_scale.cpu().numpy(), k)["out"]
    routed = seen["forward"][0][2]
    assert np.linalg.norm(f64(routed) - ref) <= 5e-3 * np.linalg.norm(ref)
    # shared expert
    (a0, _, h), (a1, _, shared) = seen["mxfp4_linear"]
    assert a0[0] is normed and a1[0] is h
    check_product(h, O.values(*O.quantize(f64(normed))), O.values(W.shared_w13.cpu().numpy(), W.shared_w13_scale.cpu().numpy()),
                  True, "shared W13")
    check_product(shared, O.values(*O.quantize(f64(h))), O.values(W.shared_w2.cpu().numpy(), W.shared_w2_scale.cpu().numpy()),
                  False, "shared W2")
    o, oe, n, ne = reference(residual, routed, shared, True, W.post_norm, W.gate[None], False, 0.5, W.next_norm, 1e-6)
    close(out, o, oe, "out")
    close(nxt, n, ne, "normed")


@pytest.mark.parametrize("T", [1, 40])
def test_routed_experts_in_mxfp4(T):
    rng = np.random.default_rng(T)
    d, I, E, k = 256, 128, 8, 3
    W = make(rng, d, I, E, 64, shared=False).prepare(mxfp4_experts=True)
    x = rows(rng, T, d)
    logits = gpu(rng.standard_normal((T, E)).astype(np.float32))
    got = block.routed_mxfp4(x, logits, W, k)
    assert torch.equal(got, block.routed_mxfp4(x, logits, W, k))
    ids, w, off, slot = (t.cpu().numpy() for t in moe.route(logits, k))
    h = moe.mxfp4_linear(x, W.w13, W.w13_tiled, offsets=gpu(off), row_index=gpu(slot), index_div=k, swiglu=True)
    a = O.values(*O.quantize(f64(h)))                 # the second product's operand, from the GPU's h
    want, bound = np.zeros((T, d)), np.zeros((T, d))
    for r, s in enumerate(slot):
        e = ids[s // k, s % k]
        y, S = O.matmul(a[r:r + 1], O.values(W.w2[e].cpu().numpy(), W.w2_scale[e].cpu().numpy()))
        want[s // k] += w[s // k, s % k] * y[0]
        # the product's bound, and the fp32 product and sum of k terms
        bound[s // k] += w[s // k, s % k] * ((I / 64 + 64) * 2.0 ** -23 * S[0] + (k + 1) * 2.0 ** -23 * np.abs(y[0]))
    assert (np.abs(f64(got) - want) <= bound + 1e-30).all()
    residual, normed = block.block_forward(x, x, W, k, mxfp4_experts=True)
    assert residual.shape == normed.shape == (T, d) and torch.isfinite(normed.float()).all()
