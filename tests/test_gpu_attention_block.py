"""The attention block (page slots, FP8 projections, the cache, latent attention,
block end) and the MoE block with an FP8 shared expert, against the fp64
definitions, stage by stage on the GPU's own intermediate values."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import block
from oracle import fp8 as O
from tests._latent_util import attend, check
from tests.test_gpu_block import make as moe_weights
from tests.test_gpu_block_norm import close, reference, rms
from tests.test_gpu_fp8_linear import check_product, weights
from tests.test_gpu_mxfp4_ops import f64, gpu, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, R, H, PAGE = 256, 160, 5, 16


def fp8(rng, E, N, K):
    codes, s = weights(rng, E, N, K)
    w = gpu(codes).view(torch.float8_e4m3fn)
    return (w, gpu(s)) if E > 1 else (w[0], gpu(s)[0])


def attention_weights(seed=0):
    rng = np.random.default_rng(seed)
    norm = lambda n: (1 + 0.1 * torch.randn(n, device=DEV)).to(torch.bfloat16)  # noqa: E731
    m = {"w_down": fp8(rng, 1, R + 576, D), "w_q": fp8(rng, 1, 192 * H, R), "w_kv": fp8(rng, 1, 256 * H, 512),
         "w_k": fp8(rng, H, 512, 128), "w_v": fp8(rng, H, 128, 512), "w_o": fp8(rng, 1, D, 128 * H)}
    kw = {}
    for name, (w, s) in m.items():
        kw[name], kw[name + "_scale"] = w, s
    return block.AttentionWeights(q_norm=norm(R), kv_norm=norm(512), next_norm=norm(D), **kw).prepare()


def values(w, s):
    return O.weight_values(w.view(torch.uint8).cpu().numpy(), s.cpu().numpy())


def quantised(x):
    return O.row_values(*O.quantize(f64(x)))


def turned(x, positions, base=10000.0):
    """rotary in fp64"""
    angle = positions.double()[:, None] * base ** (-torch.arange(32, dtype=torch.float64, device=DEV) / 32)
    while angle.dim() < x.dim():
        angle = angle[:, None]
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2)


def seen_calls(monkeypatch):
    seen = {}
    for name in ("fp8_linear", "latent_attention", "latent_decode", "block_residual", "rms_norm"):
        def keep(*a, _f=getattr(block, name), _n=name, **kw):
            seen.setdefault(_n, []).append((a, kw, _f(*a, **kw)))
            return seen[_n][-1][2]
        monkeypatch.setattr(block, name, keep)
    return seen


def step(W, cache, table, lens, new, free, residual, prompt, monkeypatch, some_cached=False):
    """one call, held to the definitions; returns the page slots"""
    T = sum(new)
    p = moe.page_slots(torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(new, dtype=torch.int32, device=DEV), table, free,
                       PAGE, T)
    normed = moe.rms_norm(residual, W.next_norm)
    kept = cache.clone()
    with monkeypatch.context() as m:
        seen = seen_calls(m)
        out, nxt = block.attention_forward(residual, normed, W, cache, table, p, prompt,
                                           cached_tokens=int(p.k_offsets[-1]) if some_cached else None)
    lin = [c for c in seen["fp8_linear"]]
    assert lin[0][0][0] is normed
    down = lin[0][2]
    check_product(down, quantised(normed), values(W.w_down, W.w_down_scale), False, "down")
    # what the cache holds now: the new tokens' latent vectors at their slots, all else as it was
    c = f64(down[:, R:R + 512])
    c = c * rms(c, 1e-6) * f64(W.kv_norm)
    flat = cache.view(-1, 576)
    close(flat[p.slots][:, :512], c, 2.0 ** -17 * np.abs(c), "latent vectors")
    kr = turned(down[:, R + 512:], p.positions)
    pair = kr.abs().unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1)
    assert ((flat[p.slots][:, 512:].double() - kr).abs() <= 2.0 ** -8 * kr.abs() + 2.0 ** -22 * pair).all()
    other = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
    other[p.slots] = False
    assert torch.equal(flat[other].view(torch.int16), kept.view(-1, 576)[other].view(torch.int16))
    ql = f64(down[:, :R])
    ql = ql * rms(ql, 1e-6) * f64(W.q_norm)
    close(lin[1][0][0], ql, 2.0 ** -17 * np.abs(ql), "the queries' latent vector")
    q = lin[1][2]
    check_product(q, quantised(lin[1][0][0]), values(W.w_q, W.w_q_scale), False, "queries")
    q = q.view(T, H, 192)
    qr = turned(q[..., 128:], p.positions)
    qr_pair = qr.abs().unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1)
    rows_of = []                                      # each sequence's latent vectors, from the table
    for b, (n, t) in enumerate(zip(lens, new)):
        i = torch.arange(n + t, device=DEV)
        rows_of.append(cache[table[b, i // PAGE].long(), i % PAGE])
    if prompt:
        (ac, akw, o), = seen["latent_attention"]
        assert torch.equal(lin[2][0][0], torch.cat(rows_of)[:, :512])
        check_product(lin[2][2], quantised(lin[2][0][0]), values(W.w_kv, W.w_kv_scale), False, "keys and values")
        kv = lin[2][2].view(-1, H, 256)
        assert torch.equal(ac[0][..., :128], q[..., :128])
        assert ((ac[0][..., 128:].double() - qr).abs() <= 2.0 ** -8 * qr.abs() + 2.0 ** -22 * qr_pair).all()
        q0 = k0 = 0
        for b, (n, t) in enumerate(zip(lens, new)):
            seen_keys = torch.arange(t, device=DEV)[:, None] + n >= torch.arange(n + t, device=DEV)[None]
            for h in range(H) if t else ():
                k = torch.cat([kv[k0:k0 + n + t, h, :128], rows_of[b][:, 512:]], 1)
                check(o[q0:q0 + t, h], *attend(ac[0][q0:q0 + t, h], k, kv[k0:k0 + n + t, h, 128:], 192 ** -0.5, seen_keys), f"{b} {h}")
            q0, k0 = q0 + t, k0 + n + t
    else:
        (dc, dkw, ol), = seen["latent_decode"]
        by_head = lin[2][2].view(H, T, 512)
        back = lin[3][2].view(H, T, 128)
        for h in range(H):
            check_product(by_head[h], quantised(q[:, h, :128]), values(W.w_k[h], W.w_k_scale[h]), False, "into the latent space")
            check_product(back[h], quantised(ol[:, h]), values(W.w_v[h], W.w_v_scale[h]), False, "values of a head")
        assert torch.equal(dc[0][..., :512], by_head.transpose(0, 1))
        assert ((dc[0][..., 512:].double() - qr).abs() <= 2.0 ** -8 * qr.abs() + 2.0 ** -22 * qr_pair).all()
        for b in range(T):
            check(ol[b], *attend(dc[0][b], rows_of[b], rows_of[b][:, :512], 192 ** -0.5), f"sequence {b}")
        o = back.transpose(0, 1)
    a, kw, y = lin[-1]
    assert torch.equal(a[0], o.reshape(T, H * 128))
    check_product(y, quantised(a[0]), values(W.w_o, W.w_o_scale), False, "output projection")
    want, we, n, ne = reference(residual, y, None, False, None, None, False, 1.0, W.next_norm, 1e-6)
    close(out, want, we, "residual")
    close(nxt, n, ne, "normed")
    moe.ops_check()
    return p


def test_prompts_then_decoded_tokens(monkeypatch):
    rng = np.random.default_rng(1)
    W = attention_weights()
    new = [40, 1, 33]
    free = torch.randperm(40, device=DEV).to(torch.int32)
    cache = torch.full((40, PAGE, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    lens = [0, 0, 0]
    p = step(W, cache, table, lens, new, free, rows(rng, sum(new), D), True, monkeypatch)
    for _ in range(3):
        lens, free = p.lengths.tolist(), free[int(p.taken):].clone()
        p = step(W, cache, table, lens, [1, 1, 1], free, rows(rng, 3, D), False, monkeypatch)
    # more of a prompt behind what the cache holds, one sequence without new tokens
    lens, free = p.lengths.tolist(), free[int(p.taken):].clone()
    step(W, cache, table, lens, [17, 0, 30], free, rows(rng, 47, D), True, monkeypatch, some_cached=True)


@pytest.mark.parametrize("T", [1, 40])
def test_shared_expert_in_fp8(T, monkeypatch):
    rng = np.random.default_rng(T)
    d, Is = 256, 192
    W = moe_weights(rng, d, 128, 8, Is, shared=False)
    W.shared_w13, W.shared_w13_scale = fp8(rng, 1, 2 * Is, d)
    W.shared_w2, W.shared_w2_scale = fp8(rng, 1, d, Is)
    W.prepare()
    residual = rows(rng, T, d)
    seen = seen_calls(monkeypatch)
    normed = block.first_norm(residual, W)
    block.block_forward(residual, normed, W, 2)
    (a0, _, h), (a1, _, shared) = seen["fp8_linear"]
    assert a0[0] is normed and a1[0] is h
    check_product(h, quantised(normed), values(W.shared_w13, W.shared_w13_scale), True, "shared W13")
    check_product(shared, quantised(h), values(W.shared_w2, W.shared_w2_scale), False, "shared W2")
    (_, kw, _), = seen["block_residual"]
    assert kw["y2"] is shared
    moe.ops_check()
