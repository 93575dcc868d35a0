"""The end of a block (norm, gate, residual, next norm) on the GPU against its
definition in fp64.

Error bound: every factor of b (the reciprocal root of a mean of d squares in
fp32, weight, gate, sigmoid, scale) is within a few ulp: the mean is a sum of
non-negative terms, off by at most (d / threads + 12) 2^-24 <= 2^-18 relative,
its root by half of that; the sigmoid's fast exponential by 2^-20 (1 + |g|).
So b's magnitude errs by at most 2^-17 (1 + |g|), the sum out by that much of
|scale b| plus 2^-23 |out|, and normed by the error of out times its factor plus
2^-17 of itself; bf16 results add 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(DEV).to(dtype)


def rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)


def reference(r, y, y2, post, pw, gate, sig, scale, nw, eps):
    b = f64(y) + (0 if y2 is None else f64(y2))
    mag = np.abs(f64(y)) + (0 if y2 is None else np.abs(f64(y2)))
    f = np.ones_like(b)
    if post:
        f = f * rms(b, eps)
    if pw is not None:
        f = f * f64(pw)
    g = np.zeros(())
    if gate is not None:
        g = f64(gate)
        if g.ndim == 1:
            g = g[:, None] if g.shape[0] == b.shape[0] and g.shape[0] != b.shape[1] else g[None, :]
        f = f * (1 / (1 + np.exp(-g)) if sig else g)
    out = f64(r) + scale * b * f
    err = 2.0 ** -17 * (1 + np.abs(g)) * np.abs(scale * f) * mag + 2.0 ** -23 * np.abs(out)
    n = rms(out, eps) * (1 if nw is None else f64(nw))
    normed = out * n
    # a change of out also moves the mean: relatively by at most ||err|| / ||out||
    with np.errstate(invalid="ignore", divide="ignore"):
        moved = np.linalg.norm(err, axis=-1, keepdims=True) / np.linalg.norm(out, axis=-1, keepdims=True)
    moved = np.where(np.isfinite(moved), moved, 0)
    return out, err, normed, err * np.abs(n) + (2.0 ** -17 + moved) * np.abs(normed)


def close(got, ref, err, what):
    if got.dtype == BF:
        err = err + 2.0 ** -8 * (np.abs(ref) + err)
    bad = ~(np.abs(f64(got) - ref) <= err + 1e-30)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def run(T, d, rt=BF, yt=F32, two=True, post=True, pw=BF, gate=None, gt=F32, sig=False, scale=0.5, nw=BF, eps=1e-6, seed=0):
    rng = np.random.default_rng(seed)
    r, y = rand(rng, (T, d), rt, 3.0), rand(rng, (T, d), yt, 0.7)
    y2 = rand(rng, (T, d), BF) if two else None
    pw = None if pw is None else rand(rng, (d,), pw)
    nw = None if nw is None else rand(rng, (d,), nw)
    shape = {None: None, "token": (T,), "channel": (d,), "element": (T, d)}[gate]
    g = None if shape is None else rand(rng, shape, gt)
    out, normed = moe.block_residual(r, y, y2=y2, post_norm=post, post_weight=pw, gate=g, gate_sigmoid=sig,
                                     scale=scale, next_weight=nw, eps=eps)
    assert out.dtype == rt and normed.dtype == BF
    o, oe, n, ne = reference(r, y, y2, post, pw, g, sig, scale, nw, eps)
    close(out, o, oe, "out")
    close(normed, n, ne, "normed")


@pytest.mark.parametrize("T", [1, 2, 33])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 64, 100, 256, 1001, 1024, 4096, 4104, 7168, 8191, 8200, 16384])
def test_widths(T, d):
    if T == d:
        T += 1
    run(T, d, gate="token", sig=True, seed=d)


@pytest.mark.parametrize("gate", [None, "token", "channel", "element"])
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("d", [520, 333])
def test_gates_and_norms(gate, sig, post, d):
    run(9, d, gate=gate, sig=sig, post=post, seed=d)


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32, None])
@pytest.mark.parametrize("gt", [BF, F32])
def test_types(rt, yt, wt, gt):
    for d in (768, 250):
        run(5, d, rt=rt, yt=yt, two=yt == BF, pw=wt, nw=wt, gate="element", gt=gt)
        run(5, d, rt=rt, yt=yt, two=yt != BF, pw=wt, nw=wt, gate="channel", gt=gt, sig=True)


def test_strided_rows_in_place_and_no_next_norm():
    rng = np.random.default_rng(2)
    for d, pad in ((256, 64), (250, 3)):
        buf = rand(rng, (12, d + pad), BF)
        y = rand(rng, (12, d + pad), F32)[:, pad:]
        g = rand(rng, (12, d + pad), BF)[:, :d]
        r = buf[:, :d]
        keep = buf[:, d:].clone()
        o, oe, n, ne = reference(r, y, None, True, None, g, True, 1.0, None, 1e-5)
        out, normed = moe.block_residual(r, y, gate=g, gate_sigmoid=True, eps=1e-5, out=r)
        assert out is r
        close(out, o, oe, "out")
        close(normed, n, ne, "normed")
        assert torch.equal(buf[:, d:], keep)
        out2, none = moe.block_residual(r.contiguous(), y, next_norm=False)
        assert none is None and out2.shape == (12, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [5, 4096, 4100])
def test_rms_norm(d, dtype):
    rng = np.random.default_rng(d)
    x, w = rand(rng, (17, d), dtype, 5.0), rand(rng, (d,), BF)
    n = f64(x) * rms(f64(x), 1e-6) * f64(w)
    close(moe.rms_norm(x, w), n, 2.0 ** -17 * np.abs(n), "rms_norm")


def test_zero_rows_large_values_and_nan():
    x = torch.zeros(4, 512, dtype=F32, device=DEV)
    x[1] = 1e18                                   # its square sum still fits fp32
    x[2, 5] = float("nan")
    got = f64(moe.rms_norm(x))
    assert (got[0] == 0).all() and (got[1] == 1).all() and np.isnan(got[2]).all() and (got[3] == 0).all()


def test_the_same_bits_again():
    rng = np.random.default_rng(9)
    r, y = rand(rng, (50, 4096), BF), rand(rng, (50, 4096), F32)
    a, b = moe.block_residual(r, y), moe.block_residual(r, y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows():
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    out, normed = moe.block_residual(e, e)
    assert out.shape == normed.shape == (0, 64)


@pytest.mark.parametrize("T,d", [(2600, 64), (5000, 8), (5001, 520), (1300, 1032), (1250, 4096), (620, 7168), (700, 8192),
                                 (650, 8200), (4900, 250), (640, 16384)])
@pytest.mark.parametrize("gate,sig,post", [("token", True, True), ("element", False, False), ("channel", True, True),
                                           (None, False, True)])
def test_many_rows(T, d, gate, sig, post):
    """enough rows for the persistent form (and widths that it does not take)"""
    run(T, d, rt=F32 if gate == "channel" else BF, yt=BF if gate == "element" else F32, two=gate != "channel", gate=gate, sig=sig,
        post=post, seed=T)


@pytest.mark.parametrize("d", [512, 4096])
def test_many_rows_strided_in_place_without_norms_and_rms_norm(d):
    rng = np.random.default_rng(d)
    T = 20000 if d == 512 else 3000
    buf = rand(rng, (T, d + 64), BF, 3.0)
    r, keep = buf[:, :d], buf[:, d:].clone()
    y = rand(rng, (T, d + 8), F32)[:, 8:]
    w = rand(rng, (d,), BF)
    n = f64(r) * rms(f64(r), 1e-6) * f64(w)
    close(moe.rms_norm(r, w), n, 2.0 ** -17 * np.abs(n), "rms_norm")
    ref, err, _, _ = reference(r, y, None, False, None, None, False, 2.0, None, 1e-6)
    out, none = moe.block_residual(r, y, post_norm=False, scale=2.0, next_norm=False, out=r)
    assert none is None
    close(out, ref, err, "out")
    assert torch.equal(buf[:, d:], keep)
    moe.ops_check()


@pytest.mark.parametrize("T,d", [(9800, 33), (9729, 1), (5003, 604), (4900, 1001), (620, 7167), (650, 12001), (610, 16383)])
@pytest.mark.parametrize("gate,sig,post", [("token", True, True), ("element", False, False), ("channel", True, True)])
def test_many_rows_that_do_not_start_on_16_bytes(T, d, gate, sig, post):
    run(T, d, rt=F32 if gate == "channel" else BF, yt=BF if gate == "element" else F32, two=gate != "channel",
        pw=None if d == 1 else BF, gate=gate, sig=sig, post=post, seed=T)


@pytest.mark.parametrize("d,off", [(1001, 1), (4096, 3), (604, 0)])
def test_many_rows_at_odd_addresses_in_place(d, off):
    """rows packed tightly behind an odd start: a copy of whole 16 bytes would reach beside the first and the last row"""
    rng = np.random.default_rng(d)
    T = 5000

    def packed(dtype):
        flat = rand(rng, (off + T * d,), dtype, 2.0)
        return flat, flat[off:].view(T, d)

    (flat, r), (_, y), (_, g) = packed(BF), packed(F32), packed(BF)
    head = flat[:off].clone()
    o, oe, n, ne = reference(r, y, None, True, None, g, True, 0.5, None, 1e-6)
    first = moe.block_residual(r.clone(), y, gate=g, gate_sigmoid=True, scale=0.5)
    out, normed = moe.block_residual(r, y, gate=g, gate_sigmoid=True, scale=0.5, out=r)
    close(out, o, oe, "out")
    close(normed, n, ne, "normed")
    assert torch.equal(flat[:off], head)
    assert torch.equal(out, first[0]) and torch.equal(normed, first[1])
    moe.ops_check()


@pytest.mark.parametrize("T,d", [(3000, 4096), (700, 7167)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T, d):
    """host-planted: the first CTA of the persistent form never loads its first row (no fault on the GPU)"""
    rng = np.random.default_rng(T)
    r, y = rand(rng, (T, d), BF), rand(rng, (T, d), F32)
    want = moe.block_residual(r, y)
    moe.ops_check()
    moe.set_fault_injection(moe.FAULT_TC_TOKEN_TILE, 2000)
    try:
        moe.block_residual(r, y)
        torch.cuda.synchronize()
    finally:
        moe.set_fault_injection(moe.FAULT_NONE)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    again = moe.block_residual(r, y)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    moe.ops_check()


def test_offsets_beyond_32_bits():
    rng = np.random.default_rng(4)
    T, d = 140000, 16384
    r = torch.zeros(T, d, dtype=BF, device=DEV)
    y = torch.zeros(T, d, dtype=BF, device=DEV)
    r[-3:], y[-3:] = rand(rng, (3, d), BF), rand(rng, (3, d), BF)
    o, oe, n, ne = reference(r[-3:], y[-3:], None, True, None, None, False, 1.0, None, 1e-6)
    out, normed = moe.block_residual(r, y)
    close(out[-3:], o, oe, "out")
    close(normed[-3:], n, ne, "normed")
    assert not out[:16].any()
