"""Latent attention in fp64 (torch, on the inputs' device) with its error bound.

softmax(z) v with z = scale q k^T, values of bf16 inputs exact.  An element of z is
a sum of D products in fp32, 16 a tensor-core instruction: off by at most (D / 16 +
16) 2^-23 sum |q k|, times scale, and by 2^-22 |z| more for the scale and its
log2 e, two roundings of z and one of the difference to the maximum (|z| and the
maximum: 2^-23 each).  exp2's own error is 2^-22; so a weight p is off by d_j = e^(dz)
- 1 + 2^-22 relative to itself, and its rounding to bf16 adds 2^-8.  With a = sum p
|v| / sum p, the result is within
    (2^-8 + 2 max d_j + (n / 16 + 16 + 2 pieces) 2^-23 + 2^-20) a
of the definition (the denominator's error, max d_j again, included), and its
rounding to bf16 adds 2^-8 of it.
"""
import torch


def attend(q, k, v, scale, seen=None):
    """q [R, D], k [L, D], v [L, V] (any type), seen [R, L] or None: (result, bound), fp64 [R, V]"""
    q, k, v = q.double(), k.double(), v.double()
    z = q @ k.t() * scale
    D, n = q.shape[1], k.shape[0]
    mag = q.abs() @ k.abs().t() * abs(scale)
    top = z.abs().amax(1, keepdim=True)
    dz = (D / 16 + 16) * 2.0 ** -23 * mag + 2.0 ** -22 * z.abs() + 2.0 ** -23 * (z.abs() + top)
    if seen is not None:
        z = z.masked_fill(~seen, -torch.inf)
        dz = dz.masked_fill(~seen, 0)
    m = z.amax(1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(z - m)
    l = p.sum(1, keepdim=True)
    empty = (l == 0).squeeze(1)
    l = l.clamp(min=1e-300)
    o, a = p @ v / l, p @ v.abs() / l
    d = (torch.expm1(dz) + 2.0 ** -22).amax(1, keepdim=True)
    err = (2.0 ** -8 + 2 * d + (n / 16 + 16 + 2 * (n // 256 + 1)) * 2.0 ** -23 + 2.0 ** -20) * a
    o[empty] = 0
    return o, err + 2.0 ** -8 * (o.abs() + err) + 1e-37


def check(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(want[i])}, bound {float(bound[i])}")
