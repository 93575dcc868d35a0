"""The definition of rows in 8-bit floating point (oracle/fp8.py), held to hand-worked values and to PyTorch's own
conversion."""
import numpy as np
import torch

from oracle import fp8


def test_the_codes_are_pytorchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8.VALUES, t)
    assert fp8.VALUES[0x7E] == 448 and fp8.VALUES[1] == 2.0 ** -9 and fp8.VALUES[0x38] == 1


def test_hand_worked_scales():
    x = np.zeros((8, 256))
    x[0, 0] = 448                 # exactly the largest code at scale 1
    x[1, 0] = 448.0001            # one more: scale 2
    x[2, 0], x[2, 128] = -896, 3  # scale 2; 3 <= 448 2^-7 = 3.5: scale 2^-7
    x[3, 0] = 3.500001            # scale 2^-6
    x[4, 0] = 2.0 ** -130         # below 448 2^-127: the least scale
    x[5, 0] = np.inf
    x[6, 130] = np.nan
    codes, s = fp8.quantize(x)
    assert s[0, 0] == 127 and codes[0, 0] == 0x7E
    assert s[1, 0] == 128 and codes[1, 0] == fp8.VALUES.tolist().index(224.0)
    assert s[2, 0] == 128 and codes[2, 0] == 0xFE and s[2, 1] == 120
    assert s[3, 0] == 121 and s[4, 0] == 0 and s[7, 0] == 0 and s[7, 1] == 0
    assert s[5, 0] == 255 and (codes[5, :128] == 127).all() and s[5, 1] == 0 and s[6].tolist() == [0, 255]


def test_rounding_is_pytorchs():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 200)) * np.exp2(rng.integers(-12, 12, (40, 200)))).astype(np.float32)
    codes, s = fp8.quantize(x)
    scale = np.repeat(np.exp2(s.astype(np.float64) - 127), 128, axis=1)[:, :200]
    want = torch.from_numpy((x / scale).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(codes, want)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 128))
    x[0, 0] = 448
    x[0, 1:5] = [17, 19, 2.0 ** -10, 3 * 2.0 ** -10]  # between 16 and 18, 18 and 20, 0 and 2^-9, 2^-9 and 2^-8
    c, _ = fp8.quantize(x)
    assert fp8.VALUES[c[0, 1:5]].tolist() == [16, 20, 0, 2.0 ** -8]


def test_tiles():
    s = np.arange(6, dtype=np.uint8).reshape(1, 3, 2) + 1
    t = fp8.tile_scales(s, 300)
    assert (t[0, 0, 1] == 2).all() and t[0, 2, 0, 16 * 5] == 5 and t[0, 2, 0, 16 * 5 + 4] == 5 and t[0, 2, 0, 16 * 12 + 4] == 0
    g = fp8.tile_scales(s, 300, swiglu=True)          # rows 0, 150, 1, 151, ..
    assert g[0, 0, 0, 0] == 1 and g[0, 0, 0, 16] == 3 and g[0, 2, 0, 16 * 11 + 4 + 3] == 5
