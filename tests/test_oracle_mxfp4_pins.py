"""The MXFP4 oracle against hand-worked rows and brute force (no GPU)."""
import numpy as np

from oracle import mxfp4 as O


def test_hand_worked_row():
    x = np.zeros((1, 32))
    # amax 5: floor(log2) = 2, scale 2^0; 2.5 is a tie between 2 (code 4) and 3 (code 5): even code 4
    x[0, :10] = [5.0, -0.2, 0.25, 0.3, 0.75, 2.5, -3.5, 5.0, 4.9, -0.0]
    codes, scales = O.quantize(x)
    assert scales.tolist() == [[127]]
    c = np.stack([codes[0] & 15, codes[0] >> 4], axis=1).reshape(-1)
    assert c[:10].tolist() == [6, 8, 0, 1, 2, 4, 14, 6, 6, 8]
    assert O.values(codes, scales)[0, :9].tolist() == [4.0, 0.0, 0.0, 0.5, 1.0, 2.0, -4.0, 4.0, 4.0]


def test_scales_of_extreme_blocks():
    x = np.zeros((5, 32))
    x[1, 0] = 2.0 ** -133
    x[2, 0] = 3.3895313892515355e38
    x[3, 0] = np.inf
    x[4, 0] = np.nan
    codes, scales = O.quantize(x)
    assert scales[:, 0].tolist() == [0, 0, 252, 255, 255]
    v = O.values(codes, scales)
    assert (v[0] == 0).all() and np.isnan(v[3:]).all() and v[2, 0] == 6 * 2.0 ** 125


def test_every_value_goes_to_the_nearest():
    x = np.random.default_rng(0).standard_normal((64, 32)) * 3
    codes, scales = O.quantize(x)
    v = O.values(codes, scales)
    scale = np.exp2(scales.astype(np.float64) - 127)
    grid = np.concatenate([-O.MAGNITUDES, O.MAGNITUDES])
    best = np.abs(x[:, :, None] - grid * scale[:, :, None]).min(axis=-1)
    np.testing.assert_allclose(np.abs(v - x), best, rtol=0, atol=0)


def test_a_value_that_is_representable_stays():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (40, 16), dtype=np.uint8)
    codes[:, 0] |= 0x07                             # a 6 in every block: the scale is then the block's own
    scales = rng.integers(1, 252, (40, 1), dtype=np.uint8)
    v = O.values(codes, scales)
    c2, s2 = O.quantize(v)
    np.testing.assert_array_equal(s2, scales)
    np.testing.assert_array_equal(O.values(c2, s2), v)


def test_tiled_layout_by_hand():
    s = np.arange(130 * 5, dtype=np.uint16).astype(np.uint8).reshape(1, 130, 5)
    t = O.tile_scales(s)
    assert t.shape == (1, 2, 2, 512)
    assert t[0, 0, 0, 0:4].tolist() == s[0, 0, :4].tolist()          # row 0
    assert t[0, 0, 0, 4:8].tolist() == s[0, 32, :4].tolist()         # row 32 beside it
    assert t[0, 0, 0, 16:20].tolist() == s[0, 1, :4].tolist()        # row 1 in the next 16 bytes
    assert t[0, 1, 1, 16:20].tolist() == [s[0, 129, 4], 0, 0, 0]     # row 129, past the end of K zeros
    g = O.tile_scales(s, swiglu=True)
    assert g[0, 0, 0, 16:20].tolist() == s[0, 65, :4].tolist()       # row 1 is the first up row


def test_swiglu_and_product():
    a = np.array([[1.0, 2.0]])
    w = np.array([[3.0, -1.0], [0.5, 0.5]])
    y, S = O.matmul(a, w)
    assert y.tolist() == [[1.0, 1.5]] and S.tolist() == [[5.0, 1.5]]
    h = O.swiglu(y)
    np.testing.assert_allclose(h, [[1.5 / (1 + np.exp(-1.0))]])
