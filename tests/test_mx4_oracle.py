"""Pins of the oracle's MX4 quantizer (32-column blocks of e2m1 codes under one
power-of-two scale): worked blocks, numpy's rounding and frexp, brute force over all 16
codes, the error bounds that follow from the grid, and the special blocks."""
import numpy as np
import pytest

import oracle as O

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nibbles(codes):
    c = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    return c


def test_worked_block():
    """Maximum 7.9 = 2^2 x 1.975: scale 2^0, byte 127; every tie of the grid goes to the
    even code, and magnitudes above 6 saturate."""
    v = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.26, -0.74, -1.0, -6.0, 4.99, 5.01, -0.0, 0.0]
    want = [0, 2, 2, 4, 4, 6, 6, 7, 9, 9, 10, 15, 6, 7, 8, 0]
    w = np.zeros((1, 64), np.float32)
    w[0, :16] = v
    codes, scales = O.mx4_quantize(w)
    assert nibbles(codes)[0, :16].tolist() == want
    assert scales.shape == (1, 16) and scales[0].tolist() == [127] + [0] * 15
    assert codes[0, 0] == 0 | 2 << 4  # the lower column in the low nibble
    assert np.array_equal(O.mx4_dequantize(codes, scales)[0, :8], [0, 1, 1, 2, 2, 4, 4, 6])


@pytest.mark.parametrize("power", [-126, -40, 0, 40, 120])
def test_scale_and_codes_against_numpy_and_brute_force(power):
    rng = np.random.default_rng(power + 200)
    w = np.ldexp(rng.normal(size=(7, 192)), power).astype(np.float32)
    codes, scales = O.mx4_quantize(w)
    b = w.astype(np.float64).reshape(7, 6, 32)
    e = np.maximum(np.frexp(np.abs(b).max(axis=2))[1] - 3, -127)
    assert np.array_equal(scales[:, :6].astype(int), e + 127)
    assert not scales[:, 6:].any()
    r = b / np.ldexp(1.0, e)[:, :, None]
    c = nibbles(codes).reshape(7, 6, 32)
    # brute force: no code of the grid is nearer; a tie leaves the even code
    d = np.abs(np.abs(r)[..., None] - GRID)
    got = np.take_along_axis(d, (c & 7)[..., None].astype(int), axis=3)[..., 0]
    assert np.array_equal(got, d.min(axis=3))
    ties = (d == d.min(axis=3, keepdims=True)).sum(axis=3) > 1
    assert np.all((c[ties] & 1) == 0)
    assert np.array_equal(c >> 3, np.signbit(r))
    # the grid's steps: 1/2 below 2, 1 below 4, 2 below 8 (6 to 8 saturate: at most 2 off)
    a = np.abs(r)
    bound = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    err = np.abs(O.mx4_dequantize(codes, scales).reshape(7, 6, 32) - b)
    assert np.all(err <= bound * np.ldexp(1.0, e)[:, :, None])


def test_quantizing_the_values_again_changes_nothing():
    """Values on a block's grid whose maximum is 4 or 6 steps keep codes and scale."""
    w = np.random.default_rng(3).normal(size=(5, 512)).astype(np.float32)
    codes, scales = O.mx4_quantize(w)
    v = O.mx4_dequantize(codes, scales)
    again = O.mx4_dequantize(*O.mx4_quantize(v.astype(np.float32)))
    assert np.array_equal(v, again)


def test_bf16_and_fp32_inputs_agree():
    w = np.random.default_rng(4).normal(size=(4, 128)).astype(np.float32)
    bits = (w.view(np.uint32) >> 16).astype(np.uint16)
    wide = (bits.astype(np.uint32) << 16).view(np.float32)
    a, b = O.mx4_quantize(bits, dtype=O.BF16), O.mx4_quantize(wide)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_special_blocks():
    w = np.random.default_rng(5).normal(size=(3, 128)).astype(np.float32)
    clean_c, clean_s = O.mx4_quantize(w)
    w[0, 3], w[1, 40], w[2, 127] = np.nan, np.inf, -np.inf
    w[1, 64:96] = 0.0
    codes, scales = O.mx4_quantize(w)
    assert scales[0, 0] == scales[1, 1] == scales[2, 3] == 255 and scales[1, 2] == 0
    v = O.mx4_dequantize(codes, scales)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:64]).all() and np.isnan(v[2, 96:]).all()
    assert not v[1, 64:96].any()
    keep = np.ones((3, 4), bool)
    keep[0, 0] = keep[1, 1] = keep[1, 2] = keep[2, 3] = False
    assert np.array_equal(scales[:, :4][keep], clean_s[:, :4][keep])
    assert np.array_equal(nibbles(codes).reshape(3, 4, 32)[keep], nibbles(clean_c).reshape(3, 4, 32)[keep])
    # subnormals: the scale stays at 2^-127, the grid's step there is 2^-128
    t = np.full((1, 64), np.float32(2.0 ** -128))
    t[0, 1] = 2.0 ** -130
    codes, scales = O.mx4_quantize(t)
    assert scales[0, 0] == 0 and nibbles(codes)[0, :2].tolist() == [1, 0]
