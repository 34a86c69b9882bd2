"""Pins of the MX oracle: the formats' grids, the powers of blocks, ties, layout
and non-finite blocks, against values written out by hand and PyTorch's own
8-bit conversion."""

import numpy as np
import pytest
import torch

from oracle import mx_oracle as mx


def test_grids_hold_the_formats_values():
    g8, g4 = mx.mx_grid("mxfp8"), mx.mx_grid("mxfp4")
    assert g8[-1] == 448 and g8[0] == 0 and g8[1] == 2.0 ** -9 and g8[8] == 2.0 ** -6
    assert list(g4) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.all(np.diff(g8) > 0) and np.all(np.diff(g4) > 0)


@pytest.mark.parametrize("value,code", [
    (0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
    (5.0000001, 7), (6.0, 7), (-0.25, 8), (-5.0, 14), (-6.0, 15),
])
def test_four_bit_ties_go_to_the_even_code(value, code):
    assert mx.mx_round(np.array([value]), "mxfp4")[0] == code


def test_eight_bit_rounding_is_that_of_torch():
    g = torch.Generator().manual_seed(0)
    v = torch.cat([torch.randn(4000, generator=g) * 100, torch.randn(4000, generator=g) * 0.01])
    v = v.clamp(-448, 448)
    # exact ties between neighbouring elements too
    grid = torch.tensor(mx.mx_grid("mxfp8"))
    v = torch.cat([v.double(), (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2])
    v = v.float().double()
    want = v.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(mx.mx_round(v.numpy(), "mxfp8"), want)


@pytest.mark.parametrize("fmt,amax,p", [
    ("mxfp8", 448.0, 0), ("mxfp8", 449.0, 1), ("mxfp8", 224.0, -1), ("mxfp8", 1.0, -8),
    ("mxfp8", 1.75, -8), ("mxfp8", 1.7578125, -7), ("mxfp8", 0.0, -127),
    ("mxfp4", 6.0, 0), ("mxfp4", 6.03125, 1), ("mxfp4", 3.0, -1), ("mxfp4", 4.0, 0),
    ("mxfp4", 1.0, -2), ("mxfp4", 2.0 ** -130, -127), ("mxfp4", 2.0 ** 127, 125),
])
def test_powers_of_blocks(fmt, amax, p):
    assert mx.mx_power(amax, fmt) == p


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_layout_round_trip_and_errors(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 160)) * np.exp(rng.standard_normal((5, 1)))
    codes, scales = mx.mx_quantize(x, fmt)
    sc, ss = mx.mx_store(codes, scales, fmt)
    assert sc.shape == (5, 160 if fmt == "mxfp8" else 80) and ss.shape == (2, 5, 4)
    assert np.all(ss[1, :, 1:] == 0)  # 5 blocks: three of the last word lie past K
    c2, s2 = mx.mx_load(sc, ss, 160, fmt)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    v = mx.mx_values(codes, scales, fmt)
    amax = np.abs(x).reshape(5, 5, 32).max(2).repeat(32, axis=1)
    # half a step of the grid at the block's largest element (E4M3: 16 of 448; E2M1: 1 of
    # 6), where the block's power lets that element lie anywhere above half the largest
    step = (16 / 224 if fmt == "mxfp8" else 1 / 3)
    assert np.all(np.abs(v - x) <= step * amax)
    assert np.all(np.abs(v).reshape(5, 5, 32).max(2) <= np.abs(x).reshape(5, 5, 32).max(2) * 2)


def test_non_finite_blocks():
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40], x[0, 70] = 1.0, np.inf, np.nan
    codes, scales = mx.mx_quantize(x, "mxfp8")
    assert scales[0, 0] != 255 and scales[0, 1] == 255 and scales[0, 2] == 255
    assert not codes[0, 32:].any()
    v = mx.mx_values(codes, scales, "mxfp8")
    assert np.all(np.isnan(v[0, 32:])) and v[0, 3] == 1.0


def test_grouped_product_and_norm_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    w = np.array([[[1.0, 0.0]], [[0.0, 10.0]], [[1.0, 1.0]]])
    y = mx.grouped_mm(x, w, [0, 1, 1, 2])
    assert y[0, 0] == 1.0 and y[1, 0] == 7.0 and np.isnan(y[2, 0])
    s, xn = mx.add_rmsnorm(np.array([[1.0, 4.0]]), np.array([[2.0, 0.0]]), eps=0.0)
    # (3, 4): mean square 12.5
    assert np.array_equal(s, [[3.0, 4.0]])
    assert np.allclose(xn, np.array([[3.0, 4.0]]) / np.sqrt(12.5), rtol=1e-15)
    assert np.allclose(mx.swiglu(np.array([[0.0, 2.0, 5.0, 3.0]])),
                       [[0.0, 2.0 / (1 + np.exp(-2.0)) * 3.0]], rtol=1e-15)
