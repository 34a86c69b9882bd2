"""Outputs of the narrow-format operators that lie over what the call reads are refused
before any CUDA call (the pointers below are not followed)."""

import pytest
import torch

from routed_moe_layer_b200 import build, ops

INVALID, WORKSPACE = 1, 3
P = 1 << 24  # 16 MB apart: no range below reaches the next pointer


@pytest.fixture(scope="module")
def L():
    if build.needs_build():
        build.build_library()
    return ops.lib()


def touching(at, n, out):
    """Where an output of `out` bytes may and may not lie beside the n bytes at `at`: 64-byte
    steps, so that nothing but the overlap is wrong."""
    free = [at - out, at + -(-n // 64) * 64]
    taken = [at, at - out + 64, at + (n - 1) // 64 * 64]
    return [(y, False) for y in free] + [(y, True) for y in taken]


# the workspace is missing, which is tested last: a call that is not refused for its
# output comes back with that
def expect(over):
    return INVALID if over else WORKSPACE


def test_grouped_mm(L):
    R, E, N, K = 7, 3, 64, 96
    x, w = P, 2 * P
    for at, n in ((x, R * K * 2), (w, E * N * K * 2)):
        for y, over in touching(at, n, R * N * 2):
            got = L.moe_grouped_mm(x, 4 * P, R, E, N, K, w, y, None, 0, None)
            assert got == expect(over), (at, y)


@pytest.mark.parametrize("fmt", [1, 2])
def test_grouped_mm_mx(L, fmt):
    R, E, N, K, y_rows = 7, 3, 64, 160, 9
    x, xs, w, ws = P, 2 * P, 3 * P, 4 * P
    row = K if fmt == 1 else K // 2
    for at, n in ((x, R * row), (xs, 2 * R * 4), (w, E * N * row), (ws, E * 2 * N * 4)):
        for y, over in touching(at, n, y_rows * N * 2):
            got = L.moe_grouped_mm_mx(x, xs, 5 * P, R, E, N, K, fmt, w, ws, None, 6 * P, y, y_rows,
                                      None, 0, None)
            assert got == expect(over), (at, y)


@pytest.mark.parametrize("fmt", [1, 2])
def test_expert_rows_mx(L, fmt):
    T, R, E, H, I, y_rows = 4, 8, 3, 96, 160, 8
    x, xs, w13, w13s, w2, w2s = (i * P for i in range(1, 7))
    h, i = (H, I) if fmt == 1 else (H // 2, I // 2)
    for at, n in ((w13, E * 2 * I * h), (w13s, E * 2 * I * 4), (w2, E * H * i), (w2s, E * 2 * H * 4)):
        for y, over in touching(at, n, y_rows * H * 2):
            got = L.moe_expert_rows_mx(x, xs, T, 7 * P, 8 * P, R, E, H, I, fmt, w13, w13s, w2, w2s,
                                       None, 9 * P, y, y_rows, None, 0, None)
            assert got == expect(over), (at, y)
    assert L.moe_expert_rows_mx(x, xs, T, 7 * P, 8 * P, R, E, H, I, fmt, w13, w13s, w2, w2s, None,
                                9 * P, x, y_rows, None, 0, None) == INVALID


# These have no workspace that could be missing, so only what is refused is tried, and not where
# a refusal that got lost would make a kernel follow the pointers.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that nothing may follow")


@no_gpu
@pytest.mark.parametrize("fmt", [1, 2])
def test_quantisation(L, fmt):
    groups, rows, K = 2, 5, 160
    n = groups * rows
    row = K if fmt == 1 else K // 2
    x, c, s = P, 2 * P, 3 * P
    sizes = {"x": n * K * 2, "c": n * row, "s": n * 2 * 4}

    def both(x, c, s):
        return [L.moe_mx_quantize(x, groups, rows, K, fmt, c, s, None),
                L.moe_mx_dequantize(c, s, groups, rows, K, fmt, x, None)]
    for name, at in (("c", c), ("s", s)):
        for y, over in touching(at, sizes[name], sizes["x"]):
            if over:
                assert both(y, c, s) == [INVALID] * 2
    for y, over in touching(c, sizes["c"], sizes["s"]):
        if over:  # the scales over the codes
            assert L.moe_mx_quantize(x, groups, rows, K, fmt, c, y, None) == INVALID


@no_gpu
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_add_rmsnorm(L, fmt):
    T, H = 5, 192
    n, row = T * H * 2, H if fmt == 1 else H // 2
    at = dict(x=P, residual=2 * P, gamma=3 * P, sum=4 * P, xn=5 * P)
    size = dict(x=n, residual=n, gamma=H * 4, sum=n, xn=n)
    if fmt:
        at |= dict(codes=6 * P, scales=7 * P)
        size |= dict(codes=T * row, scales=2 * T * 4)

    def call(**kw):
        a = dict(codes=None, scales=None) | at | kw
        return L.moe_add_rmsnorm(a["x"], a["residual"], a["gamma"], 1e-6, T, H, fmt, a["sum"],
                                 a["xn"], a["codes"], a["scales"], None)
    outs = [o for o in ("sum", "xn", "codes", "scales") if o in at]
    for o in outs:
        for other in at:
            if other == o:
                continue
            for y, over in touching(at[other], size[other], size[o]):
                if over and not (o == "sum" and other in ("x", "residual") and y == at[other]):
                    assert call(**{o: y}) == INVALID, (o, other, y - at[other])
    # in place over x, whose other rows are the residual's
    assert call(sum=P, residual=P + H * 2) == INVALID
