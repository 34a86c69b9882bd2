"""The narrow-format operators on a B200 against the float64 oracle.

Quantisation, its inverse and the norm's codes are compared bit for bit.  A
product's output is held to its own rounding, 2^-8 of the value (bf16, to
nearest), plus the fp32 accumulation: the products of two elements are exact
in fp32 (at most 8 bits of mantissa; bf16 products: 16), and every one of K additions
loses at most 2^-23 of the sum of magnitudes S (truncation allowed): K * 2^-23 * S."""

import numpy as np
import pytest
import torch

from oracle import bf16_round, fp8_block_dequant, mx_oracle as mx
from routed_moe_layer_b200 import inputs, ops
from routed_moe_layer_b200.ops import BlockConfig
from tests.parity import to_np
from tests.test_zz_write_guards import guarded

pytestmark = pytest.mark.gpu

DEV = "cuda"
FMTS = ["mxfp8", "mxfp4"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(rows, K, seed):
    """bf16 rows of different sizes, with zeros, ties, subnormals and large values."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x = x.bfloat16().float()
    flat = x.view(-1)
    special = torch.tensor([0.0, -0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 448.0, 17.0,
                            2.0 ** -130, -2.0 ** -133, 3e38, -3e38, 1.1875, 1.0625])
    at = torch.randint(0, flat.numel(), (max(1, flat.numel() // 40),), generator=g)
    flat[at] = special[torch.randint(0, len(special), (len(at),), generator=g)]
    return x.bfloat16()


def stored(codes, scales, fmt):
    c, s = mx.mx_store(codes, scales, fmt)
    return torch.from_numpy(c), torch.from_numpy(s)


def operands(rows, K, fmt, seed, lead=None, scale=1.0):
    """Random MX operands made by the oracle: device arrays and their float64 values."""
    g = gen(seed)
    n = rows if lead is None else lead * rows
    x = (scale * torch.randn(n, K, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).numpy()
    codes, scales = fast_quantize(x, fmt)
    v = mx.mx_values(codes, scales, fmt)
    if lead is None:
        c, s = stored(codes, scales, fmt)
        return c.to(DEV), s.to(DEV), v
    parts = [stored(codes[i * rows:(i + 1) * rows], scales[i * rows:(i + 1) * rows], fmt)
             for i in range(lead)]
    return (torch.stack([p[0] for p in parts]).to(DEV), torch.stack([p[1] for p in parts]).to(DEV),
            v.reshape(lead, rows, K))


def fast_quantize(x, fmt):
    """The oracle's quantisation, blocks at once (finite values)."""
    b = x.astype(np.float64).reshape(x.shape[0], -1, 32)
    amax = np.abs(b).max(2)
    p = np.vectorize(lambda a: mx.mx_power(a, fmt))(amax) if amax.size else np.zeros(amax.shape, int)
    codes = mx.mx_round(b / (2.0 ** p)[:, :, None], fmt).reshape(x.shape)
    return codes, (p + 127).astype(np.uint8)


def groups(R, E, seed, lead_rows=0, tail_rows=0):
    """Ragged offsets over R rows: some groups empty, rows before and after the groups."""
    g = np.random.default_rng(seed)
    cuts = np.sort(g.integers(lead_rows, R - tail_rows + 1, E - 1)) if E > 1 else np.zeros(0, int)
    return np.concatenate([[lead_rows], cuts, [R - tail_rows]]).astype(np.int32)


def check_product(y, x, w, off, row_w=None, dest=None):
    ref = mx.grouped_mm(x, w, off)
    S = mx.grouped_mm(np.abs(x), np.abs(w), off)
    K = x.shape[1]
    if row_w is not None:
        ref, S = ref * row_w[:, None], S * np.abs(row_w)[:, None]
    got = to_np(y).astype(np.float64)
    if dest is not None:
        got = got[dest]
    rows = slice(off[0], off[-1])
    # one more fp32 rounding for the row weight
    tol = 2.0 ** -8 * np.abs(ref) + (K + 2) * 2.0 ** -23 * S
    err = np.abs(got - ref)[rows]
    assert np.all(err <= tol[rows] * (1 + 1e-6)), (np.max(err / np.maximum(tol[rows], 1e-300)))


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 128), (33, 160), (257, 224), (64, 1024),
                                    (2, 16384)])
def test_quantize_is_the_oracles(rows, K, fmt):
    x = values(rows, K, rows * 1000 + K)
    want_c, want_s = stored(*mx.mx_quantize(to_np(x), fmt), fmt)
    c, s = ops.mx_quantize(x.to(DEV), fmt)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(c.cpu(), want_c)
    back = ops.mx_dequantize(c, s, fmt)
    v = mx.mx_values(*mx.mx_load(c.cpu().numpy(), s.cpu().numpy(), K, fmt), fmt)
    assert np.array_equal(to_np(back), bf16_round(v))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_every_bf16_value(fmt):
    """Each of the 65,536 bf16 patterns alone in its block (zeros beside it), and
    beside a 1.0: every scale byte, subnormals, infinities, NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536, 64, dtype=torch.bfloat16)
    x[:, 5] = bits
    x[:, 40] = bits
    x[:, 41] = 1.0
    c, s = ops.mx_quantize(x.to(DEV), fmt)
    xn = x.double().numpy()
    finite = np.isfinite(xn).all(1)
    codes, scales = np.zeros(x.shape, np.uint8), np.full((65536, 2), 255, np.uint8)
    codes[finite], scales[finite] = fast_quantize(xn[finite], fmt)
    want_c, want_s = stored(codes, scales, fmt)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(c.cpu(), want_c)
    back = to_np(ops.mx_dequantize(c, s, fmt))
    assert np.array_equal(np.isnan(back).any(1), ~finite)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_stack_is_its_matrices(fmt):
    x = torch.stack([values(33, 96, 7), values(33, 96, 8), values(33, 96, 9)]).to(DEV)
    c, s = ops.mx_quantize(x, fmt)
    assert s.shape == (3, 1, 33, 4)
    for i in range(3):
        ci, si = ops.mx_quantize(x[i].contiguous(), fmt)
        assert torch.equal(c[i], ci) and torch.equal(s[i], si)
    assert torch.equal(ops.mx_dequantize(c, s, fmt)[1], ops.mx_dequantize(c[1], s[1], fmt))


def test_quantize_offsets_past_32_bits():
    rows, K = 140000, 16384  # 2.29e9 elements
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[rows - 1] = values(1, K, 3)[0].to(DEV)
    c, s = ops.mx_quantize(x, "mxfp8")
    c1, s1 = ops.mx_quantize(x[rows - 1:].contiguous(), "mxfp8")
    assert torch.equal(c[rows - 1:], c1) and torch.equal(s[:, rows - 1:], s1)
    assert not c[rows - 2].any()
    del x
    assert torch.equal(ops.mx_dequantize(c, s, "mxfp8")[rows - 1:], ops.mx_dequantize(c1, s1, "mxfp8"))


def test_empty_and_misaligned_calls():
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    c, s = ops.mx_quantize(none, "mxfp4")
    assert c.shape == (0, 32) and s.shape == (1, 0, 4)
    assert ops.mx_dequantize(c, s, "mxfp4").shape == (0, 64)
    assert [t.shape[0] for t in ops.add_rmsnorm(none, none, fmt="mxfp8")] == [0, 0, 0, 1]
    w = torch.ones(2, 32, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert ops.grouped_mm(none, w, off).shape == (0, 32)
    wc, ws = ops.mx_quantize(w, "mxfp4")
    assert ops.grouped_mm_mx(c, s, wc, ws, off, "mxfp4").shape == (0, 32)
    # rows, but none of them in a group
    y = torch.full((5, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(5, 64, dtype=torch.bfloat16, device=DEV)
    ops.grouped_mm(x, w, off, out=y)
    ops.grouped_mm_mx(*ops.mx_quantize(x, "mxfp4"), wc, ws, off, "mxfp4", out=y)
    assert (y == 7).all()
    buf = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        ops.mx_quantize(buf[4:4 + 256].view(4, 64), "mxfp8")  # 8 bytes off
    with pytest.raises(ValueError, match="contiguous"):
        ops.mx_quantize(torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV).t(), "mxfp8")


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("fmt", [None] + FMTS)
@pytest.mark.parametrize("T,H", [(1, 64), (3, 192), (17, 1024), (5, 1088), (300, 2048), (9, 4096),
                                 (2, 8192), (3, 16384)])
def test_add_rmsnorm(T, H, fmt):
    g = gen(T + H)
    x = torch.randn(T, H, generator=g).bfloat16()
    r = (3 * torch.randn(T, H, generator=g)).bfloat16()
    x[T // 2] = 0
    r[T // 2] = 0  # an all-zero row
    gamma = 1 + 0.2 * torch.randn(H, generator=g)
    for res, gm, eps in ((r, gamma, 1e-6), (None, None, 1e-5), (r, None, 0.1)):
        ref_s, ref = mx.add_rmsnorm(to_np(x), None if res is None else to_np(res), eps,
                                    None if gm is None else gm.numpy())
        d = [None if t is None else t.to(DEV) for t in (x, res, gm)]
        out = ops.add_rmsnorm(d[0], d[1], d[2], eps=eps, fmt=fmt)
        assert np.array_equal(to_np(out[0]), ref_s)
        # half a bf16 step, and in fp32: the sum of squares loses at most H * 2^-24 of itself
        # (half of that after the root), the quotient, root and two products half a step each
        tol = (2.0 ** -8 + (H / 2 + 6) * 2.0 ** -24) * np.abs(ref)
        assert np.all(np.abs(to_np(out[1]) - ref) <= tol * (1 + 1e-6) + 1e-40)
        if fmt:
            c, s = ops.mx_quantize(out[1], fmt)
            assert torch.equal(out[2], c) and torch.equal(out[3], s)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_add_rmsnorm_in_place(which):
    g = gen(5)
    x, r = torch.randn(40, 640, generator=g).bfloat16().to(DEV), torch.randn(40, 640, generator=g).bfloat16().to(DEV)
    want = ops.add_rmsnorm(x, r, fmt="mxfp8")
    a, b = x.clone(), r.clone()
    got = ops.add_rmsnorm(a, b, fmt="mxfp8", sum_out=a if which == "x" else b)
    assert got[0].data_ptr() == (a if which == "x" else b).data_ptr()
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    assert torch.equal(b if which == "x" else a, r if which == "x" else x)
    # a row alone gives the row's bits in the batch
    one = ops.add_rmsnorm(x[7:8], r[7:8], fmt="mxfp8")
    assert torch.equal(one[1], want[1][7:8]) and torch.equal(one[2], want[2][7:8])
    assert torch.equal(one[3][:, 0], want[3][:, 7])


def test_add_rmsnorm_propagates_nan_to_its_row_alone():
    x = torch.ones(4, 128, dtype=torch.bfloat16, device=DEV)
    x[2, 77] = float("nan")
    _, xn, c, s = ops.add_rmsnorm(x, fmt="mxfp4")
    assert torch.isnan(xn[2]).all() and not torch.isnan(xn[[0, 1, 3]]).any()
    assert (s[:, 2] == 255).all() and (s[:, [0, 1, 3]] != 255).all()


# ------------------------------------------------------------------ products
SHAPES = [  # R, E, N, K: swapped operands, items of 64 and of 128 rows (bf16: pair tiles too)
    (1, 1, 32, 32), (8, 16, 64, 96), (40, 3, 96, 160), (257, 5, 160, 352), (300, 2, 544, 512),
    (600, 1, 256, 128), (1000, 7, 288, 1056), (515, 128, 64, 256), (65, 1, 32, 32),
    (130, 2, 128, 2112), (128, 2, 128, 2112), (64, 1, 416, 1184), (200, 4, 64, 64),
]


@pytest.mark.parametrize("R,E,N,K", SHAPES)
def test_grouped_mm(R, E, N, K):
    g = gen(R + N)
    x = torch.randn(R, K, generator=g).bfloat16()
    w = torch.randn(E, N, K, generator=g).bfloat16()
    lead, tail = (2, 3) if R > 30 else (0, 0)
    off = groups(R, E, R, lead, tail)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.alloc_workspace(4096, DEV)
    y = ops.grouped_mm(x.to(DEV), w.to(DEV), torch.from_numpy(off).to(DEV), out=out, workspace=ws)
    assert ops.read_device_status(ws)[0] == 0
    check_product(y, to_np(x), to_np(w), off)
    assert (y[:lead] == 7).all() and (y[R - tail:] == 7).all()  # rows outside the groups


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,N,K", SHAPES)
def test_grouped_mm_mx(R, E, N, K, fmt):
    xc, xs, x = operands(R, K, fmt, R + K)
    wc, wsc, w = operands(N, K, fmt, N + K, lead=E, scale=0.1)
    lead, tail = (2, 3) if R > 30 else (0, 0)
    off = groups(R, E, R, lead, tail)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.alloc_workspace(256, DEV)
    y = ops.grouped_mm_mx(xc, xs, wc, wsc, torch.from_numpy(off).to(DEV), fmt, out=out, workspace=ws)
    assert ops.read_device_status(ws)[0] == 0
    check_product(y, x, w, off)
    assert (y[:lead] == 7).all() and (y[R - tail:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_mm_mx_weights_and_destinations(fmt):
    R, E, N, K, rows = 300, 6, 128, 256, 350
    xc, xs, x = operands(R, K, fmt, 1)
    wc, wsc, w = operands(N, K, fmt, 2, lead=E)
    off = groups(R, E, 4)
    g = gen(9)
    row_w = torch.randn(R, generator=g)
    dest = torch.randperm(rows, generator=g)[:R].int()
    dest[10], dest[20] = -1, rows  # not stored
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.grouped_mm_mx(xc, xs, wc, wsc, torch.from_numpy(off).to(DEV), fmt, row_w=row_w.to(DEV),
                      row_dest=dest.to(DEV), out=out)
    kept = np.ones(R, bool)
    kept[[10, 20]] = False
    ref, S = mx.grouped_mm(x, w, off), mx.grouped_mm(np.abs(x), np.abs(w), off)
    rw = row_w.numpy().astype(np.float64)[:, None]
    got = to_np(out)[dest.numpy()[kept]]
    tol = 2.0 ** -8 * np.abs(ref * rw) + (K + 2) * 2.0 ** -23 * S * np.abs(rw)
    assert np.all(np.abs(got - (ref * rw)[kept]) <= tol[kept] * (1 + 1e-6))
    free = np.setdiff1d(np.arange(rows), dest.numpy()[kept])
    assert (out[torch.from_numpy(free).to(DEV)] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_every_element_and_scale_reaches_the_product(fmt):
    """One-hot rows against matrices of every code: the product reads each
    element, each row's and each column's scale from the right place."""
    K, N = 512, 256
    grid = mx.mx_grid(fmt)
    n = 2 * len(grid)
    signed = np.array([c if c < len(grid) else c - len(grid) + (128 if fmt == "mxfp8" else 8)
                       for c in range(n)], np.uint8)
    rng = np.random.default_rng(3)
    wc = signed[rng.integers(0, n, (N, K))]
    wsb = rng.integers(117, 137, (N, K // 32)).astype(np.uint8)
    xc = np.zeros((K, K), np.uint8)
    one = 0x38 if fmt == "mxfp8" else 2  # 1.0
    xc[np.arange(K), np.arange(K)] = one
    xsb = rng.integers(117, 137, (K, K // 32)).astype(np.uint8)
    xd, xsd = stored(xc, xsb, fmt)
    wd, wsd = stored(wc, wsb, fmt)
    off = torch.tensor([0, K], dtype=torch.int32, device=DEV)
    y = ops.grouped_mm_mx(xd.to(DEV), xsd.to(DEV), wd[None].to(DEV), wsd[None].to(DEV), off, fmt)
    ref = mx.mx_values(xc, xsb, fmt) @ mx.mx_values(wc, wsb, fmt).T  # one term each: exact
    assert np.array_equal(to_np(y), ref)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [24, 96])
def test_powers_far_from_each_other(R, fmt):
    """Blocks of rows with powers from 2^-126 to 2^120 against columns with the
    opposite ones: each product lies near 1 and is exact, however far its
    factors' scales lie apart."""
    K, N = 256, 64
    rng = np.random.default_rng(5)
    one = 0x38 if fmt == "mxfp8" else 2  # 1.0
    xc, wc = np.full((R, K), one, np.uint8), np.full((N, K), one, np.uint8)
    blocks = K // 32
    # one nonzero block a row; in it the row's power p, and the columns' -p in that block
    p = rng.integers(-120, 121, blocks)
    at = np.arange(R) % blocks
    xc[np.arange(K)[None, :] // 32 != at[:, None]] = 0
    xsb = np.full((R, blocks), 127, np.uint8)
    xsb[np.arange(R), at] = 127 + p[at]
    wsb = np.broadcast_to(127 - p, (N, blocks)).astype(np.uint8) + rng.integers(0, 5, (N, blocks)).astype(np.uint8)
    xd, xsd = stored(xc, xsb, fmt)
    wd, wsd = stored(wc, wsb, fmt)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    y = ops.grouped_mm_mx(xd.to(DEV), xsd.to(DEV), wd[None].to(DEV), wsd[None].to(DEV), off, fmt)
    ref = 32.0 * 2.0 ** (wsb.astype(int) - (127 - p))[:, at].T
    assert np.array_equal(to_np(y), ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_one_expert_takes_every_row(fmt):
    """Skewed as far as it goes: the forms are chosen by the average."""
    E, H, I = 64, 160, 64
    w13c, w13s, w13 = operands(2 * I, H, fmt, 2, lead=E, scale=H ** -0.5)
    w2c, w2s, w2 = operands(H, I, fmt, 3, lead=E, scale=I ** -0.5)
    for R, e in ((100, 63), (100, 0), (900, 31), (1500, 7)):
        xc, xs, x = operands(R, H, fmt, R)
        off = np.where(np.arange(E + 1) > e, R, 0).astype(np.int32)
        tok = torch.randperm(R, generator=gen(1)).int()
        ref, tol = experts_tolerance(x[tok.numpy()], w13, w2, off, fmt, np.ones(R))
        y = ops.expert_rows_mx(xc, xs, torch.from_numpy(off).to(DEV), w13c, w13s, w2c, w2s, None,
                               fmt, tok_of=tok.to(DEV))
        assert np.all(np.abs(to_np(y) - ref) <= tol * (1 + 1e-6))


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_blocks_reach_their_rows_and_columns_alone(fmt):
    R, N, K = 200, 96, 160
    xc, xs, _ = operands(R, K, fmt, 3)
    wc, wsc, _ = operands(N, K, fmt, 4, lead=1)
    xs[1, 150, 0] = 255   # block 4 of row 150
    wsc[0, 0, 17, 2] = 255
    y = ops.grouped_mm_mx(xc, xs, wc, wsc, torch.tensor([0, R], dtype=torch.int32, device=DEV), fmt)
    nan = torch.isnan(y)
    assert nan[150].all() and nan[:, 17].all()
    nan[150] = False
    nan[:, 17] = False
    assert not nan.any()


def test_block_scaled_fp8_weights_are_mx_weights():
    """The weights of forward_fp8 (one scale per 128 x 128 block), their scales spread."""
    E, N, K, R = 3, 320, 384, 150
    w = inputs.make_fp8_weights(K, seed=1, E=E, I=N // 2, I_shared=0)
    codes, blocks = w["w13_q"], w["w13_s"]
    assert codes.shape == (E, N, K)
    xc, xs, x = operands(R, K, "mxfp8", 2)
    off = groups(R, E, 3)
    y = ops.grouped_mm_mx(xc, xs, codes.to(DEV), ops.mx_block_scales(blocks.to(DEV), N),
                          torch.from_numpy(off).to(DEV), "mxfp8")
    check_product(y, x, fp8_block_dequant(codes.numpy(), blocks.numpy()), off)


def test_bad_offsets_are_reported_and_write_nothing_outside():
    R, E, N, K = 600, 4, 64, 64
    x = torch.ones(R, K, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(E, N, K, dtype=torch.bfloat16, device=DEV)
    xc, xs = ops.mx_quantize(x, "mxfp8")
    wc, wsc = ops.mx_quantize(w, "mxfp8")
    buf = torch.full((R + 64, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.alloc_workspace(4096, DEV)
    for bad in ([0, 100, 300, 500, R + 50], [-5, 10, 20, 30, 40], [0, 400, 200, 500, 600],
                [2 ** 30, 2 ** 31 - 1, 5, 6, 7]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        ops.grouped_mm(x, w, off, out=buf[:R], workspace=ws)
        assert ops.read_device_status(ws)[0] == 6
        ops.grouped_mm_mx(xc, xs, wc, wsc, off, "mxfp8", out=buf[:R], workspace=ws)
        assert ops.read_device_status(ws)[0] == 6
        assert (buf[R:] == 7).all()
    ok = torch.tensor([0, 100, 100, 500, R], dtype=torch.int32, device=DEV)
    ops.grouped_mm(x, w, ok, out=buf[:R], workspace=ws)
    assert ops.read_device_status(ws)[0] == 0  # cleared by the next call
    assert (buf[:R] == K).all()


# R, E, N, K of pair tiles: over 192 rows an expert, and more items of 128 x 128 than SMs
PAIR_SHAPES = [(1000, 1, 2720, 352), (1500, 5, 1312, 1056), (3000, 3, 800, 96), (7800, 40, 416, 32),
               (1100, 1, 2560, 2112), (700, 1, 3200, 160)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,N,K", PAIR_SHAPES)
def test_grouped_mm_mx_pair_tiles(R, E, N, K, fmt):
    assert R > 192 * E and (R // 128 + E) * -(-N // 128) > 148
    xc, xs, x = operands(R, K, fmt, R + K)
    wc, wsc, w = operands(N, K, fmt, N + K, lead=E, scale=0.1)
    lead, tail = 2, 3
    off = groups(R, E, R, lead, tail)
    offd = torch.from_numpy(off).to(DEV)
    ws = ops.alloc_workspace(256, DEV)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = ops.grouped_mm_mx(xc, xs, wc, wsc, offd, fmt, out=out, workspace=ws)
    assert ops.read_device_status(ws)[0] == 0
    check_product(y, x, w, off)
    assert (y[:lead] == 7).all() and (y[R - tail:] == 7).all()
    # weights that scale exactly, destinations in any order, two of them nowhere
    g = gen(9)
    row_w = 2.0 ** torch.randint(-2, 3, (R,), generator=g).float()
    dest = torch.randperm(R + 50, generator=g)[:R].int()
    dest[10], dest[20] = -1, R + 50
    z = torch.full((R + 50, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.grouped_mm_mx(xc, xs, wc, wsc, offd, fmt, row_w=row_w.to(DEV), row_dest=dest.to(DEV), out=z)
    kept = torch.ones(R, dtype=torch.bool)
    kept[[10, 20]] = False
    kept[:lead] = False
    kept[R - tail:] = False
    want = (y.float() * row_w.to(DEV)[:, None]).bfloat16()
    assert torch.equal(z[dest[kept].long().to(DEV)], want[kept.to(DEV)])
    free = np.setdiff1d(np.arange(R + 50), dest.numpy()[kept.numpy()])
    assert (z[torch.from_numpy(free).to(DEV)] == 7).all()
    # the bits of the swapped form
    lo, hi = int(off[0]), min(int(off[1]), int(off[0]) + 50)
    part = torch.full((E + 1,), hi - lo, dtype=torch.int32, device=DEV)
    part[0] = 0
    a = ops.grouped_mm_mx(xc[lo:hi].contiguous(), xs[:, lo:hi].contiguous(), wc, wsc, part, fmt)
    assert torch.equal(a, y[lo:hi])


@pytest.mark.parametrize("fmt", FMTS)
def test_pair_tiles_read_every_element_and_scale(fmt):
    """As test_every_element_and_scale_reaches_the_product; a NaN block of a row and one
    of a column besides."""
    K, N = 512, 3840
    grid = mx.mx_grid(fmt)
    n = 2 * len(grid)
    signed = np.array([c if c < len(grid) else c - len(grid) + (128 if fmt == "mxfp8" else 8)
                       for c in range(n)], np.uint8)
    rng = np.random.default_rng(3)
    wc = signed[rng.integers(0, n, (N, K))]
    wsb = rng.integers(117, 137, (N, K // 32)).astype(np.uint8)
    xc = np.zeros((K, K), np.uint8)
    xc[np.arange(K), np.arange(K)] = 0x38 if fmt == "mxfp8" else 2  # 1.0
    xsb = rng.integers(117, 137, (K, K // 32)).astype(np.uint8)
    ref = mx.mx_values(xc, xsb, fmt) @ mx.mx_values(wc, wsb, fmt).T  # one term each: exact
    off = torch.tensor([0, K], dtype=torch.int32, device=DEV)

    def product():
        xd, xsd = stored(xc, xsb, fmt)
        wd, wsd = stored(wc, wsb, fmt)
        return ops.grouped_mm_mx(xd.to(DEV), xsd.to(DEV), wd[None].to(DEV), wsd[None].to(DEV), off, fmt)
    assert np.array_equal(to_np(product()), ref)
    xsb[300, 7] = 255
    wsb[2000, 3] = 255
    got = to_np(product())
    ref[300] = np.nan
    ref[:, 2000] = np.nan
    assert np.array_equal(got, ref, equal_nan=True)


def test_pair_tiles_bad_offsets():
    R, E, N, K = 2000, 4, 1280, 64
    x = torch.ones(R, K, dtype=torch.bfloat16, device=DEV)
    xc, xs = ops.mx_quantize(x, "mxfp4")
    wc, wsc = ops.mx_quantize(torch.ones(E, N, K, dtype=torch.bfloat16, device=DEV), "mxfp4")
    buf = torch.full((R + 64, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.alloc_workspace(256, DEV)
    for bad in ([0, 100, 300, 500, R + 50], [-5, 10, 20, 30, 40], [0, 400, 200, 500, 600],
                [2 ** 30, 2 ** 31 - 1, 5, 6, 7]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        ops.grouped_mm_mx(xc, xs, wc, wsc, off, "mxfp4", out=buf[:R], workspace=ws)
        assert ops.read_device_status(ws)[0] == 6
        assert (buf[R:] == 7).all()
    ok = torch.tensor([0, 100, 100, 1900, R], dtype=torch.int32, device=DEV)
    ops.grouped_mm_mx(xc, xs, wc, wsc, ok, "mxfp4", out=buf[:R], workspace=ws)
    assert ops.read_device_status(ws)[0] == 0 and (buf[:R] == K).all()


# ------------------------------------------------------------------ experts
def experts_tolerance(x, w13, w2, off, fmt, row_w):
    """ref and the bound of |y - ref|: h's fp32 errors move an element over a
    rounding border only where it lies that near to one; each such element may be
    one step of its grid off (its block's power too, where the block's largest
    element lies that near to the power's border)."""
    H, I = x.shape[1], w13.shape[1] // 2
    gu, S = mx.grouped_mm(x, w13, off), mx.grouped_mm(np.abs(x), np.abs(w13), off)
    h = mx.swiglu(gu)
    g, u = gu[:, :I], gu[:, I:]
    eg, eu = H * 2.0 ** -23 * S[:, :I], H * 2.0 ** -23 * S[:, I:]
    silu = g / (1 + np.exp(-g))
    # silu' lies within +-1.1; its fast exponential and divide are within 2^-19 of it
    d = 1.1 * eg * np.abs(u) + (np.abs(silu) + 1.1 * eg) * eu + 2.0 ** -19 * np.abs(h)
    codes, scales = fast_quantize(h, fmt)
    q = mx.mx_values(codes, scales, fmt)
    lo, hi = nearest(h - d, h, fmt), nearest(h + d, h, fmt)
    slack = np.maximum(np.abs(lo - q), np.abs(hi - q))
    b = np.abs(h).reshape(len(h), -1, 32)
    top = mx.mx_grid(fmt)[-1] * 2.0 ** (scales.astype(int) - 127)
    amax, dm = b.max(2), d.reshape(b.shape).max(2)
    border = (amax + dm > top) | (amax - dm <= top / 2)
    # the whole block may then lie on the neighbouring power's grid: at most one step of the
    # wider one at its largest element (E4M3 2^-3, E2M1 1/2 of the element's binade, doubled)
    step = (0.25 if fmt == "mxfp8" else 1.0) * 2 * amax
    slack = np.maximum(slack, np.repeat(np.where(border, step, 0.0), 32, axis=1))
    ref = mx.grouped_mm(q, w2, off) * row_w[:, None]
    Sh = mx.grouped_mm(np.abs(q) + slack, np.abs(w2), off)
    tol = mx.grouped_mm(slack, np.abs(w2), off) + (I + 2) * 2.0 ** -23 * Sh
    tol = tol * np.abs(row_w)[:, None]
    return ref, tol + 2.0 ** -8 * (np.abs(ref) + tol)


def nearest(v, like, fmt):
    """v rounded on the grids (powers) that ``like`` has, saturated there."""
    _, scales = fast_quantize(like, fmt)
    p = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)
    top = mx.mx_grid(fmt)[-1]
    codes = mx.mx_round(np.clip(v / p, -top, top), fmt)
    return mx.mx_values(codes, scales, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 4, 64, 32), (30, 32, 4, 288, 160), (13, 16, 3, 1184, 64), (9, 4, 2, 160, 96), (70, 16, 4, 256, 160),
                                       (400, 3, 2, 512, 288), (333, 1, 1, 96, 128)])
def test_expert_rows_mx(T, E, k, H, I, fmt):
    xc, xs, x = operands(T, H, fmt, T + H)
    w13c, w13s, w13 = operands(2 * I, H, fmt, H + I, lead=E, scale=H ** -0.5)
    w2c, w2s, w2 = operands(H, I, fmt, I, lead=E, scale=I ** -0.5)
    g = gen(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).reshape(-1)
    order = torch.argsort(ids, stable=True)
    off = np.concatenate([[0], np.cumsum(np.bincount(ids.numpy(), minlength=E))]).astype(np.int32)
    tok = (order // k).int()
    row_w = torch.rand(T, k, generator=g).reshape(-1)[order]
    offd = torch.from_numpy(off).to(DEV)
    rows = x[tok.numpy()]
    ref, tol = experts_tolerance(rows, w13, w2, off, fmt, row_w.numpy().astype(np.float64))
    y = ops.expert_rows_mx(xc, xs, offd, w13c, w13s, w2c, w2s, order.int().to(DEV), fmt,
                           row_w=row_w.to(DEV), tok_of=tok.to(DEV))
    got = to_np(y).astype(np.float64)[order.numpy()]
    assert np.all(np.abs(got - ref) <= tol * (1 + 1e-6)), np.max(np.abs(got - ref) / tol)
    # the rows already grouped, in their own order: the same bits
    cs, ss = xc[tok.long().to(DEV)].contiguous(), xs[:, tok.long().to(DEV)].contiguous()
    y2 = ops.expert_rows_mx(cs, ss, offd, w13c, w13s, w2c, w2s, None, fmt, row_w=row_w.to(DEV))
    assert torch.equal(y2, y[order.to(DEV)])


@pytest.mark.parametrize("fmt", FMTS)
def test_a_rows_bits_do_not_depend_on_the_other_rows(fmt):
    """The forms for few and for many rows per expert, with and without a gathered
    copy: every row has the same bits in a call of 3, 40 and 700 rows."""
    E, H, I, R = 2, 288, 160, 700
    xc, xs, _ = operands(R, H, fmt, 1)
    w13c, w13s, _ = operands(2 * I, H, fmt, 2, lead=E, scale=H ** -0.5)
    w2c, w2s, _ = operands(H, I, fmt, 3, lead=E, scale=I ** -0.5)
    rows = torch.arange(R, dtype=torch.int32, device=DEV)

    def call(lo, mid, hi):  # rows [lo, mid) with expert 0, [mid, hi) with expert 1
        off = torch.tensor([0, mid - lo, hi - lo], dtype=torch.int32, device=DEV)
        y = ops.expert_rows_mx(xc, xs, off, w13c, w13s, w2c, w2s, None, fmt, tok_of=rows[lo:hi])
        z = ops.grouped_mm_mx(xc[lo:hi].contiguous(), xs[:, lo:hi].contiguous(), w13c, w13s, off, fmt)
        return y, z
    full = call(0, 300, R)
    for lo, mid, hi in ((298, 300, 301), (290, 300, 330), (0, 300, 400)):
        part = call(lo, mid, hi)
        for a, b in zip(part, full):
            assert torch.equal(a, b[lo:hi])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E", [(100, 2), (200, 2), (380, 4), (250, 2), (1400, 2)])
def test_expert_rows_mx_between_the_forms(R, E, fmt):
    """Rows on either side of where the up and the down product change their form (1,400
    rows: both pair tiles): the bits of calls of at most 30 rows."""
    H, I = 1664, 64
    xc, xs, _ = operands(R, H, fmt, 1)
    w13c, w13s, _ = operands(2 * I, H, fmt, 2, lead=E, scale=H ** -0.5)
    w2c, w2s, _ = operands(H, I, fmt, 3, lead=E, scale=I ** -0.5)
    off = groups(R, E, 3)
    tok = torch.randperm(R, generator=gen(2)).int().to(DEV)
    row_w = torch.rand(R, generator=gen(3)).to(DEV)
    y = ops.expert_rows_mx(xc, xs, torch.from_numpy(off).to(DEV), w13c, w13s, w2c, w2s, None, fmt,
                           row_w=row_w, tok_of=tok)
    for e in range(E):
        for lo in range(int(off[e]), int(off[e + 1]), 90):
            hi = min(lo + 30, int(off[e + 1]))
            part = torch.tensor([0] * (e + 1) + [hi - lo] * (E - e), dtype=torch.int32, device=DEV)
            a = ops.expert_rows_mx(xc, xs, part, w13c, w13s, w2c, w2s, None, fmt,
                                   row_w=row_w[lo:hi].contiguous(), tok_of=tok[lo:hi].contiguous())
            assert torch.equal(a, y[lo:hi])


def test_expert_rows_mx_token_outside_counts_as_zeros():
    xc, xs, _ = operands(4, 64, "mxfp8", 1)
    w13c, w13s, _ = operands(64, 64, "mxfp8", 2, lead=2)
    w2c, w2s, _ = operands(64, 32, "mxfp8", 3, lead=2)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    tok = torch.tensor([0, -1, 4, 3], dtype=torch.int32, device=DEV)
    y = ops.expert_rows_mx(xc, xs, off, w13c, w13s, w2c, w2s, None, "mxfp8", tok_of=tok)
    assert (y[1:3] == 0).all() and (y[0] != 0).any() and (y[3] != 0).any()


# ------------------------------------------------------------------ together
def block(T, H, E, I, Is, k, seed):
    cfg = BlockConfig(T=T, H=H, E=E, I=I, I_shared=Is, top_k=k, n_group=4, topk_group=2)
    d = inputs.make_block_inputs(T, H, seed=seed, E=E, I=I, I_shared=Is, unit_scale=True)
    return cfg, {n: (None if v is None else v.to(DEV)) for n, v in d.items()}


def run_layer(d, cfg, w13, w2, stream_in, gamma, fmt):
    """One layer of a stack: norm of the stream with the last block's output, the block."""
    s, xn, c, sc = ops.add_rmsnorm(d["x"], stream_in, gamma, fmt=fmt)
    return s, xn, c, sc, ops.forward_mx(xn, d["Wr"], d["bias"], w13, w2, d["ws13"], d["ws2"], cfg,
                                        fmt, x_mx=(c, sc), residual=s)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 50, 700])
def test_norm_router_experts_restore_together(T, fmt):
    H, E, I, k = 256, 16, 96, 4
    cfg, d = block(T, H, E, 128, 0, k, T)  # its bf16 experts are not used
    w13c, w13s, w13 = operands(2 * I, H, fmt, 7, lead=E, scale=H ** -0.5)
    w2c, w2s, w2 = operands(H, I, fmt, 8, lead=E, scale=I ** -0.5)
    res = inputs.make_tokens(T, H, seed=3).to(DEV)
    gamma = (1 + 0.1 * torch.randn(H, generator=gen(4))).to(DEV)
    s, xn, c, sc, out = run_layer(d, cfg, (w13c, w13s), (w2c, w2s), res, gamma, fmt)
    ids, w = ops.route(xn, d["Wr"], d["bias"], cfg)
    # the oracle under the GPU's routing, from the GPU's narrow tokens (tested bit for bit above)
    x = mx.mx_values(*mx.mx_load(c.cpu().numpy(), sc.cpu().numpy(), H, fmt), fmt)
    flat = ids.cpu().reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat.numpy(), minlength=E))])
    rw = w.cpu().reshape(-1)[order].numpy().astype(np.float64)
    y, tol = experts_tolerance(x[(order // k).numpy()], w13, w2, off, fmt, rw)
    ref, bound = to_np(s).astype(np.float64), np.zeros((T, H))
    for row, slot in enumerate(order.tolist()):
        ref[slot // k] += y[row]
        bound[slot // k] += tol[row]
    # the restore: k + 1 terms added in fp32 (half a step of the partial sums each), one rounding
    mag = np.abs(to_np(s)) + sum(np.abs(y[np.argsort(order.numpy())][j::k]) for j in range(k))
    bound += (k + 1) * 2.0 ** -24 * (mag + bound)
    bound += 2.0 ** -8 * (np.abs(ref) + bound)
    assert np.all(np.abs(to_np(out) - ref) <= bound * (1 + 1e-6))


@pytest.mark.parametrize("Is", [0, 96 * 2])
def test_forward_mx_is_its_steps(Is):
    T, H, E, I, k = 300, 256, 16, 128, 4
    cfg, d = block(T, H, E, I, Is, k, 5)
    w13, w2 = ops.mx_quantize(d["w13"], "mxfp8"), ops.mx_quantize(d["w2"], "mxfp8")
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[250:] = 0
    out = ops.forward_mx(d["x"], d["Wr"], d["bias"], w13, w2, d["ws13"], d["ws2"], cfg, "mxfp8",
                         token_mask=mask)
    full = ops.forward_mx(d["x"], d["Wr"], d["bias"], w13, w2, d["ws13"], d["ws2"], cfg, "mxfp8")
    assert torch.equal(out[:250], full[:250])  # real tokens: the bits of the call without padding
    shared = ops.dense_ffn(d["x"], d["ws13"], d["ws2"]) if Is else torch.zeros_like(d["x"])
    assert torch.equal(out[250:], shared[250:])
    # near the bf16 block: what eight bits change is a few percent of the output
    ref = ops.forward(d["x"], d["Wr"], d["bias"], d["w13"], d["w2"], d["ws13"], d["ws2"], cfg)
    assert (full - ref).float().norm() < 0.2 * ref.float().norm()


@pytest.mark.parametrize("T", [6, 32, 96])  # rows from the tokens, swapped products, pair tiles
def test_captured_replayed_and_on_two_streams(T):
    H, E, I, k = 512, 16, 128, 4
    cfg, d = block(T, H, E, I, 0, k, 6)
    w13, w2 = ops.mx_quantize(d["w13"], "mxfp4"), ops.mx_quantize(d["w2"], "mxfp4")
    res = inputs.make_tokens(T, H, seed=3).to(DEV)
    gamma = torch.ones(H, device=DEV)
    want = [t.clone() for t in run_layer(d, cfg, w13, w2, res, gamma, "mxfp4")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):  # two graphs of the same leaves, each with its own workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(run_layer(d, cfg, w13, w2, res, gamma, "mxfp4"))
        graphs.append(g)
    keep = d["x"].clone()
    for _ in range(3):
        d["x"].copy_(res)  # other inputs, then the first ones again: nothing is kept
        graphs[0].replay()
        assert not torch.equal(outs[0][4], want[4])
        d["x"].copy_(keep)
        for g, o in zip(graphs, outs):
            g.replay()
            for a, b in zip(o, want):
                assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):  # overlapping calls
        with torch.cuda.stream(streams[i % 2]):
            got.append(run_layer(d, cfg, w13, w2, res, gamma, "mxfp4"))
    torch.cuda.synchronize()
    for o in got:
        for a, b in zip(o, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [60, 900])  # swapped operands, pair tiles
def test_products_write_only_their_rows_and_leave_inputs(R, fmt):
    E, N, K = 4, 96, 160
    xc, xs, _ = operands(R, K, fmt, 1)
    wc, wsc, _ = operands(N, K, fmt, 2, lead=E)
    off = torch.from_numpy(groups(R, E, 3)).to(DEV)
    before = [t.clone() for t in (xc, xs, wc, wsc, off)]
    y, c_y = guarded((R, N), torch.bfloat16, DEV)
    ws, c_ws = guarded((256,), torch.uint8, DEV)
    ops.grouped_mm_mx(xc, xs, wc, wsc, off, fmt, out=y, workspace=ws)
    c, s = operands(2 * N, K, fmt, 5, lead=E)[:2]
    w2c, w2s = operands(K, N, fmt, 6, lead=E)[:2]
    z, c_z = guarded((R, K), torch.bfloat16, DEV)
    n = ops.lib().moe_expert_rows_mx_workspace_bytes(R, K, E, N, ops.MX_FORMATS[fmt], 1)
    ws2, c_ws2 = guarded((n,), torch.uint8, DEV)
    tok = torch.arange(R, dtype=torch.int32, device=DEV).flip(0).contiguous()
    ops.expert_rows_mx(xc, xs, off, c, s, w2c, w2s, None, fmt, tok_of=tok, y=z, workspace=ws2)
    assert ops.read_device_status(ws2)[0] == 0
    for check in (c_y, c_ws, c_z, c_ws2):
        check()
    for a, b in zip((xc, xs, wc, wsc, off), before):
        assert torch.equal(a, b)


def test_products_with_outputs_past_32_bits():
    R, N, K = 140000, 16384, 32  # 2.29e9 outputs
    g = gen(1)
    x = torch.randn(R, K, generator=g).bfloat16().to(DEV)
    w = torch.randn(1, N, K, generator=g).bfloat16().to(DEV)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    y = ops.grouped_mm(x, w, off)
    last = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    assert torch.equal(y[-5:], ops.grouped_mm(x[-5:].contiguous(), w, last))
    for fmt in FMTS:
        xc, xs = ops.mx_quantize(x, fmt)
        wc, wsc = ops.mx_quantize(w, fmt)
        ops.grouped_mm_mx(xc, xs, wc, wsc, off, fmt, out=y)
        tail = ops.grouped_mm_mx(xc[-5:].contiguous(), xs[:, -5:].contiguous(), wc, wsc, last, fmt)
        assert torch.equal(y[-5:], tail)
