"""Refusals of the narrow-format operators that need no GPU: the C entry points
return before any CUDA call, and the Python functions refuse host tensors,
wrong types, shapes and layouts."""

import ctypes

import pytest
import torch

from routed_moe_layer_b200 import build, ops

OK, INVALID, SHAPE, WORKSPACE = 0, 1, 2, 3
P = 1 << 20  # a pointer that no call below follows (512-byte aligned)


@pytest.fixture(scope="module")
def L():
    if build.needs_build():
        build.build_library()
    return ops.lib()


@pytest.mark.parametrize("kw,expect", [
    ({"rows": 0}, OK), ({"groups": 0}, OK),
    ({"rows": -1}, INVALID), ({"groups": -1}, INVALID), ({"K": 0}, INVALID),
    ({"fmt": 0}, INVALID), ({"fmt": 3}, INVALID),
    ({"K": 48}, SHAPE), ({"K": 16416}, SHAPE),
    ({"x": 0}, INVALID), ({"codes": 0}, INVALID), ({"scales": 0}, INVALID),
    ({"x": P + 8}, INVALID), ({"codes": 2 * P + 4}, INVALID), ({"scales": 3 * P + 2}, INVALID),
    ({"codes": P}, INVALID),  # in place
    ({"x": P + 16}, INVALID), ({"groups": 2 ** 20, "rows": 2 ** 12}, SHAPE),
])
def test_quantize_checks(L, kw, expect):
    a = dict(x=P, groups=1, rows=4, K=64, fmt=1, codes=2 * P, scales=3 * P) | kw
    assert L.moe_mx_quantize(a["x"], a["groups"], a["rows"], a["K"], a["fmt"], a["codes"],
                             a["scales"], None) == expect
    assert L.moe_mx_dequantize(a["codes"], a["scales"], a["groups"], a["rows"], a["K"], a["fmt"],
                               a["x"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"T": 0}, OK), ({"T": -1}, INVALID), ({"H": 0}, INVALID), ({"H": 96}, SHAPE),
    ({"H": 16448}, SHAPE), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"fmt": 5}, INVALID), ({"x": 0}, INVALID), ({"codes": 0}, INVALID), ({"scales": 0}, INVALID),
    ({"fmt": 0}, INVALID),                              # codes without a format
    ({"fmt": 0, "codes": 0, "scales": 0, "xn": 0}, INVALID),  # nothing to compute
    ({"xn": P}, INVALID), ({"xn": 4 * P}, INVALID),     # xn over x or the sum
    ({"gamma": 6 * P + 4}, INVALID), ({"residual": 7 * P + 2}, INVALID),
    ({"sum": 4 * P + 8}, INVALID),
])
def test_add_rmsnorm_checks(L, kw, expect):
    a = dict(x=P, residual=0, gamma=0, eps=1e-6, T=4, H=64, fmt=1, sum=4 * P, xn=5 * P,
             codes=2 * P, scales=3 * P) | kw
    got = L.moe_add_rmsnorm(a["x"], a["residual"] or None, a["gamma"] or None, a["eps"], a["T"],
                            a["H"], a["fmt"], a["sum"], a["xn"] or None, a["codes"] or None,
                            a["scales"] or None, None)
    assert got == expect


GROUPED = [
    ({"R": 0}, OK), ({"R": -1}, INVALID), ({"E": 0}, INVALID), ({"N": 0}, INVALID),
    ({"K": 0}, INVALID), ({"E": 129}, SHAPE), ({"N": 48}, SHAPE), ({"K": 40}, SHAPE),
    ({"N": 16416}, SHAPE), ({"K": 16416}, SHAPE), ({"R": 2 ** 31 - 1}, SHAPE),
    ({"x": 0}, INVALID), ({"w": 0}, INVALID), ({"off": 0}, INVALID), ({"y": 0}, INVALID),
    ({"y": P}, INVALID), ({"y": 2 * P}, INVALID), ({"x": P + 8}, INVALID),
    ({"w": 2 * P + 8}, INVALID), ({"y": 3 * P + 16}, INVALID), ({"off": 4 * P + 2}, INVALID),
    ({"ws": 0}, WORKSPACE), ({"ws": 5 * P + 64}, WORKSPACE), ({"ws_bytes": 128}, WORKSPACE),
]


@pytest.mark.parametrize("kw,expect", GROUPED)
def test_grouped_mm_checks(L, kw, expect):
    a = dict(x=P, off=4 * P, R=8, E=4, N=64, K=96, w=2 * P, y=3 * P, ws=5 * P, ws_bytes=1 << 16) | kw
    assert L.moe_grouped_mm(a["x"], a["off"], a["R"], a["E"], a["N"], a["K"], a["w"], a["y"],
                            a["ws"], a["ws_bytes"], None) == expect
    if expect == SHAPE:
        assert L.moe_grouped_mm_workspace_bytes(a["R"], a["E"], a["N"], a["K"]) == 0


@pytest.mark.parametrize("kw,expect", GROUPED + [
    ({"fmt": 0}, INVALID), ({"xs": 0}, INVALID), ({"wsc": 0}, INVALID), ({"xs": 6 * P + 1}, INVALID),
    ({"y_rows": 7}, INVALID), ({"y_rows": -1}, INVALID),
])
def test_grouped_mm_mx_checks(L, kw, expect):
    a = dict(x=P, xs=6 * P, off=4 * P, R=8, E=4, N=64, K=96, fmt=2, w=2 * P, wsc=7 * P, y=3 * P,
             y_rows=8, ws=5 * P, ws_bytes=1 << 16) | kw
    if a["R"] > a["y_rows"] and "y_rows" not in kw:
        a["y_rows"] = a["R"]
    assert L.moe_grouped_mm_mx(a["x"], a["xs"], a["off"], a["R"], a["E"], a["N"], a["K"], a["fmt"],
                               a["w"], a["wsc"], None, None, a["y"], a["y_rows"], a["ws"],
                               a["ws_bytes"], None) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"R": 0}, OK), ({"R": -1}, INVALID), ({"T": -1}, INVALID), ({"E": 200}, SHAPE),
    ({"H": 100}, SHAPE), ({"I": 33}, SHAPE), ({"fmt": 7}, INVALID), ({"w2": 0}, INVALID),
    ({"w2s": 0}, INVALID), ({"tok": 0}, INVALID),      # rows not gathered, but T != R
    ({"dest": 0, "y_rows": 5}, INVALID), ({"w13": 9 * P + 8}, INVALID),
    ({"tok": 3 * P + 1}, INVALID), ({"dest": 8 * P + 2}, INVALID), ({"w2s": 7 * P + 4}, INVALID),
    ({"y": 10 * P + 16}, INVALID), ({"ws_bytes": 64}, WORKSPACE), ({"ws": 0}, WORKSPACE),
])
def test_expert_rows_mx_checks(L, kw, expect):
    a = dict(x=P, xs=2 * P, T=4, tok=3 * P, off=4 * P, R=8, E=4, H=64, I=96, fmt=1, w13=9 * P,
             w13s=5 * P, w2=6 * P, w2s=7 * P, dest=8 * P, y=10 * P, y_rows=8, ws=11 * P,
             ws_bytes=1 << 20) | kw
    got = L.moe_expert_rows_mx(a["x"], a["xs"], a["T"], a["tok"] or None, a["off"], a["R"], a["E"],
                               a["H"], a["I"], a["fmt"], a["w13"], a["w13s"], a["w2"] or None,
                               a["w2s"] or None, None, a["dest"] or None, a["y"], a["y_rows"],
                               a["ws"], a["ws_bytes"], None)
    assert got == expect
    need = L.moe_expert_rows_mx_workspace_bytes(a["R"], a["H"], a["E"], a["I"], a["fmt"], 1)
    assert (need == 0) == (expect == SHAPE or a["R"] < 0 or a["fmt"] == 7)


def test_python_functions_refuse_host_tensors_and_wrong_layouts():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8)
    w = torch.zeros((2, 64, 64), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ops.mx_quantize(x, "mxfp8"), lambda: ops.mx_dequantize(q, s, "mxfp8"),
                 lambda: ops.add_rmsnorm(x), lambda: ops.grouped_mm(x, w, off),
                 lambda: ops.grouped_mm_mx(q, s, q[None], s[None], off, "mxfp8"),
                 lambda: ops.expert_rows_mx(q, s, off, q[None], s[None], q[None], s[None], None,
                                            "mxfp8")):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="fmt"):
        ops.mx_quantize(x, "int8")
    with pytest.raises(ValueError, match="matrix"):
        ops.mx_quantize(x[0], "mxfp8")
    with pytest.raises(TypeError):
        ops.mx_quantize(None, "mxfp8")
    with pytest.raises(TypeError):
        ops.grouped_mm(x, None, off)
    with pytest.raises(ValueError):
        ops.grouped_mm(x, w[0], off)


def test_tensors_of_two_devices_are_refused(monkeypatch):
    class On(torch.Tensor):  # a host tensor that says it is on a device
        def get_device(self):
            return self.on

        @property
        def is_cuda(self):
            return True

    def on(dev, *shape, dtype=torch.bfloat16):
        t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
        t.on = dev
        return t
    called = []
    monkeypatch.setattr(ops, "_call", lambda *a: called.append(a))
    ops._is(on(1, 4, 64), "x", torch.bfloat16, (4, 64), 1)
    with pytest.raises(ValueError, match="cuda:0"):
        ops._is(on(1, 4, 64), "x", torch.bfloat16, (4, 64), 0)
    with pytest.raises(ValueError, match="cuda:0"):
        ops.add_rmsnorm(on(0, 4, 64), on(1, 4, 64))
    with pytest.raises(ValueError, match="cuda:0"):
        ops.grouped_mm(on(0, 4, 64), on(1, 2, 64, 64), on(0, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="cuda:0"):
        ops.mx_dequantize(on(0, 4, 64, dtype=torch.uint8), on(1, 1, 4, 4, dtype=torch.uint8), "mxfp8")
    assert not called
