"""Calls of the narrow-format operators that the Python functions refuse before
the library is reached, tried on host tensors that say they are on a device
(the library's calls are replaced by a list of those that got through)."""

import pytest
import torch

from routed_moe_layer_b200 import ops

BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class On(torch.Tensor):
    """A host tensor that says it is on a device."""

    on = 0

    def get_device(self):
        return self.on

    @property
    def is_cuda(self):
        return True


def on(*shape, dtype=U8, dev=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.on = dev
    return t


@pytest.fixture
def called(monkeypatch):
    """Names of the entry points that a call reached."""
    names = []
    monkeypatch.setattr(ops, "_call", lambda name, *a: names.append(name))
    monkeypatch.setattr(ops, "_ws_bytes", lambda *a: 256)
    return names


def mx(rows, K, fmt, lead=()):
    """Codes and scales of zeros, laid out for rows of K elements."""
    return (on(*lead, rows, K if fmt == "mxfp8" else K // 2), on(*lead, -(-K // 128), rows, 4))


# the rows' format and K, the weights' format and K: the scales' shapes are those of
# the rows' K in all of them, so the codes alone tell
WRONG_WIDTHS = [
    ("mxfp8", 1024, "mxfp4", 1024),  # half the bytes that K elements take
    ("mxfp4", 1024, "mxfp8", 1024),  # twice the bytes
    ("mxfp8", 1024, "mxfp8", 928),   # another K in the same word of scales
    ("mxfp4", 1024, "mxfp4", 992),
    ("mxfp8", 96, "mxfp8", 1),
    ("mxfp8", 96, "mxfp8", 128),
]


@pytest.mark.parametrize("fmt,K,w_fmt,w_K", WRONG_WIDTHS)
def test_grouped_mm_mx_refuses_weights_of_another_width(called, fmt, K, w_fmt, w_K):
    E, N = 2, 64
    x, xs = mx(8, K, fmt)
    off = on(E + 1, dtype=I32)
    w, ws = mx(N, K, fmt, (E,))
    out = on(8, N, dtype=BF16)
    ops.grouped_mm_mx(x, xs, w, ws, off, fmt, out=out)  # of the same width: goes through
    assert called == ["moe_grouped_mm_mx"]
    bad = mx(N, w_K, w_fmt, (E,))[0]
    assert bad.shape != w.shape
    with pytest.raises(ValueError, match="w_codes must have shape"):
        ops.grouped_mm_mx(x, xs, bad, ws, off, fmt, out=out)
    assert called == ["moe_grouped_mm_mx"]


@pytest.mark.parametrize("fmt,K,w_fmt,w_K", WRONG_WIDTHS)
def test_expert_rows_mx_refuses_weights_of_another_width(called, fmt, K, w_fmt, w_K):
    E, other = 2, 64  # K as H for w13, as I for w2
    off = on(E + 1, dtype=I32)
    bad = mx(2 * other, w_K, w_fmt, (E,))[0]
    for H, I in ((K, other), (other, K)):
        x, xs = mx(8, H, fmt)
        w13, w13s = mx(2 * I, H, fmt, (E,))
        w2, w2s = mx(H, I, fmt, (E,))
        y = on(8, H, dtype=BF16)
        called.clear()
        ops.expert_rows_mx(x, xs, off, w13, w13s, w2, w2s, None, fmt, y=y)
        assert called == ["moe_expert_rows_mx"]
        with pytest.raises(ValueError, match="must have shape"):
            if H == K:
                ops.expert_rows_mx(x, xs, off, bad, w13s, w2, w2s, None, fmt, y=y)
            else:
                ops.expert_rows_mx(x, xs, off, w13, w13s, bad[:, :H], w2s, None, fmt, y=y)
        assert called == ["moe_expert_rows_mx"]


@pytest.mark.parametrize("w_K", [1, 32, 96, 160, 256])
def test_grouped_mm_refuses_weights_of_another_width(called, w_K):
    x, off = on(8, 128, dtype=BF16), on(3, dtype=I32)
    ops.grouped_mm(x, on(2, 64, 128, dtype=BF16), off, out=on(8, 64, dtype=BF16))
    assert called == ["moe_grouped_mm"]
    with pytest.raises(ValueError, match="w must have shape"):
        ops.grouped_mm(x, on(2, 64, w_K, dtype=BF16), off, out=on(8, 64, dtype=BF16))
    assert called == ["moe_grouped_mm"]


STEPS = ("route", "permute", "mx_quantize", "expert_rows_mx", "dense_ffn", "combine_rows")


@pytest.fixture
def steps(monkeypatch):
    """(step, current device) of every step that forward_mx takes; device 0 is current
    outside of it."""
    taken, current = [], [0]

    class Device:  # torch.cuda.device
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()

    def step(name, result):
        def f(*a, **k):
            taken.append((name, current[-1]))
            return result
        monkeypatch.setattr(ops, name, f)
    monkeypatch.setattr(torch.cuda, "device", Device)
    step("route", (None, None))
    step("permute", dict(expert_offsets=None, row_of=None, tok_of=None, w_of=None))
    step("mx_quantize", (None, None))
    for name in STEPS[3:]:
        step(name, name)
    return taken


def block(dev, T=6, H=128, Is=64, E=8, I=32):
    cfg = ops.BlockConfig(T=T, H=H, E=E, I=I, I_shared=Is, top_k=2)
    return dict(x=on(T, H, dtype=BF16, dev=dev), Wr=on(E, H, dtype=F32, dev=dev),
                bias=on(E, dtype=F32, dev=dev), w13=(None, None), w2=(None, None),
                ws13=on(2 * Is, H, dtype=BF16, dev=dev), ws2=on(H, Is, dtype=BF16, dev=dev), cfg=cfg,
                fmt="mxfp8")


@pytest.mark.parametrize("dev", [0, 1])
def test_forward_mx_takes_every_step_on_its_tensors_device(steps, dev):
    assert ops.forward_mx(**block(dev)) == "combine_rows"
    assert steps == [(name, dev) for name in STEPS]


@pytest.mark.parametrize("name", ["Wr", "bias", "ws13", "ws2", "residual", "out", "token_mask"])
def test_forward_mx_refuses_tensors_of_two_devices(steps, name):
    a = block(1) | {"residual": on(6, 128, dtype=BF16, dev=1), "out": on(6, 128, dtype=BF16, dev=1),
                    "token_mask": on(6, dev=1)}
    assert ops.forward_mx(**a) == "combine_rows"
    steps.clear()
    a[name].on = 0
    with pytest.raises(ValueError, match=f"cuda:1, {name} is on"):
        ops.forward_mx(**a)
    with pytest.raises(TypeError, match=f"{name} must be a tensor"):
        ops.forward_mx(**a | {name: "x"})
    assert not steps


def test_forward_mx_without_a_shared_expert_does_not_look_at_its_weights(steps):
    a = block(0) | {"ws13": None, "ws2": on(1, dev=1)}
    a["cfg"].I_shared = 0
    assert ops.forward_mx(**a) == "combine_rows"
    assert "dense_ffn" not in [name for name, _ in steps]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,H", [(5, 128), (7, 128), (0, 128), (6, 64), (6, 160), (6, 256)])
def test_forward_mx_refuses_codes_of_other_tokens(steps, T, H, fmt):
    a = block(0) | {"fmt": fmt}
    good, bad = mx(6, 128, fmt), mx(T, H, fmt)
    assert ops.forward_mx(**a, x_mx=good) == "combine_rows"
    assert "mx_quantize" not in [name for name, _ in steps]
    steps.clear()
    for x_mx in (bad, (bad[0], good[1]), (good[0], bad[1])):
        if [t.shape for t in x_mx] != [t.shape for t in good]:
            with pytest.raises(ValueError, match="must have shape"):
                ops.forward_mx(**a, x_mx=x_mx)
    other = "mxfp4" if fmt == "mxfp8" else "mxfp8"
    with pytest.raises(ValueError, match="x_codes must have shape"):
        ops.forward_mx(**a, x_mx=mx(6, 128, other))
    with pytest.raises(ValueError, match="cuda:0"):
        ops.forward_mx(**a, x_mx=(on(*good[0].shape, dev=1), good[1]))
    assert not steps


def test_workspaces_that_are_not_whole_are_refused(called):
    E, N, K = 2, 64, 64
    x, off = on(8, K, dtype=BF16), on(E + 1, dtype=I32)
    c, s = mx(8, K, "mxfp8")
    w, ws = mx(N, K, "mxfp8", (E,))
    w13, w13s = mx(2 * N, K, "mxfp8", (E,))
    calls = (
        lambda k: ops.grouped_mm(x, on(E, N, K, dtype=BF16), off, out=on(8, N, dtype=BF16), workspace=k),
        lambda k: ops.grouped_mm_mx(c, s, w, ws, off, "mxfp8", out=on(8, N, dtype=BF16), workspace=k),
        lambda k: ops.expert_rows_mx(c, s, off, w13, w13s, w, ws, None, "mxfp8",
                                     y=on(8, K, dtype=BF16), workspace=k),
    )
    one = torch.zeros(1, dtype=U8).expand(1 << 16).as_subclass(On)  # 65,536 elements of one byte
    for i, call in enumerate(calls):
        call(on(1 << 16))
        assert len(called) == i + 1
        for bad in (one, on(1 << 16)[::2]):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                call(bad)
        with pytest.raises(ValueError, match="workspace must be on cuda:0"):
            call(on(1 << 16, dev=1))
        assert len(called) == i + 1
