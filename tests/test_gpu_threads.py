"""Every entry point as the first CUDA call of a new host thread: a thread has no
current context until a call makes one so, and the outputs and workspaces are
allocated (and torch's caching allocator filled) by another thread."""

import threading

import pytest
import torch

from routed_moe_layer_b200 import inputs, ops
from routed_moe_layer_b200.ops import BlockConfig
from tests.test_gpu_mx import FMTS, gen

pytestmark = pytest.mark.gpu

DEV = "cuda"


def in_a_new_thread(call):
    out, err = [], []

    def work():
        try:
            out.append(call())
        except BaseException as e:  # shown by the test's own thread
            err.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if err:
        raise err[0]
    return out[0]


def check(call):
    """The bits of the same call made here."""
    want = call()
    torch.cuda.synchronize()
    got = in_a_new_thread(call)
    torch.cuda.synchronize()
    want, got = ((v if isinstance(v, tuple) else (v,)) for v in (want, got))
    assert len(want) == len(got)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 40, 2500])
def test_block_and_its_parts(T):
    cfg = BlockConfig(T=T, H=256, E=16, I=128, I_shared=128, top_k=4, n_group=4, topk_group=2)
    d = {n: v.to(DEV) for n, v in inputs.make_block_inputs(T, 256, seed=1, E=16, I=128, I_shared=128,
                                                           unit_scale=True).items()}
    x, Wr, bias = d["x"], d["Wr"], d["bias"]
    ws = ops.alloc_workspace(ops.workspace_bytes(cfg), DEV)
    args = (x, Wr, bias, d["w13"], d["w2"], d["ws13"], d["ws2"], cfg)
    check(lambda: ops.forward(*args, out=torch.empty_like(x), workspace=ws))
    check(lambda: ops.route(x, Wr, bias, cfg))
    check(lambda: ops.dense_ffn(x, d["ws13"], d["ws2"]))
    check(lambda: ops.rmsnorm(x))
    ids, w = ops.route(x, Wr, bias, cfg)
    p = ops.permute(ids, cfg, topk_w=w, x=x)
    check(lambda: tuple(ops.permute(ids, cfg, topk_w=w, x=x)[n] for n in ("expert_offsets", "row_of", "xp")))
    dest = torch.arange(T * 4, dtype=torch.int32, device=DEV)
    check(lambda: ops.expert_rows(p["xp"], p["expert_offsets"], d["w13"], d["w2"], dest, row_w=p["w_of"]))
    check(lambda: ops.grouped_mm(p["xp"], d["w13"], p["expert_offsets"]))
    y = ops.expert_rows(p["xp"], p["expert_offsets"], d["w13"], d["w2"], dest, row_w=p["w_of"])
    check(lambda: ops.combine_rows(y, p["row_of"], 4))
    q = {n: None if v is None else v.to(DEV) for n, v in
         inputs.make_fp8_weights(256, 1, E=16, I=128, I_shared=128).items()}
    check(lambda: ops.forward_fp8(x, Wr, bias, q, cfg, out=torch.empty_like(x), workspace=ws))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 40, 2500])  # rows from the tokens, swapped, pair tiles
def test_narrow_operators(T, fmt):
    H, E, I, k = 512, 8, 128, 2
    x = torch.randn(T, H, generator=gen(1)).bfloat16().to(DEV)
    c, s = ops.mx_quantize(x, fmt)
    w13 = ops.mx_quantize(torch.randn(E, 2 * I, H, generator=gen(2)).bfloat16().to(DEV), fmt)
    w2 = ops.mx_quantize(torch.randn(E, H, I, generator=gen(3)).bfloat16().to(DEV), fmt)
    R = T * k
    off = torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32, device=DEV)
    tok = torch.arange(T, dtype=torch.int32, device=DEV).repeat(k)
    rows = ops.mx_quantize(x.repeat(k, 1), fmt)
    y = torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
    ws = ops.alloc_workspace(1 << 24, DEV)
    check(lambda: ops.expert_rows_mx(c, s, off, *w13, *w2, None, fmt, tok_of=tok, y=y, workspace=ws).clone())
    check(lambda: ops.grouped_mm_mx(*rows, *w13, off, fmt, workspace=ws))
    check(lambda: ops.mx_quantize(x, fmt))
    check(lambda: ops.mx_dequantize(c, s, fmt))
    check(lambda: ops.add_rmsnorm(x, x, fmt=fmt))
