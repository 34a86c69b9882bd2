"""The forms of the MX products (operands swapped, rows loaded from the tokens, pair
tiles) captured, replayed, on two streams, from two threads, with guarded outputs
and with operands written right before the call.  Each test asserts which forms its
sizes take, by the library's own rule, which the first test reads from the source."""

import os
import threading

import numpy as np
import pytest
import torch

from routed_moe_layer_b200 import build, inputs, ops
from tests.test_gpu_mx import FMTS, block, check_product, gen, groups, operands, run_layer
from tests.test_zz_write_guards import guarded

gpu = pytest.mark.gpu

DEV = "cuda"


# ------------------------------------------------------------------ which form a call takes
RULE = """
  if (epi == MX_SWIGLU) return rows <= 112 * groups;
  return rows <= (fmt == MOE_MXFP8 ? 192 : 128) * groups ||
         (rows / 128 + groups) * ((n + 127) / 128) <= num_sms();
"""


def up_form(R, E, gathered=True):
    if gathered and R <= 4 * E:
        return "tokens"
    return "swapped" if R <= 112 * E else "pair"


def rows_form(R, E, N, fmt):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few = R <= (192 if fmt == "mxfp8" else 128) * E or (R // 128 + E) * -(-N // 128) <= sms
    return "swapped" if few else "pair"


def test_the_forms_are_chosen_as_here():
    source = open(os.path.join(build.CSRC, "api.cu")).read()
    assert RULE in source
    assert "constexpr int64_t GATHER_ROWS_PER_EXPERT = 4;" in source
    assert "return R <= GATHER_ROWS_PER_EXPERT * (int64_t)E;" in source


# ------------------------------------------------------------------ the layer
@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,up,down", [(12, 512, "tokens", "swapped"), (96, 512, "swapped", "swapped"),
                                         (600, 512, "pair", "swapped"), (1024, 1024, "pair", "pair")])
def test_captured_replayed_and_on_two_streams(T, H, up, down, fmt):
    E, I, k = 16, 128, 4
    assert (up_form(T * k, E), rows_form(T * k, E, H, fmt)) == (up, down)
    cfg, d = block(T, H, E, I, 0, k, 6)
    w13, w2 = ops.mx_quantize(d["w13"], fmt), ops.mx_quantize(d["w2"], fmt)
    res = inputs.make_tokens(T, H, seed=3).to(DEV)
    gamma = torch.ones(H, device=DEV)
    layer = lambda: run_layer(d, cfg, w13, w2, res, gamma, fmt)
    want = [t.clone() for t in layer()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):  # two graphs of the same leaves, each with its own workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append([layer() for _ in range(3)])  # one call starts while another ends
        graphs.append(g)
    keep = d["x"].clone()
    for _ in range(3):
        d["x"].copy_(res)  # other inputs, then the first ones again: nothing is kept
        graphs[0].replay()
        assert not torch.equal(outs[0][0][4], want[4])
        d["x"].copy_(keep)
        for g, o in zip(graphs, outs):
            g.replay()
            for got in o:
                for a, b in zip(got, want):
                    assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(8):  # overlapping calls
        with torch.cuda.stream(streams[i % 2]):
            got.append(layer())
    torch.cuda.synchronize()
    for o in got:
        for a, b in zip(o, want):
            assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,N,K,form", [(60, 4, 96, 160, "swapped"), (1500, 5, 1312, 1056, "pair"),
                                          (3000, 3, 800, 96, "pair")])
def test_products_write_only_their_rows_and_leave_inputs(R, E, N, K, form, fmt):
    assert rows_form(R, E, N, fmt) == form
    xc, xs, x = operands(R, K, fmt, 1)
    wc, wsc, w = operands(N, K, fmt, 2, lead=E)
    off = groups(R, E, 3)
    offd = torch.from_numpy(off).to(DEV)
    before = [t.clone() for t in (xc, xs, wc, wsc, offd)]
    y, c_y = guarded((R, N), torch.bfloat16, DEV)
    ws, c_ws = guarded((256,), torch.uint8, DEV)
    ops.grouped_mm_mx(xc, xs, wc, wsc, offd, fmt, out=y, workspace=ws)
    assert ops.read_device_status(ws)[0] == 0
    check_product(y, x, w, off)
    c_y()
    c_ws()
    for a, b in zip((xc, xs, wc, wsc, offd), before):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,H,I,up,down", [(12, 4, 160, 96, "tokens", "swapped"), (60, 4, 160, 96, "swapped", "swapped"),
                                             (900, 4, 160, 96, "pair", "swapped"), (1000, 2, 2176, 160, "pair", "pair")])
def test_experts_write_only_their_rows_and_leave_inputs(R, E, H, I, up, down, fmt):
    assert (up_form(R, E), rows_form(R, E, H, fmt)) == (up, down)
    xc, xs, _ = operands(R, H, fmt, 1)
    w13 = operands(2 * I, H, fmt, 5, lead=E, scale=H ** -0.5)[:2]
    w2 = operands(H, I, fmt, 6, lead=E, scale=I ** -0.5)[:2]
    off = torch.from_numpy(groups(R, E, 3)).to(DEV)
    tok = torch.arange(R, dtype=torch.int32, device=DEV).flip(0).contiguous()
    leaves = (xc, xs, *w13, *w2, off, tok)
    before = [t.clone() for t in leaves]
    want = ops.expert_rows_mx(xc, xs, off, *w13, *w2, None, fmt, tok_of=tok)
    y, c_y = guarded((R, H), torch.bfloat16, DEV)
    n = ops.lib().moe_expert_rows_mx_workspace_bytes(R, H, E, I, ops.MX_FORMATS[fmt], 1)
    ws, c_ws = guarded((n,), torch.uint8, DEV)
    ops.expert_rows_mx(xc, xs, off, *w13, *w2, None, fmt, tok_of=tok, y=y, workspace=ws)
    assert ops.read_device_status(ws)[0] == 0
    assert torch.equal(y, want)
    c_y()
    c_ws()
    for a, b in zip(leaves, before):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ written right before
def routing(T, E, k, seed):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    order = np.argsort(ids, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=E))]).astype(np.int32)
    return [torch.from_numpy(a).to(DEV) for a in (off, (order // k).astype(np.int32), order.astype(np.int32))]


WRITTEN = [(4, "tokens", "swapped"), (40, "swapped", "swapped"), (460, "pair", "swapped"),
           (1100, "pair", "pair")]


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,up,down", WRITTEN)
def test_operands_copied_in_right_before_the_call(T, up, down, fmt):
    """The down product reads its weights, their scales and the offsets while the up
    product runs: they may have been written by the kernel before the call, on its stream,
    with other contents every time."""
    E, k, H, I = 8, 2, 2176, 192
    assert (up_form(T * k, E), rows_form(T * k, E, H, fmt)) == (up, down)
    sets, wants = [], []
    for seed in (1, 2, 3):
        x = torch.randn(T, H, generator=gen(seed)).bfloat16().to(DEV)
        w13 = (H ** -0.5 * torch.randn(E, 2 * I, H, generator=gen(seed + 10))).bfloat16().to(DEV)
        w2 = (I ** -0.5 * torch.randn(E, H, I, generator=gen(seed + 20))).bfloat16().to(DEV)
        sets.append([*ops.mx_quantize(x, fmt), *ops.mx_quantize(w13, fmt), *ops.mx_quantize(w2, fmt),
                     *routing(T, E, k, seed)])

    def call(x, xs, w13, w13s, w2, w2s, off, tok, dest):
        return ops.expert_rows_mx(x, xs, off, w13, w13s, w2, w2s, dest, fmt, tok_of=tok)
    for s in sets:
        torch.cuda.synchronize()
        wants.append(call(*s))
        torch.cuda.synchronize()
    assert not torch.equal(wants[0], wants[1])
    live = [t.clone() for t in sets[0]]
    for first in range(len(live)):  # each operand once as the last one written
        turn = list(range(first + 1, len(live))) + list(range(first + 1))
        got = []
        for i in range(6):
            for j in turn:
                live[j].copy_(sets[i % 3][j])
            got.append(call(*live))
        for i, y in enumerate(got):
            assert torch.equal(y, wants[i % 3])
    # the same, captured
    src = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for a, b in zip(live, src):
            a.copy_(b)
        y = call(*live)
    for i in range(6):
        for a, b in zip(src, sets[i % 3]):
            a.copy_(b)
        g.replay()
        assert torch.equal(y, wants[i % 3])


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,up,down", WRITTEN)
def test_weights_quantised_right_before_the_call(T, up, down, fmt):
    """The quantisation lets the kernel after it start at once; its outputs lie where the
    last ones did."""
    E, k, H, I = 8, 2, 2176, 192
    assert (up_form(T * k, E), rows_form(T * k, E, H, fmt)) == (up, down)
    xc, xs = ops.mx_quantize(torch.randn(T, H, generator=gen(1)).bfloat16().to(DEV), fmt)
    w13 = ops.mx_quantize((H ** -0.5 * torch.randn(E, 2 * I, H, generator=gen(2))).bfloat16().to(DEV), fmt)
    wide = [(I ** -0.5 * torch.randn(E, H, I, generator=gen(3 + i))).bfloat16().to(DEV) for i in range(3)]
    off, tok, dest = routing(T, E, k, 4)

    def call(w):
        w2 = ops.mx_quantize(w, fmt)
        return ops.expert_rows_mx(xc, xs, off, *w13, *w2, dest, fmt, tok_of=tok), w2[0].data_ptr()
    wants = []
    for w in wide:
        w2 = ops.mx_quantize(w, fmt)
        torch.cuda.synchronize()
        wants.append(ops.expert_rows_mx(xc, xs, off, *w13, *w2, dest, fmt, tok_of=tok))
        torch.cuda.synchronize()
    del w2
    got = [call(wide[i % 3]) for i in range(30)]
    assert len({at for _, at in got}) < 30  # memory used again
    for i, (y, _) in enumerate(got):
        assert torch.equal(y, wants[i % 3])


@gpu
@pytest.mark.parametrize("T,up,down", WRITTEN)
def test_two_threads_on_one_stream(T, up, down):
    """Two host threads whose calls' kernels interleave on one stream."""
    E, k, H, I, fmt = 8, 2, 2176, 192, "mxfp8"
    assert (up_form(T * k, E), rows_form(T * k, E, H, fmt)) == (up, down)
    jobs = []
    for seed in (1, 2):
        x = ops.mx_quantize(torch.randn(T, H, generator=gen(seed)).bfloat16().to(DEV), fmt)
        w13 = ops.mx_quantize((H ** -0.5 * torch.randn(E, 2 * I, H, generator=gen(seed + 2))).bfloat16().to(DEV), fmt)
        w2 = ops.mx_quantize((I ** -0.5 * torch.randn(E, H, I, generator=gen(seed + 4))).bfloat16().to(DEV), fmt)
        off, tok, dest = routing(T, E, k, seed)
        jobs.append(lambda x=x, w13=w13, w2=w2, off=off, tok=tok, dest=dest: ops.expert_rows_mx(
            *x, off, *w13, *w2, dest, fmt, tok_of=tok))
    wants = [job() for job in jobs]
    torch.cuda.synchronize()
    stream, got, start = torch.cuda.Stream(), [[], []], threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(60):
                got[i].append(jobs[i]())
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 60
        for y in got[i]:
            assert torch.equal(y, wants[i])


# ------------------------------------------------------------------ side by side in memory
@gpu
def test_outputs_may_lie_beside_what_is_read_but_not_over_it():
    T, H, K, N, E = 6, 128, 64, 64, 2
    g = gen(1)
    buf = torch.empty(3 * T + 1, H, dtype=torch.bfloat16, device=DEV)
    x, r = buf[:T], buf[T:2 * T]
    x.copy_(torch.randn(T, H, generator=g).bfloat16())
    r.copy_(torch.randn(T, H, generator=g).bfloat16())
    keep = buf[:2 * T].clone()
    want = ops.add_rmsnorm(x.clone(), r.clone(), fmt="mxfp8")
    got = ops.add_rmsnorm(x, r, fmt="mxfp8", sum_out=buf[2 * T:3 * T])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(buf[:2 * T], keep)
    for bad in (buf[1:T + 1], buf[T - 1:2 * T - 1], buf[2 * T - 1:3 * T - 1]):
        with pytest.raises(RuntimeError, match="INVALID_ARG"):
            ops.add_rmsnorm(x, r, fmt="mxfp8", sum_out=bad)
    assert torch.equal(buf[:2 * T], keep)
    rows = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    w = torch.randn(E, N, K, generator=g).bfloat16().to(DEV)
    off = torch.tensor([0, 2, T], dtype=torch.int32, device=DEV)
    both = torch.empty(2 * T, K, dtype=torch.bfloat16, device=DEV)
    both[:T].copy_(rows)
    assert torch.equal(ops.grouped_mm(both[:T], w, off, out=both[T:]), ops.grouped_mm(rows, w, off))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        ops.grouped_mm(both[:T], w, off, out=both[T - 1:2 * T - 1])
    assert torch.equal(both[:T], rows)


# ------------------------------------------------------------------ bad indices
INDEXED = [(12, 4, 160, 96, "tokens", "swapped"), (60, 4, 160, 96, "swapped", "swapped"),
           (900, 4, 160, 96, "pair", "swapped"), (1000, 2, 2176, 160, "pair", "pair")]


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,H,I,up,down", INDEXED)
def test_experts_with_bad_offsets_report_them_and_stay_inside(R, E, H, I, up, down, fmt):
    assert (up_form(R, E), rows_form(R, E, H, fmt)) == (up, down)
    xc, xs, _ = operands(R, H, fmt, 1)
    w13 = operands(2 * I, H, fmt, 5, lead=E, scale=H ** -0.5)[:2]
    w2 = operands(H, I, fmt, 6, lead=E, scale=I ** -0.5)[:2]
    tok = torch.arange(R, dtype=torch.int32, device=DEV).flip(0).contiguous()
    y, check = guarded((R, H), torch.bfloat16, DEV)
    n = ops.lib().moe_expert_rows_mx_workspace_bytes(R, H, E, I, ops.MX_FORMATS[fmt], 1)
    ws, c_ws = guarded((n,), torch.uint8, DEV)

    def call(off):
        ops.expert_rows_mx(xc, xs, torch.tensor(off, dtype=torch.int32, device=DEV), *w13, *w2, None,
                           fmt, tok_of=tok, y=y, workspace=ws)
        return ops.read_device_status(ws)[0]
    even = [R * e // E for e in range(E + 1)]
    assert call(even) == 0
    want = y.clone()
    for bad in (even[:-1] + [R + 50], [-5] + even[1:], [even[0], R, *even[2:]] if E > 2 else [R, 0, R],
                [2 ** 30, 2 ** 31 - 1] + [5] * (E - 1), [-2 ** 31] * (E + 1)):
        assert call(bad) == 6
        check()
        c_ws()
    assert call(even) == 0  # cleared by the next call
    assert torch.equal(y, want)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,E,H,I,up,down", INDEXED)
def test_experts_tokens_and_destinations_outside(R, E, H, I, up, down, fmt):
    """A token outside counts as zeros, a row whose destination lies outside is not stored; the
    other rows have the bits of the call without them."""
    assert (up_form(R, E), rows_form(R, E, H, fmt)) == (up, down)
    T = R // 2
    xc, xs, _ = operands(T, H, fmt, 1)
    w13 = operands(2 * I, H, fmt, 5, lead=E, scale=H ** -0.5)[:2]
    w2 = operands(H, I, fmt, 6, lead=E, scale=I ** -0.5)[:2]
    off = torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32, device=DEV)
    tok = torch.randint(0, T, (R,), generator=gen(2)).int()
    want = ops.expert_rows_mx(xc, xs, off, *w13, *w2, None, fmt, tok_of=tok.to(DEV))
    none = torch.zeros(R, dtype=torch.bool)
    for at, t in ((0, -1), (R // 3, T), (R // 2, 2 ** 31 - 1), (R - 1, -2 ** 31)):
        tok[at], none[at] = t, True
    dest = torch.randperm(R, generator=gen(3)).int()
    lost = torch.zeros(R, dtype=torch.bool)
    free = []
    for at, to in ((1, -1), (R // 3 + 1, R), (R // 2 + 1, 2 ** 31 - 1), (R - 2, -2 ** 31)):
        free.append(int(dest[at]))
        dest[at], lost[at] = to, True
    y, check = guarded((R, H), torch.bfloat16, DEV)
    y.fill_(7.0)
    ops.expert_rows_mx(xc, xs, off, *w13, *w2, dest.to(DEV), fmt, tok_of=tok.to(DEV), y=y)
    check()
    kept = ~lost
    got = y[dest[kept].long().to(DEV)]
    zero = none[kept].to(DEV)
    assert (got[zero] == 0).all()
    assert torch.equal(got[~zero], want[kept.to(DEV)][~zero])
    assert (y[torch.tensor(free, device=DEV)] == 7).all()
