"""What is measured of the narrow-format operators: inputs, plain forms and exact values.

The operators are add_rmsnorm, mx_quantize / mx_dequantize, grouped_mm, grouped_mm_mx and
expert_rows_mx of ``routed_moe_layer_b200.ops``.  ``run`` computes them in their plain form,
elementary torch operations in 32 bits, or, where ``own`` is true, by the library's kernels.

Formats ("mxfp8": E4M3 elements, "mxfp4": E2M1 elements, two to a byte, the even element in the
low nibble): every 32 consecutive elements of a row share one power of two 2^(s - 127).  Codes are
uint8 [rows, K] or [rows, K / 2]; scales uint8 [ceil(K / 128), rows, 4], the byte of block b of
row r at [b // 4, r, b % 4]; bytes of blocks past K are 0.  A stack of matrices has one more
leading dimension in both.
"""

import math

import torch

own = False

TOP = {"mxfp8": 448.0, "mxfp4": 6.0}  # largest element of each format
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm before the experts of one decoded token: latency
        {"name": "norm_1x2048", "op": "norm", "T": 1, "H": 2048, "fmt": "mxfp8"},
        # the same in the largest prefill batch (video and text tokens of one request)
        {"name": "norm_19412x2048", "op": "norm", "T": 19412, "H": 2048, "fmt": "mxfp8"},
        # activations of a small batch to four bits and back: what the format costs in accuracy
        {"name": "round_trip_240x1024", "op": "round_trip", "rows": 240, "K": 1024, "fmt": "mxfp4"},
        # the stacked gate and up weights of 16 experts to eight bits, as when a model is loaded
        {"name": "quantize_24576x2048", "op": "quantize", "rows": 24576, "K": 2048, "fmt": "mxfp8"},
        # one projection of the routed rows in bf16: a single token, then the largest batch
        {"name": "grouped_1", "op": "grouped", "T": 1, "K": 1024, "N": 1536, "E": 128, "k": 8},
        {"name": "grouped_19412", "op": "grouped", "T": 19412, "K": 768, "N": 2048, "E": 128, "k": 8},
        # the same projection with both operands narrow: few rows an expert, the largest batch
        {"name": "grouped_mx8_240", "op": "grouped_mx", "T": 240, "K": 1024, "N": 1536, "E": 128,
         "k": 8, "fmt": "mxfp8"},
        {"name": "grouped_mx4_19412", "op": "grouped_mx", "T": 19412, "K": 2048, "N": 1536, "E": 128,
         "k": 8, "fmt": "mxfp4"},
        # the routed experts from gathered narrow tokens: decode, a short clip, the largest batch
        {"name": "experts_mx8_1", "op": "experts", "T": 1, "H": 2048, "I": 768, "E": 128, "k": 8,
         "fmt": "mxfp8"},
        {"name": "experts_mx4_784", "op": "experts", "T": 784, "H": 2048, "I": 768, "E": 128, "k": 8,
         "fmt": "mxfp4"},
        {"name": "experts_mx8_19412", "op": "experts", "T": 19412, "H": 2048, "I": 768, "E": 128,
         "k": 8, "fmt": "mxfp8"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "round_trip", "quantize", "grouped", "grouped_mx", "experts"])
    fmt = rng.choice(["mxfp8", "mxfp4"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 19412), "H": 64 * rng.randint(4, 32), "fmt": "mxfp8"}
    if op in ("round_trip", "quantize"):
        fmt = "mxfp8" if op == "quantize" else fmt
        return {"op": op, "rows": _log(rng, 1, 24576), "K": 32 * rng.randint(4, 64), "fmt": fmt}
    E = rng.choice([8, 16, 32, 64, 128])
    case = {"op": op, "T": _log(rng, 1, 19412), "E": E, "k": rng.randint(1, 8)}
    if op == "experts":
        case |= {"H": 64 * rng.randint(4, 32), "I": 32 * rng.randint(4, 24)}
    else:
        case |= {"K": 32 * rng.randint(4, 64), "N": 32 * rng.randint(4, 48)}
    return case if op == "grouped" else case | {"fmt": fmt}


# ------------------------------------------------------------------ inputs
def _routing(T, E, k, g, device):
    """A batch's tokens on their experts, some of them more popular: the rows sorted by expert,
    each with its token, its slot and its weight, and the most rows that one expert has."""
    scores = torch.randn(T, E, generator=g, device=device) + 0.3 * torch.randn(E, generator=g, device=device)
    ids = scores.topk(k, dim=1).indices.reshape(-1)
    dest = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=device)
    offsets[1:] = counts.cumsum(0)
    w = torch.rand(T, k, generator=g, device=device) + 0.1
    w = 2.5 * w / w.sum(1, keepdim=True)
    return {"offsets": offsets, "tok_of": (dest // k).int(), "row_dest": dest.int(),
            "row_w": w.reshape(-1)[dest].contiguous(), "most": int(counts.max())}


def _weights(E, N, K, fmt, g, device):
    """The experts' matrices as they are kept: narrow codes and scales, made one expert at a time."""
    codes, scales = [], []
    for _ in range(E):
        c, s = _quantize(0.02 * torch.randn(N, K, generator=g, device=device), fmt)
        codes.append(c)
        scales.append(s)
    return torch.stack(codes), torch.stack(scales)


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    state = dict(case)
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        state |= {"x": normal(T, H).bfloat16(), "residual": (3.0 * normal(T, H)).bfloat16(),
                  "gamma": 1.0 + 0.2 * normal(H)}
    elif op in ("round_trip", "quantize"):
        # rows of different sizes, as activations and weights have
        x = normal(case["rows"], case["K"]) * torch.exp(normal(case["rows"], 1))
        state["x"] = x.bfloat16()
    elif op == "grouped":
        T, K, N, E, k = (case[n] for n in ("T", "K", "N", "E", "k"))
        state |= _routing(T, E, k, g, device)
        state["x"] = normal(T * k, K).bfloat16()
        state["w"] = torch.stack([(0.02 * normal(N, K)).bfloat16() for _ in range(E)])
    elif op == "grouped_mx":
        T, K, N, E, k = (case[n] for n in ("T", "K", "N", "E", "k"))
        state |= _routing(T, E, k, g, device)
        state["x"], state["xs"] = _quantize(normal(T * k, K), case["fmt"])
        state["w"], state["ws"] = _weights(E, N, K, case["fmt"], g, device)
    else:
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        state |= _routing(T, E, k, g, device)
        state["x"], state["xs"] = _quantize(normal(T, H), case["fmt"])
        state["w13"], state["w13s"] = _weights(E, 2 * I, H, case["fmt"], g, device)
        state["w2"], state["w2s"] = _weights(E, H, I, case["fmt"], g, device)
    return state


# ------------------------------------------------------------------ plain forms
def _values4(device):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _quantize(x, fmt):
    """codes, scales of x [rows, K]: the smallest power of two under which no element passes the
    format's largest, elements rounded to nearest, ties to the even code."""
    rows, K = x.shape
    b = x.float().reshape(rows, K // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9, 6 = 3/4 2^3
    p = e - 9 + (m > 0.875).int() if fmt == "mxfp8" else e - 3 + (m > 0.75).int()
    p = torch.where(m == 0, -127, p).clamp(-127, 127)
    v = (b.double() * torch.exp2(-p.double()).unsqueeze(2)).float()  # exact: a power of two
    if fmt == "mxfp8":
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, K)
    else:
        a = v.abs()
        n = (a > .25).byte() + (a >= .75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() \
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte() + 8 * torch.signbit(v).byte()
        n = n.reshape(rows, K // 2, 2)
        codes = n[..., 0] + 16 * n[..., 1]
    words = -(-K // 128)
    scales = torch.zeros(rows, words * 4, dtype=torch.uint8, device=x.device)
    scales[:, :K // 32] = (p + 127).byte()
    return codes, scales.reshape(rows, words, 4).transpose(0, 1).contiguous()


def _values(codes, scales, fmt):
    """The fp32 values of codes [..., rows, K] and scales [..., words, rows, 4]."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = _values4(codes.device)
        v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    K = v.shape[-1]
    s = scales.transpose(-3, -2).flatten(-2)[..., :K // 32].contiguous()
    s = s.view(torch.float8_e8m0fnu).float()
    return (v.unflatten(-1, (K // 32, 32)) * s.unsqueeze(-1)).flatten(-2)


def _rows_by_expert(offsets, rows):
    """The expert of every row and its place among that expert's rows."""
    at = torch.arange(rows, device=offsets.device)
    expert = torch.searchsorted(offsets[1:].long(), at, right=True)
    return expert, at - offsets.long()[expert]


def _grouped(x, w, offsets, most):
    """fp32 x_r . W_e^T: the rows of every expert in a padded batch, one batched product."""
    expert, place = _rows_by_expert(offsets, x.shape[0])
    batch = torch.zeros(w.shape[0], most, x.shape[1], device=x.device)
    batch[expert, place] = x
    return torch.bmm(batch, w.transpose(1, 2))[expert, place]


def _run_plain(s):
    op, fmt = s["op"], s.get("fmt")
    if op == "norm":
        total = (s["x"].float() + s["residual"].float()).bfloat16()
        t = total.float()
        xn = (t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["gamma"]).bfloat16()
        return {"sum": total, "xn": xn, **_told(*_quantize(xn, fmt))}
    if op == "quantize":
        return _told(*_quantize(s["x"], fmt))
    if op == "round_trip":
        return _values(*_quantize(s["x"], fmt), fmt).bfloat16()
    if op == "grouped":
        return _grouped(s["x"].float(), s["w"].float(), s["offsets"], s["most"]).bfloat16()
    if op == "grouped_mx":
        x, w = _values(s["x"], s["xs"], fmt), _values(s["w"], s["ws"], fmt)
        return _grouped(x, w, s["offsets"], s["most"]).bfloat16()
    I = s["I"]
    x = _values(s["x"], s["xs"], fmt)[s["tok_of"].long()]
    gu = _grouped(x, _values(s["w13"], s["w13s"], fmt), s["offsets"], s["most"])
    gate, up = gu[:, :I], gu[:, I:]
    h = _values(*_quantize(gate / (1 + torch.exp(-gate)) * up, fmt), fmt)
    y = s["row_w"].unsqueeze(1) * _grouped(h, _values(s["w2"], s["w2s"], fmt), s["offsets"], s["most"])
    out = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)
    out[s["row_dest"].long()] = y.bfloat16()
    return out


def _told(codes, scales):
    """Eight-bit codes and scales as the values they stand for (the same bytes)."""
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        return _run_plain(state)
    from routed_moe_layer_b200 import ops

    s, op, fmt = state, state["op"], state.get("fmt")
    if op == "norm":
        total, xn, codes, scales = ops.add_rmsnorm(s["x"], s["residual"], s["gamma"], eps=EPS, fmt=fmt)
        return {"sum": total, "xn": xn, **_told(codes, scales)}
    if op == "quantize":
        return _told(*ops.mx_quantize(s["x"], fmt))
    if op == "round_trip":
        return ops.mx_dequantize(*ops.mx_quantize(s["x"], fmt), fmt)
    if op == "grouped":
        return ops.grouped_mm(s["x"], s["w"], s["offsets"])
    if op == "grouped_mx":
        return ops.grouped_mm_mx(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], fmt)
    return ops.expert_rows_mx(s["x"], s["xs"], s["offsets"], s["w13"], s["w13s"], s["w2"], s["w2s"],
                              s["row_dest"], fmt, row_w=s["row_w"], tok_of=s["tok_of"])


def _narrow(fmt):
    """Bytes of one element with its share of the scale."""
    return (1 if fmt == "mxfp8" else 0.5) + 1 / 32


def work(case):
    op, fmt = case["op"], case.get("fmt")
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": n * (8 + _narrow(fmt)) + 4 * case["H"], "flops": 8 * n}
    if op in ("round_trip", "quantize"):
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 + _narrow(fmt)) if op == "quantize" else 4 * n, "flops": 4 * n}
    T, E, k = case["T"], case["E"], case["k"]
    R = T * k
    used = E * (1 - (1 - k / E) ** T)  # experts that hold a row, on the average
    if op == "experts":
        H, I = case["H"], case["I"]
        per = _narrow(fmt)
        return {"bytes": used * 3 * H * I * per + T * H * per + 2 * R * H + 12 * R, "flops": 6 * R * H * I}
    K, N = case["K"], case["N"]
    per = 2 if op == "grouped" else _narrow(fmt)
    return {"bytes": (used * N + R) * K * per + 2 * R * N, "flops": 2 * R * K * N}


# ------------------------------------------------------------------ exact values, in 64 bits
def _grid(fmt):
    """The nonnegative elements of a format, in the order of their codes."""
    if fmt == "mxfp4":
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    values = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    return torch.tensor(values[:-1], dtype=torch.float64, device="cuda")  # the last one is NaN


def _powers(blocks, fmt):
    """log2 of each block's shared power of two, from its largest element [..., 32]."""
    top, biggest = TOP[fmt], blocks.abs().amax(-1)
    p = torch.ceil(torch.log2(biggest.clamp_min(1e-300) / top))
    p = torch.where(top * torch.exp2(p) < biggest, p + 1, p)
    p = torch.where(top * torch.exp2(p - 1) >= biggest, p - 1, p)
    return p.clamp(-127, 127)


def _rounded(x, fmt):
    """(elements, powers) of x [rows, K]: the elements on the format's grid, not multiplied."""
    grid = _grid(fmt)
    blocks = x.unflatten(-1, (-1, 32))
    p = _powers(blocks, fmt)
    v = blocks / torch.exp2(p).unsqueeze(-1)
    hi = torch.searchsorted(grid, v.abs()).clamp(1, grid.numel() - 1)
    down, up = v.abs() - grid[hi - 1], grid[hi] - v.abs()
    pick = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)
    return torch.copysign(grid[pick], v).flatten(-2), p


def _product(x, w, bounds):
    """Rows of each expert times its matrix, expert by expert; w(e) is expert e's matrix."""
    parts = [x[lo:hi] @ w(e).T for e, (lo, hi) in enumerate(zip(bounds, bounds[1:]))]
    return torch.cat(parts)


def _wide(codes, scales, fmt):
    """64-bit values of codes [rows, K], element by element from the format's definition."""
    grid = _grid(fmt)
    if fmt == "mxfp8":
        n, sign = (codes & 127).long(), codes >= 128
    else:
        n = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.long, device=codes.device)
        n[:, 0::2], n[:, 1::2] = (codes % 16).long(), (codes // 16).long()
        n, sign = n % 8, n >= 8
    v = torch.where(sign, -grid[n], grid[n])
    s = torch.exp2(scales.double() - 127).permute(1, 0, 2).reshape(v.shape[0], -1)
    return v * s.repeat_interleave(32, dim=1)[:, :v.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case.get("fmt")
    if op == "norm":
        t = (s["x"].double() + s["residual"].double()).bfloat16().double()
        xn = t / torch.sqrt((t * t).sum(1, keepdim=True) / t.shape[1] + EPS) * s["gamma"].double()
        p = _powers(xn.bfloat16().double().unflatten(-1, (-1, 32)), fmt)
        # the elements before their rounding; the scales are a choice, not a value
        return {"sum": s["x"].double() + s["residual"].double(), "xn": xn,
                "codes": xn / torch.exp2(p).repeat_interleave(32, dim=1), "scales": None}
    if op == "quantize":
        v, p = _rounded(s["x"].double(), fmt)
        words = -(-p.shape[1] // 4)
        scales = torch.full((p.shape[0], words * 4), -127.0, dtype=torch.float64, device=p.device)
        scales[:, :p.shape[1]] = p
        return {"codes": v, "scales": torch.exp2(scales).reshape(-1, words, 4).transpose(0, 1)}
    if op == "round_trip":
        v, p = _rounded(s["x"].double(), fmt)
        return v * torch.exp2(p).repeat_interleave(32, dim=1)
    bounds = s["offsets"].tolist()
    if op == "grouped":
        return _product(s["x"].double(), lambda e: s["w"][e].double(), bounds)
    if op == "grouped_mx":
        return _product(_wide(s["x"], s["xs"], fmt), lambda e: _wide(s["w"][e], s["ws"][e], fmt), bounds)
    I, x = case["I"], _wide(s["x"], s["xs"], fmt)[s["tok_of"].long()]
    gu = _product(x, lambda e: _wide(s["w13"][e], s["w13s"][e], fmt), bounds)
    h, p = _rounded(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:], fmt)
    h = h * torch.exp2(p).repeat_interleave(32, dim=1)
    y = _product(h, lambda e: _wide(s["w2"][e], s["w2s"][e], fmt), bounds) * s["row_w"].double().unsqueeze(1)
    out = torch.empty_like(y)
    out[s["row_dest"].long()] = y
    return out
