"""Expert products and 4-bit microscaled products, case by case.

Two operators that stand beside the layer's own kernels:

* matrix products grouped by expert with ragged sizes, for experts that are not quantised:
  with rows sorted by expert and `offsets` their E + 1 borders,
      forward  y[r]    = w[e] x[r]           for offsets[e] <= r < offsets[e + 1]
      dgrad    dx[r]   = w[e]^T dy[r]
      wgrad    dw[e]   = sum over the rows r of e of dy[r] x[r]^T
* microscaled 4-bit floating point (MXFP4: E2M1 values, one power of two per 32; NVFP4: E2M1
  values, one E4M3 scale per 16 and one FP32 scale per tensor): the quantiser, its inverse and
  the product of two quantised operands.

Sizes: hidden 5120, 256 experts, 8 of them for a token, expert sizes 1536 and 2560, and the
small layer of the tests (hidden 256, 16 experts, inner size 128); token counts 1, 8, 1024 and
16384 are one sequence's decoding step, its step with 7 drafted tokens, 128 sequences of 8 and
a prefill of 8 x 2048.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
ALPHA_X = 2.0 ** -9  # tensor scale of N(0, 1) activations: about their largest value / 2688


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one small layer's step: 4 tokens x 2 experts; the call's own latency
        dict(name="grouped_fwd_tiny", op="fwd", rows=8, groups=16, n=256, k=256, skew=0.0, type="bf16", out="bf16"),
        # decoding with 7 drafted tokens: 64 rows over 256 experts, bound by reading their weights
        dict(name="grouped_fwd_decode8", op="fwd", rows=64, groups=256, n=1536, k=5120, skew=0.0, type="bf16",
             out="bf16"),
        # 128 sequences x 8 tokens, down projection
        dict(name="grouped_fwd_spec1024", op="fwd", rows=8192, groups=256, n=5120, k=1536, skew=0.0, type="fp16",
             out="fp16"),
        # 8 x 2048 tokens, gate and up projections of inner size 2560 in one product
        dict(name="grouped_fwd_prefill16k", op="fwd", rows=131072, groups=256, n=5120, k=5120, skew=0.0,
             type="bf16", out="bf16"),
        # a training step's gradients on one of four expert-parallel ranks, uneven experts
        dict(name="grouped_dgrad_rank", op="dgrad", rows=32768, groups=64, n=1536, k=5120, skew=0.5, type="bf16",
             out="bf16"),
        dict(name="grouped_wgrad_rank", op="wgrad", rows=32768, groups=64, n=1536, k=5120, skew=0.5, type="bf16",
             out="bf16"),
        # odd sizes, some experts without rows, FP32 gradients
        dict(name="grouped_wgrad_odd", op="wgrad", rows=3001, groups=48, n=520, k=1000, skew=1.0, type="fp16",
             out="fp32"),
        # a decoding step's activations, there and back
        dict(name="fp4_values_decode8", op="values", rows=8, k=5120, format="mxfp4", type="bf16"),
        # a prefill's activations, there and back (what a calibration looks at)
        dict(name="fp4_values_prefill16k", op="values", rows=16384, k=5120, format="nvfp4", type="bf16"),
        # one projection hidden -> hidden: quantise the activations, multiply by 4-bit weights
        dict(name="fp4_linear_decode1", op="linear", rows=1, n=5120, k=5120, format="mxfp4", type="bf16"),
        dict(name="fp4_linear_odd", op="linear", rows=1031, n=2044, k=1568, format="nvfp4", type="fp16"),
        dict(name="fp4_linear_prefill16k", op="linear", rows=16384, n=5120, k=5120, format="mxfp4", type="bf16"),
    ]


def _log(rng, low, high, multiple=1):
    return max(1, round(math.exp(rng.uniform(math.log(low), math.log(high))) / multiple)) * multiple


def draw(rng):
    op = rng.choice(["fwd", "fwd", "dgrad", "wgrad", "values", "linear", "linear"])
    kind = rng.choice(["bf16", "fp16"])
    if op == "values":
        return dict(op=op, rows=_log(rng, 1, 16384), k=_log(rng, 64, 5120, 32), format=rng.choice(list(BLOCK)),
                    type=kind)
    if op == "linear":
        return dict(op=op, rows=_log(rng, 1, 16384), n=_log(rng, 64, 5120), k=_log(rng, 64, 5120, 32),
                    format=rng.choice(list(BLOCK)), type=kind)
    return dict(op=op, rows=_log(rng, 1, 32768), groups=_log(rng, 1, 128), n=_log(rng, 64, 2560, 8),
                k=_log(rng, 64, 5120, 8), skew=rng.choice([0.0, 0.5, 1.0]), type=kind, out=kind)


def work(case):
    rows, k = case["rows"], case["k"]
    if case["op"] == "values":
        return {"bytes": 4 * rows * k, "flops": 0}
    n = case["n"]
    flops = 2 * rows * n * k
    if case["op"] == "linear":
        weight = n * k * (0.5 + 1.0 / BLOCK[case["format"]])
        return {"bytes": int(2 * rows * k + weight + 2 * rows * n), "flops": flops}
    groups, size = case["groups"], torch.empty(0, dtype=TYPES[case["out"]]).element_size()
    # the experts that some row goes to, on average: only their weights are read
    used = sum(1.0 - (1.0 - p) ** rows for p in _shares(case))
    moved = {"fwd": 2 * rows * k + 2 * used * n * k + size * rows * n,
             "dgrad": 2 * rows * n + 2 * used * n * k + size * rows * k,
             "wgrad": 2 * rows * n + 2 * rows * k + size * groups * n * k}[case["op"]]
    return {"bytes": int(moved) + 4 * (groups + 1), "flops": flops}


def _shares(case):
    p = [(e + 1.0) ** -case["skew"] for e in range(case["groups"])]
    return [v / sum(p) for v in p]


# ------------------------------------------------------------------------------ inputs
def _normal(gen, shape, std, kind):
    out = torch.empty(shape, dtype=kind, device="cuda")
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 28) // shape[-1])
    for i in range(0, flat.shape[0], step):  # in pieces: the FP32 draws of a large tensor take twice its memory
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(std))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = TYPES[case["type"]]
    rows, k = case["rows"], case["k"]
    state = {"case": dict(case)}
    if case["op"] in ("values", "linear"):
        x = _normal(gen, (rows, k), 1.0, kind)
        # a few channels are larger than the rest, as in a residual stream
        x.mul_(1.0 + 7.0 * (torch.rand(k, generator=gen, device="cuda") < 0.01).to(kind))
        state["x"] = x
        if case["op"] == "linear":
            state["w_codes"], state["w_sf"], state["w_alpha"] = _weights_fp4(
                _normal(gen, (case["n"], k), 0.02, torch.float32), case["format"])
        return state
    groups, n = case["groups"], case["n"]
    shares = torch.tensor(_shares(case), dtype=torch.float64, device="cuda")
    shares = shares[torch.randperm(groups, generator=gen, device="cuda")]
    ids = torch.multinomial(shares, rows, replacement=True, generator=gen)
    counts = torch.bincount(ids, minlength=groups)
    state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    # for the plain form: the experts that have rows, and the most rows of one
    state["present"] = torch.nonzero(counts).flatten()
    state["most"] = int(counts.max())
    if case["op"] != "dgrad":
        state["x"] = _normal(gen, (rows, k), 1.0, kind)
    if case["op"] != "fwd":
        state["dy"] = _normal(gen, (rows, n), 1.0 / 16, kind)
    if case["op"] != "wgrad":
        state["w"] = _normal(gen, (groups, n, k), 0.02, kind)
    return state


def _weights_fp4(w, form):
    """Codes [n, k / 2] (value 2i in the low half of a byte), scale bytes [n, k / block] in rows
    of a multiple of 16 bytes, and the tensor scale [1] (NVFP4)."""
    n, k = w.shape
    alpha = w.abs().amax().reshape(1) / 2688.0 if form == "nvfp4" else None
    q, scale = _fp4(w, form, alpha)
    index = (q.abs() * 2).long()
    code = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=w.device)[index]
    code = (code + 8 * torch.signbit(q)).to(torch.uint8).view(n, k)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    blocks = k // BLOCK[form]
    sf = torch.zeros((n, (blocks + 15) // 16 * 16), dtype=torch.uint8, device=w.device)[:, :blocks]
    if form == "mxfp4":
        sf.copy_((torch.frexp(scale)[1] + 126).to(torch.uint8).view(n, blocks))
    else:
        sf.copy_(scale.to(torch.float8_e4m3fn).view(torch.uint8).view(n, blocks))
    return codes.contiguous(), sf, alpha


# ------------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return {"fwd": _fwd, "dgrad": _dgrad, "wgrad": _wgrad, "values": _values, "linear": _linear}[case["op"]](
        state, case)


def _fwd(s, case):
    if own:
        import sparse_moe_layer_fp32_b200 as bm
        return bm.beam_moe_grouped_gemm(s["x"], s["w"], s["offsets"], out_dtype=TYPES[case["out"]])
    x, at = _by_expert(s["x"], s)
    y = torch.bmm(x, _weights(s).transpose(1, 2))
    return _by_row(y, at, case["rows"], TYPES[case["out"]])


def _dgrad(s, case):
    if own:
        import sparse_moe_layer_fp32_b200 as bm
        return bm.beam_moe_grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"], out_dtype=TYPES[case["out"]])
    dy, at = _by_expert(s["dy"], s)
    return _by_row(torch.bmm(dy, _weights(s)), at, case["rows"], TYPES[case["out"]])


def _wgrad(s, case):
    if own:
        import sparse_moe_layer_fp32_b200 as bm
        return bm.beam_moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], out_dtype=TYPES[case["out"]])
    dy, _ = _by_expert(s["dy"], s)
    x, _ = _by_expert(s["x"], s)
    dw = torch.zeros((case["groups"], case["n"], case["k"]), dtype=TYPES[case["out"]], device=x.device)
    dw[s["present"]] = torch.bmm(dy.transpose(1, 2), x).to(dw.dtype)
    return dw


def _by_expert(rows, s):
    """Rows in FP32 as [experts with rows, most, columns], zeros behind each expert's last, and
    the row that each place holds (the number of rows where it holds none)."""
    start, end = s["offsets"][s["present"]].long(), s["offsets"][s["present"] + 1].long()
    at = start[:, None] + torch.arange(s["most"], device=rows.device)
    held = at < end[:, None]
    out = rows[at.clamp(max=rows.shape[0] - 1)].float() * held[..., None]
    return out, torch.where(held, at, rows.shape[0])


def _weights(s):
    w = s["w"]
    return w.float() if s["present"].numel() == w.shape[0] else w[s["present"]].float()


def _by_row(y, at, rows, kind):
    out = torch.empty((rows + 1, y.shape[-1]), dtype=kind, device=y.device)
    out[at] = y.to(kind)
    return out[:rows]


def _values(s, case):
    form = case["format"]
    if own:
        import sparse_moe_layer_fp32_b200 as bm
        codes, sf, alpha = bm.beam_moe_quantize_fp4(s["x"], form, alpha=ALPHA_X if form == "nvfp4" else None)
        return bm.beam_moe_dequantize_fp4(codes, sf, form, alpha=alpha, out_dtype=s["x"].dtype)
    return _fp4_values(s["x"], form).to(s["x"].dtype)


def _linear(s, case):
    form = case["format"]
    if own:
        import sparse_moe_layer_fp32_b200 as bm
        codes, sf, alpha = bm.beam_moe_quantize_fp4(s["x"], form, alpha=ALPHA_X if form == "nvfp4" else None)
        return bm.beam_moe_gemm_fp4(codes, sf, s["w_codes"], s["w_sf"], form, alpha_a=alpha, alpha_b=s["w_alpha"],
                                    out_dtype=s["x"].dtype)
    return torch.matmul(_fp4_values(s["x"], form), _decoded(s, form, torch.float32).t()).to(s["x"].dtype)


def _fp4(x, form, alpha):
    """E2M1 values and block scales, [blocks, block] and [blocks, 1], of an FP32 tensor."""
    v = x.reshape(-1, BLOCK[form])
    amax = v.abs().amax(1, keepdim=True)
    if form == "mxfp4":  # the smallest power of two, from 2^-127 on, with amax <= 6 * 2^e
        part, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - torch.where(part <= 0.75, 3, 2), -127).clamp(min=-127)
        return _e2m1(torch.ldexp(v, -e)), torch.ldexp(torch.ones_like(amax), e)
    scale = (amax / (6.0 * alpha)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    return torch.where(scale > 0, _e2m1(v / (scale * alpha)), 0.0), scale


def _e2m1(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, ties to the even code."""
    size = v.abs()
    step = 0.5 + 0.5 * (size >= 2) + (size >= 4)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _fp4_values(x, form):
    alpha = torch.full((1,), ALPHA_X, device=x.device)
    q, scale = _fp4(x.float(), form, alpha)
    return (q * (scale * alpha if form == "nvfp4" else scale)).view(x.shape)


def _decoded(s, form, kind):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=kind,
                         device=s["w_codes"].device)
    codes = s["w_codes"]
    q = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    q = q.view(codes.shape[0], -1, BLOCK[form])
    if form == "mxfp4":
        scale = torch.ldexp(torch.ones((), dtype=kind, device=codes.device), s["w_sf"].int() - 127)
    else:
        scale = s["w_sf"].view(torch.float8_e4m3fn).to(kind) * s["w_alpha"].to(kind)
    return (q * scale[..., None]).view(codes.shape[0], -1)


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("values", "linear"):
        x = s["x"].double()
        values = torch.empty_like(x)
        block = BLOCK[case["format"]]
        step = max(1, (1 << 25) // x.shape[1])
        for i in range(0, x.shape[0], step):
            v = x[i:i + step].reshape(-1, block)
            if case["format"] == "mxfp4":
                d = _smallest_power(v.abs().amax(1, keepdim=True) / 6.0)
            else:
                d = ALPHA_X * _nearest(v.abs().amax(1, keepdim=True) / (6.0 * ALPHA_X), _e4m3_table(v.device))
            q = torch.where(d > 0, v / torch.where(d > 0, d, 1.0), 0.0)
            grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
            values[i:i + step] = (torch.sign(q) * _nearest(q.abs(), grid) * d).view(-1, x.shape[1])
        if case["op"] == "values":
            return values
        return values @ _decoded(s, case["format"], torch.float64).t()
    border = s["offsets"].tolist()
    groups, n, k = case["groups"], case["n"], case["k"]
    shape = {"fwd": (case["rows"], n), "dgrad": (case["rows"], k), "wgrad": (groups, n, k)}[case["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    for e in range(groups):
        a, b = border[e], border[e + 1]
        if a == b:
            continue
        if case["op"] == "fwd":
            out[a:b] = s["x"][a:b].double() @ s["w"][e].double().t()
        elif case["op"] == "dgrad":
            out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        else:
            out[e] = s["dy"][a:b].double().t() @ s["x"][a:b].double()
    return out


def _smallest_power(v):
    """The smallest 2^e >= v with e >= -127, found by trying; 0 for 0 (every code is 0 there)."""
    e = torch.floor(torch.log2(v.clamp(min=2.0 ** -127))) - 1
    for _ in range(3):
        e = torch.where(torch.pow(2.0, e) < v, e + 1, e)
    return torch.where(v > 0, torch.pow(2.0, e.clamp(min=-127)), 0.0)


def _e4m3_table(device):
    code = torch.arange(127, device=device)
    e, m = code // 8, (code % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))


def _nearest(v, table):
    """The nearest value of an ascending table of a float format's codes 0, 1, 2, ..., ties to
    the even code, the last one above it."""
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, table.numel() - 1)
    lo = hi - 1
    down, up = v - table[lo], table[hi] - v
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return table[pick]
