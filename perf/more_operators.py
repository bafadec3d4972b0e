"""Cases, plain forms and exact values of the operators around a layer's projections: the
root-mean-square norm with the residual's addition, quantisation to 8-bit floating point with
a scale for each block of 128, and the matrix product of such tensors.

Notation.  A norm adds first, h = x + residual (rounded to the tensors' type, as the residual
stream keeps it), then out = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps).
8-bit tensors hold q = x / scale rounded to e4m3 (at most 448) or e5m2 (at most 57344); the
scale of 128 neighbours along a row is the smallest power of two that their largest finite
magnitude allows.  Such a block lies in one row, or with `tile` spans 128 rows too (weights).
The transposed form of a tensor has its blocks along the tensor's columns.
The product is out[m, n] = add[m, n] + sum_k a[m, k] b[n, k] of the values that the operands
stand for.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BLOCK = 128
EPS = 1e-6


def _norm(name, way, dtype, rows, D, res=True, out8=None):
    return {"name": name, "op": "norm", "dir": way, "dtype": dtype, "rows": rows, "D": D, "res": res, "out8": out8}


def _quant(name, dtype, rows, cols, to="e4m3", both=True, tile=False):
    return {"name": name, "op": "quant", "dtype": dtype, "rows": rows, "cols": cols, "to": to, "both": both, "tile": tile}


def _mm(name, M, N, K, dtype="bf16", a="e4m3", b="e4m3", tile=True, add=False):
    return {"name": name, "op": "mm", "M": M, "N": N, "K": K, "dtype": dtype, "a": a, "b": b, "tile": tile, "add": add}


def listed():
    return [
        # one decode token of 64 sequences, 64 heads of 128: the norm in front of a projection,
        # in 8 bits for it, and the residual stream: latency
        _norm("norm_step", "fwd", "bf16", 64, 8192, out8="e4m3"),
        # the same on a prefill of 8192 tokens
        _norm("norm_prefill", "fwd", "bf16", 8192, 8192, out8="e4m3"),
        # odd rows without a residual
        _norm("norm_odd", "fwd", "fp16", 4999, 1537, res=False),
        # training: the gradient of the prefill's norm and its residual
        _norm("norm_train", "bwd", "bf16", 8192, 8192),
        # training: an output gradient for the two products of a projection's backward pass
        _quant("quant_grad", "bf16", 8192, 8192, to="e5m2"),
        # a projection's 32-bit weights after an optimizer's step, for both passes
        _quant("quant_weight", "fp32", 8192, 2048, tile=True),
        # one token through a projection, and one token of 64 sequences: reading the weights
        _mm("mm_token", 1, 8192, 8192),
        _mm("mm_step", 64, 8192, 8192),
        # a prefill of 8192 tokens through a projection
        _mm("mm_prefill", 8192, 8192, 8192),
        # a ragged prompt through a projection to odd heads, added to the residual stream
        _mm("mm_ragged", 4999, 1537, 2111, dtype="fp16", add=True),
        # a prompt of 512 tokens: few tiles for many SMs
        _mm("mm_prompt", 512, 2048, 8192),
        # a weight gradient over 16384 tokens, added to the gradient so far in 32 bits
        _mm("mm_wgrad", 8192, 2048, 16384, dtype="fp32", a="e5m2", tile=False, add=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _extent(rng, lo, hi):
    """A size of a model's: multiples of 128 and 16, powers of two, odd ones."""
    n = _log_uniform(rng, lo, hi)
    return rng.choice([max(BLOCK, n // BLOCK * BLOCK), max(16, n // 16 * 16), 1 << n.bit_length() - 1, n | 1])


def draw(rng):
    op = rng.choice(["norm", "quant", "mm", "mm"])
    if op == "norm":
        way, dtype = rng.choice(["fwd", "bwd"]), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        D = min(_extent(rng, 64, 16384), 16384)
        rows = _log_uniform(rng, 1, max(1, min(32768, (1 << (25 if dtype == "fp32" else 26)) // D)))
        c = _norm("", way, dtype, rows, D, rng.random() < 0.7,
                  rng.choice([None, "e4m3", "e5m2"]) if way == "fwd" else None)
    elif op == "quant":
        cols = min(_extent(rng, 16, 16384), 16384)
        rows = _log_uniform(rng, 1, min(32768, (1 << 25) // cols))
        c = _quant("", rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows, cols, rng.choice(["e4m3", "e4m3", "e5m2"]),
                   rng.random() < 0.6, rng.random() < 0.3)
    else:
        N, K = (min(_extent(rng, 16, 16384), 16384) for _ in range(2))
        M = _log_uniform(rng, 1, max(1, min(16384, (1 << 37) // (N * K))))
        c = _mm("", M, N, K, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["e4m3", "e4m3", "e5m2"]),
                rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.6, rng.random() < 0.3)
    return {k: v for k, v in c.items() if k != "name"}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    e = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        n = rows * D
        if case["dir"] == "bwd":                           # dout, h, dx, and the residual's gradient
            return {"bytes": (4 if case["res"] else 3) * n * e + 4 * rows + 8 * D, "flops": 10 * n}
        # x, and with a residual that and the sum; the output, in 8 bits with its scales (the
        # values that it stands for, which come back beside it, are not counted)
        out = n + rows * _blocks(D) if case["out8"] else n * e
        return {"bytes": (3 if case["res"] else 1) * n * e + out + 4 * rows + 4 * D, "flops": 6 * n}
    if case["op"] == "quant":
        R, C = case["rows"], case["cols"]
        n = R * C
        if case["tile"]:
            scales = _blocks(R) * _blocks(C) * (2 if case["both"] else 1)
        else:
            scales = R * _blocks(C) + (C * _blocks(R) if case["both"] else 0)
        return {"bytes": n * (e + (2 if case["both"] else 1)) + scales, "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    rows = _blocks(N) if case["tile"] else N
    return {"bytes": (M + N) * K + (M + rows) * _blocks(K) + M * N * e * (2 if case["add"] else 1), "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- inputs
def _empty8(rows, cols, to, tile=False):
    """An 8-bit tensor and its scales, rows 16 and 4 bytes aligned as the product reads them."""
    lines, blocks = _blocks(rows) if tile else rows, _blocks(cols)
    q = torch.empty(rows, -(-cols // 16) * 16, dtype=TYPES[to], device="cuda")[:, :cols]
    s = torch.empty(lines, -(-blocks // 4) * 4, dtype=torch.float8_e8m0fnu, device="cuda")[:, :blocks]
    return q, s


def _operand(x, to, tile):
    q, s = _empty8(*x.shape, to, tile)
    e = _exponents(x, to, tile)
    q.copy_(_over(x, e).to(TYPES[to]))
    s.view(torch.uint8).copy_((e[::BLOCK] if tile else e) + 127)
    return q, s


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).add_(mean)

    def tokens(rows, cols, std=1.0):
        """Rows of different size, a few channels far larger than the others."""
        return normal(rows, cols, std=std) * normal(rows, 1, std=0.5).exp() * normal(1, cols, std=0.5).exp()

    s = {"case": dict(case)}
    if case["op"] == "norm":
        rows, D, dt = case["rows"], case["D"], TYPES[case["dtype"]]
        s["weight"] = normal(D, std=0.1, mean=1.0)
        s["x"] = tokens(rows, D).to(dt)
        if case["dir"] == "bwd":
            s["rstd"] = _rstd(s["x"].float())
            s["dout"] = normal(rows, D).to(dt)
            s["dres"] = normal(rows, D).to(dt) if case["res"] else None
            return s
        s["res"] = tokens(rows, D).to(dt) if case["res"] else None
        s["res_out"] = torch.empty_like(s["x"]) if case["res"] else None
        s["rstd"] = torch.empty(rows, device=dev)
        if case["out8"]:
            s["out"], s["scales"] = _empty8(rows, D, case["out8"])
            s["values"] = torch.empty(rows, D, dtype=torch.bfloat16, device=dev)
        else:
            s["out"], s["scales"] = torch.empty_like(s["x"]), None
        return s
    if case["op"] == "quant":
        R, C = case["rows"], case["cols"]
        x = normal(R, C, std=C ** -0.5) if case["tile"] else tokens(R, C, std=1e-3 if case["to"] == "e5m2" else 1.0)
        s["x"] = x.to(TYPES[case["dtype"]])
        s["q"], s["scales"] = _empty8(R, C, case["to"], case["tile"])
        s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device=dev)
        s["qt"], s["scales_t"], s["values_t"] = None, None, None
        if case["both"]:
            s["qt"], s["scales_t"] = _empty8(C, R, case["to"], case["tile"])
            s["values_t"] = torch.empty(C, R, dtype=torch.bfloat16, device=dev)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["a"], s["sa"] = _operand(tokens(M, K), case["a"], False)
    s["b"], s["sb"] = _operand(normal(N, K, std=K ** -0.5) if case["tile"] else tokens(N, K, std=K ** -0.5), case["b"], case["tile"])
    s["add"] = tokens(M, N).to(TYPES[case["dtype"]]) if case["add"] else None
    s["out"] = torch.empty(M, N, dtype=TYPES[case["dtype"]], device=dev)
    return s


# ----------------------------------------------------------------------------- the calls
def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "norm":
            return _norm_fwd(s) if c["dir"] == "fwd" else _norm_bwd(s)
        return _quant_plain(s) if c["op"] == "quant" else _mm_plain(s)
    from gated_delta_rule_52_gb300 import fp8, rms_norm
    if c["op"] == "norm":
        if c["dir"] == "bwd":
            return rms_norm.rms_norm_bwd(s["dout"], s["x"], s["weight"], s["rstd"], dresidual=s["dres"])
        rms_norm.rms_norm_fwd(s["x"], s["weight"], EPS, s["out"], residual=s["res"], residual_out=s["res_out"],
                              rstd=s["rstd"], scales=s["scales"])
        out = s["out"]
        if c["out8"]:                                      # the values that the 8 bits stand for
            fp8.dequantize(s["out"], s["scales"], s["values"])
            out = s["values"]
        return {"out": out, "res_out": s["res_out"], "rstd": s["rstd"]}
    if c["op"] == "quant":
        fp8.quantize(s["x"], s["q"], s["scales"], qt=s["qt"], scales_t=s["scales_t"], tile=c["tile"])
        fp8.dequantize(s["q"], s["scales"], s["values"])
        if c["both"]:
            fp8.dequantize(s["qt"], s["scales_t"], s["values_t"])
        return {"values": s["values"], "values_t": s["values_t"]}
    fp8.matmul(s["a"], s["sa"], s["b"], s["sb"], s["out"], add=s["add"])
    return {"out": s["out"]}


# ----------------------------------------------------------------------------- plain forms
def _power(e):
    """2^e in 32 bits, from its bits."""
    return (e + 127).to(torch.int32).mul(1 << 23).view(torch.float32)


def _exponents(x, to, tile):
    """The scales' exponents of x [R, C], one for each row and block of 128 columns (with
    `tile` the same in 128 rows)."""
    R, C = x.shape
    x = torch.where(x.isfinite(), x.abs(), 0.0)
    x = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % BLOCK if tile else 0))
    if tile:
        top = x.view(_blocks(R), BLOCK, _blocks(C), BLOCK).amax((1, 3)).repeat_interleave(BLOCK, 0)[:R]
    else:
        top = x.view(R, _blocks(C), BLOCK).amax(2)
    m, k = torch.frexp(top)                                # top = m 2^k, 1/2 <= m < 1; 448 = 7/8 2^9, 57344 = 7/8 2^16
    e = k - (9 if to == "e4m3" else 16) + (m > 0.875).int()
    return torch.where(top < 2.0 ** -126, 0, e.clamp(min=-126)).int()


def _over(x, e):
    return x * _power(-e).repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def _rounded(x, to, tile=False):
    """The values that x stands for in 8 bits."""
    e = _exponents(x, to, tile)
    return _over(_over(x, e).to(TYPES[to]).float(), -e)


def _rstd(h):
    return 1 / ((h * h).mean(-1) + EPS).sqrt()


def _norm_fwd(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(s["x"].dtype).float()
    rstd = _rstd(h)
    y = h * rstd[:, None] * s["weight"]
    y = _rounded(y, s["case"]["out8"]).to(torch.bfloat16) if s["case"]["out8"] else y.to(s["x"].dtype)
    return {"out": y, "res_out": None if s["res"] is None else h.to(s["x"].dtype), "rstd": rstd}


def _norm_bwd(s):
    h, dy, rstd = s["x"].float(), s["dout"].float(), s["rstd"][:, None]
    hat = h * rstd
    d = dy * s["weight"]
    dx = rstd * (d - hat * (d * hat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * hat).sum(0)}


def _quant_plain(s):
    x, c = s["x"].float(), s["case"]
    turned = _rounded(x.T, c["to"], c["tile"]).to(torch.bfloat16).contiguous() if c["both"] else None
    return {"values": _rounded(x, c["to"], c["tile"]).to(torch.bfloat16), "values_t": turned}


def _values(q, scales, tile):
    e = scales.view(torch.uint8).int() - 127
    return _over(q.float(), -(e.repeat_interleave(BLOCK, 0)[:q.shape[0]] if tile else e))


def _mm_plain(s):
    y = _values(s["a"], s["sa"], False) @ _values(s["b"], s["sb"], s["case"]["tile"]).T
    if s["add"] is not None:
        y = y + s["add"].float()
    return {"out": y.to(s["out"].dtype)}


# ----------------------------------------------------------------------------- 64 bits
def _eight_bits(x, to, tile=False):
    """What the 8 bits of x [R, C] stand for, from the formats' definitions: e4m3 has 3 bits
    behind the leading one and steps of 2^-9 at least, e5m2 2 bits and 2^-16."""
    bits, low, most = (3, -9, 448.0) if to == "e4m3" else (2, -16, 57344.0)
    R, C = x.shape
    out = torch.empty_like(x)
    for c in range(0, C, BLOCK):
        part = x[:, c:c + BLOCK]
        top = part.abs().amax(1)
        if tile:
            top = torch.cat([top[r:r + BLOCK].amax().expand(min(BLOCK, R - r)) for r in range(0, R, BLOCK)])
        e = torch.log2(top.clamp(min=2.0 ** -126) / most).ceil()
        e = torch.where(torch.exp2(e) * most < top, e + 1, torch.where(torch.exp2(e - 1) * most >= top, e - 1, e))
        scale = torch.where(top < 2.0 ** -126, 1.0, torch.exp2(e.clamp(min=-126)))[:, None]
        v = part / scale
        step = torch.exp2((torch.frexp(v)[1] - 1 - bits).clamp(min=low).double())
        out[:, c:c + BLOCK] = (v / step).round() * step * scale      # halves go to the even one
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        w = s["weight"].double()
        if case["dir"] == "bwd":
            # rstd belongs to the inputs as it is: its own derivative is -rstd^3 mean(h dh)
            h, dy, r = s["x"].double(), s["dout"].double(), s["rstd"].double()[:, None]
            dx = dy * w * r - h * r.pow(3) * (dy * w * h).sum(-1, keepdim=True) / case["D"]
            if s["dres"] is not None:
                dx = dx + s["dres"].double()
            return {"dx": dx, "dweight": torch.einsum("rd,rd->d", dy, h * r)}
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["x"].dtype).double()
        r = (h.square().sum(-1) / case["D"] + EPS).rsqrt()
        y = h * r[:, None] * w
        return {"out": _eight_bits(y, case["out8"]) if case["out8"] else y,
                "res_out": h if s["res"] is not None else None, "rstd": r}
    if case["op"] == "quant":
        x, to, tile = s["x"].double(), case["to"], case["tile"]
        return {"values": _eight_bits(x, to, tile), "values_t": _eight_bits(x.T.contiguous(), to, tile) if case["both"] else None}

    def stands_for(q, scales, tile):
        f = scales.to(torch.float64).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
        return q.to(torch.float64) * (f.repeat_interleave(BLOCK, 0)[:q.shape[0]] if tile else f)

    y = torch.matmul(stands_for(s["a"], s["sa"], False), stands_for(s["b"], s["sb"], case["tile"]).T)
    return {"out": y if s["add"] is None else y + s["add"].double()}
