"""Cases, plain forms and exact values of the layer operators next to the delta rule: the
gated linear recurrence, layer norm and the short causal convolution, forward and backward.

Notation of the recurrence, per channel c of head h (sigma is the logistic function):
  gk_t = lower_bound * sigma(exp(A_log[h]) * (g_t + dt_bias))     bounded gate
  gk_t = -exp(A_log[h]) * log(1 + exp(g_t + dt_bias))             gate without a lower bound
  h_t  = exp(gk_t) * h_{t-1} + sigma(i_t) * x_t,  out_t = h_t
Layer norm: y = (x - mean) * rstd * weight + bias over the last axis.
Short convolution, W taps per channel: y_t = silu(bias + sum_j weight[j] * x_{t-W+1+j}), the
rows before a sequence's first being its initial state.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
# Rows from one checkpoint of the recurrence's state to the next: the forward pass of a
# training step leaves the state that every 64th packed row starts from, in 32 bits.
CHECKPOINT_ROWS = 64


def _glr(name, way, dtype, B, T, H, K, seqs=0, gate="bounded", state="fp32", fused=False):
    return {"name": name, "op": "glr", "dir": way, "dtype": dtype, "B": B, "T": T, "H": H, "K": K,
            "seqs": seqs, "gate": gate, "state": state, "fused": fused}


def _norm(name, way, dtype, rows, D, affine=True):
    return {"name": name, "op": "norm", "dir": way, "dtype": dtype, "rows": rows, "D": D, "affine": affine}


def _conv(name, way, dtype, B, T, D, W=4, seqs=0, state=True, fused=False):
    return {"name": name, "op": "conv", "dir": way, "dtype": dtype, "B": B, "T": T, "D": D, "W": W,
            "seqs": seqs, "state": state, "fused": fused}


def listed():
    return [
        # one decode token for 64 sequences, 32-bit states: latency
        _glr("glr_step", "fwd", "bf16", 64, 1, 64, 128),
        # the long prefill of 8192 tokens and 64 heads; the three inputs are slices of one
        # projection's output
        _glr("glr_prefill", "fwd", "bf16", 1, 8192, 64, 128, state="bf16", fused=True),
        # few channels and many tokens (8 heads of a tensor-parallel group): the scan has
        # to be split over the tokens; the gate without a lower bound
        _glr("glr_long", "fwd", "bf16", 1, 65536, 8, 128, gate="unbounded"),
        # the backward pass of the long prefill in training
        _glr("glr_train", "bwd", "bf16", 1, 8192, 64, 128),
        # ragged packed documents of odd widths in 32 bits, training
        _glr("glr_train_ragged", "bwd", "fp32", 1, 20011, 11, 77, seqs=48, gate="unbounded"),
        # the norm in front of a layer: prefill, a decode step, and training
        _norm("norm_prefill", "fwd", "bf16", 8192, 8192),
        _norm("norm_step", "fwd", "fp16", 64, 2048),
        _norm("norm_train", "bwd", "bf16", 8192, 8192),
        _norm("norm_train_odd", "bwd", "fp32", 4999, 1537),
        # the convolution on q, k, v: a ragged serving batch read in place from a wider
        # projection, one decode token for 64 sequences, and training
        _conv("conv_ragged", "fwd", "fp16", 1, 16384, 4096, seqs=32, fused=True),
        _conv("conv_step", "fwd", "bf16", 64, 1, 8192),
        _conv("conv_train", "bwd", "bf16", 1, 8192, 8192),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    most = 1 << (25 if dtype == "fp32" else 26)          # elements of one tensor
    op, way = rng.choice(["glr", "glr", "norm", "conv"]), rng.choice(["fwd", "bwd"])
    if op == "norm":
        D = rng.choice([rng.choice([1, 5]) << rng.randint(6, 11), 1 << rng.randint(9, 14), _log_uniform(rng, 64, 16000) | 1])
        rows = _log_uniform(rng, 1, max(1, min(65536, most // D)))
        return {k: v for k, v in _norm("", way, dtype, rows, D, rng.random() < 0.8).items() if k != "name"}
    K = rng.choice([64, 128, 128, rng.randrange(33, 128, 2)])
    H = rng.choice([1 << rng.randint(0, 6), _log_uniform(rng, 1, 62) | 1])
    room = most // (H * K)
    seqs = B = 0
    if rng.random() < 0.4:                               # a packed batch
        B, T = 1, _log_uniform(rng, 64, min(room, 65536))
        seqs = _log_uniform(rng, 2, 64)
    elif rng.random() < 0.3:                             # a step of one to a few tokens
        B, T = _log_uniform(rng, 1, min(256, room // 8)), _log_uniform(rng, 1, 8)
    else:
        B = _log_uniform(rng, 1, 8)
        T = _log_uniform(rng, 16, min(room // B, 65536))
    if op == "glr":
        c = _glr("", way, dtype, B, T, H, K, seqs, rng.choice(["bounded", "unbounded"]),
                 rng.choice(["fp32", "bf16", "none"]), rng.random() < 0.3)
    else:
        c = _conv("", way, dtype, B, T, H * K, rng.choice([4, 4, 3, 2]), seqs, rng.random() < 0.7,
                  rng.random() < 0.3)
    return {k: v for k, v in c.items() if k != "name"}


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        par = 4 * case["D"] * (2 if case["affine"] else 0)
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * e + par + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + (3 * 4 * case["D"] if case["affine"] else 0), "flops": 14 * n}
    seqs = case["seqs"] or case["B"]
    rows = case["B"] * case["T"]
    if case["op"] == "glr":
        D = case["H"] * case["K"]
        n, st = rows * D, seqs * D * {"fp32": 4, "bf16": 2, "none": 0}[case["state"]]
        par = 4 * (D + case["H"])
        if case["dir"] == "fwd":
            return {"bytes": 4 * n * e + 2 * st + par, "flops": 16 * n}
        ck = 4 * D * -(-rows // CHECKPOINT_ROWS)
        grads = 2 * 4 * seqs * D if st else 0            # of the final and the initial state
        return {"bytes": 7 * n * e + ck + st + grads + 2 * par, "flops": 40 * n}
    D, W = case["D"], case["W"]
    n, st = rows * D, seqs * (W - 1) * D * (1 if case["state"] else 0)
    par = 4 * D * (W + 1)
    if case["dir"] == "fwd":
        return {"bytes": 2 * n * e + 2 * st * e + par, "flops": (2 * W + 6) * n}
    return {"bytes": 3 * n * e + st * e + 2 * st * 4 + 2 * par, "flops": (6 * W + 12) * n}


# ----------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Lengths of the packed sequences, from random cuts (a few come out very short)."""
    rng, T, n = random.Random(seed), case["T"], case["seqs"]
    cuts = [0] + sorted(rng.randint(0, T) for _ in range(n - 1)) + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _sequences(case, seed, dev):
    """cu_seqlens (or None), the longest sequence, and of every packed row its sequence and
    its place in that sequence."""
    if case["seqs"]:
        lens = _lengths(case, seed)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(dev)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), cu[1:] - cu[:-1], output_size=case["T"])
        return cu, max(lens), seq, torch.arange(case["T"], device=dev) - cu[seq]
    rows = torch.arange(case["B"] * case["T"], device=dev)
    return None, case["T"], rows // case["T"], rows % case["T"]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).add_(mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        # a residual stream: rows of different size, some channels far from zero
        x = normal(rows, D) * normal(rows, 1, std=0.5).exp() + normal(D, std=0.4)
        s.update(x=x.to(dt), weight=normal(D, std=0.1, mean=1.0) if case["affine"] else None,
                 bias=normal(D, std=0.1) if case["affine"] else None)
        if case["dir"] == "fwd":
            s.update(out=torch.empty(rows, D, dtype=dt, device=dev), mean=torch.empty(rows, device=dev),
                     rstd=torch.empty(rows, device=dev))
        else:
            s["mean"], s["rstd"] = _norm_stats(s["x"].float())
            s["dout"] = normal(rows, D, dtype=dt)
        return s
    B, T = case["B"], case["T"]
    cu, longest, seq, place = _sequences(case, seed, dev)
    N = case["seqs"] or B
    s.update(cu=cu, longest=longest, seq=seq, place=place)
    if case["op"] == "glr":
        H, K = case["H"], case["K"]
        if case["fused"]:
            s["x"], s["i"], s["g"] = normal(B, T, 3, H, K, dtype=dt).unbind(2)
        else:
            s["x"], s["i"], s["g"] = (normal(B, T, H, K, dtype=dt) for _ in range(3))
        # gates that forget over a few to a few hundred tokens
        s["A_log"] = normal(H, std=0.3)
        s["dt_bias"] = normal(H, K, std=1.0, mean=-3.0)
        s["lb"] = -5.0 if case["gate"] == "bounded" else None
        st = {"fp32": torch.float32, "bf16": torch.bfloat16, "none": None}[case["state"]]
        s["init"] = normal(N, H, K, dtype=st) if st else None
        if case["dir"] == "fwd":
            s["out"] = torch.empty(B, T, H, K, dtype=dt, device=dev)
            s["final"] = torch.empty(N, H, K, dtype=st, device=dev) if st else None
        else:
            s["dout"] = normal(B, T, H, K, dtype=dt)
            s["dfinal"] = normal(N, H, K) if st else None
            h, start = _glr_states(s)
            s["checkpoints"] = start[::CHECKPOINT_ROWS].contiguous().view(-1, H, K)
            del h, start
        return s
    D, W = case["D"], case["W"]
    s["x"] = normal(B, T, 2 * D, dtype=dt)[:, :, :D] if case["fused"] else normal(B, T, D, dtype=dt)
    s["weight"], s["bias"] = normal(D, W, std=0.5), normal(D, std=0.1)
    s["init"] = normal(N, W - 1, D, dtype=dt) if case["state"] else None
    if case["dir"] == "fwd":
        s["out"] = torch.empty(B, T, D, dtype=dt, device=dev)
        s["final"] = torch.empty(N, W - 1, D, dtype=dt, device=dev) if case["state"] else None
    else:
        s["dout"] = normal(B, T, D, dtype=dt)
        s["dfinal"] = normal(N, W - 1, D) if case["state"] else None
    return s


# ----------------------------------------------------------------------------- the calls
def run(s):
    c = s["case"]
    if not own:
        return {"glr": {"fwd": _glr_fwd, "bwd": _glr_bwd}, "norm": {"fwd": _norm_fwd, "bwd": _norm_bwd},
                "conv": {"fwd": _conv_fwd, "bwd": _conv_bwd}}[c["op"]][c["dir"]](s)
    from gated_delta_rule_52_gb300 import glr, layer_norm, short_conv
    if c["op"] == "glr":
        if c["dir"] == "fwd":
            glr.glr_fwd(s["x"], s["i"], s["g"], s["out"], s["A_log"], s["dt_bias"], s["lb"],
                        initial_state=s["init"], final_state=s["final"], cu_seqlens=s["cu"])
            return {"out": s["out"], "final": s["final"]}
        return glr.glr_bwd(s["x"], s["i"], s["g"], s["A_log"], s["dt_bias"], s["lb"], s["dout"],
                           initial_state=s["init"], dfinal=s["dfinal"], cu_seqlens=s["cu"],
                           checkpoints=s["checkpoints"], want_dinit=s["init"] is not None)
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            layer_norm.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS, s["out"], mean=s["mean"], rstd=s["rstd"])
            return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
        return layer_norm.layer_norm_bwd(s["dout"], s["x"], s["weight"], s["mean"], s["rstd"])
    if c["dir"] == "fwd":
        short_conv.short_conv_fwd(s["x"], s["weight"], s["bias"], s["out"], activation="silu",
                                  initial_state=s["init"], final_state=s["final"], cu_seqlens=s["cu"])
        return {"out": s["out"], "final": s["final"]}
    return short_conv.short_conv_bwd(s["x"], s["weight"], s["bias"], s["dout"], activation="silu",
                                     initial_state=s["init"], dfinal=s["dfinal"], cu_seqlens=s["cu"],
                                     want_dinit=s["init"] is not None)


# ----------------------------------------------------------------------------- plain forms
def _sigma(x):
    t = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + t), t / (1 + t))


def _rows(t):
    """[B, T, ...] in 32 bits with packed rows and flat channels."""
    return t.float().reshape(t.shape[0] * t.shape[1], -1)


def _gate(s, g):
    """Log decay of every packed row, and what its derivative needs: exp(A_log) per channel,
    the argument of the gate's function, and that function's slope."""
    eA = s["A_log"].exp().repeat_interleave(s["case"]["K"])
    u = g + s["dt_bias"].reshape(-1)
    if s["lb"] is None:
        return -eA * (u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))), eA, u, _sigma(u)
    z = eA * u
    sg = _sigma(z)
    return s["lb"] * sg, eA, z, sg * _sigma(-z)


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t over axis 0, by doubling; a is 0 at a sequence's first row."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _glr_states(s):
    """States after every packed row, and the states that every row starts from."""
    x, i, g = _rows(s["x"]), _rows(s["i"]), _rows(s["g"])
    a = _gate(s, g)[0].exp()
    first = (s["place"] == 0)[:, None]
    init = torch.zeros_like(x[:1]) if s["init"] is None else s["init"].float().flatten(1)[s["seq"]]
    b = _sigma(i) * x + torch.where(first, a * init, 0.0)
    h = _scan(torch.where(first, 0.0, a), b, s["longest"])
    return h, torch.where(first, init, h.roll(1, 0))


def _last(s):
    """The last packed row of every sequence, and whether the sequence has any."""
    c, N = s["case"], s["case"]["seqs"] or s["case"]["B"]
    if s["cu"] is None:
        end = torch.arange(1, N + 1, device="cuda") * c["T"]
        return end - 1, torch.ones(N, dtype=torch.bool, device="cuda")
    return (s["cu"][1:] - 1).clamp(min=0), s["cu"][1:] > s["cu"][:-1]


def _glr_fwd(s):
    h, _ = _glr_states(s)
    out = h.view(s["out"].shape).to(s["out"].dtype)
    if s["final"] is None:
        return {"out": out, "final": None}
    at, some = _last(s)
    fin = torch.where(some[:, None], h[at], s["init"].float().flatten(1))
    return {"out": out, "final": fin.view(s["final"].shape).to(s["final"].dtype)}


def _glr_bwd(s):
    x, i, g, dout = _rows(s["x"]), _rows(s["i"]), _rows(s["g"]), _rows(s["dout"])
    shape, dt = s["x"].shape, s["x"].dtype
    H, K = s["case"]["H"], s["case"]["K"]
    _, start = _glr_states(s)
    gk, eA, z, slope = _gate(s, g)
    a, si = gk.exp(), _sigma(i)
    at, some = _last(s)
    if s["dfinal"] is not None:
        dout = dout.index_add(0, at, torch.where(some[:, None], s["dfinal"].flatten(1), 0.0))
    after = torch.cat([torch.where((s["place"] == 0)[1:, None], 0.0, a[1:]), torch.zeros_like(a[:1])])
    e = _scan(after.flip(0), dout.flip(0), s["longest"]).flip(0)
    dl = e * start * a
    if s["lb"] is None:
        dg, dA = -dl * eA * slope, dl * gk
    else:
        dz = dl * s["lb"] * slope
        dg, dA = dz * eA, dz * z
    r = {"dx": (e * si).view(shape).to(dt), "di": (e * x * si * _sigma(-i)).view(shape).to(dt),
         "dg": dg.view(shape).to(dt), "dA_log": dA.view(-1, H, K).sum((0, 2)), "ddt_bias": dg.sum(0).view(H, K),
         "dinit": None}
    if s["init"] is not None:
        first = (at + 1 - torch.bincount(s["seq"], minlength=at.numel())).clamp(max=x.shape[0] - 1)
        dinit = torch.where(some[:, None], (a * e)[first], s["dfinal"].flatten(1))
        r["dinit"] = dinit.view(s["dfinal"].shape)
    return r


def _norm_stats(x):
    mean = x.mean(-1)
    return mean, 1 / (((x - mean[:, None]) ** 2).mean(-1) + EPS).sqrt()


def _norm_fwd(s):
    x = s["x"].float()
    mean, rstd = _norm_stats(x)
    y = (x - mean[:, None]) * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return {"out": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dout"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    d = dy * s["weight"] if s["weight"] is not None else dy
    dx = rstd * (d - d.mean(-1, keepdim=True) - xhat * (d * xhat).mean(-1, keepdim=True))
    r = {"dx": dx.to(s["x"].dtype), "dweight": None, "dbias": None}
    if s["weight"] is not None:
        r["dweight"], r["dbias"] = (dy * xhat).sum(0), dy.sum(0)
    return r


def _taps(s, x):
    """x_{t-W+1+j} of every packed row for each tap j, and of the rows before a sequence's
    first the initial state's."""
    W, place, got = s["case"]["W"], s["place"], []
    for j in range(W):
        back = W - 1 - j
        before = torch.zeros_like(x[:1]) if s["init"] is None else \
            s["init"].float()[s["seq"], (place + j).clamp(max=W - 2)]
        got.append(torch.where((place >= back)[:, None], x.roll(back, 0), before) if back else x)
    return got


def _conv_sum(s, taps):
    y = s["bias"] + torch.zeros_like(taps[0])
    for j, t in enumerate(taps):
        y = y + s["weight"][:, j] * t
    return y


def _window(s):
    """For every sequence and row of its state: the packed row that the final state holds
    there, and the row of the initial state that it holds where the sequence is too short."""
    N, W = s["case"]["seqs"] or s["case"]["B"], s["case"]["W"]
    length = torch.bincount(s["seq"], minlength=N)
    end = length.cumsum(0)
    j = torch.arange(W - 1, device="cuda")
    inside = length[:, None] + j >= W - 1
    row = (end[:, None] - (W - 1) + j).clamp(min=0)
    return inside, row, (length[:, None] + j).clamp(max=W - 2)


def _conv_fwd(s):
    x = _rows(s["x"])
    y = _conv_sum(s, _taps(s, x))
    out = (y * _sigma(y)).view(s["out"].shape).to(s["out"].dtype)
    if s["final"] is None:
        return {"out": out, "final": None}
    inside, row, old = _window(s)
    n = torch.arange(inside.shape[0], device="cuda")[:, None]
    fin = torch.where(inside[..., None], x[row], s["init"].float()[n, old])
    return {"out": out, "final": fin.to(s["final"].dtype)}


def _conv_bwd(s):
    x, dy = _rows(s["x"]), _rows(s["dout"])
    W, R, place = s["case"]["W"], x.shape[0], s["place"]
    taps = _taps(s, x)
    y = _conv_sum(s, taps)
    sg = _sigma(y)
    d = dy * (sg + y * sg * _sigma(-y))
    dx = s["weight"][:, W - 1] * d
    for back in range(1, min(W, R)):
        reach = (place[back:] >= back)[:, None]
        dx[:-back] += torch.where(reach, s["weight"][:, W - 1 - back] * d[back:], 0.0)
    dinit = None
    if s["init"] is not None:
        inside, row, old = _window(s)
        n = torch.arange(inside.shape[0], device="cuda")[:, None].expand_as(row)
        dx = dx.index_add(0, row[inside], s["dfinal"][inside])
        dinit = torch.zeros_like(s["dfinal"]).index_put((n[~inside], old[~inside]), s["dfinal"][~inside], accumulate=True)
        for j in range(W - 1):                           # a tap j at place p reads row p + j
            early = place < W - 1 - j
            dinit.index_put_((s["seq"][early], place[early] + j), s["weight"][:, j] * d[early], accumulate=True)
    return {"dx": dx.view(s["x"].shape).to(s["x"].dtype),
            "dweight": torch.stack([(d * t).sum(0) for t in taps], 1), "dbias": d.sum(0), "dinit": dinit}


# ----------------------------------------------------------------------------- 64 bits
def _bounds(s):
    c = s["case"]
    ends = [c["T"] * (n + 1) for n in range(c["B"])] if s["cu"] is None else s["cu"][1:].tolist()
    return list(zip([0] + ends[:-1], ends))


def exact(case, seed):
    s = prepare(case, seed)
    return {"glr": _glr_exact, "norm": _norm_exact, "conv": _conv_exact}[case["op"]](s)


def _glr_exact(s):
    """The recurrence row by row: all sequences of a batch at once, packed ones in turn."""
    c, dd = s["case"], torch.float64
    H, K, D = c["H"], c["K"], c["H"] * c["K"]
    x, i, g = (s[k].to(dd).reshape(-1, D) for k in "xig")
    A = s["A_log"].to(dd).exp().repeat_interleave(K)
    v = g + s["dt_bias"].to(dd).reshape(-1)
    gk = -A * torch.nn.functional.softplus(v, threshold=1e4) if s["lb"] is None else s["lb"] * torch.sigmoid(A * v)
    a, si = gk.exp(), torch.sigmoid(i)
    b = si * x
    bounds = _bounds(s)
    N = len(bounds)
    init = torch.zeros(N, D, dtype=dd, device="cuda") if s["init"] is None else s["init"].to(dd).view(N, D)
    if s["cu"] is None:                                  # [T, B, D], one step for the whole batch
        runs = [(list(range(N)), [torch.arange(N, device="cuda") * c["T"] + t for t in range(c["T"])])] if N > 1 else \
            [([0], [slice(t, t + 1) for t in range(c["T"])])]
    else:
        runs = [([n], [slice(t, t + 1) for t in range(*bounds[n])]) for n in range(N)]
    start, out, fin = torch.empty_like(b), torch.empty_like(b), init.clone()
    for who, steps in runs:
        h = init[who]
        for t in steps:
            start[t] = h
            h = torch.addcmul(b[t], a[t], h)
            out[t] = h
        fin[who] = h
    shape = s["x"].shape
    if c["dir"] == "fwd":
        return {"out": out.view(shape), "final": fin.view(N, H, K) if s["final"] is not None else None}
    del out, b
    do = s["dout"].to(dd).reshape(-1, D)
    e, dinit = torch.empty_like(do), torch.zeros(N, D, dtype=dd, device="cuda")
    for who, steps in runs:
        back = s["dfinal"].to(dd).view(N, D)[who] if s["dfinal"] is not None else torch.zeros(len(who), D, dtype=dd, device="cuda")
        for t in reversed(steps):
            back = back + do[t]
            e[t] = back
            back = back * a[t]
        dinit[who] = back
    dl = e * start * a
    if s["lb"] is None:
        dg, dA = -dl * A * torch.sigmoid(v), dl * gk
    else:
        dv = dl * s["lb"] * torch.sigmoid(A * v) * torch.sigmoid(-A * v)
        dg, dA = dv * A, dv * A * v
    return {"dx": (e * si).view(shape), "di": (e * x * si * torch.sigmoid(-i)).view(shape), "dg": dg.view(shape),
            "dA_log": dA.sum(0).view(H, K).sum(1), "ddt_bias": dg.sum(0).view(H, K),
            "dinit": dinit.view(N, H, K) if s["init"] is not None else None}


def _norm_exact(s):
    x = s["x"].double().requires_grad_(s["case"]["dir"] == "bwd")
    w, b = (None if s[k] is None else s[k].double().requires_grad_(s["case"]["dir"] == "bwd") for k in ("weight", "bias"))
    mean = x.mean(-1, keepdim=True)
    rstd = (x.var(-1, unbiased=False, keepdim=True) + EPS).rsqrt()
    y = (x - mean) * rstd
    y = y * w + b if w is not None else y
    if s["case"]["dir"] == "fwd":
        return {"out": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    got = torch.autograd.grad(y, [x] + ([w, b] if w is not None else []), s["dout"].double())
    return dict(zip(("dx", "dweight", "dbias"), list(got) + [None] * (3 - len(got))))


def _conv_exact(s):
    """Every sequence with its state's rows in front of it, by differentiation."""
    c, bwd = s["case"], s["case"]["dir"] == "bwd"
    D, W = c["D"], c["W"]
    leaf = lambda t: t.double().detach().clone().requires_grad_(bwd)  # noqa: E731
    x, w, b = leaf(s["x"].reshape(-1, D)), leaf(s["weight"]), leaf(s["bias"])
    bounds = _bounds(s)
    init = leaf(s["init"]) if s["init"] is not None else torch.zeros(len(bounds), W - 1, D, dtype=torch.float64, device="cuda")
    ys, fins = [], []
    for n, (lo, hi) in enumerate(bounds):
        rows = torch.cat([init[n], x[lo:hi]])
        y = b + sum(w[:, j] * rows[j:j + hi - lo] for j in range(W))
        ys.append(torch.nn.functional.silu(y))
        fins.append(rows[hi - lo:])
    out, fin = torch.cat(ys), torch.stack(fins)
    if not bwd:
        return {"out": out.view(s["x"].shape), "final": fin if s["final"] is not None else None}
    loss = (out * s["dout"].double().reshape(-1, D)).sum()
    if s["dfinal"] is not None:
        loss = loss + (fin * s["dfinal"].double()).sum()
    got = torch.autograd.grad(loss, [x, w, b] + ([init] if s["init"] is not None else []))
    return {"dx": got[0].view(s["x"].shape), "dweight": got[1], "dbias": got[2], "dinit": got[3] if len(got) > 3 else None}
