"""The operators around the delta rule on the GPU against 64-bit references, every element
within the bound that the reference carries for it (tests/layer_ref.py)."""
import pytest
import torch

from gated_delta_rule_52_gb300 import glr, kda, layer_norm, short_conv
from tests import layer_ref as ref
from tests.layer_ref import assert_close

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cu(lens):
    return None if lens is None else torch.tensor([0] + list(lens)).cumsum(0).cuda()


def _place(t, how):
    """The same values on the GPU: contiguous, as a slice of a wider tensor, or as a slice
    that starts one element off (what lies beside it is NaN)."""
    if how == "dense":
        return t.cuda()
    pad = {"slice": 16, "odd": 1}[how]
    lead, tail = (t.shape[:2], t.shape[2:]) if t.dim() == 4 else (t.shape[:-1], t.shape[-1:])
    width = tail.numel()
    wide = torch.full((*lead, width + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
    part = wide[..., pad:pad + width].unflatten(-1, tuple(tail))
    part.copy_(t)
    return part


def _status():
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK


# ------------------------------------------------------------------ gated recurrence
def _glr_inputs(B, T, H, K, dt, lens, sd, seed):
    g = _gen(seed)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(s, generator=g) * std + mean  # noqa: E731
    N = B if lens is None else len(lens)
    d = {k: n(B, T, H, K).to(dt) for k in ("x", "i", "g", "dout")}
    d["A_log"], d["dt_bias"] = n(H, std=0.3), n(H, K, mean=-2.0)
    d["init"] = None if sd is None else n(N, H, K).to(sd)
    d["dfinal"] = n(N, H, K)
    d["cu"], d["N"], d["seqs"] = _cu(lens), N, ref.bounds_of(B, T, lens)
    return d


def _glr_ref(d, lb, bwd=True):
    r = lambda t: None if t is None else t.double().reshape(-1, *d["x"].shape[2:])  # noqa: E731
    return ref.glr(r(d["x"]), r(d["i"]), r(d["g"]), d["A_log"].double(), d["dt_bias"].double(), lb, d["seqs"],
                   None if d["init"] is None else d["init"].double(), r(d["dout"]) if bwd else None,
                   d["dfinal"].double() if bwd else None)


def _glr_run(d, lb, how="dense", checkpoints=True, in_place=False, stream=None, bwd=True):
    x, i, g, dout = (_place(d[k], how) for k in ("x", "i", "g", "dout"))
    B, T, H, K = x.shape
    A, tb = d["A_log"].cuda(), d["dt_bias"].cuda()
    init = None if d["init"] is None else d["init"].cuda()
    out = _place(torch.full(x.shape, float("nan"), dtype=x.dtype), how)
    sd = F if init is None else init.dtype
    fin = init.clone() if in_place else torch.full((d["N"], H, K), float("nan"), dtype=sd, device="cuda")
    ck = torch.full(glr.checkpoint_shape(B, T, H, K), float("nan"), device="cuda") if checkpoints else None
    dfinal = d["dfinal"].cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    glr.glr_fwd(x, i, g, out, A, tb, lb, initial_state=fin if in_place else init, final_state=fin,
                cu_seqlens=d["cu"], checkpoints=ck, stream=stream)
    r = {"out": out, "final": fin, "ck": ck}
    if bwd:
        r.update(glr.glr_bwd(x, i, g, A, tb, lb, dout, initial_state=init, dfinal=dfinal,
                             cu_seqlens=d["cu"], checkpoints=ck, stream=stream))
    _status()
    return r


def _glr_check(got, want):
    for name in ("out", "final", "dx", "di", "dg", "dA_log", "ddt_bias", "dinit"):
        if name in got:
            assert_close(name, got[name], *want[name])
    if got.get("ck") is not None:
        start, E = want["start"]
        assert_close("checkpoints", got["ck"], start[::64], E[::64])


@pytest.mark.parametrize("B,T,H,K,dt,sd,lb,how", [
    (2, 1, 3, 128, BF, F, -5.0, "dense"),          # one token
    (64, 1, 2, 64, BF, BF, None, "dense"),
    (3, 2, 2, 32, HF, F, -5.0, "slice"),
    (2, 7, 1, 1, F, F, None, "dense"),             # one channel
    (1, 63, 2, 32, BF, None, -5.0, "dense"),
    (1, 64, 2, 32, BF, BF, -5.0, "slice"),
    (2, 65, 2, 40, HF, F, None, "dense"),
    (5, 33, 5, 77, BF, F, -3.0, "odd"),            # odd width, rows off by one element
    (1, 300, 3, 43, F, F, -5.0, "odd"),
    (1, 1023, 2, 128, BF, F, None, "slice"),
    (2, 1100, 1, 96, F, None, -5.0, "dense"),
    (1, 5000, 1, 20, BF, F, None, "dense"),
    (2, 200, 1, 600, BF, F, -5.0, "dense"),        # one wide head
    (1, 130, 40, 3, F, BF, None, "dense"),         # many narrow ones
    (1, 4500, 1, 8, HF, F, -5.0, "slice"),         # few channels, many tiles
    (1, 2100, 2, 29, HF, F, None, "odd"),
    (1, 200, 1, 65, BF, F, -5.0, "dense"),         # unaligned, one channel in the last block
    (1, 200, 5, 26, BF, F, None, "dense"),         # rows of 4-byte alignment
])
def test_glr(B, T, H, K, dt, sd, lb, how):
    d = _glr_inputs(B, T, H, K, dt, None, sd, T + H)
    _glr_check(_glr_run(d, lb, how), _glr_ref(d, lb))


@pytest.mark.parametrize("lens,H,K,dt,sd,lb", [
    ((0, 5, 0, 0, 70, 1, 1, 200, 0), 2, 32, BF, F, -5.0),
    ((64, 64, 128, 1), 1, 64, F, BF, None),
    ((1,) * 37 + (0, 300), 3, 24, HF, F, -5.0),
    ((0, 0, 0), 2, 16, BF, F, None),               # sequences without tokens only
    ((900, 3, 1200, 130, 129, 128, 127), 2, 33, BF, F, None),
    ((2, 3), 1, 33, BF, F, -5.0),                  # fewer unaligned rows than 16 bytes have elements
    ((1, 70), 3, 33, F, None, -5.0),
    ((65, 7, 0, 191), 5, 51, HF, BF, -5.0),
])
def test_glr_ragged(lens, H, K, dt, sd, lb):
    d = _glr_inputs(1, sum(lens), H, K, dt, lens, sd, len(lens))
    _glr_check(_glr_run(d, lb), _glr_ref(d, lb))


@pytest.mark.parametrize("T", [1, 6, 700])
def test_glr_state_in_place_and_states_recomputed(T):
    d = _glr_inputs(3, T, 2, 48, BF, None, F, 9)
    _glr_check(_glr_run(d, -5.0, checkpoints=False, in_place=True), _glr_ref(d, -5.0))


@pytest.mark.parametrize("lb", [-5.0, 0.0, None])
@pytest.mark.parametrize("T", [3, 260])
def test_glr_masked_tokens(T, lb):
    # i = -inf adds nothing, g = -inf keeps the state, g = +inf forgets the most that the
    # gate allows; the type's lowest values act as they do
    d = _glr_inputs(2, T, 2, 32, BF, None, F, 21)
    low = torch.finfo(BF).min
    d["i"][:, 1::5] = float("-inf")
    d["i"][:, 2::7] = low
    d["g"][:, 1::3] = float("-inf")
    d["g"][:, 2::11] = float("inf")
    d["g"][:, 0::13] = low
    _glr_check(_glr_run(d, lb, bwd=False), _glr_ref(d, lb, bwd=False))


@pytest.mark.parametrize("lb", [-5.0, None])
def test_glr_gradient_at_masked_tokens(lb):
    # infinite logits have the gradients of very large ones: 0 for the masked token's own
    d = _glr_inputs(2, 200, 2, 32, BF, None, F, 22)
    d["i"][:, 1::5] = float("-inf")
    d["g"][:, 1::3] = float("-inf")
    d["g"][:, 2::11] = float("inf")
    got = _glr_run(d, lb)
    for k in ("i", "g"):
        d[k] = d[k].float().clamp(-1e4, 1e4)
    _glr_check(got, _glr_ref(d, lb))


@pytest.mark.parametrize("B", [0, 3])
def test_glr_without_tokens(B):
    d = _glr_inputs(B, 0, 2, 16, BF, None, F, 23)
    got = _glr_run(d, -5.0)
    assert torch.equal(got["final"].cpu(), d["init"]) and torch.equal(got["dinit"].cpu(), d["dfinal"])
    assert not got["dA_log"].any() and not got["ddt_bias"].any()


@pytest.mark.parametrize("lb", [-5.0, None])
def test_glr_sequences_do_not_reach_each_other(lb):
    lens = (100, 3, 64, 64, 200, 1, 1, 90)
    d = _glr_inputs(1, sum(lens), 2, 40, BF, lens, F, 5)
    bad, (lo, hi) = 4, (231, 431)
    for k in ("x", "i", "g", "dout"):
        d[k][0, lo:hi:3] = float("nan")
        d[k][0, lo + 1:hi:3] = float("inf")
    d["init"][bad] = float("inf")
    d["dfinal"][bad] = float("nan")
    got = _glr_run(d, lb)
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[lo:hi] = False
    for k in ("x", "i", "g", "dout"):
        d[k][0, lo:hi] = 0
    d["init"][bad] = d["dfinal"][bad] = 0
    want = _glr_ref(d, lb)
    for name in ("out", "dx", "di", "dg"):
        assert_close(name, got[name].reshape(-1, 2, 40)[keep.cuda()], *(t[keep] for t in want[name]))
    others = [n for n in range(len(lens)) if n != bad]
    for name in ("final", "dinit"):
        assert_close(name, got[name][others], *(t[others] for t in want[name]))
    assert not torch.isfinite(got["final"][bad]).any()


def test_glr_same_bits_every_time_and_on_another_stream():
    d = _glr_inputs(1, 3000, 2, 64, BF, (1000, 0, 1999, 1), F, 6)
    a = _glr_run(d, -5.0)
    b = _glr_run(d, -5.0, stream=torch.cuda.Stream())
    for k, v in a.items():
        assert torch.equal(v, b[k]), k


def test_glr_repeated_input_rows():
    # a gate shared by every token: stride 0 over the rows
    d = _glr_inputs(1, 150, 2, 32, F, None, F, 8)
    first = d["g"][:, :1]
    d["g"] = first.expand(1, 150, 2, 32)
    x, i, g = d["x"].cuda(), d["i"].cuda(), first.cuda().expand(1, 150, 2, 32)
    out = torch.empty_like(x)
    glr.glr_fwd(x, i, g, out, d["A_log"].cuda(), d["dt_bias"].cuda(), -5.0, initial_state=d["init"].cuda())
    _status()
    assert_close("out", out, *_glr_ref(d, -5.0, bwd=False)["out"])


@pytest.mark.parametrize("lb", [-5.0, None])
def test_glr_gradient_against_differences(lb):
    # the loss of the 64-bit reference along a random direction of every input
    d = _glr_inputs(2, 90, 2, 16, F, None, F, 11)
    got = _glr_run(d, lb)
    names = {"x": "dx", "i": "di", "g": "dg", "A_log": "dA_log", "dt_bias": "ddt_bias", "init": "dinit"}

    def loss(k, e, way):
        m = dict(d, **{k: d[k].double() + e * way})
        r = _glr_ref(m, lb, bwd=False)
        return float((r["out"][0].reshape(d["dout"].shape) * d["dout"].double()).sum() + (r["final"][0] * d["dfinal"].double()).sum())

    for k, dk in names.items():
        way = torch.randn(d[k].shape, generator=_gen(3), dtype=torch.float64)
        want = (loss(k, 1e-5, way) - loss(k, -1e-5, way)) / 2e-5
        dot = got[dk].cpu().double().reshape(way.shape) * way
        # steps of 1e-5 leave about 1e-8 of the loss' scale; the gradient's own bound is below 2^-12 of its terms
        assert abs(float(dot.sum()) - want) <= 2.0 ** -12 * float(dot.abs().sum()) + 1e-6, k


def test_glr_in_a_cuda_graph():
    d = _glr_inputs(1, 700, 2, 32, BF, None, F, 14)
    e = {k: d[k].cuda() for k in ("x", "i", "g", "A_log", "dt_bias", "init")}
    out, fin = torch.empty_like(e["x"]), torch.empty_like(e["init"])

    def call():
        glr.glr_fwd(e["x"], e["i"], e["g"], out, e["A_log"], e["dt_bias"], -5.0, initial_state=e["init"], final_state=fin)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (15, 16):
        d2 = _glr_inputs(1, 700, 2, 32, BF, None, F, seed)
        for k in ("x", "i", "g", "init"):
            e[k].copy_(d2[k])
        d2.update(A_log=d["A_log"], dt_bias=d["dt_bias"])
        graph.replay()
        _status()
        want = _glr_ref(d2, -5.0, bwd=False)
        assert_close("out", out, *want["out"])
        assert_close("final", fin, *want["final"])


# ------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("rows,D,dt,how,affine", [
    (1, 1, F, "dense", True), (3, 2, BF, "dense", True), (7, 33, HF, "odd", True), (1, 129, F, "odd", True),
    (64, 64, BF, "dense", False), (5, 1000, HF, "slice", True), (200, 256, BF, "dense", True),
    (2, 1537, F, "dense", True), (9, 4096, BF, "slice", True), (300, 2049, BF, "odd", True), (70, 4097, BF, "odd", True), (3, 8191, HF, "odd", True),
    (5, 8191, F, "odd", True), (2, 15001, BF, "odd", True),
    (3, 8192, BF, "dense", True), (4, 16384, HF, "dense", True), (2, 16385, F, "dense", False),
    (2, 70001, BF, "dense", True), (1300, 24, F, "dense", True), (0, 64, BF, "dense", True),
])
def test_layer_norm(rows, D, dt, how, affine):
    g = _gen(rows + D)
    x = (torch.randn(rows, D, generator=g) * 2 + 1.5).to(dt)
    dy = torch.randn(rows, D, generator=g).to(dt)
    w = 1 + 0.2 * torch.randn(D, generator=g) if affine else None
    b = 0.2 * torch.randn(D, generator=g) if affine else None
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    d = lambda t: None if t is None else t.double()  # noqa: E731
    want = ref.norm(x.double(), d(w), d(b), 1e-5, dy.double())
    xg, dyg = _place(x, how), _place(dy, how)
    out = _place(torch.full((rows, D), float("nan"), dtype=dt), how)
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    layer_norm.layer_norm_fwd(xg, c(w), c(b), 1e-5, out, mean=mean, rstd=rstd)
    got = layer_norm.layer_norm_bwd(dyg, xg, c(w), mean, rstd, want_params=True)
    again = layer_norm.layer_norm_bwd(dyg, xg, c(w), mean, rstd)
    torch.cuda.synchronize()
    for name, t in (("out", out), ("mean", mean), ("rstd", rstd), *got.items()):
        assert_close(name, t, *want[name])
    assert torch.equal(again["dx"], got["dx"])
    assert (again["dweight"] is None) == (w is None)
    if affine:
        assert torch.equal(again["dweight"], got["dweight"])


def test_layer_norm_in_place_and_leading_dimensions():
    x = torch.randn(2, 3, 5, 96, generator=_gen(1)).to(BF)
    want = ref.norm(x.double().reshape(-1, 96), None, None, 1e-6)
    y = x.cuda()
    layer_norm.layer_norm_fwd(y, None, None, 1e-6, y)
    torch.cuda.synchronize()
    assert_close("out", y.reshape(-1, 96), *want["out"])


def test_layer_norm_rows_do_not_reach_each_other():
    x = torch.randn(50, 130, generator=_gen(2))
    x[7], x[20, 3], x[21, 5] = 1e30, float("nan"), float("inf")
    x[30] = 4.0                                    # a constant row: variance 0
    out, mean, rstd = torch.empty(50, 130).cuda(), torch.empty(50).cuda(), torch.empty(50).cuda()
    layer_norm.layer_norm_fwd(x.cuda(), None, None, 1e-5, out, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    fine = [r for r in range(50) if r not in (7, 20, 21)]
    want = ref.norm(x[fine].double(), None, None, 1e-5)
    for name, t in (("out", out), ("mean", mean), ("rstd", rstd)):
        assert_close(name, t[fine], *want[name])
    assert torch.isnan(out[20]).all() and torch.isnan(out[21]).all()


def test_layer_norm_gradient_against_differences():
    g = _gen(4)
    x, dy, w, b = (torch.randn(*s, generator=g) for s in ((6, 70), (6, 70), (70,), (70,)))
    mean, rstd, out = torch.empty(6).cuda(), torch.empty(6).cuda(), torch.empty(6, 70).cuda()
    layer_norm.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), 1e-5, out, mean=mean, rstd=rstd)
    got = layer_norm.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    at = {"dx": x.double(), "dweight": w.double(), "dbias": b.double()}

    def loss(name, e, v):
        m = dict(at, **{name: at[name] + e * v})
        return float((ref.norm(m["dx"], m["dweight"], m["dbias"], 1e-5)["out"][0] * dy.double()).sum())

    for name, t in at.items():
        v = torch.randn(t.shape, generator=g, dtype=torch.float64)
        want = (loss(name, 1e-5, v) - loss(name, -1e-5, v)) / 2e-5
        dot = got[name].cpu().double() * v
        assert abs(float(dot.sum()) - want) <= 2.0 ** -12 * float(dot.abs().sum()) + 1e-6, name


# ------------------------------------------------------------------ short convolution
def _conv_inputs(B, T, D, W, dt, lens, state, seed, bias=True):
    g = _gen(seed)
    N = B if lens is None else len(lens)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": n(B, T, D).to(dt), "dout": n(B, T, D).to(dt), "w": n(D, W) * 0.6, "b": n(D) * 0.2 if bias else None,
            "init": n(N, W - 1, D).to(dt) if state else None, "dfinal": n(N, W - 1, D), "cu": _cu(lens),
            "N": N, "seqs": ref.bounds_of(B, T, lens)}


def _conv_ref(d, act):
    D = d["x"].shape[2]
    o = lambda t: None if t is None else t.double()  # noqa: E731
    return ref.conv(d["x"].double().reshape(-1, D), o(d["w"]), o(d["b"]), d["seqs"], act == "silu", o(d["init"]),
                    d["dout"].double().reshape(-1, D), o(d["dfinal"]))


def _conv_run(d, act, how="dense", in_place=False, stream=None):
    x, dout = _place(d["x"], how), _place(d["dout"], how)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    w, b, init, dfinal = c(d["w"]), c(d["b"]), c(d["init"]), c(d["dfinal"])
    out = _place(torch.full(d["x"].shape, float("nan"), dtype=x.dtype), how)
    fin = init.clone() if in_place else torch.full((d["N"], w.shape[1] - 1, x.shape[2]), float("nan"), dtype=x.dtype, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    short_conv.short_conv_fwd(x, w, b, out, activation=act, initial_state=fin if in_place else init,
                              final_state=fin, cu_seqlens=d["cu"], stream=stream)
    r = {"out": out, "final": fin}
    r.update(short_conv.short_conv_bwd(x, w, b, dout, activation=act, initial_state=init, dfinal=dfinal,
                                       cu_seqlens=d["cu"], stream=stream))
    torch.cuda.synchronize()
    return r


def _conv_check(got, want):
    for name, t in got.items():
        if t is not None:
            assert_close(name, t, *want[name])


@pytest.mark.parametrize("B,T,D,W,dt,lens,state,act,how", [
    (2, 1, 256, 4, BF, None, True, "silu", "dense"),
    (64, 1, 72, 4, HF, None, True, "silu", "slice"),
    (3, 2, 40, 4, BF, None, True, None, "dense"),
    (1, 5, 1, 2, F, None, False, "silu", "dense"),
    (2, 33, 77, 3, BF, None, True, "silu", "odd"),
    (2, 71, 66, 4, HF, None, True, "silu", "odd"),
    (1, 20, 131, 3, BF, (7, 0, 13), True, None, "dense"),
    (1, 64, 128, 4, HF, None, False, "silu", "slice"),
    (4, 65, 129, 2, F, None, True, None, "odd"),
    (1, 1000, 200, 4, BF, None, True, "silu", "dense"),
    (2, 513, 96, 3, F, None, True, "silu", "slice"),
    (1, 0, 64, 4, BF, None, True, "silu", "dense"),
    (1, 277, 64, 4, BF, (0, 5, 0, 0, 70, 1, 1, 200, 0), True, "silu", "dense"),
    (1, 30, 33, 4, HF, (1, 2, 3, 1, 1, 0, 2, 20), True, "silu", "odd"),
    (1, 257, 48, 4, F, (64, 64, 128, 1), False, "silu", "dense"),
    (1, 600, 24, 2, BF, (599, 1), True, None, "slice"),
])
def test_short_conv(B, T, D, W, dt, lens, state, act, how):
    d = _conv_inputs(B, T, D, W, dt, lens, state, T + D)
    _conv_check(_conv_run(d, act, how), _conv_ref(d, act))


@pytest.mark.parametrize("lens", [(1, 1, 1), (0, 2, 1), (300, 2, 40)])
def test_short_conv_state_in_place_without_bias(lens):
    d = _conv_inputs(1, sum(lens), 64, 4, BF, lens, True, 3, bias=False)
    _conv_check(_conv_run(d, "silu", in_place=True), _conv_ref(d, "silu"))


def test_short_conv_sequences_do_not_reach_each_other():
    lens = (40, 3, 64, 2, 90)
    d = _conv_inputs(1, sum(lens), 64, 4, BF, lens, True, 6)
    for k in ("x", "dout"):
        d[k][0, 43:107:2], d[k][0, 44:107:2] = float("nan"), float("inf")
    d["init"][2], d["dfinal"][2] = float("nan"), float("inf")
    got = _conv_run(d, "silu")
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[43:107] = False
    for k in ("x", "dout"):
        d[k][0, 43:107] = 0
    d["init"][2] = d["dfinal"][2] = 0
    want = _conv_ref(d, "silu")
    for name in ("out", "dx"):
        assert_close(name, got[name][0][keep.cuda()], *(t[keep] for t in want[name]))
    for name in ("final", "dinit"):
        assert_close(name, got[name][[0, 1, 3, 4]], *(t[[0, 1, 3, 4]] for t in want[name]))


def test_short_conv_same_bits_every_time_and_on_another_stream():
    d = _conv_inputs(1, 2000, 96, 4, BF, (700, 0, 1299, 1), True, 6)
    a = _conv_run(d, "silu")
    b = _conv_run(d, "silu", stream=torch.cuda.Stream())
    for k, v in a.items():
        assert torch.equal(v, b[k]), k


def test_short_conv_gradient_against_differences():
    d = _conv_inputs(2, 30, 20, 4, F, None, True, 13)
    got = _conv_run(d, "silu")

    def loss(k, e, v):
        r = _conv_ref(dict(d, **{k: d[k].double() + e * v}), "silu")
        return float((r["out"][0].reshape(d["dout"].shape) * d["dout"].double()).sum() + (r["final"][0] * d["dfinal"].double()).sum())

    for k, dk in {"x": "dx", "w": "dweight", "b": "dbias", "init": "dinit"}.items():
        v = torch.randn(d[k].shape, generator=_gen(3), dtype=torch.float64)
        want = (loss(k, 1e-5, v) - loss(k, -1e-5, v)) / 2e-5
        dot = got[dk].cpu().double().reshape(v.shape) * v
        assert abs(float(dot.sum()) - want) <= 2.0 ** -12 * float(dot.abs().sum()) + 1e-6, k


def test_offsets_beyond_32_bits():
    # rows 2^21 elements apart: the last row starts past element 2^31
    rows, D = 1100, 64
    wide = torch.zeros(1, rows, 1 << 21, dtype=BF, device="cuda")
    part = wide[:, :, 5:5 + D]
    part.copy_(torch.randn(1, rows, D, generator=_gen(2)).to(BF))
    dense = part.contiguous()
    w, A, tb = torch.randn(D, 4, generator=_gen(3)).cuda(), torch.zeros(1).cuda(), torch.full((1, D), -2.0).cuda()
    outs = []
    for t in (part, dense):
        o = [torch.empty_like(dense) for _ in range(3)]
        t4 = t.unflatten(2, (1, D))
        glr.glr_fwd(t4, t4, t4, o[0].unflatten(2, (1, D)), A, tb, -5.0)
        short_conv.short_conv_fwd(t, w, None, o[1])
        layer_norm.layer_norm_fwd(t, None, None, 1e-5, o[2])
        outs.append(o)
    _status()
    for a, b in zip(*outs):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=0)   # two roundings to bf16


# ------------------------------------------------------------------ together
def test_block_trains_and_serves():
    from gated_delta_rule_52_gb300 import block
    gen = _gen(0)
    blocks = [block.Block(kind, 128, gen) for kind in ("glr", "kda")]
    losses = block.train(blocks, 25, 2, 200, gen)
    assert all(b < a for a, b in zip(losses[::8], losses[8::8])), losses
    u = torch.randn(2, 90, 128, generator=gen).to("cuda", BF)
    whole, stepped = block.serve(blocks, u, 90), block.serve(blocks, u, 70)
    _status()
    # both round every operator's output to bf16 (2^-9 each, a dozen in a row), the delta
    # rule's chunked form besides holds its operands in fp16
    assert float((whole.float() - stepped.float()).norm()) <= 2.0 ** -6 * float(whole.float().norm())
    # and what was trained is what is served
    h = u
    for b in blocks:
        h = b.train(h)
    assert float((whole.float() - h.float()).norm()) <= 2.0 ** -6 * float(whole.float().norm())
