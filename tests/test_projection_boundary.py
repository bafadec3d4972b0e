"""Refusals of the operators around a layer's projections, without a GPU: every call here
carries at least one invalid argument (or has no work), so nothing touches a device; calls
whose tensors or stream are elsewhere; and the 64-bit references against differentiation and
torch's own 8-bit types."""
import ctypes

import pytest
import torch

from gated_delta_rule_52_gb300 import _args, fp8, kda, rms_norm
from gated_delta_rule_52_gb300 import build as kbuild
from tests import projection_ref as ref
from tests.projection_ref import E4, E5, E8
from tests.test_layer_devices import _OnGpu, _Stream

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(20)]   # never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    kbuild.build_library()
    return kda.lib()


def test_rms_norm_refusals(L):
    def fwd(x=P[0], xs=64, r=P[1], rs=64, w=P[2], eps=1e-6, out=P[3], os=64, od=1, s=None, ss=0, ro=P[4], ros=64, rstd=P[5], dt=1,
            rows=4, D=64):
        return L.kda_rms_norm_fwd(x, xs, r, rs, w, eps, out, os, od, s, ss, ro, ros, rstd, dt, rows, D, None)

    def bwd(dy=P[0], ds=64, x=P[1], xs=64, w=P[2], rstd=P[3], dr=P[4], drs=64, dx=P[5], dw=P[6], dt=1, rows=4, D=64):
        return L.kda_rms_norm_bwd(dy, ds, x, xs, w, rstd, dr, drs, dx, dw, dt, rows, D, None)

    for call, names, odd in ((fwd, ("x", "out"), ("x", "r", "w", "out", "ro", "rstd")),
                             (bwd, ("dy", "x", "rstd", "dx"), ("dy", "x", "w", "rstd", "dr", "dx", "dw"))):
        for name in names:
            assert call(**{name: None}) == kda.KDA_ERR_NULL
        for name in odd:
            assert call(**{name: ODD}) == kda.KDA_ERR_ALIGN
        for o in (dict(rows=-1), dict(D=-1), dict(D=0), dict(rows=1 << 31), dict(D=1 << 31), dict(xs=-1)):
            assert call(**o) == kda.KDA_ERR_SHAPE, o
        for dt in (0, 4, 5, -1):
            assert call(dt=dt) == kda.KDA_ERR_DTYPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(eps=eps) == kda.KDA_ERR_VALUE
    for o in (dict(os=63), dict(ros=63), dict(rs=-1), dict(od=4, s=P[6], ss=0), dict(od=4, s=P[6], ss=1, D=129, xs=129, os=129, ros=129)):
        assert fwd(**o) == kda.KDA_ERR_SHAPE, o
    assert fwd(od=2) == kda.KDA_ERR_DTYPE and fwd(od=6) == kda.KDA_ERR_DTYPE
    assert fwd(od=4) == kda.KDA_ERR_NULL and fwd(r=None) == kda.KDA_ERR_NULL
    assert bwd(ds=-1) == kda.KDA_ERR_SHAPE and bwd(drs=-1) == kda.KDA_ERR_SHAPE
    assert fwd(rows=0, x=None, out=None) == kda.KDA_OK
    assert bwd(D=0, rows=0) == kda.KDA_OK and bwd(rows=0, dw=None) == kda.KDA_OK


def test_quantize_refusals(L):
    def quant(x=P[0], xs=64, dt=1, q=P[1], qs=64, s=P[2], ss=1, qt=P[3], qts=4, st=P[4], sts=1, qd=4, tile=0, rows=4, cols=64):
        return L.kda_fp8_quantize(x, xs, dt, q, qs, s, ss, qt, qts, st, sts, qd, tile, rows, cols, None)

    def back(q=P[0], qs=64, qd=4, s=P[1], ss=1, tile=0, out=P[2], os=64, dt=1, rows=4, cols=64):
        return L.kda_fp8_dequantize(q, qs, qd, s, ss, tile, out, os, dt, rows, cols, None)

    for o in (dict(x=None), dict(s=None), dict(st=None), dict(q=None), dict(qt=None), dict(q=None, s=None, qt=None, st=None)):
        assert quant(**o) == kda.KDA_ERR_NULL, o
    for o in (dict(q=None), dict(s=None), dict(out=None)):
        assert back(**o) == kda.KDA_ERR_NULL, o
    for call in (quant, back):
        for o in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=1 << 31), dict(rows=1 << 30, cols=1 << 30)):
            assert call(**o) == kda.KDA_ERR_SHAPE, o
        for o in (dict(dt=0), dict(dt=4), dict(qd=1), dict(qd=6), dict(qd=0)):
            assert call(**o) == kda.KDA_ERR_DTYPE, o
        assert call(rows=0) == kda.KDA_OK and call(cols=0) == kda.KDA_OK
    for o in (dict(xs=-1), dict(qs=63), dict(ss=0), dict(qts=3), dict(sts=0)):
        assert quant(**o) == kda.KDA_ERR_SHAPE, o
    for o in (dict(qs=-1), dict(ss=-1), dict(os=63)):
        assert back(**o) == kda.KDA_ERR_SHAPE, o
    assert quant(x=ODD) == kda.KDA_ERR_ALIGN and back(out=ODD) == kda.KDA_ERR_ALIGN


def test_matmul_refusals(L):
    def mm(a=P[0], as_=256, ad=4, sa=P[1], sas=4, at=0, b=P[2], bs=256, bd=5, sb=P[3], sbs=4, bt=1, out=P[4], os=200, add=P[5],
           adds=200, dt=1, M=8, N=200, K=256):
        return L.kda_fp8_matmul(a, as_, ad, sa, sas, at, b, bs, bd, sb, sbs, bt, out, os, add, adds, dt, M, N, K, None)

    for name in ("a", "sa", "b", "sb", "out"):
        assert mm(**{name: None}) == kda.KDA_ERR_NULL
    for o in (dict(a=HALF), dict(b=HALF), dict(sa=ODD), dict(sb=ODD), dict(out=ODD), dict(add=ODD), dict(as_=264), dict(bs=257),
              dict(sas=6), dict(sbs=3)):
        assert mm(**o) == kda.KDA_ERR_ALIGN, o
    for o in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(as_=240), dict(bs=0), dict(sas=1),
              dict(sbs=0), dict(os=199), dict(adds=-1), dict(M=(1 << 31) - 1, N=(1 << 31) - 1, os=1 << 31)):
        assert mm(**o) == kda.KDA_ERR_SHAPE, o
    for o in (dict(ad=1), dict(bd=2), dict(ad=6), dict(dt=4), dict(dt=0)):
        assert mm(**o) == kda.KDA_ERR_DTYPE, o
    assert mm(M=0, a=None, out=None) == kda.KDA_OK and mm(N=0, b=None, out=None) == kda.KDA_OK


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=torch.uint8 if dtype in (E4, E5, E8) else dtype).view(dtype).as_subclass(_OnGpu)


BF = torch.bfloat16
CALLS = {
    "rms_norm_fwd": (rms_norm.rms_norm_fwd, lambda: {
        "x": _t(6, 256, dtype=BF), "weight": _t(256), "eps": 1e-6, "out": _t(6, 256, dtype=E4), "residual": _t(6, 256, dtype=BF),
        "residual_out": _t(6, 256, dtype=BF), "rstd": _t(6), "scales": _t(6, 2, dtype=E8), "stream": _Stream(0)}),
    "rms_norm_bwd": (rms_norm.rms_norm_bwd, lambda: {
        "dout": _t(6, 8), "x": _t(6, 8), "weight": _t(8), "rstd": _t(6), "dresidual": _t(6, 8), "stream": _Stream(0)}),
    "fp8_quantize": (fp8.quantize, lambda: {
        "x": _t(6, 256), "q": _t(6, 256, dtype=E5), "scales": _t(6, 2, dtype=E8), "qt": _t(256, 6, dtype=E5),
        "scales_t": _t(256, 1, dtype=E8), "stream": _Stream(0)}),
    "fp8_dequantize": (fp8.dequantize, lambda: {
        "q": _t(300, 256, dtype=E5), "scales": _t(3, 2, dtype=E8), "out": _t(300, 256), "stream": _Stream(0)}),
    "fp8_matmul": (fp8.matmul, lambda: {
        "a": _t(2, 3, 512, dtype=E5), "a_scales": _t(2, 3, 4, dtype=E8), "b": _t(200, 512, dtype=E4), "b_scales": _t(2, 4, dtype=E8),
        "out": _t(2, 3, 200), "add": _t(2, 3, 200), "stream": _Stream(0)}),
}


@pytest.fixture
def calls(monkeypatch):
    made, current = [], [0]
    monkeypatch.setattr(_args, "entry", lambda name: lambda *a: made.append(name) or 0)
    monkeypatch.setattr(_args, "current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(_args, "new", lambda stream, t, *shapes: [None if s is None else _t(*s, dtype=t.dtype) for s in shapes])
    return made, current


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_and_the_stream_on_the_current_gpu(name, calls):
    made, current = calls
    call, arguments = CALLS[name]
    call(**arguments())
    assert made == ["kda_" + name]
    made.clear()
    for k, v in arguments().items():
        if not isinstance(v, (torch.Tensor, _Stream)):
            continue
        a = arguments()
        if k == "stream":
            a[k] = _Stream(1)
        else:
            a[k].gpu = 1
        with pytest.raises(ValueError, match="cuda:1"):
            call(**a)
        assert not made, k
    current[0] = 1
    with pytest.raises(ValueError, match="cuda:1"):
        call(**arguments())
    assert not made


# arguments changed to a wrong shape, type or absence
BAD = {
    "rms_norm_fwd": [{"scales": None}, {"scales": _t(6, 1, dtype=E8)}, {"scales": _t(6, 2)}, {"out": _t(6, 256)}, {"residual": None},
                     {"weight": _t(255)}, {"residual": _t(6, 256)}, {"residual_out": _t(5, 256, dtype=BF)}, {"rstd": _t(5)},
                     {"out": _t(6, 256, dtype=BF)}, {"x": _t(6, 256, dtype=torch.float64)}, {"out": None}],
    "rms_norm_bwd": [{"rstd": _t(6, 1)}, {"dout": _t(6, 9)}, {"dresidual": _t(6, 8, dtype=BF)}, {"weight": _t(8, dtype=BF)}],
    "fp8_quantize": [{"q": None}, {"scales": None}, {"scales_t": None}, {"qt": None}, {"qt": _t(256, 6, dtype=E4)}, {"tile": True},
                     {"q": None, "scales": None, "qt": None, "scales_t": None}, {"x": _t(256)}, {"q": _t(6, 255, dtype=E5)},
                     {"q": _t(6, 256)}, {"scales_t": _t(6, 2, dtype=E8)}],
    "fp8_dequantize": [{"scales": _t(300, 3, dtype=E8)}, {"scales": _t(3, 2)}, {"out": _t(256, 300)}, {"q": _t(300, 256)}, {"scales": None},
                       {"out": _t(300, 256, dtype=E4)}],
    "fp8_matmul": [{"a": _t(2, 3, 500, dtype=E5)}, {"b": _t(200, 2, 256, dtype=E4)}, {"out": _t(6, 200)}, {"add": _t(2, 3, 200, dtype=BF)},
                   {"a_scales": _t(2, 3, 3, dtype=E8)}, {"b_scales": _t(199, 4, dtype=E8)}, {"b": _t(200, 512)}, {"a": _t(512, dtype=E5)},
                   {"out": _t(2, 3, 200, dtype=E4)}, {"out": _t(2, 3, 400)[..., ::2]}],
}


@pytest.mark.parametrize("name", BAD)
def test_bindings_refuse(name, calls):
    made, _ = calls
    call, arguments = CALLS[name]
    for bad in BAD[name]:
        with pytest.raises((ValueError, TypeError)):
            call(**{**arguments(), **bad})
        assert not made, bad


# matrices on the current stream, whose checks are the short ones
PLAIN = {
    "rms_norm_fwd": lambda: {k: v for k, v in CALLS["rms_norm_fwd"][1]().items() if k != "stream"},
    "rms_norm_bwd": lambda: {k: v for k, v in CALLS["rms_norm_bwd"][1]().items() if k != "stream"},
    "fp8_quantize": lambda: {k: v for k, v in CALLS["fp8_quantize"][1]().items() if k != "stream"},
    "fp8_dequantize": lambda: {k: v for k, v in CALLS["fp8_dequantize"][1]().items() if k != "stream"},
    "fp8_matmul": lambda: {"a": _t(6, 512, dtype=E5), "a_scales": _t(6, 4, dtype=E8), "b": _t(200, 512, dtype=E4),
                           "b_scales": _t(2, 4, dtype=E8), "out": _t(6, 200), "add": _t(6, 200)},
}
NEW = {"rms_norm_bwd": (9, 10)}   # pointers of tensors that the call makes
WIDER = {   # strides that the short checks pass on, and those of which they make nothing
    "rms_norm_fwd": [{"x": _t(6, 300, dtype=BF)[:, 9:265]}, {"out": _t(6, 256, dtype=BF), "scales": None}, {"residual": _t(1, 256, dtype=BF).expand(6, 256)},
                     {"residual": None, "residual_out": None}, {"weight": None, "rstd": None}],
    "rms_norm_bwd": [{"x": _t(6, 12)[:, 1:9]}, {"dout": _t(1, 8).expand(6, 8), "dresidual": None}, {"weight": None}, {"want_dweight": False},
                     {"weight": None, "want_dweight": True}, {"dresidual": _t(6, 9)[:, :8]}],
    "fp8_quantize": [{"x": _t(6, 300)[:, :256]}, {"q": None, "scales": None}, {"qt": None, "scales_t": None}, {"scales": _t(6, 4, dtype=E8)[:, :2]},
                     {"tile": True, "scales": _t(1, 2, dtype=E8), "scales_t": _t(2, 1, dtype=E8)}],
    "fp8_dequantize": [{"q": _t(300, 272, dtype=E5)[:, :256]}, {"scales": _t(300, 2, dtype=E8)}, {"out": _t(300, 999, dtype=BF)[:, 1:257]}],
    "fp8_matmul": [{"add": None}, {"add": _t(200).expand(6, 200)}, {"out": _t(6, 400)[:, 200:]}, {"b_scales": _t(200, 8, dtype=E8)[:, :4]},
                   {"a_scales": _t(1, 4, dtype=E8)}, {"a": _t(0, 512, dtype=E5), "a_scales": _t(0, 4, dtype=E8), "out": _t(0, 200), "add": None}],
}
WRONG = {
    "rms_norm_fwd": [b for b in BAD["rms_norm_fwd"]] + [{"x": _t(6, 512, dtype=BF)[:, ::2]}],
    "rms_norm_bwd": [b for b in BAD["rms_norm_bwd"]] + [{"x": _t(6, 16)[:, ::2]}, {"dout": _t(8, 6).T}, {"dout": None}],
    "fp8_quantize": [b for b in BAD["fp8_quantize"]] + [{"qt": _t(6, 256, dtype=E5).T}, {"scales": _t(6, 4, dtype=E8)[:, ::2]}],
    "fp8_dequantize": [b for b in BAD["fp8_dequantize"]] + [{"out": _t(256, 300).T}],
    "fp8_matmul": [{"a": _t(6, 500, dtype=E5)}, {"b": _t(200, 512)}, {"b": _t(199, 512, dtype=E4)}, {"out": _t(6, 200, dtype=E4)}, {"out": _t(5, 200)},
                   {"add": _t(6, 200, dtype=BF)}, {"add": _t(200)}, {"a_scales": _t(6, 3, dtype=E8)}, {"a_scales": _t(2, 4, dtype=E8)},
                   {"b_scales": _t(200, 4)}, {"b_scales": None}, {"out": _t(6, 400)[:, ::2]}, {"add": _t(200, 6).T}, {"a": None}],
}


@pytest.fixture
def passed(calls, monkeypatch):
    """What reaches the entry points, on the current stream and on a given one."""
    seen = []
    monkeypatch.setattr(_args, "entry", lambda name: lambda *a: seen.append((name, *a[:-1])) or 0)
    monkeypatch.setattr(_args, "stream_handle", lambda stream, dev: 0)
    return seen


@pytest.mark.parametrize("name", PLAIN)
def test_short_checks_pass_on_what_the_long_ones_do(name, passed):
    call = CALLS[name][0]
    for change in ({}, *WIDER[name]):
        a = {**PLAIN[name](), **change}
        call(**a)
        call(**a, stream=_Stream(0))
        assert len(passed) == 2 and passed[0][0] == "kda_" + name
        short, long = ([bool(v) if i in NEW.get(name, ()) else v for i, v in enumerate(c)] for c in passed)
        assert short == long, change
        passed.clear()


@pytest.mark.parametrize("name", PLAIN)
def test_short_checks_refuse(name, passed, calls):
    call, current = CALLS[name][0], calls[1]
    for bad in WRONG[name]:
        for stream in ({}, {"stream": _Stream(0)}):
            with pytest.raises((ValueError, TypeError)):
                call(**{**PLAIN[name](), **bad}, **stream)
        assert not passed, bad
    for k, v in PLAIN[name]().items():
        if isinstance(v, torch.Tensor):
            for gpu in (1, -1):
                a = PLAIN[name]()
                a[k].gpu = gpu
                with pytest.raises(ValueError):
                    call(**a)
                assert not passed, k
    current[0] = 1
    with pytest.raises(ValueError, match="cuda:1"):
        call(**PLAIN[name]())
    assert not passed


def test_empty_lays_rows_out_for_the_product():
    q, s = fp8.empty(5, 300, E5, device="cpu")
    assert q.shape == (5, 300) and q.stride() == (304, 1) and q.dtype == E5
    assert s.shape == (5, 3) and s.stride() == (4, 1) and s.dtype == E8
    q, s = fp8.empty(129, 128, tile=True, device="cpu")
    assert q.shape == (129, 128) and q.is_contiguous() and s.shape == (2, 1) and s.stride() == (4, 1)
    with pytest.raises(ValueError):
        fp8.empty(1, 1, torch.float32, device="cpu")


@pytest.mark.parametrize("to", [E4, E5])
def test_reference_rounds_like_the_type(to):
    """All values of the type, and neighbours of the points half-way between two."""
    all_ = torch.arange(256, dtype=torch.uint8).view(to).double()
    v = all_[all_.isfinite()].unique()
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = torch.nn.functional.pad(x, (0, -len(x) % 128)).view(-1, 128)
    x = torch.cat([x, torch.full((len(x), 1), ref.FORMAT[to][2])], 1)[:, 1:].contiguous()   # the largest in every block: scale 1
    got, e = ref.quantized(x, to)
    assert (e == 0).all()
    assert torch.equal(got, x.float().to(to).double())


@pytest.mark.parametrize("to", [E4, E5])
def test_reference_scales(to):
    most = ref.FORMAT[to][2]
    for top, want in ((most, 0), (most * (1 + 2.0 ** -23), 1), (most / 2, -1), (most * 2.0 ** 30, 30), (0.0, 0), (2.0 ** -127, 0),
                      (2.0 ** -126, -126), (1.0, -8 if to == E4 else -15), (3.4e38, 120 if to == E4 else 113)):
        assert ref.scale_exponent(top, to) == want, top
    x = torch.zeros(130, 200, dtype=torch.float64)
    x[0, 0], x[129, 199], x[1, 1] = most, most / 4, float("inf")
    assert ref.exponents(x, to).shape == (130, 2) and ref.exponents(x, to, True).tolist() == [[0, 0], [0, -2]]


def test_reference_gradients_against_autograd():
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy, dres = n(4, 9), n(9), n(4, 9), n(4, 9)
    v = [t.clone().requires_grad_() for t in (x, w)]
    r = (v[0].square().mean(-1) + 1e-6).rsqrt()
    want = torch.autograd.grad((v[0] * r[:, None] * v[1] * dy).sum() + (v[0] * dres).sum(), v)
    h, y, rr = ref.rms(x, None, w, 1e-6)
    for got, ww in zip(ref.rms_grads(h, w, rr, dy, dres), want):
        torch.testing.assert_close(got, ww, rtol=1e-10, atol=1e-12)
    # and against differences of the formula
    f = lambda t: float((ref.rms(t, None, w, 1e-6)[1] * dy).sum() + (t * dres).sum())  # noqa: E731
    dx = ref.rms_grads(h, w, rr, dy, dres)[0]
    for i, j in ((0, 0), (2, 5), (3, 8)):
        e = torch.zeros_like(x)
        e[i, j] = 1e-6
        assert abs((f(x + e) - f(x - e)) / 2e-6 - float(dx[i, j])) < 1e-7 * (1 + abs(float(dx[i, j])))
