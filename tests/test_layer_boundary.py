"""Refusals of the operators around the delta rule, without a GPU: every call here carries
at least one invalid argument (or has no work), so nothing touches a device; and the 64-bit
references' gradients against differentiation of their formulas."""
import ctypes
import math

import pytest
import torch

from gated_delta_rule_52_gb300 import _args, glr, kda, layer_norm, short_conv
from gated_delta_rule_52_gb300 import build as kbuild
from tests import layer_ref as ref

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(20)]   # never dereferenced
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    kbuild.build_library()
    return kda.lib()


def glr_fwd(L, **o):
    a = dict(x=P[0], i=P[1], g=P[2], xs=64, is_=64, gs=64, out=P[3], os=64, dt=1, A=P[4], tb=P[5], lb=-5.0, ub=0,
             init=None, fin=None, sd=0, cu=None, ns=0, B=1, T=8, H=2, K=32, ck=None)
    a.update(o)
    return L.kda_glr_fwd(a["x"], a["i"], a["g"], a["xs"], a["is_"], a["gs"], a["out"], a["os"], a["dt"], a["A"], a["tb"],
                         a["lb"], a["ub"], a["init"], a["fin"], a["sd"], a["cu"], a["ns"], a["B"], a["T"], a["H"],
                         a["K"], a["ck"], None)


def glr_bwd(L, **o):
    a = dict(x=P[0], i=P[1], g=P[2], xs=64, is_=64, gs=64, dt=1, A=P[4], tb=P[5], lb=-5.0, ub=0, init=None, sd=0,
             ck=None, dout=P[6], ds=64, dfin=None, cu=None, ns=0, B=1, T=8, H=2, K=32, dx=P[7], di=P[8], dg=P[9],
             dA=P[10], dtb=P[11], dinit=None)
    a.update(o)
    return L.kda_glr_bwd(a["x"], a["i"], a["g"], a["xs"], a["is_"], a["gs"], a["dt"], a["A"], a["tb"], a["lb"], a["ub"],
                         a["init"], a["sd"], a["ck"], a["dout"], a["ds"], a["dfin"], a["cu"], a["ns"], a["B"], a["T"],
                         a["H"], a["K"], a["dx"], a["di"], a["dg"], a["dA"], a["dtb"], a["dinit"], None)


@pytest.mark.parametrize("call", [glr_fwd, glr_bwd])
def test_glr_refusals(L, call):
    for name in ("x", "i", "g", "A", "tb"):
        assert call(L, **{name: None}) == kda.KDA_ERR_NULL
        assert call(L, **{name: ODD}) == kda.KDA_ERR_ALIGN
    for o in (dict(B=-1), dict(T=-1), dict(H=-1), dict(K=-2), dict(B=2, cu=P[12], ns=2), dict(cu=P[12], ns=0),
              dict(B=1 << 20, T=1 << 12), dict(H=1 << 20, K=1 << 12), dict(B=1 << 20, T=1, H=1 << 6, K=1 << 7),
              dict(xs=-64), dict(gs=-1), dict(B=1 << 62, T=1 << 62)):
        assert call(L, **o) == kda.KDA_ERR_SHAPE, o
    for o in (dict(dt=0), dict(dt=4), dict(init=P[13], sd=0), dict(init=P[13], sd=3), dict(sd=9)):
        assert call(L, **o) == kda.KDA_ERR_DTYPE, o
    for lb in (-5.5, 0.1, float("nan")):
        assert call(L, lb=lb) == kda.KDA_ERR_VALUE
    assert call(L, cu=ODD, ns=1) == kda.KDA_ERR_ALIGN
    assert call(L, init=ODD, sd=2) == kda.KDA_ERR_ALIGN


def test_glr_refusals_of_one_direction(L):
    assert glr_fwd(L, out=None) == kda.KDA_ERR_NULL
    assert glr_fwd(L, os=63) == kda.KDA_ERR_SHAPE
    assert glr_fwd(L, fin=P[13]) == kda.KDA_ERR_DTYPE
    assert glr_fwd(L, ck=ODD) == kda.KDA_ERR_ALIGN
    assert glr_fwd(L, B=0, x=None, i=None, g=None, out=None) == kda.KDA_OK
    for name in ("dout", "dx", "di", "dg", "dA", "dtb"):
        assert glr_bwd(L, **{name: None}) == kda.KDA_ERR_NULL
        assert glr_bwd(L, **{name: ODD}) == kda.KDA_ERR_ALIGN
    for name in ("ck", "dfin", "dinit"):
        assert glr_bwd(L, **{name: ODD}) == kda.KDA_ERR_ALIGN
    assert glr_bwd(L, ds=-1) == kda.KDA_ERR_SHAPE
    assert glr_bwd(L, H=0, dA=None, dtb=None) == kda.KDA_OK


def test_layer_norm_refusals(L):
    def fwd(x=P[0], xs=64, w=P[1], b=P[2], eps=1e-5, out=P[3], os=64, m=None, r=None, dt=1, rows=4, D=64):
        return L.kda_layer_norm_fwd(x, xs, w, b, eps, out, os, m, r, dt, rows, D, None)

    def bwd(dy=P[4], ds=64, x=P[0], xs=64, w=P[1], m=P[5], r=P[6], dx=P[7], dw=P[8], db=P[9], dt=1, rows=4, D=64):
        return L.kda_layer_norm_bwd(dy, ds, x, xs, w, m, r, dx, dw, db, dt, rows, D, None)

    for call, names in ((fwd, ("x", "out")), (bwd, ("dy", "x", "m", "r", "dx"))):
        for name in names:
            assert call(**{name: None}) == kda.KDA_ERR_NULL
            assert call(**{name: ODD}) == kda.KDA_ERR_ALIGN
        for o in (dict(rows=-1), dict(D=-1), dict(D=0), dict(rows=1 << 31), dict(D=1 << 31), dict(xs=-1)):
            assert call(**o) == kda.KDA_ERR_SHAPE, o
        for dt in (0, 4, -1):
            assert call(dt=dt) == kda.KDA_ERR_DTYPE
        assert call(w=ODD) == kda.KDA_ERR_ALIGN
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(eps=eps) == kda.KDA_ERR_VALUE
    assert fwd(os=63) == kda.KDA_ERR_SHAPE
    assert bwd(ds=-1) == kda.KDA_ERR_SHAPE
    assert fwd(rows=0, x=None, out=None) == kda.KDA_OK
    assert bwd(D=0, rows=0) == kda.KDA_OK


def test_short_conv_refusals(L):
    def fwd(x=P[0], xs=64, w=P[1], b=P[2], act=1, out=P[3], os=64, dt=1, init=None, fin=None, cu=None, ns=0, B=1, T=8,
            D=64, W=4):
        return L.kda_short_conv_fwd(x, xs, w, b, act, out, os, dt, init, fin, cu, ns, B, T, D, W, None)

    def bwd(x=P[0], xs=64, w=P[1], b=P[2], act=1, dt=1, init=None, dy=P[4], ds=64, dfin=None, cu=None, ns=0, B=1, T=8,
            D=64, W=4, dx=P[5], dw=P[6], db=P[7], dinit=None):
        return L.kda_short_conv_bwd(x, xs, w, b, act, dt, init, dy, ds, dfin, cu, ns, B, T, D, W, dx, dw, db, dinit, None)

    for call, names in ((fwd, ("x", "w", "out")), (bwd, ("x", "w", "dy", "dx", "dw"))):
        for name in names:
            assert call(**{name: None}) == kda.KDA_ERR_NULL
            assert call(**{name: ODD}) == kda.KDA_ERR_ALIGN
        for W in (-1, 0, 1, 5):
            assert call(W=W) == kda.KDA_ERR_UNSUPPORTED
        for act in (-1, 2):
            assert call(act=act) == kda.KDA_ERR_VALUE
        for dt in (0, 4):
            assert call(dt=dt) == kda.KDA_ERR_DTYPE
        for o in (dict(B=-1), dict(T=-1), dict(D=-1), dict(D=1 << 31), dict(B=2, cu=P[12], ns=2), dict(cu=P[12], ns=0),
                  dict(B=1 << 20, T=1 << 12), dict(B=1 << 20, T=1, D=1 << 12), dict(xs=-1)):
            assert call(**o) == kda.KDA_ERR_SHAPE, o
        for name in ("b", "init", "cu"):
            assert call(**{name: ODD}, **({"ns": 1} if name == "cu" else {})) == kda.KDA_ERR_ALIGN
    assert fwd(os=63) == kda.KDA_ERR_SHAPE
    assert fwd(fin=ODD) == kda.KDA_ERR_ALIGN
    assert bwd(ds=-1) == kda.KDA_ERR_SHAPE
    assert bwd(dfin=ODD) == kda.KDA_ERR_ALIGN and bwd(dinit=ODD) == kda.KDA_ERR_ALIGN
    assert fwd(B=0, x=None, out=None) == kda.KDA_OK
    assert bwd(D=0, w=None, dw=None) == kda.KDA_OK


def test_bindings_refuse():
    x = torch.zeros(1, 4, 2, 8, dtype=torch.bfloat16)
    A, tb = torch.zeros(2), torch.zeros(2, 8)
    with pytest.raises(ValueError):
        glr.glr_fwd(x, x, x, x, A, tb, -5.0)                       # not on a GPU
    with pytest.raises(ValueError):
        glr.glr_fwd(x.double(), x, x, x, A, tb, -5.0)              # element type
    with pytest.raises(ValueError):
        glr.glr_bwd(x[0], x, x, A, tb, -5.0, x)                    # dimensions
    with pytest.raises(TypeError):
        glr.glr_fwd(None, x, x, x, A, tb, -5.0)
    with pytest.raises(ValueError):
        layer_norm.layer_norm_fwd(x, None, None, 1e-5, x)
    with pytest.raises(ValueError):
        short_conv.short_conv_fwd(x, torch.zeros(8, 4), None, x)   # dimensions
    with pytest.raises(ValueError):
        short_conv.short_conv_bwd(x[0], torch.zeros(8), None, x[0])
    assert glr.checkpoint_shape(2, 33, 3, 5) == (2, 3, 5) and glr.checkpoint_shape(1, 64, 1, 1) == (1, 1, 1)
    assert glr.checkpoint_shape(1, 0, 1, 1) == (0, 1, 1)


class _SaysGpu(torch.Tensor):                                      # a CPU tensor that says it is on a GPU
    is_cuda = True


def test_row_strides():
    def stride(t, lead):
        f = t.as_subclass(_SaysGpu)
        return _args.rows("t", f, t.dtype, t.shape, lead, math.prod(t.shape[lead:]))

    t = torch.zeros(3, 5, 4, 8)
    assert stride(t, 2) == 32
    assert stride(torch.zeros(3, 5, 100)[:, :, 3:35].unflatten(2, (4, 8)), 2) == 100
    assert stride(torch.zeros(1, 5, 100)[:, :, 3:35].unflatten(2, (4, 8)), 2) == 100
    assert stride(torch.zeros(3, 5, 3, 4, 8)[:, :, 1], 2) == 96
    assert stride(torch.zeros(1, 1, 32).expand(3, 5, 32), 2) == 0
    assert stride(torch.zeros(7, 0), 1) == 0
    for bad in (t.transpose(0, 1), t.transpose(2, 3), t[..., ::2], torch.zeros(3, 7, 4, 8)[:, :5]):
        with pytest.raises(ValueError):
            stride(bad, 2)


@pytest.mark.parametrize("lb", [-5.0, None])
def test_reference_gradients_against_autograd(lb):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    seqs = ref.bounds_of(1, 12, [5, 0, 7])
    x, i, gg, A, tb, init, do, df = n(12, 2, 3), n(12, 2, 3), n(12, 2, 3), n(2), n(2, 3), n(3, 2, 3), n(12, 2, 3), n(3, 2, 3)
    got = ref.glr(x, i, gg, A, tb, lb, seqs, init, do, df)
    v = [t.clone().requires_grad_() for t in (x, i, gg, A, tb, init)]
    outs, fins = [], []
    e, u = v[3].exp()[:, None], v[2] + v[4]
    a = (-e * torch.log1p(u.exp()) if lb is None else lb * torch.sigmoid(e * u)).exp()
    for k, (lo, hi) in enumerate(seqs):
        h = v[5][k]
        for t in range(lo, hi):
            h = a[t] * h + torch.sigmoid(v[1][t]) * v[0][t]
            outs.append(h)
        fins.append(h)
    grads = torch.autograd.grad((torch.stack(outs) * do).sum() + (torch.stack(fins) * df).sum(), v)
    for name, want in zip(("dx", "di", "dg", "dA_log", "ddt_bias", "dinit"), grads):
        torch.testing.assert_close(got[name][0], want, rtol=1e-10, atol=1e-12)
    # layer norm and the convolution
    x, w, b, dy = n(4, 9), n(9), n(9), n(4, 9)
    v = [t.clone().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(torch.nn.functional.layer_norm(v[0], (9,), v[1], v[2], 1e-5), v, dy)
    r = ref.norm(x, w, b, 1e-5, dy)
    for name, want in zip(("dx", "dweight", "dbias"), grads):
        torch.testing.assert_close(r[name][0], want, rtol=1e-9, atol=1e-11)
    seqs = ref.bounds_of(1, 9, [2, 0, 7])
    x, w, b, init, dy, df = n(9, 5), n(5, 4), n(5), n(3, 3, 5), n(9, 5), n(3, 3, 5)
    v = [t.clone().requires_grad_() for t in (x, w, b, init)]
    loss = 0
    for k, (lo, hi) in enumerate(seqs):
        rows = torch.cat([v[3][k], v[0][lo:hi]])
        if hi > lo:
            y = torch.nn.functional.conv1d(rows.T[None], v[1][:, None], v[2], groups=5)[0].T
            loss = loss + (torch.nn.functional.silu(y) * dy[lo:hi]).sum()
        loss = loss + (rows[hi - lo:] * df[k]).sum()
    grads = torch.autograd.grad(loss, v)
    r = ref.conv(x, w, b, seqs, True, init, dy, df)
    for name, want in zip(("dx", "dweight", "dbias", "dinit"), grads):
        torch.testing.assert_close(r[name][0], want, rtol=1e-9, atol=1e-11)
