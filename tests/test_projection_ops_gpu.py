"""The operators around a layer's projections on the GPU against 64-bit references: every
element of the product within a bound on fp32 sums, and exactly where sums are exact; the 8-bit
tensors bit for bit; the norm within its arithmetic's bound."""
import pytest
import torch

from gated_delta_rule_52_gb300 import fp8, kda, rms_norm
from tests import projection_ref as ref
from tests.layer_ref import D32, assert_close
from tests.projection_ref import E4, E5, E8

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _status():
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK


def _place(t, how):
    """The same values on the GPU: dense, or a slice of a wider tensor of NaN (one element off
    for "odd")."""
    if how == "dense":
        return t.cuda()
    pad = {"slice": 16, "odd": 1}[how]
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 2 * pad), float("nan"), dtype=t.dtype, device="cuda")
    part = wide[..., pad:pad + t.shape[-1]]
    part.copy_(t)
    return part


# ------------------------------------------------------------------ product
def _small_operand(rows, K, to, tile, g):
    """Whole numbers of -3 to 3 times scales of 1/2, 1 and 2: fp32 sums of them are exact."""
    q, s = fp8.empty(rows, K, to, tile)
    q.copy_(torch.randint(-3, 4, (rows, K), generator=g).float().cuda())
    s.view(torch.uint8).copy_(torch.randint(126, 129, s.shape, generator=g).to(torch.uint8).cuda())
    return q, s


def _normal_operand(rows, K, to, tile, g):
    x = torch.randn(rows, K, generator=g) * torch.randn(rows, 1, generator=g).exp()
    q, s = fp8.empty(rows, K, to, tile)
    fp8.quantize(x.cuda(), q, s, tile=tile)
    return q, s


MM = [  # M, N, K, a, b, a_tile, b_tile, dtype, add
    (1, 128, 128, E4, E4, False, True, F, False),
    (1, 1, 1, E4, E4, False, False, F, False),
    (16, 128, 512, E4, E4, False, False, F, True),
    (1, 1000, 4096, E4, E4, False, True, BF, False),
    (17, 129, 130, E4, E5, False, False, F, True),
    (2, 77, 65, E5, E4, True, False, HF, True),
    (33, 256, 1024, E5, E5, False, True, F, False),
    (64, 640, 2111, E4, E4, False, True, BF, True),
    (100, 300, 513, E5, E4, False, False, F, False),
    (128, 128, 128, E4, E4, True, True, F, False),
    (129, 257, 640, E4, E4, False, True, F, True),
    (255, 1537, 384, E4, E4, True, False, HF, False),
    (300, 100, 4097, E5, E4, False, False, F, True),
    (513, 700, 256, E4, E4, False, True, BF, False),
    (1100, 520, 1200, E4, E5, True, True, F, False),
    (400, 264, 640, E4, E4, False, True, BF, True),
    (700, 1000, 384, E5, E4, False, False, HF, True),
    (520, 1032, 4300, E4, E4, False, False, F, True),        # fp32 sums of several segments
    (2049, 513, 130, E4, E4, False, True, BF, True),
    (1537, 2048, 256, E4, E4, True, True, HF, False),
]


@pytest.mark.parametrize("M,N,K,ta,tb,a_tile,b_tile,dt,add", MM)
def test_exact_products(M, N, K, ta, tb, a_tile, b_tile, dt, add):
    g = _gen(M + N + K)
    a, sa = _small_operand(M, K, ta, a_tile, g)
    b, sb = _small_operand(N, K, tb, b_tile, g)
    plus = torch.randint(-8, 9, (M, N), generator=g).to(dt).cuda() if add else None
    out = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    fp8.matmul(a, sa, b, sb, out, add=plus)
    _status()
    want = ref.product(a, sa, b, sb, plus)
    assert float(want.abs().max()) < 2.0 ** 20              # in steps of 1/4: exact in fp32
    assert torch.equal(out.cpu(), want.float().to(dt))


@pytest.mark.parametrize("M,N,K,ta,tb,a_tile,b_tile,dt,add", MM)
def test_products(M, N, K, ta, tb, a_tile, b_tile, dt, add):
    g = _gen(M + N + K + 1)
    a, sa = _normal_operand(M, K, ta, a_tile, g)
    b, sb = _normal_operand(N, K, tb, b_tile, g)
    plus = torch.randn(M, N, generator=g).to(dt).cuda() if add else None
    out = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    fp8.matmul(a, sa, b, sb, out, add=plus)
    _status()
    want = ref.product(a, sa, b, sb, plus)
    assert_close("out", out, want, ref.product_bound(a, sa, b, sb) + 2.0 ** -23 * want.abs())


# ------------------------------------------------------------------ 8-bit tensors
QUANT = [  # rows, cols, dtype, type, how
    (1, 1, BF, E4, "dense"), (1, 128, F, E4, "dense"), (3, 130, HF, E5, "dense"), (128, 128, BF, E4, "dense"),
    (129, 257, BF, E4, "odd"), (200, 384, F, E5, "slice"), (77, 1000, HF, E4, "slice"), (300, 65, F, E4, "odd"),
    (130, 512, BF, E5, "dense"),
]


def _quant_input(rows, cols, dt, seed):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-20, 12, (rows, 1), generator=g).float())
    x = (x * torch.exp2(torch.randint(-3, 3, (1, cols), generator=g).float())).to(dt)
    x[rows // 2] = 0
    if cols > 100:
        x[-1, :60] = torch.tensor([448.0, 1.75, -448.0], dtype=dt).repeat(20)   # the border of a scale
    return x


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("rows,cols,dt,to,how", QUANT)
def test_quantize(rows, cols, dt, to, how, tile):
    x = _quant_input(rows, cols, dt, rows + cols)
    q, s = fp8.empty(rows, cols, to, tile)
    qt, st = fp8.empty(cols, rows, to, tile)
    fp8.quantize(_place(x, how), q, s, qt=qt, scales_t=st, tile=tile)
    _status()
    for name, got, gs, src in (("q", q, s, x), ("qt", qt, st, x.T)):
        want, e = ref.quantized(src.double(), to, tile)
        assert torch.equal(gs.cpu().view(torch.uint8), ref.bytes_of(e)), name
        assert torch.equal(ref.values(got, gs), want), name
        back = torch.full(got.shape, float("nan"), dtype=F, device="cuda")
        fp8.dequantize(got, gs, back)
        assert torch.equal(back.cpu().double(), want), name


@pytest.mark.parametrize("to", [E4, E5])
@pytest.mark.parametrize("dt", [BF, HF, F])
def test_quantize_what_is_not_finite(dt, to):
    """Infinities and NaN take no part in a scale and stay in their places; blocks of nothing
    else; magnitudes below the normal numbers."""
    g = _gen(7)
    x = torch.randn(140, 300, generator=g).to(dt)
    inf, nan = float("inf"), float("nan")
    x[0, 5], x[1, 130], x[2, 299], x[130, 0] = inf, -inf, nan, -nan
    x[3], x[4, :128], x[5, 128:] = nan, inf, -inf
    x[:, 77] = inf
    x[6] = 0
    if dt != HF:
        x[8, :128] = 2.0 ** -128                                # in e5m2 and e4m3 below a scale's reach: 0
    if dt == F:
        x[9, :128] = torch.randn(128, generator=g) * 2.0 ** -120
    q, s = fp8.empty(140, 300, to)
    qt, st = fp8.empty(300, 140, to)
    fp8.quantize(x.cuda(), q, s, qt=qt, scales_t=st)
    tq, ts = fp8.empty(140, 300, to, True)
    fp8.quantize(x.cuda(), tq, ts, tile=True)
    _status()
    z = torch.where(x.abs() < 2.0 ** -126, 0, x).double()       # what is not normal counts as 0
    for name, got, gs, src, tile in (("q", q, s, z, False), ("qt", qt, st, z.T, False), ("tile", tq, ts, z, True)):
        want, e = ref.quantized(src, to, tile)
        assert torch.equal(gs.cpu().view(torch.uint8), ref.bytes_of(e)), name
        have = ref.values(got, gs)
        assert torch.equal(have.isnan(), want.isnan()) and torch.equal(have.nan_to_num(nan=0, posinf=inf), want.nan_to_num(nan=0, posinf=inf)), name


# ------------------------------------------------------------------ norm
def _close8(name, q, s, y, err):
    """8-bit values of y, known to within err: the scale of some block within that, and the
    value as near as that scale allows."""
    e = s.cpu().view(torch.uint8).long() - 127
    lo, hi = ref.exponents((y.abs() - err).clamp(min=0), q.dtype), ref.exponents(y.abs() + err, q.dtype)
    assert ((e >= lo) & (e <= hi)).all(), f"{name}: scales"
    scale = torch.exp2(ref.spread(e, y.shape).double())
    off = (ref.values(q, s) - y).abs()
    tol = ref.half_step((y.abs() + err) / scale, q.dtype) * scale + err
    assert (off <= tol).all(), f"{name}: {float((off / tol).max())} of its bound"


RMS = [  # rows, D, dtype, out8, residual, weight, how
    (1, 1, BF, None, False, True, "dense"), (2, 128, BF, E4, True, True, "dense"), (3, 130, HF, E5, True, True, "dense"),
    (5, 1000, F, E4, False, True, "slice"), (4, 2048, BF, None, True, True, "slice"), (7, 777, BF, E4, True, False, "odd"),
    (2, 8192, BF, E4, True, True, "dense"), (3, 1537, HF, None, False, True, "odd"), (2, 16385, F, None, True, True, "dense"),
    (2, 20000, BF, E4, True, True, "dense"), (9, 136, BF, E4, True, True, "slice"), (17, 264, BF, E5, False, True, "dense"),
    (11, 1096, HF, E4, True, True, "dense"), (5, 4100, F, E4, True, True, "dense"), (3, 16384, BF, E4, True, True, "dense"),
    (600, 8192, BF, E5, True, True, "dense"), (400, 520, F, None, True, True, "dense"), (1000, 8184, BF, None, False, False, "dense"),
    (170, 7000, F, None, True, True, "dense"), (9, 4099, BF, E4, True, True, "odd"), (700, 1537, HF, E5, True, True, "dense"),
    (3, 9001, HF, None, True, True, "dense"), (2, 16383, F, E4, True, True, "odd"), (2, 20001, BF, None, True, True, "odd"),
    (650, 260, BF, None, True, True, "odd"), (5, 8192, BF, E4, True, True, "odd"), (33, 64, F, None, True, False, "dense"), (700, 512, BF, E5, True, True, "dense"),
]


def _rms_inputs(rows, D, dt, seed):
    g = _gen(seed)
    x = (torch.randn(rows, D, generator=g) * torch.randn(rows, 1, generator=g).exp()).to(dt)
    return x, torch.randn(rows, D, generator=g).to(dt), 1 + torch.randn(D, generator=g) * 0.2, g


def _sum_err(D):
    # a thread's chain of at most D / 128 + 2 terms, 10 joins, a division, a root and products:
    # relative units of 2^-24; the approximate division and root count 4 each
    return (D / 128 + 2 + 10 + 16) * 2.0 ** -24


@pytest.mark.parametrize("rows,D,dt,out8,residual,weight,how", RMS)
def test_rms_norm(rows, D, dt, out8, residual, weight, how):
    x, res, w, g = _rms_inputs(rows, D, dt, rows + D)
    res, w = res if residual else None, w if weight else None
    h, y, r = ref.rms(x, res, w, EPS)
    wg = None if w is None else w.cuda()
    out, scales = fp8.empty(rows, D, out8) if out8 else (_place(torch.full((rows, D), float("nan"), dtype=dt), how), None)
    total = _place(torch.full((rows, D), float("nan"), dtype=dt), how) if residual else None
    rstd = torch.full((rows,), float("nan"), device="cuda")
    rms_norm.rms_norm_fwd(_place(x, how), wg, EPS, out, residual=None if res is None else _place(res, how), residual_out=total,
                          rstd=rstd, scales=scales)
    _status()
    err = _sum_err(D)
    assert_close("rstd", rstd, r, err * r)
    if residual:
        assert torch.equal(total.cpu().double(), h)
    if out8:
        _close8("out", out, scales, y, 2 * err * y.abs())
    else:
        assert_close("out", out, y, 2 * err * y.abs())
    # gradients
    dy, dres = torch.randn(rows, D, generator=g).to(dt), torch.randn(rows, D, generator=g).to(dt)
    dres = dres if residual else None
    got = rms_norm.rms_norm_bwd(_place(dy, how), _place(h.to(dt), how), wg, rstd, dresidual=None if dres is None else _place(dres, how),
                                want_dweight=True)
    _status()
    rd, ww = rstd.cpu().double(), None if w is None else w.double()
    dx, dw = ref.rms_grads(h, ww, rd, dy.double(), None if dres is None else dres.double())
    d, hat = (dy.double() if w is None else dy.double() * ww), h * rd[:, None]
    E = rd[:, None] * (D32 * d.abs() + hat.abs() * (D / 128 + 28) * 2.0 ** -23 * (d * hat).abs().mean(-1, keepdim=True))
    assert_close("dx", got["dx"], dx, E + 2.0 ** -23 * (0 if dres is None else dres.double().abs()))
    # the columns' sums: rows one after the other in a part, parts in turn
    assert_close("dweight", got["dweight"], dw, (min(rows, 512) + 40) * 2.0 ** -23 * (dy.double() * hat).abs().sum(0))
