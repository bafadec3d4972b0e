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
    (520, 1032, 4300, E4, E4, False, False, F, True),
    (300, 136, 8400, E4, E4, False, True, F, True),          # fp32 sums of several segments of K
    (8300, 1033, 8400, E4, E4, False, True, F, True),        # and of more tiles than pairs of SMs
    (4999, 1920, 16600, E4, E5, False, False, F, False),
    (4999, 1921, 300, E4, E4, False, True, F, True),
    (5000, 1928, 300, E4, E4, False, True, BF, True),
    (3000, 2001, 140, E4, E4, False, True, HF, True),
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


# long K of operands beyond the L2.  Odd numbers of tiles, one tile above none, rows that end inside a
# tile and inside a half of it, both tile widths
LONG = [
    (7800, 301, 8300, E5, E4, False, False, F, True),
    (8192, 256, 8192, E4, E4, False, True, BF, False),
    (8100, 448, 8192, E4, E5, True, True, HF, True),
    (300, 8000, 8320, E4, E4, False, True, F, False),
    (200, 6500, 10240, E5, E5, False, False, F, True),
    (8192, 2048, 8192, E4, E4, False, True, BF, True),
]


@pytest.mark.parametrize("M,N,K,ta,tb,a_tile,b_tile,dt,add", LONG)
def test_exact_products_of_long_rows(M, N, K, ta, tb, a_tile, b_tile, dt, add):
    test_exact_products(M, N, K, ta, tb, a_tile, b_tile, dt, add)


def test_shared_rows_back_to_back_and_captured():
    """The same product three times in a row, and from a graph: the same bits."""
    g = _gen(77)
    a, sa = _normal_operand(8000, 8192, E4, False, g)
    b, sb = _normal_operand(384, 8192, E4, True, g)
    outs = [torch.full((8000, 384), float("nan"), device="cuda") for _ in range(4)]
    for o in outs[:3]:
        fp8.matmul(a, sa, b, sb, o)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(3):
            fp8.matmul(a, sa, b, sb, outs[3])
    graph.replay()
    graph.replay()
    _status()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


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


@pytest.mark.parametrize("rows,cols,tile", [(77, 131, False), (140, 264, True), (33, 520, False)])
def test_quantize_one_way_and_to_rows_of_any_alignment(rows, cols, tile):
    x = _quant_input(rows, cols, BF, 3).cuda()
    want, e = ref.quantized(x.cpu().double(), E4, tile)
    want_t, e_t = ref.quantized(x.cpu().double().T, E4, tile)
    for off in (0, 1, 8):                                     # dense rows, from some element on
        room = torch.zeros(rows * cols + 16, dtype=torch.uint8, device="cuda")
        for q, shape, value, ex in ((True, (rows, cols), want, e), (False, (cols, rows), want_t, e_t)):
            room.zero_()
            t = room[off:off + rows * cols].view(shape).view(E4)
            s = torch.zeros(ex.shape, dtype=torch.uint8, device="cuda").view(E8)
            fp8.quantize(x, *((t, s) if q else (None, None)), **({} if q else {"qt": t, "scales_t": s}), tile=tile)
            _status()
            assert torch.equal(s.cpu().view(torch.uint8), ref.bytes_of(ex)) and torch.equal(ref.values(t, s), value)
            assert not room[:off].any() and not room[off + rows * cols:].any()
            back = torch.empty(shape, dtype=BF, device="cuda")
            fp8.dequantize(t, s, back)
            assert torch.equal(back.cpu().double(), value)


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


# few rows: one CTA's (up to 4 KB a tensor), one cluster's (256 KB, 128 where they are not aligned), and
# more; few and many elements to a thread
FEW = [(2, 1024, BF), (3, 1024, BF), (8, 16384, BF), (9, 16384, BF), (7, 96, F), (128, 1024, HF), (129, 1024, HF), (64, 1023, BF), (65, 1023, BF),
       (3, 8191, HF), (32, 2048, F), (33, 2048, F), (1, 8192, F), (16384, 8, BF), (16385, 8, BF), (4, 4096, BF), (5, 4096, BF), (64, 256, HF), (65, 256, HF), (16, 512, F), (17, 512, F), (8, 1023, BF), (9, 1023, BF), (2, 4096, F),
       (1, 16384, BF), (63, 8, BF), (2048, 8, BF), (2049, 8, BF), (608, 1032, BF), (609, 1032, BF), (300, 4104, HF), (620, 8192, BF)]


@pytest.mark.parametrize("rows,D,dt", FEW)
def test_rms_norm_of_few_rows(rows, D, dt):
    test_rms_norm(rows, D, dt, None, True, True, "dense")


# ------------------------------------------------------------------ calls of other kinds
def test_norm_product_and_gradients_in_a_row():
    """A norm in 8 bits, the product that reads it, and the backward pass's: each step against its
    64-bit reference on what the step before wrote."""
    M, K, N = 150, 384, 300
    g = _gen(11)
    x, res, w = torch.randn(M, K, generator=g).to(BF), torch.randn(M, K, generator=g).to(BF), 1 + 0.2 * torch.randn(K, generator=g)
    W, dy = torch.randn(N, K, generator=g) * K ** -0.5, torch.randn(M, N, generator=g).to(BF) * 1e-3
    q, s = fp8.empty(M, K)
    h, rstd = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(M, device="cuda")
    rms_norm.rms_norm_fwd(x.cuda(), w.cuda(), EPS, q, residual=res.cuda(), residual_out=h, rstd=rstd, scales=s)
    wq, ws = fp8.empty(N, K, tile=True)
    wt, wts = fp8.empty(K, N, tile=True)
    fp8.quantize(W.cuda(), wq, ws, qt=wt, scales_t=wts, tile=True)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    fp8.matmul(q, s, wq, ws, y)
    d, ds = fp8.empty(M, N, E5)
    dt, dts = fp8.empty(N, M, E5)
    fp8.quantize(dy.cuda(), d, ds, qt=dt, scales_t=dts)
    xt, xts = fp8.empty(K, M)
    plain = torch.empty(M, K, dtype=BF, device="cuda")
    fp8.dequantize(q, s, plain)
    fp8.quantize(plain, qt=xt, scales_t=xts)
    dn, dW = torch.empty(M, K, dtype=BF, device="cuda"), torch.ones(N, K, device="cuda")
    fp8.matmul(d, ds, wt, wts, dn)
    fp8.matmul(dt, dts, xt, xts, dW, add=dW)
    r = rms_norm.rms_norm_bwd(dn, h, w.cuda(), rstd, dresidual=h)
    _status()
    hh, yy, rr = ref.rms(x, res, w, EPS)
    _close8("norm", q, s, yy, 2 * _sum_err(K) * yy.abs())
    for name, got, a, sa, b, sb, add in (("y", y, q, s, wq, ws, None), ("dn", dn, d, ds, wt, wts, None), ("dW", dW, dt, dts, xt, xts, torch.ones(N, K))):
        want = ref.product(a, sa, b, sb, add)
        assert_close(name, got, want, ref.product_bound(a, sa, b, sb) + 2.0 ** -23 * want.abs())
    dx, dw = ref.rms_grads(hh, w.double(), rstd.cpu().double(), dn.cpu().double(), hh)
    mag = rr[:, None] * (dn.cpu().double() * w.double()).abs() * (1 + (hh * rr[:, None]).abs()) + hh.abs()
    assert_close("dx", r["dx"], dx, D32 * mag.amax(1, keepdim=True).expand_as(mag))


def _everything(M=70, K=640, N=520, big=300):
    """Every operator on inputs of its own: the call, and the tensors that it writes."""
    g = _gen(5)
    c = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    x, res, w = c(M, K), c(M, K), c(K).float()
    q, s = fp8.empty(M, K)
    h, rstd, y16 = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, K, dtype=BF, device="cuda")
    qt, st = fp8.empty(K, M)
    b, sb = fp8.empty(N, K, tile=True)
    a2, sa2 = fp8.empty(big, K)
    fp8.quantize(c(N, K), b, sb, tile=True)
    fp8.quantize(c(big, K), a2, sa2)
    few, many = torch.zeros(M, N, dtype=BF, device="cuda"), torch.zeros(big, N, device="cuda")
    one = torch.zeros(1, N, dtype=BF, device="cuda")

    def call(stream=None):
        rms_norm.rms_norm_fwd(x, w, EPS, q, residual=res, residual_out=h, rstd=rstd, scales=s, stream=stream)
        fp8.matmul(q, s, b, sb, few, stream=stream)
        fp8.matmul(q[:1], s[:1], b, sb, one, stream=stream)
        fp8.matmul(a2, sa2, b, sb, many, stream=stream)
        fp8.quantize(h, qt=qt, scales_t=st, stream=stream)
        fp8.dequantize(q, s, y16, stream=stream)
        return rms_norm.rms_norm_bwd(x, h, w, rstd, dresidual=res, stream=stream)

    return call, (x, res), (q, s, h, rstd, few, one, many, qt, st, y16)


def _bits(t):
    return t.contiguous().view(torch.uint8).clone()


def test_same_bits_every_time_and_on_another_stream():
    call, _, outs = _everything()
    r = call()
    want = [_bits(t) for t in (*outs, r["dx"], r["dweight"])]
    for t in outs:
        t.view(torch.uint8).zero_() if t.element_size() == 1 else t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = call(side)
    torch.cuda.current_stream().wait_stream(side)
    for t, w in zip((*outs, r["dx"], r["dweight"]), want):
        assert torch.equal(_bits(t), w)
    _status()


def test_captured_and_replayed_on_new_inputs():
    call, (x, res), outs = _everything()
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                        # two graphs of the same calls
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = call()
        graphs.append((g, r))
    x.copy_(-2 * x)
    res.copy_(res.flip(0))
    for g, r in graphs:
        g.replay()
        torch.cuda.synchronize()
        got = [_bits(t) for t in (*outs, r["dx"], r["dweight"])]
        e = call()
        torch.cuda.synchronize()
        for a, b in zip(got, (*outs, e["dx"], e["dweight"])):
            assert torch.equal(a, _bits(b))
    _status()


def test_two_streams_at_once():
    first, second = _everything(), _everything(M=64, K=512, N=1000, big=600)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for call, _, outs in (first, second):
        call()
        want.append([_bits(t) for t in outs])
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (call, _, _) in zip(streams, (first, second)):
            call(st)
    torch.cuda.synchronize()
    for w, (_, _, outs) in zip(want, (first, second)):
        for a, b in zip(w, outs):
            assert torch.equal(a, _bits(b))
    _status()


@pytest.mark.parametrize("M", [1, 40, 200, 600])
@pytest.mark.parametrize("N", [264, 301])
def test_addend_in_place_and_rows_of_a_wider_tensor(M, N):
    g = _gen(M + N)
    a, sa = _small_operand(M, 300, E4, False, g)
    b, sb = _small_operand(N, 300, E4, True, g)
    wide = torch.full((M, N + 24), 7.0, dtype=BF, device="cuda")
    out = wide[:, 8:8 + N]
    out.copy_(torch.randint(-5, 6, (M, N), generator=g).to(BF))
    want = ref.product(a, sa, b, sb, out).float().to(BF)
    fp8.matmul(a, sa, b, sb, out, add=out)
    _status()
    assert torch.equal(out.cpu(), want)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + N:] == 7).all()


@pytest.mark.parametrize("M", [3, 70, 300])
def test_rows_that_are_not_finite_stay_alone(M):
    g = _gen(M)
    a, sa = _small_operand(M, 200, E4, False, g)
    b, sb = _small_operand(260, 200, E5, True, g)
    out = torch.empty(M, 260, device="cuda")
    want = ref.product(a, sa, b, sb)
    a.view(torch.uint8)[1, 130] = 0x7f                        # NaN
    sa.view(torch.uint8)[2, 0] = 255                          # a scale of NaN
    b.view(torch.uint8)[9, 3] = 0x7c                          # infinity in e5m2
    fp8.matmul(a, sa, b, sb, out)
    _status()
    got = out.cpu()
    assert got[1:3].isnan().all()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert not got[keep][:, 9].isfinite().any()
    cols = [j for j in range(260) if j != 9]
    assert torch.equal(got[keep][:, cols].double(), want[keep][:, cols])


def test_nothing_to_sum_and_nothing_to_write():
    for M, N in ((5, 300), (300, 5)):
        a, sa = fp8.empty(M, 0)
        b, sb = fp8.empty(N, 0)
        add = torch.randn(M, N, device="cuda")
        out = torch.full((M, N), float("nan"), device="cuda")
        fp8.matmul(a, sa, b, sb, out, add=add)
        assert torch.equal(out, add)
        fp8.matmul(a, sa, b, sb, out)
        assert (out == 0).all()
    a, sa = fp8.empty(0, 128)
    b, sb = fp8.empty(4, 128)
    fp8.matmul(a, sa, b, sb, torch.empty(0, 4, device="cuda"))
    fp8.quantize(torch.empty(0, 128, device="cuda"), a, sa)
    r = rms_norm.rms_norm_bwd(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"), torch.ones(8, device="cuda"), torch.empty(0, device="cuda"))
    assert r["dx"].shape == (0, 8) and (r["dweight"] == 0).all()
    _status()


def test_norm_in_place():
    g = _gen(3)
    for D in (512, 333, 20000):
        x, res, w = torch.randn(6, D, generator=g).to(BF), torch.randn(6, D, generator=g).to(BF), torch.randn(D, generator=g).cuda()
        out, total = torch.empty(6, D, dtype=BF, device="cuda"), torch.empty(6, D, dtype=BF, device="cuda")
        rms_norm.rms_norm_fwd(x.cuda(), w, EPS, out, residual=res.cuda(), residual_out=total)
        a, b = x.cuda(), res.cuda()
        rms_norm.rms_norm_fwd(a, w, EPS, a, residual=b, residual_out=b)          # out over x, the sum over the residual
        assert torch.equal(a, out) and torch.equal(b, total)
        a, b = x.cuda(), res.cuda()
        rms_norm.rms_norm_fwd(a, w, EPS, b, residual=b, residual_out=a)          # the other way round
        assert torch.equal(b, out) and torch.equal(a, total)
        a = x.cuda()
        rms_norm.rms_norm_fwd(a, w, EPS, a, residual=res.cuda())
        assert torch.equal(a, out)
    _status()


def test_norm_of_one_row_and_to_dense_rows_of_8_bits():
    g = _gen(4)
    for shape in ((640,), (3, 2, 264), (5, 333), (4, 1004)):
        x, w = torch.randn(shape, generator=g).to(BF), 1 + 0.2 * torch.randn(shape[-1], generator=g)
        D, rows = shape[-1], x.numel() // shape[-1]
        out = torch.zeros(x.numel(), dtype=torch.uint8, device="cuda").view(shape).view(E4)
        s = torch.zeros(*shape[:-1], ref.blocks(D), dtype=torch.uint8, device="cuda").view(E8)
        rstd = torch.empty(shape[:-1], device="cuda")
        rms_norm.rms_norm_fwd(x.cuda(), w.cuda(), EPS, out, rstd=rstd, scales=s)
        _status()
        _, y, r = ref.rms(x.view(rows, D), None, w, EPS)
        assert_close("rstd", rstd.view(rows), r, _sum_err(D) * r)
        _close8("out", out.view(torch.uint8).view(rows, D).view(E4), s.view(torch.uint8).view(rows, -1).view(E8), y, 2 * _sum_err(D) * y.abs())
        got = rms_norm.rms_norm_bwd(x.cuda(), x.cuda(), w.cuda(), rstd)
        assert got["dx"].shape == x.shape and got["dweight"].shape == (D,)


@pytest.mark.parametrize("M", [2, 100, 700])
def test_one_row_added_to_all(M):
    g = _gen(M)
    a, sa = _small_operand(M, 256, E4, False, g)
    b, sb = _small_operand(264, 256, E4, True, g)
    bias = torch.randint(-5, 6, (264,), generator=g).float().cuda()
    out = torch.empty(M, 264, device="cuda")
    fp8.matmul(a, sa, b, sb, out, add=bias.expand(M, 264))
    _status()
    assert torch.equal(out.cpu().double(), ref.product(a, sa, b, sb, bias.expand(M, 264)))


@pytest.mark.parametrize("M", [2, 129])
def test_offsets_beyond_32_bits(M):
    """Rows of a, of the output and of a quantised tensor 2^25 bytes or more apart, so that the last
    ones lie beyond 2^32."""
    K, N = 256, 136
    g = _gen(M)
    step = (1 << 32) // (M - 1) // 16 * 16 + 4096
    room = torch.empty(step * (M - 1) + 4096, dtype=torch.uint8, device="cuda")
    a = room.view(E4).as_strided((M, K), (step, 1))
    small, sa = _small_operand(M, K, E4, False, g)
    a.copy_(small)
    b, sb = _small_operand(N, K, E4, False, g)
    out = torch.empty(M, N, device="cuda")
    fp8.matmul(a, sa, b, sb, out)
    want = ref.product(small, sa, b, sb)
    assert torch.equal(out.cpu().double(), want)
    back = torch.empty(M, K, device="cuda")
    fp8.dequantize(a, sa, back)
    assert torch.equal(back.cpu().double(), ref.values(small, sa))
    far = room.view(F).as_strided((M, N), (step // 4, 1))      # the output there
    fp8.matmul(small, sa, b, sb, far)
    assert torch.equal(far.cpu().double(), want)
    q, s = a, fp8.empty(M, K)[1]
    fp8.quantize(back, q, s)
    assert torch.equal(ref.values(q, s), ref.quantized(back.cpu().double(), E4)[0])
    x = room.view(BF).as_strided((M, K), (step // 2, 1))       # the norm's rows
    x.copy_(torch.randn(M, K, generator=g).to(BF))
    y = torch.empty(M, K, dtype=BF, device="cuda")
    rms_norm.rms_norm_fwd(x, None, EPS, y)
    z = torch.empty_like(y)
    rms_norm.rms_norm_fwd(x.contiguous(), None, EPS, z)
    assert torch.equal(y, z)
    _status()
