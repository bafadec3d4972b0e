"""The operators around a layer's projections, called in the ways that their documentation allows: every
kernel of the product with every way into and out of it, strided and far tensors, graphs that fork and
join, graphs and host threads at once, all bytes."""
import threading

import pytest
import torch

from gated_delta_rule_52_gb300 import block, fp8, rms_norm
from tests import projection_ref as ref
from tests.layer_ref import D32, assert_close
from tests.projection_ref import E4, E5, E8
from tests.test_projection_ops_gpu import EPS, _bits, _everything, _gen, _status, _sum_err

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ every kernel of the product
def _whole(rows, K, to, tile, g):
    """Whole numbers of -3 to 3 times scales of 1/2, 1 and 2, and their values in doubles."""
    q, s = fp8.empty(rows, K, to, tile)
    q.copy_(torch.randint(-3, 4, (rows, K), generator=g, device="cuda").float())
    s.view(torch.uint8).copy_(torch.randint(126, 129, s.shape, generator=g, device="cuda"))
    e = torch.exp2(s.view(torch.uint8).double() - 127)
    if tile:
        e = e.repeat_interleave(128, 0)[:rows]
    return q, s, q.float().double() * e.repeat_interleave(128, 1)[:, :K]


# rows of few, of one round and of several, parts of K; an output row of 16 bytes and one that is not
SHAPES = [(10, 304, 1100), (10, 301, 1100), (30, 504, 700), (30, 501, 700), (50, 504, 2111), (50, 501, 2111), (64, 264, 8200), (300, 200, 4000),
          (300, 203, 4000), (130, 6504, 4100), (130, 6501, 4100), (520, 1040, 4300), (520, 1030, 4300), (400, 264, 640), (400, 261, 640),
          (1537, 2048, 256), (1537, 2045, 256), (3000, 2008, 140), (3000, 2001, 140), (5000, 4008, 130), (5000, 4003, 130)]
ADD = ["none", "own", "off16", "off1", "row", "out"]


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_kernel_and_addend(M, N, K, dt):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, sa, va = _whole(M, K, E4, False, g)
    b, sb, vb = _whole(N, K, E5, True, g)
    product = va @ vb.T
    for add in ADD:
        plus = None
        if add != "none":
            off = {"off16": 16 // dt.itemsize, "off1": 1}.get(add, 0)   # addends 16 and 2 or 4 bytes off
            room = torch.full((M, N + 40), float("nan"), dtype=dt, device="cuda")
            plus = room[:, off:off + N]
            plus.copy_(torch.randint(-8, 9, (1 if add == "row" else M, N), generator=g, device="cuda"))
            if add == "row":
                plus = plus[:1].expand(M, N)
        want = (product if plus is None else product + plus.double()).float().to(dt)
        assert float(product.abs().max()) < 2.0 ** 21
        out = plus if add == "out" else torch.full((M, N), float("nan"), dtype=dt, device="cuda")
        fp8.matmul(a, sa, b, sb, out, add=plus)
        assert torch.equal(out, want), add
        if add == "out":
            assert room[:, N:].isnan().all()
    _status()


def test_tensors_of_tokens_by_batch():
    """[B, T, K] operands that are slices of wider tensors, and addends of each token."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, T, K, N = 3, 50, 272, 200
    q, _, _ = _whole(B * T, K + 32, E4, False, g)
    b, sb, vb = _whole(N, K, E4, True, g)
    a, sa = q.view(B, T, -1)[..., 16:16 + K], torch.full((B, T, 4), 127, dtype=torch.uint8, device="cuda")[..., :3]
    va = q.float().double()[:, 16:16 + K]
    wide = torch.full((B, T, N + 9), float("nan"), device="cuda")
    bias = torch.randint(-5, 6, (N,), generator=g, device="cuda").float()
    fp8.matmul(a, sa.view(E8), b, sb, wide[..., 3:3 + N], add=bias.expand(B, T, N))
    assert torch.equal(wide[..., 3:3 + N].double().reshape(B * T, N), va @ vb.T + bias.double())
    x = torch.randn(B, T, 2 * K, generator=g, device="cuda").to(BF)[..., 5:5 + K]
    y = torch.empty(B, T, K, dtype=BF, device="cuda")
    rms_norm.rms_norm_fwd(x, None, EPS, y)
    want = ref.rms(x.reshape(-1, K).cpu(), None, None, EPS)[1]
    assert_close("y", y.view(-1, K), want, 2 * _sum_err(K) * want.abs())
    q1, s1 = torch.zeros(B, T, K, dtype=torch.uint8, device="cuda").view(E4), torch.zeros(B, T, 3, dtype=torch.uint8, device="cuda").view(E8)
    q2, s2 = fp8.empty(B * T, K)
    fp8.quantize(x, q1, s1)
    fp8.quantize(x.reshape(-1, K), q2, s2)
    assert torch.equal(_bits(q1).view(-1), _bits(q2).view(-1)) and torch.equal(_bits(s1).view(-1), _bits(s2).view(-1))
    _status()


def test_far_rows_that_are_not_aligned():
    """Output and addend with rows 40 MB apart, so that the last ones lie beyond 2^32 bytes, element by element."""
    g = torch.Generator(device="cuda").manual_seed(2)
    M, N, K = 110, 131, 200
    a, sa, va = _whole(M, K, E4, False, g)
    b, sb, vb = _whole(N, K, E4, True, g)
    step = 40 << 20
    room = torch.zeros(step * M, dtype=torch.uint8, device="cuda")
    for dt in (BF, F):
        out = room.view(dt).as_strided((M, N), (step // dt.itemsize, 1), 1)
        out.copy_(torch.randint(-5, 6, (M, N), generator=g, device="cuda"))
        want = (va @ vb.T + out.double()).float().to(dt)
        fp8.matmul(a, sa, b, sb, out, add=out)
        assert torch.equal(out, want)
        x = out                                                # and the norm's, both ways
        y, r = torch.empty(M, N, dtype=dt, device="cuda"), torch.empty(M, device="cuda")
        z = torch.empty_like(y)
        rms_norm.rms_norm_fwd(x, None, EPS, y, rstd=r)
        rms_norm.rms_norm_fwd(x.contiguous(), None, EPS, z)
        assert torch.equal(y, z)
        got, near = (rms_norm.rms_norm_bwd(t, t, None, r, dresidual=t, want_dweight=True) for t in (x, x.contiguous()))
        assert torch.equal(got["dx"], near["dx"]) and torch.equal(got["dweight"], near["dweight"])
        qt = room.view(E4).as_strided((N, M), (35000000, 1), 3)
        st, near_qt, near_st = fp8.empty(N, M)[1], *fp8.empty(N, M)
        src = y.clone()
        fp8.quantize(src, qt=qt, scales_t=st)
        fp8.quantize(src, qt=near_qt, scales_t=near_st)
        assert torch.equal(_bits(qt), _bits(near_qt)) and torch.equal(_bits(st), _bits(near_st))
    _status()


# ------------------------------------------------------------------ bytes
@pytest.mark.parametrize("to", [E4, E5])
def test_every_byte_under_every_scale(to):
    """Values from 2^-126 on are exact in fp32 (or infinite), smaller ones are those or 0."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2).cuda()
    want = q.cpu().view(to).double() * torch.exp2(s.cpu().double() - 127).repeat_interleave(128, 1)
    want[255] = float("nan")
    for cols in (256, 255):                                    # groups of 8, single elements
        for dt in (F, BF):
            out = torch.full((256, 256), 7.0, dtype=dt, device="cuda")[:, :cols]
            fp8.dequantize(q.view(to)[:, :cols], s.view(E8), out)
            got, w = out.cpu().double(), want[:, :cols]
            assert torch.equal(got.isnan(), w.isnan())
            small = w.abs() < 2.0 ** -126
            keep = ~small & ~w.isnan()
            assert torch.equal(got[keep], w[keep].float().to(dt).double())
            assert ((got == 0) | (got == w) | ~small).all()
    _status()


def test_products_of_extreme_scales():
    """2^-127 and 2^127 meet: what the scales' product leaves is exact, in every kernel."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for M, N, K in ((3, 40, 256), (200, 140, 256), (300, 136, 4096)):
        a, sa, _ = _whole(M, K, E4, False, g)
        b, sb, _ = _whole(N, K, E4, False, g)
        sa.view(torch.uint8).fill_(0)
        sb.view(torch.uint8).fill_(254)
        out = torch.empty(M, N, device="cuda")
        fp8.matmul(a, sa, b, sb, out)
        assert torch.equal(out.double(), a.float().double() @ b.float().double().T)
    _status()


# ------------------------------------------------------------------ norm
def _grad_err(hat, d, r, D):
    """dx = r (d - hat mean(d hat)): a dozen operations on d, and the mean's chain of sums."""
    return r * (D32 * d.abs() + hat.abs() * (D / 128 + 28) * 2.0 ** -23 * (d * hat).abs().mean(-1, keepdim=True))


@pytest.mark.parametrize("rows,D,dt", [(200, 16400, BF), (130, 20001, HF), (150, 8200, F), (200, 16384, F), (130, 8193, F), (700, 9001, BF)])
def test_norm_gradients_of_long_rows(rows, D, dt):
    """Rows too long for registers, more than one part of them in the weight's gradient."""
    g = _gen(rows + D)
    h, dy, dres = (torch.randn(rows, D, generator=g).to(dt) for _ in range(3))
    w = 1 + 0.2 * torch.randn(D, generator=g)
    rstd = (1 / (h.double().square().mean(-1) + EPS).sqrt()).float()
    got = rms_norm.rms_norm_bwd(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dresidual=dres.cuda())
    _status()
    r, hh, d = rstd.double()[:, None], h.double(), dy.double()
    dx, dw = ref.rms_grads(hh, w.double(), rstd.double(), d, dres.double())
    assert_close("dx", got["dx"], dx, _grad_err(hh * r, d * w.double(), r, D) + 2.0 ** -23 * dres.double().abs())
    assert_close("dweight", got["dweight"], dw, (rows + 40) * 2.0 ** -23 * (d * hh * r).abs().sum(0))


def test_norm_of_expanded_rows_and_odd_weights():
    """One gradient, residual or row for all, and a weight that starts 4 bytes off: the bits of dense tensors."""
    g = torch.Generator(device="cuda").manual_seed(4)
    for rows, D, dt in ((70, 512, BF), (40, 333, HF), (2, 20000, F), (900, 2048, BF)):
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        x, one, w = n(rows, D).to(dt), n(1, D).to(dt), n(D + 1)
        got = []
        for r, weight in ((one.expand(rows, D), w[1:]), (one.repeat(rows, 1), w[1:].clone())):
            out, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
            rms_norm.rms_norm_fwd(x, weight, EPS, out, residual=r, residual_out=h, rstd=rstd)
            grads = rms_norm.rms_norm_bwd(r, h, weight, rstd, dresidual=r)
            got.append((h, rstd, out, grads["dx"], grads["dweight"]))
        assert torch.equal(got[0][0], got[1][0])               # a weight off its alignment takes another kernel
        H, y, R = ref.rms(x.cpu(), one.cpu().expand(rows, D), w[1:].cpu(), EPS)
        for h, rstd, out, dx, dw in got:
            assert_close("out", out, y, 2 * _sum_err(D) * y.abs())
            want, want_w = ref.rms_grads(H, w[1:].cpu().double(), rstd.cpu().double(), one.cpu().double().expand(rows, D), one.cpu().double().expand(rows, D))
            hat, d = H * R[:, None], one.cpu().double() * w[1:].cpu().double()
            assert_close("dx", dx, want, _grad_err(hat, d, R[:, None], D) + 2.0 ** -23 * one.cpu().double().abs())
            assert_close("dweight", dw, want_w, (min(rows, 512) + 40) * 2.0 ** -23 * (one.cpu().double() * hat).abs().sum(0))
    _status()


def test_norm_through_autograd():
    g = _gen(9)
    for shape in ((2, 5, 256), (7, 130)):
        x, w, dy = torch.randn(shape, generator=g).to(BF), 1 + 0.2 * torch.randn(shape[-1], generator=g), torch.randn(shape, generator=g).to(BF)
        leaf, weight = x.cuda().requires_grad_(), w.cuda().requires_grad_()
        out = block.RmsNorm.apply(leaf, weight)
        dx, dw = torch.autograd.grad(out, [leaf, weight], dy.cuda())
        D = shape[-1]
        v = [x.double().view(-1, D).requires_grad_(), w.double().requires_grad_()]
        y = v[0] * (v[0].square().mean(-1, keepdim=True) + block.EPS).rsqrt() * v[1]
        want = torch.autograd.grad(y, v, dy.double().view(-1, D))
        assert_close("out", out.detach().view(-1, D), y.detach(), 2 * _sum_err(D) * y.detach().abs())
        r = (v[0].detach().square().mean(-1, keepdim=True) + block.EPS).rsqrt()
        hat, d = v[0].detach() * r, dy.double().view(-1, D) * v[1].detach()
        # rstd is off by _sum_err, which moves both terms
        mag = r * (d.abs() + hat.abs() * (d * hat).abs().mean(-1, keepdim=True)) * 4 * (_sum_err(D) + 30 * 2.0 ** -24)
        assert_close("dx", dx.view(-1, D), want[0], mag)
        assert_close("dw", dw, want[1], 60 * 2.0 ** -23 * (dy.double().view(-1, D) * hat).abs().sum(0))
    _status()


# ------------------------------------------------------------------ order of kernels
def _big_norm():
    """A norm's backward pass that has a workspace (more than 256 KB a tensor)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, dy, w, rstd = n(700, 1024).to(BF), n(700, 1024).to(BF), n(1024), n(700).abs()
    return lambda stream=None: rms_norm.rms_norm_bwd(dy, h, w, rstd, stream=stream)


def test_captured_with_a_fork_and_a_join():
    """In a graph kernels follow those of two streams, a copy and a memset: each waits for all of them."""
    call, (x, res), outs = _everything()
    big = _big_norm()
    call()
    torch.cuda.synchronize()
    M, N = outs[4].shape
    second = torch.zeros(M, N, dtype=BF, device="cuda")
    b, sb, _ = _whole(N, 640, E4, True, torch.Generator(device="cuda").manual_seed(8))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    total = torch.zeros(M, N, device="cuda")
    q2, s2 = fp8.empty(M, 640)

    def run(main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fp8.quantize(res, q2, s2)                          # beside the others
            fp8.matmul(q2, s2, b, sb, second)
            r2 = big()
        r = call()
        main.wait_stream(side)
        fp8.matmul(outs[0], outs[1], b, sb, total.zero_(), add=total)     # behind both streams and a memset
        fp8.matmul(q2, s2, b, sb, second, add=second)
        return r, r2

    with torch.cuda.graph(graph):
        r, r2 = run(torch.cuda.current_stream())
    for _ in range(5):
        x.copy_(torch.randn_like(x))
        res.copy_(torch.randn_like(res))
        graph.replay()
        torch.cuda.synchronize()
        got = [_bits(t) for t in (*outs, second, total, r["dx"], r["dweight"], r2["dx"], r2["dweight"])]
        e, e2 = run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for i, (a, t) in enumerate(zip(got, (*outs, second, total, e["dx"], e["dweight"], e2["dx"], e2["dweight"]))):
            assert torch.equal(a, _bits(t)), i
    _status()


def test_graphs_with_workspaces_at_once():
    """Graphs of the same backward pass, which has a workspace, replayed on streams of their own at the same time."""
    call = _big_norm()
    want = [_bits(t) for t in call().values()]
    graphs, results, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for _ in streams:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(3):
                r = call()
        results.append(r)
    for _ in range(20):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        r = call()
    torch.cuda.synchronize()
    for have in (*results, r):
        assert all(torch.equal(_bits(t), w) for t, w in zip(have.values(), want))
    _status()


def test_inputs_that_change_between_calls():
    """Calls one after the other on tensors that torch's kernels write before and after: none starts early."""
    g = torch.Generator(device="cuda").manual_seed(10)
    M, K, N = 96, 1024, 520
    xs = [torch.randn(M, K, generator=g, device="cuda").to(BF) for _ in range(4)]
    b, sb, _ = _whole(N, K, E4, True, g)
    x, q, s, y = torch.empty(M, K, dtype=BF, device="cuda"), *fp8.empty(M, K), torch.empty(M, N, device="cuda")

    def step(src, wait):
        x.copy_(src)
        for f in (lambda: rms_norm.rms_norm_fwd(x, None, EPS, q, scales=s), lambda: fp8.matmul(q, s, b, sb, y), lambda: fp8.matmul(q, s, b, sb, y, add=y)):
            if wait:
                torch.cuda.synchronize()
            f()
        x.fill_(float("nan"))
        q.view(torch.uint8).fill_(0x7f)
        return y.clone()

    want = [step(t, True) for t in xs]
    for _ in range(20):
        got = [step(t, False) for t in xs]
        for a, w in zip(got, want):
            assert torch.equal(a, w)
    _status()


def test_host_threads_at_once():
    made = [_everything(), _everything(M=64, K=512, N=1000, big=600)]
    want = []
    for call, _, outs in made:
        call()
        want.append([_bits(t) for t in outs])
    torch.cuda.synchronize()
    failed = []

    def work(call):
        try:
            st = torch.cuda.Stream()
            for _ in range(30):
                call(st)
            st.synchronize()
        except Exception as e:                                 # told to the test's thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for w, (_, _, outs) in zip(want, made):
        for a, b in zip(w, outs):
            assert torch.equal(a, _bits(b))
    _status()
