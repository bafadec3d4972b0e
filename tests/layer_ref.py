"""64-bit references of the operators around the delta rule, row by row from their
definitions, on the CPU, each with a bound on what a 32-bit computation of it may be off.

A bound is carried beside each value: an elementary step that forms v from parts with
magnitude |parts| may err by D32 * |parts|, and errors of the parts propagate by the
step's derivative.  D32 = 2^-18 is 32 units of 2^-23: one step here is up to a dozen fp32
operations (a gate is two exponentials and a reciprocal with relative errors of 2^-22 to
2^-23, whose argument, up to 16 in these tests, turns a relative error of 2^-23 into an
absolute one of 2^-19 and with it a relative error of the exponential; the slopes bound
what the others pass on).  A split scan joins its parts by one more step each.  Sums over
n terms add n * 2^-24 of the sum of magnitudes.
"""
import torch

D32 = 2.0 ** -18
# Relative rounding of a stored value, and the spacing of the smallest values.
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -126), torch.bfloat16: (2.0 ** -8, 2.0 ** -126),
         torch.float16: (2.0 ** -11, 2.0 ** -24)}


def assert_close(name, got, ref, bound):
    """Every element within its bound plus one rounding to got's type (bf16 rounds to
    2^-9 of the value: 2^-8 here leaves room for a value that crosses a power of two);
    NaN and infinity where the reference has them."""
    rel, tiny = ROUND[got.dtype]
    g = got.detach().cpu().double().reshape(ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(g), fine), f"{name}: not finite at other places"
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{name}: NaN at other places"
    err = (g - ref).abs()[fine]
    tol = (bound.expand_as(ref) + rel * ref.abs() + tiny)[fine]
    bad = err > tol
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} elements off, worst {float((err / tol).max()):.3g} of its bound"


def bounds_of(B, T, lens=None):
    lens = [T] * B if lens is None else lens
    ends = torch.tensor(lens).cumsum(0).tolist()
    return list(zip([0] + ends[:-1], ends))


def sig(x):
    return torch.sigmoid(x)


def glr(x, i, g, A_log, dt_bias, lb, seqs, init=None, dout=None, dfinal=None):
    """All of the recurrence's outputs, and with dout its gradients, as {name: (value,
    bound)}.  x, i, g, dout: [R, H, K] doubles; init, dfinal: [N, H, K]."""
    R, H, K = x.shape
    N = len(seqs)
    e = A_log.exp()[:, None]
    u = g + dt_bias
    gk = -e * torch.nn.functional.softplus(u, threshold=40.0) if lb is None else lb * sig(e * u)
    a, s = gk.exp(), sig(i)
    b = s * x
    start, h, E0, E = (torch.zeros(R, H, K, dtype=torch.float64) for _ in range(4))
    fin = torch.zeros(N, H, K, dtype=torch.float64) if init is None else init.clone()
    Efin = torch.zeros_like(fin)
    for n, (lo, hi) in enumerate(seqs):
        c, ec = fin[n].clone(), torch.zeros(H, K, dtype=torch.float64)
        for t in range(lo, hi):
            start[t], E0[t] = c, ec
            ec = a[t] * ec + D32 * (a[t] * c.abs() + b[t].abs())
            c = a[t] * c + b[t]
            h[t], E[t] = c, ec
        fin[n], Efin[n] = c, ec
    r = {"out": (h, E), "final": (fin, Efin), "start": (start, E0)}
    if dout is None:
        return r
    grad, Eg = torch.zeros_like(x), torch.zeros_like(x)
    dinit, Ed = torch.zeros_like(fin), torch.zeros_like(fin)
    for n, (lo, hi) in enumerate(seqs):
        c = torch.zeros(H, K, dtype=torch.float64) if dfinal is None else dfinal[n].clone()
        ec = torch.zeros_like(c)
        for t in range(hi - 1, lo - 1, -1):
            ec = ec + D32 * (dout[t].abs() + c.abs())
            c = dout[t] + c
            grad[t], Eg[t] = c, ec
            ec = a[t] * ec + D32 * (a[t] * c).abs()
            c = a[t] * c
        dinit[n], Ed[n] = c, ec
    dl = grad * a * start
    El = a * (Eg * start.abs() + grad.abs() * E0) + D32 * dl.abs()
    ss = s * sig(-i)
    if lb is None:
        slope, rate = -e * sig(u), gk
    else:
        slope, rate = lb * sig(e * u) * sig(-e * u) * e, lb * sig(e * u) * sig(-e * u) * e * u
    dg, dA = dl * slope, dl * rate
    Edg, EdA = El * slope.abs() + D32 * dg.abs(), El * rate.abs() + D32 * dA.abs()
    round_ = 2.0 ** -24
    r.update(dx=(grad * s, Eg * s + D32 * (grad * s).abs()),
             di=(grad * x * ss, Eg * (x * ss).abs() + D32 * (grad * x * ss).abs()), dg=(dg, Edg),
             ddt_bias=(dg.sum(0), Edg.sum(0) + R * round_ * dg.abs().sum(0)),
             dA_log=(dA.sum((0, 2)), EdA.sum((0, 2)) + R * K * round_ * dA.abs().sum((0, 2))), dinit=(dinit, Ed))
    return r


def norm(x, w, b, eps, dout=None):
    """Layer norm of [rows, D] doubles."""
    D = x.shape[1]
    mean = x.mean(1, keepdim=True)
    rstd = 1 / (((x - mean) ** 2).mean(1, keepdim=True) + eps).sqrt()
    xh = (x - mean) * rstd
    # rstd's relative error: D32, and what errors of x - mean of D32 * max|x| do to it
    top = x.abs().amax(1, keepdim=True)
    Er = D32 * (1 + top * rstd)
    Exh = D32 * top * rstd + xh.abs() * Er
    ww = torch.ones(D, dtype=torch.float64) if w is None else w
    bb = torch.zeros(D, dtype=torch.float64) if b is None else b
    y = xh * ww + bb
    r = {"out": (y, Exh * ww.abs() + D32 * ((xh * ww).abs() + bb.abs())), "mean": (mean[:, 0], D32 * x.abs().mean(1)),
         "rstd": (rstd[:, 0], (Er * rstd)[:, 0])}
    if dout is None:
        return r
    d = dout * ww
    m1, m2 = d.mean(1, keepdim=True), (d * xh).mean(1, keepdim=True)
    dx = rstd * (d - m1 - xh * m2)
    a1, a2 = d.abs().mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
    Em2 = D32 * a2 + (d.abs() * Exh).mean(1, keepdim=True)
    Edx = rstd * (D32 * (d.abs() + a1 + xh.abs() * a2) + Exh * m2.abs() + xh.abs() * Em2) + Er * dx.abs()
    n, round_ = x.shape[0], 2.0 ** -24
    r.update(dx=(dx, Edx), dweight=((dout * xh).sum(0), (dout.abs() * Exh + (D32 + n * round_) * (dout * xh).abs()).sum(0)),
             dbias=(dout.sum(0), n * round_ * dout.abs().sum(0)))
    return r


def conv(x, w, b, seqs, silu=True, init=None, dout=None, dfinal=None):
    """Short convolution of [R, D] doubles."""
    R, D = x.shape
    W, N = w.shape[1], len(seqs)
    st = torch.zeros(N, W - 1, D, dtype=torch.float64) if init is None else init
    bb = torch.zeros(D, dtype=torch.float64) if b is None else b
    out, Eo = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros_like(st)
    dx, Edx = torch.zeros_like(x), torch.zeros_like(x)
    dw, Edw = torch.zeros(D, W, dtype=torch.float64), torch.zeros(D, W, dtype=torch.float64)
    db, Edb = torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
    dinit, Ed = torch.zeros_like(st), torch.zeros_like(st)
    round_ = R * 2.0 ** -24
    for n, (lo, hi) in enumerate(seqs):
        rows = torch.cat([st[n], x[lo:hi]])
        L = hi - lo
        taps = torch.stack([rows[j:j + L] for j in range(W)])            # [W, L, D]
        y = bb + sum(w[:, j] * taps[j] for j in range(W))
        Ey = D32 * (bb.abs() + sum((w[:, j] * taps[j]).abs() for j in range(W)))
        s = sig(y)
        tail = (y * s * sig(-y)) if silu else torch.zeros_like(y)
        slope = s + tail if silu else torch.ones_like(y)
        out[lo:hi] = y * s if silu else y
        Eo[lo:hi] = 1.1 * Ey + D32 * out[lo:hi].abs()                    # |silu'| <= 1.1
        fin[n] = rows[L:]
        if dout is None:
            continue
        q = dout[lo:hi] * slope
        Eq = dout[lo:hi].abs() * (0.5 * Ey + D32 * (s + tail.abs()))     # |silu''| <= 0.5
        drows, Erows = torch.zeros_like(rows), torch.zeros_like(rows)
        for j in range(W):
            drows[j:j + L] += w[:, j] * q
            Erows[j:j + L] += w[:, j].abs() * (Eq + D32 * q.abs())
            dw[:, j] += (q * taps[j]).sum(0)
            Edw[:, j] += ((Eq + (D32 + round_) * q.abs()) * taps[j].abs()).sum(0)
        db += q.sum(0)
        Edb += (Eq + round_ * q.abs()).sum(0)
        if dfinal is not None:
            drows[L:] += dfinal[n]
            Erows[L:] += D32 * dfinal[n].abs()
        dinit[n], Ed[n] = drows[:W - 1], Erows[:W - 1]
        dx[lo:hi], Edx[lo:hi] = drows[W - 1:], Erows[W - 1:]
    r = {"out": (out, Eo), "final": (fin, torch.zeros_like(fin))}
    if dout is not None:
        r.update(dx=(dx, Edx), dweight=(dw, Edw), dbias=(db, Edb), dinit=(dinit, Ed))
    return r
