"""64-bit references of the operators around a layer's projections (RMS norm, 8-bit tensors,
their product) from their definitions, on the CPU.

e4m3: 3 bits behind the leading one, normal numbers from 2^-6, steps of 2^-9 below, largest
448; e5m2: 2 bits, 2^-14, 2^-16, 57344.  A block's scale is the smallest power of two s, at
least 2^-126, with |largest finite| / s within range, and 1 where everything is below 2^-126."""
import math

import torch

E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
FORMAT = {E4: (3, -9, 448.0), E5: (2, -16, 57344.0)}      # bits, exponent of the smallest step, largest
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def scale_exponent(top, to):
    if top < 2.0 ** -126:
        return 0
    e = math.frexp(top / FORMAT[to][2])[1]                # top / most in [2^(e-1), 2^e)
    e -= top / FORMAT[to][2] == 2.0 ** (e - 1)
    return max(e, -126)


def exponents(x, to, tile=False):
    """Exponents of the scales of x [R, C] (doubles): [R or blocks(R), blocks(C)]."""
    a = torch.where(x.isfinite(), x.abs(), 0.0)
    R, C = a.shape
    step = BLOCK if tile else 1
    return torch.tensor([[scale_exponent(float(a[r:r + step, c:c + BLOCK].max()), to) for c in range(0, C, BLOCK)]
                         for r in range(0, R, step)], dtype=torch.int64).reshape(-(-R // step), blocks(C))


def spread(e, shape):
    """Exponents of the scales for every element (of rows, or of tiles, by their shape)."""
    if e.shape[0] != shape[0]:
        e = e.repeat_interleave(BLOCK, 0)[:shape[0]]
    return e.repeat_interleave(BLOCK, 1)[:, :shape[1]]


def half_step(v, to):
    """Half the spacing of the type's numbers at |v|."""
    bits, low, _ = FORMAT[to]
    k = torch.frexp(v)[1] - 1 - bits
    return torch.exp2(k.clamp(min=low).double()) / 2


def quantized(x, to, tile=False):
    """Values that x [R, C] stands for in 8 bits, and the scales' exponents."""
    e = exponents(x, to, tile)
    s = torch.exp2(spread(e, x.shape).double())
    v = x / s
    step = 2 * half_step(torch.where(v.isfinite(), v, 0.0), to)
    q = torch.where(v.isfinite(), (v / step).round() * step, v)
    if to == E4:
        q = torch.where(v.isinf(), math.nan, q)
    return q * s, e


def bytes_of(e):
    return (e + 127).to(torch.uint8)


def values(q, s):
    """Values that an 8-bit tensor with its scales stands for."""
    q, b = q.cpu(), s.cpu().view(torch.uint8).long()
    return q.double() * torch.exp2(spread(b - 127, q.shape).double())


def rms(x, res, w, eps):
    """h, y and rstd of the forward pass; x, res in their type, the rest doubles."""
    h = x.double() if res is None else (x.double() + res.double()).to(x.dtype).double()
    r = 1 / (h.square().mean(-1) + eps).sqrt()
    return h, h * r[:, None] * (1.0 if w is None else w.double()), r


def rms_grads(h, w, r, dy, dres):
    """dx and dweight for a given rstd (which depends on h), all doubles."""
    hat = h * r[:, None]
    d = dy if w is None else dy * w
    dx = r[:, None] * (d - hat * (d * hat).mean(-1, keepdim=True))
    return dx if dres is None else dx + dres, (dy * hat).sum(0)


def product(a, sa, b, sb, add=None):
    y = values(a, sa) @ values(b, sb).T
    return y if add is None else y + add.double().cpu()


def product_bound(a, sa, b, sb):
    """What an fp32 sum of the products may be off.  Products of 8-bit numbers are exact; an
    MMA adds 32 of them to the accumulator, each aligned to the largest and cut at 2^-23 of it
    or better, the sum cut again: at most 34 units of 2^-23 of the largest magnitude that a
    partial sum can have, K / 32 times.  Splits of K add up to 8 more roundings."""
    S = values(a, sa).abs() @ values(b, sb).abs().T
    return (34 * -(-a.shape[1] // 32) + 8) * 2.0 ** -23 * S
