"""A pre-norm recurrent block from the library's operators, trained and served.

  python -m gated_delta_rule_52_gb300.block [--steps 60] [--width 256] [--tokens 512]

Each block is u + Wout(mix(conv(Win(norm(u))))): layer norm, a projection, the short
convolution with SiLU on the part of it that is mixed (read in place from the projection's
output), and as the mixer either the gated linear recurrence or the delta rule (kda_fwd),
whose gate reads another part of the projection.  Training runs the operators' backward
entry points through autograd; serving carries each block's convolution and recurrent state
from a prefill to single tokens.  The task is to give back the input of three tokens ago.
"""
from __future__ import annotations

import argparse
import functools
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gated_delta_rule_52_gb300 import build, glr, kda, layer_norm, short_conv  # noqa: E402

EPS = 1e-5
LOWER_BOUND = -5.0


class _FirstOrder(torch.autograd.Function):
    """The first ``n`` tensors as they are, tied to the others; has no derivative."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the operators have first derivatives only")


def first_order(backward):
    """For a backward pass in kernels, which autograd cannot see into: under create_graph the
    gradients depend on what they were formed from, so that differentiating them again is an
    error and not a sum without their terms.  (autograd's once_differentiable does so only
    where ``dout`` has a graph of its own.)"""
    @functools.wraps(backward)
    def run(ctx, dout):
        with torch.no_grad():
            grads = backward(ctx, dout)
        return _FirstOrder.apply(len(grads), *grads, dout, *ctx.saved_tensors) if torch.is_grad_enabled() else grads
    return run


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        out, mean, rstd = torch.empty_like(x), *(torch.empty(x.shape[:-1], device=x.device) for _ in range(2))
        layer_norm.layer_norm_fwd(x, weight, bias, EPS, out, mean=mean, rstd=rstd)
        ctx.save_for_backward(x, weight, mean, rstd)
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        x, weight, mean, rstd = ctx.saved_tensors
        r = layer_norm.layer_norm_bwd(dout.contiguous(), x, weight, mean, rstd)
        return r["dx"], r["dweight"], r["dbias"]


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        short_conv.short_conv_fwd(x, weight, bias, out)
        ctx.save_for_backward(x, weight, bias)
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        x, weight, bias = ctx.saved_tensors
        r = short_conv.short_conv_bwd(x, weight, bias, dout.contiguous(), want_dinit=False)
        return r["dx"], r["dweight"], r["dbias"]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, i, g, A_log, dt_bias):
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ck = torch.empty(glr.checkpoint_shape(*x.shape), device=x.device)
        glr.glr_fwd(x, i, g, out, A_log, dt_bias, LOWER_BOUND, checkpoints=ck)
        ctx.save_for_backward(x, i, g, A_log, dt_bias, ck)
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        *inputs, ck = ctx.saved_tensors
        r = glr.glr_bwd(*inputs, LOWER_BOUND, dout.contiguous(), checkpoints=ck, want_dinit=False)
        return r["dx"], r["di"], r["dg"], r["dA_log"], r["ddt_bias"]


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, A_log, dt_bias):
        q, k, v, g, beta = (t.contiguous() for t in (q, k, v, g, beta))
        out = torch.empty_like(v)
        kda.kda_fwd(q, k, v, g, beta, 128 ** -0.5, out, A_log, dt_bias, LOWER_BOUND)
        ctx.save_for_backward(q, k, v, g, beta, A_log, dt_bias)
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        q, k, v, g, beta, A_log, dt_bias = ctx.saved_tensors
        r = kda.kda_bwd(q, k, v, g, beta, 128 ** -0.5, A_log, dt_bias, LOWER_BOUND, dout.contiguous(), want_dinit=False)
        return *(r[n].to(q.dtype) for n in ("dq", "dk", "dv", "dg", "dbeta")), r["dA_log"], r["ddt_bias"]


class Block:
    """One block of ``width`` channels; ``kind`` "glr" or "kda" (heads of 128 channels)."""

    def __init__(self, kind, width, gen, dev="cuda"):
        self.kind, self.width, self.heads = kind, width, width // 128
        n = lambda *s, std: (torch.randn(s, generator=gen) * std).to(dev)  # noqa: E731
        self.mixed = width if kind == "glr" else 3 * width       # x, or q, k, v: what the convolution reads
        wide = self.mixed + (2 * width if kind == "glr" else width + self.heads)
        bf = torch.bfloat16
        self.p = {"norm_w": torch.ones(width, device=dev), "norm_b": torch.zeros(width, device=dev),
                  "w_in": n(width, wide, std=width ** -0.5).to(bf), "w_out": n(width, width, std=width ** -0.5).to(bf),
                  "conv_w": n(self.mixed, 4, std=0.5), "conv_b": torch.zeros(self.mixed, device=dev),
                  "A_log": torch.zeros(self.heads, device=dev),
                  "dt_bias": torch.full((self.heads, 128), -3.0, device=dev)}
        for t in self.p.values():
            t.requires_grad_()

    def _parts(self, z, c):
        """The mixer's inputs from the projection's output and the convolution's."""
        heads = lambda t: t.unflatten(2, (self.heads, 128))  # noqa: E731
        rest = z[..., self.mixed:]
        if self.kind == "glr":
            return heads(c), heads(rest[..., :self.width]), heads(rest[..., self.width:])
        q, k, v = (heads(t) for t in c.split(self.width, 2))
        return q, k, v, heads(rest[..., :self.width]), rest[..., self.width:]

    def train(self, u):
        p = self.p
        z = Norm.apply(u, p["norm_w"], p["norm_b"]) @ p["w_in"]
        parts = self._parts(z, Conv.apply(z[..., :self.mixed], p["conv_w"], p["conv_b"]))
        mix = (Recurrence if self.kind == "glr" else DeltaRule).apply(*parts, p["A_log"], p["dt_bias"])
        return u + mix.flatten(2) @ p["w_out"]

    def state(self, B, dev="cuda"):
        """Zero states for serving: the convolution's last inputs and the recurrent state."""
        shape = (B, self.heads, 128) if self.kind == "glr" else (B, self.heads, 128, 128)
        return {"conv": torch.zeros(B, 3, self.mixed, dtype=torch.bfloat16, device=dev), "mix": torch.zeros(shape, device=dev)}

    @torch.no_grad()
    def serve(self, u, state):
        """Any number of tokens, one included; the states are updated in place."""
        p = self.p
        y = torch.empty_like(u)
        layer_norm.layer_norm_fwd(u, p["norm_w"], p["norm_b"], EPS, y)
        z = y @ p["w_in"]
        c = torch.empty(*u.shape[:2], self.mixed, dtype=u.dtype, device=u.device)
        short_conv.short_conv_fwd(z[..., :self.mixed], p["conv_w"], p["conv_b"], c, initial_state=state["conv"],
                                  final_state=state["conv"])
        parts = self._parts(z, c)
        if self.kind == "glr":
            mix = torch.empty_like(parts[0])
            glr.glr_fwd(*parts, mix, p["A_log"], p["dt_bias"], LOWER_BOUND, initial_state=state["mix"], final_state=state["mix"])
        else:
            parts = [t.contiguous() for t in parts]
            mix, last = torch.empty_like(parts[2]), torch.empty_like(state["mix"])
            kda.kda_fwd(*parts, 128 ** -0.5, mix, p["A_log"], p["dt_bias"], LOWER_BOUND, initial_state=state["mix"], final_state=last)
            state["mix"] = last
        return u + mix.flatten(2) @ p["w_out"]


def train(blocks, steps, B, T, gen, lr=2e-3):
    """Adam on the task's mean square error; returns the loss of every step."""
    width = blocks[0].width
    params = [t for b in blocks for t in b.p.values()]
    moments = [(torch.zeros_like(t, dtype=torch.float32), torch.zeros_like(t, dtype=torch.float32)) for t in params]
    losses = []
    for step in range(1, steps + 1):
        u = torch.randn(B, T, width, generator=gen).to("cuda", torch.bfloat16)
        h = u
        for b in blocks:
            h = b.train(h)
        loss = (h[:, 3:].float() - u[:, :-3].float()).square().mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for t, g, (m, v) in zip(params, grads, moments):
                g = g.float()
                m.lerp_(g, 0.1)
                v.lerp_(g * g, 0.01)
                t.sub_((lr * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)).to(t.dtype))
        losses.append(loss.item())
    return losses


@torch.no_grad()
def serve(blocks, u, prompt):
    """The stack's outputs with ``prompt`` tokens in one call and the others one by one."""
    states = [b.state(u.shape[0]) for b in blocks]
    outs = []
    for lo, hi in [(0, prompt)] + [(t, t + 1) for t in range(prompt, u.shape[1])]:
        h = u[:, lo:hi].contiguous()
        for b, s in zip(blocks, states):
            h = b.serve(h, s)
        outs.append(h)
    return torch.cat(outs, 1)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    build.build_library()
    gen = torch.Generator().manual_seed(0)
    blocks = [Block(kind, a.width, gen) for kind in ("glr", "kda")]
    losses = train(blocks, a.steps, a.batch, a.tokens, gen)
    u = torch.randn(a.batch, 96, a.width, generator=gen).to("cuda", torch.bfloat16)
    whole, stepped = serve(blocks, u, 96), serve(blocks, u, 80)
    off = float((whole.float() - stepped.float()).norm() / whole.float().norm())
    status = kda.get_device_status()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps; prefill against single tokens: {off:.1e} apart; "
          f"device status {status}")
    return 0 if status == kda.KDA_OK else 1


if __name__ == "__main__":
    sys.exit(main())
