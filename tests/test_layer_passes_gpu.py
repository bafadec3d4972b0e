"""The operators around the delta rule on calls so large that a CTA takes several tiles,
rows or batches of rows, their copy rings wrap, and the scans' tiles form small groups; and
captured in CUDA graphs.  Sizes follow the GPU's SM count.  Channels (of the recurrence:
heads) do not depend on each other, so some of them are compared, every row, with the 64-bit
references (tests/layer_ref.py)."""
import pytest
import torch

from gated_delta_rule_52_gb300 import glr, layer_norm, short_conv
from tests import layer_ref as ref
from tests.layer_ref import assert_close
from tests.test_layer_ops_gpu import (_conv_inputs, _conv_run, _gen, _glr_inputs, _glr_ref, _glr_run, _place)

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _ragged(T):
    """Sequences that begin and end all over T rows, some without tokens."""
    cuts = [0, 5, 5, 64, 65, T // 3, T // 3 + 1, T // 2 + 31, T // 2 + 31, T - 640, T - 100, T]
    return tuple(b - a for a, b in zip(cuts, cuts[1:]))


# A tile is 64 rows by 64 channels (32 in the backward pass of 32-bit tensors), and at most
# 5 CTAs share an SM: 16 tiles per SM are 3 and more per CTA.
@pytest.mark.parametrize("H,K,dt,lb,how,ragged", [
    (64, 64, BF, -5.0, "dense", False),
    (64, 64, HF, None, "slice", True),
    (63, 65, BF, None, "dense", True),      # unaligned rows
    (63, 65, HF, -5.0, "odd", False),
    (64, 64, F, -5.0, "dense", True),
    (63, 65, F, None, "dense", True),
    (8, 130, BF, -5.0, "dense", True),      # 17 blocks of channels: groups of 16 tiles
    (64, 128, BF, None, "dense", False),    # 128 blocks: groups of 4
])
def test_glr_many_tiles_per_cta(H, K, dt, lb, how, ragged):
    blocks = -(-H * K // 64)
    T = 64 * -(-16 * _sms() // blocks) - 7
    d = _glr_inputs(1, T, H, K, dt, _ragged(T) if ragged else None, F, K)
    got = _glr_run(d, lb, how)
    heads = [0, H // 2, H - 1]
    for k in ("x", "i", "g", "dout", "init", "dfinal"):
        d[k] = d[k][..., heads, :]
    d["A_log"], d["dt_bias"] = d["A_log"][heads], d["dt_bias"][heads]
    want = _glr_ref(d, lb)
    for name in ("out", "final", "dx", "di", "dg", "ddt_bias", "dinit"):
        assert_close(name, got[name][..., heads, :], *want[name])
    assert_close("dA_log", got["dA_log"][heads], *want["dA_log"])
    start, E = want["start"]
    assert_close("checkpoints", got["ck"][:, heads], start[::64], E[::64])


# Two CTAs per SM forward and one backward take at least four rows each, or blocks of rows
# where a row has fewer than 256 (512) threads.
@pytest.mark.parametrize("D,rows_per_sm,dt,how", [
    (1024, 65, BF, "dense"), (520, 64, HF, "dense"), (2048, 33, BF, "slice"), (5000, 9, HF, "dense"),
    (8192, 9, BF, "dense"), (1537, 9, BF, "odd"), (1000, 20, F, "dense"), (4096, 5, F, "dense"),
    (4097, 5, F, "odd"), (6001, 5, BF, "odd"), (24, 700, BF, "dense"),
])
def test_layer_norm_many_rows_per_cta(D, rows_per_sm, dt, how):
    rows, g = rows_per_sm * _sms() + 3, _gen(D)
    x = (torch.randn(rows, D, generator=g) * 2 + 1.5).to(dt)
    dy = torch.randn(rows, D, generator=g).to(dt)
    w, b = 1 + 0.2 * torch.randn(D, generator=g), 0.2 * torch.randn(D, generator=g)
    want = ref.norm(x.double(), w.double(), b.double(), 1e-5, dy.double())
    xg, dyg, wg = _place(x, how), _place(dy, how), w.cuda()
    out = _place(torch.full((rows, D), float("nan"), dtype=dt), how)
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    layer_norm.layer_norm_fwd(xg, wg, b.cuda(), 1e-5, out, mean=mean, rstd=rstd)
    got = layer_norm.layer_norm_bwd(dyg, xg, wg, mean, rstd)
    torch.cuda.synchronize()
    for name, t in (("out", out), ("mean", mean), ("rstd", rstd), *got.items()):
        assert_close(name, t, *want[name])


# 1024 lanes of 4 channels: runs of 64 rows from 64 rows per SM on, of 32 and 16 from half
# and a quarter of that; a ring holds 12 rows.
@pytest.mark.parametrize("rows_per_sm,D,W,dt,how,ragged,state", [
    (65, 4096, 4, BF, "dense", True, True), (33, 4096, 3, HF, "slice", False, True),
    (17, 4096, 4, F, "dense", True, False), (65, 4095, 4, HF, "odd", True, True),
    (33, 4095, 2, BF, "dense", True, True), (17, 4095, 4, F, "odd", False, True),
])
def test_short_conv_long_runs(rows_per_sm, D, W, dt, how, ragged, state):
    T = rows_per_sm * _sms() + 5
    d = _conv_inputs(1, T, D, W, dt, _ragged(T) if ragged else None, state, W + D)
    got = _conv_run(d, "silu", how)
    at = torch.cat([torch.arange(0, 9), torch.arange(1020, 1030), torch.arange(D - 9, D)])
    c = lambda t: None if t is None else t[..., at].double()  # noqa: E731
    want = ref.conv(c(d["x"]).reshape(T, -1), d["w"][at].double(), d["b"][at].double(), d["seqs"], True, c(d["init"]),
                    c(d["dout"]).reshape(T, -1), c(d["dfinal"]))
    for name, t in got.items():
        assert_close(name, t[at] if name == "dweight" else t[..., at], *want[name])


# ------------------------------------------------------------------ CUDA graphs
def _in_a_graph(call, inputs, others):
    """call(inputs) captured, then replayed on the values of `others`, against a plain call."""
    call(inputs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(inputs)
    for k, t in others.items():
        inputs[k].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    got = {k: t.clone() for k, t in got.items() if t is not None}
    want = call(inputs)
    torch.cuda.synchronize()
    for k, t in got.items():
        assert torch.isfinite(t).all() and torch.equal(t, want[k]), k


@pytest.mark.parametrize("T", [1, 300])
@pytest.mark.parametrize("dt", [BF, F])
def test_operators_in_cuda_graphs(T, dt):
    def inputs(seed):
        g = _gen(seed)
        n = lambda *s, dtype=F: torch.randn(s, generator=g).to("cuda", dtype)  # noqa: E731
        return {**{k: n(2, T, 2, 40, dtype=dt) for k in ("x", "i", "g", "dout")}, "A": n(2), "tb": n(2, 40), "h": n(2, 2, 40),
                "dh": n(2, 2, 40), "w": n(80, 4), "b": n(80), "s": n(2, 3, 80, dtype=dt), "ds": n(2, 3, 80), "nw": n(80)}

    def recurrence(v):
        return glr.glr_bwd(v["x"], v["i"], v["g"], v["A"], v["tb"], -5.0, v["dout"], initial_state=v["h"], dfinal=v["dh"])

    def norm(v):
        x, dout = v["x"].flatten(2), v["dout"].flatten(2)
        out, mean, rstd = torch.empty_like(x), *(torch.empty(x.shape[:2], device="cuda") for _ in range(2))
        layer_norm.layer_norm_fwd(x, v["nw"], v["b"], 1e-5, out, mean=mean, rstd=rstd)
        return {"out": out, "mean": mean, "rstd": rstd, **layer_norm.layer_norm_bwd(dout, x, v["nw"], mean, rstd)}

    def conv(v):
        x, dout = v["x"].flatten(2), v["dout"].flatten(2)
        out, last = torch.empty_like(x), torch.empty_like(v["s"])
        short_conv.short_conv_fwd(x, v["w"], v["b"], out, initial_state=v["s"], final_state=last)
        return {"out": out, "final": last, **short_conv.short_conv_bwd(x, v["w"], v["b"], dout, initial_state=v["s"], dfinal=v["ds"])}

    for call in (recurrence, norm, conv):
        _in_a_graph(call, inputs(1), inputs(2))
