"""What the rotary, group norm and input-gradient calls refuse, their workspace
sizes and the frequencies, without a GPU: every refusal precedes the first
CUDA call."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import w8a8_int8_dynamic_token_b200 as w8a8
from w8a8_int8_dynamic_token_b200 import binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    from w8a8_int8_dynamic_token_b200 import build
    build.build()
    yield


P = 256  # a pointer that is never dereferenced: argument errors come first
BIG = 1 << 40
INV, SHAPE, ALIGN, WS = (B.W8A8_ERR_INVALID_ARG, B.W8A8_ERR_UNSUPPORTED_SHAPE, B.W8A8_ERR_MISALIGNED,
                         B.W8A8_ERR_WORKSPACE)


# ----------------------------------------------------------------- input gradient

def grad(dy=P, M=4, N=32, lddy=32, Wq=P, s_w=P, K=16, dx=P, lddx=16, variant=0, ws=P, ws_bytes=BIG):
    return B.w8a8_linear_input_grad(dy, M, N, lddy, Wq, s_w, K, dx, lddx, variant, ws, ws_bytes, None)


@pytest.mark.parametrize("change,expect", [
    ({"dy": None}, INV), ({"Wq": None}, INV), ({"s_w": None}, INV), ({"dx": None}, INV),
    ({"M": 0}, INV), ({"N": 0}, INV), ({"K": 0}, INV), ({"lddy": 24}, INV), ({"lddx": 8}, INV),
    ({"variant": 7}, INV), ({"variant": -1}, INV),
    ({"N": 36, "lddy": 40}, SHAPE), ({"K": 24, "lddx": 24}, SHAPE), ({"lddy": 36}, SHAPE), ({"lddx": 20}, SHAPE),
    ({"N": 133152, "lddy": 133152}, SHAPE), ({"M": 1 << 31}, SHAPE), ({"K": 1 << 31, "lddx": 1 << 31}, SHAPE),
    ({"dy": 264}, ALIGN), ({"Wq": 257}, ALIGN), ({"s_w": 260}, ALIGN), ({"dx": 258}, ALIGN),
    ({"ws": None}, WS), ({"ws_bytes": 100}, WS), ({"ws": 264}, WS),
])
def test_input_grad_refusals(change, expect):
    assert grad(**change) == expect


def test_input_grad_one_row_has_no_stride():
    # the strides are let through: the next refusal is the workspace's
    for change in ({"lddy": 1}, {"lddx": 0}, {"lddy": 36, "lddx": 20}):
        assert grad(M=1, ws=None, **change) == WS
        assert grad(M=2, ws=None, **change) in (INV, SHAPE)


def test_input_grad_workspace():
    # codes in rows of a multiple of 16 and the scales
    assert w8a8.input_grad_workspace_size(5, 24, 16) >= 5 * 32 + 5 * 4
    for variant in (B.VARIANT_GEMV, B.VARIANT_GEMM_BN64):
        assert B.w8a8_input_grad_workspace_size(4, 64, 64, variant)[0] == SHAPE
    assert B.w8a8_input_grad_workspace_size(129, 64, 64, B.VARIANT_GEMV_TC)[0] == SHAPE
    assert B.w8a8_input_grad_workspace_size(4, 64, 64, 9)[0] == INV
    assert B.w8a8_input_grad_workspace_size(4, 60, 64, 0)[0] == SHAPE
    # a pair plan that shares K out needs more
    deep = w8a8.input_grad_workspace_size(600, 12288, 2064, B.VARIANT_GEMM_PAIR)
    assert deep > 600 * 12288 + 2400 + 4 * 32 * 128 * 16


def test_input_grad_python_checks():
    dy = torch.zeros((4, 32), dtype=torch.bfloat16)
    Wq, s_w = torch.zeros((32, 16), dtype=torch.int8), torch.zeros(32)
    with pytest.raises(ValueError, match="CUDA"):
        w8a8.linear_input_grad(dy, Wq, s_w)
    with pytest.raises(TypeError):
        w8a8.linear_input_grad(dy.float(), Wq, s_w)
    with pytest.raises(ValueError, match="mismatch"):
        w8a8.linear_input_grad(dy, Wq[:24], s_w)
    with pytest.raises(ValueError, match="mismatch"):
        w8a8.linear_input_grad(dy, Wq, s_w[:24])
    with pytest.raises(ValueError, match="stride"):
        w8a8.linear_input_grad(dy.T.contiguous().T, Wq, s_w)
    with pytest.raises(ValueError, match="out"):
        w8a8.linear_input_grad(dy, Wq, s_w, out=torch.zeros((4, 8), dtype=torch.bfloat16))


# ----------------------------------------------------------------- rotary

FREQ = (ctypes.c_double * 256)(*([0.5] * 256))


def rotary(heads=({},), count=None, dtype=0, batch=1, tokens=4, dim=16, rot=16, layout=1, positions=P, bits=64,
           axes=1, freq=FREQ, axis=None, scale=1.0):
    base = {"x": P, "y": P, "heads": 2, "x_batch": 0, "x_token": 32, "x_head": 16, "y_batch": 0, "y_token": 32, "y_head": 16}
    arr = (B.RotaryHeads * 2)()
    for i, h in enumerate(heads):
        for name, v in {**base, **h}.items():
            setattr(arr[i], name, v)
    return B.w8a8_rotary(arr, len(heads) if count is None else count, dtype, batch, tokens, dim, rot, layout,
                         positions, bits, 0, 1, axes, freq, axis, scale, 0, None)


def doubles(*v):
    return (ctypes.c_double * 256)(*v)


@pytest.mark.parametrize("change,expect", [
    ({"count": 0}, INV), ({"count": 3}, INV), ({"dtype": 3}, INV), ({"layout": 2}, INV), ({"bits": 16}, INV),
    ({"batch": 0}, INV), ({"tokens": 0}, INV), ({"rot": 0}, INV), ({"rot": 18}, INV), ({"axes": 0}, INV),
    ({"scale": math.inf}, INV), ({"scale": math.nan}, INV), ({"positions": None}, INV), ({"freq": None}, INV),
    ({"freq": doubles(-1.0)}, INV), ({"freq": doubles(math.nan)}, INV), ({"freq": doubles(math.inf)}, INV),
    ({"axis": (ctypes.c_int32 * 8)(*([1] * 8))}, INV), ({"axis": (ctypes.c_int32 * 8)(*([-1] * 8))}, INV),
    ({"heads": ({"x": None},)}, INV), ({"heads": ({"y": None},)}, INV), ({"heads": ({"heads": 0},)}, INV),
    ({"heads": ({"y_token": 0},)}, INV), ({"heads": ({"y_head": 0},)}, INV), ({"batch": 2}, INV),
    ({"heads": ({}, {"x": None})}, INV),
    ({"rot": 15}, SHAPE), ({"dim": 17}, SHAPE), ({"dim": 514, "rot": 2}, SHAPE), ({"axes": 9}, SHAPE),
    ({"tokens": 1 << 30}, SHAPE),
    ({"positions": 260}, ALIGN), ({"heads": ({"x": 257},)}, ALIGN), ({"dtype": 2, "heads": ({"y": 258},)}, ALIGN),
])
def test_rotary_refusals(change, expect):
    assert rotary(**change) == expect


@pytest.mark.parametrize("change", [{"y_head": 15}, {"y_head": 1}, {"y_head": -8}, {"y_token": 8}, {"y_token": -15}, {"y_batch": 12}])
def test_rotary_refuses_outputs_that_share_values(change):
    batch = 2 if "y_batch" in change else 1
    assert rotary(batch=batch, heads=({"y_batch": 128, **change},)) == INV
    assert rotary(batch=batch, heads=({"y_batch": 128}, {"y_batch": 128, **change})) == INV
    # an extent of one has no stride: the next refusal is the alignment's
    assert rotary(batch=1, tokens=1, heads=({"heads": 1, "y": 257, **change},)) == ALIGN


@pytest.mark.parametrize("f", [2.0 ** 64, 1e290, 1.7e308, -5e-324])
def test_rotary_refuses_frequencies_that_have_no_turns(f):
    assert rotary(freq=doubles(f)) == INV


def test_rotary_python_checks():
    x, pos, freq = torch.zeros((4, 2, 16)), torch.arange(4), torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        w8a8.rotary(x, pos, freq)
    for bad in (freq.float(), freq[None], torch.ones(16, dtype=torch.float64)[::2]):
        with pytest.raises(TypeError, match="inv_freq"):
            w8a8.rotary(x, pos, bad)
    with pytest.raises(ValueError, match="has 16"):
        w8a8.rotary(x, pos, torch.ones(9, dtype=torch.float64))
    with pytest.raises(ValueError, match="layout"):
        w8a8.rotary(x, pos, freq, layout="pairs")
    with pytest.raises(TypeError, match="positions"):
        w8a8.rotary(x, pos.float(), freq)
    for bad in (pos[:3], pos[None].expand(2, 4), pos[None, None]):
        with pytest.raises(ValueError, match="positions"):
            w8a8.rotary(x, bad, freq)
    with pytest.raises(ValueError, match="positions"):
        w8a8.rotary(x, pos, freq, axis=torch.zeros(8, dtype=torch.int32))
    with pytest.raises(TypeError, match="axis"):
        w8a8.rotary(x, pos[:, None], freq, axis=torch.zeros(7, dtype=torch.int32))
    with pytest.raises(TypeError):
        w8a8.rotary(x.double(), pos, freq)
    with pytest.raises(TypeError):
        w8a8.rotary(x, pos, freq, k=x.half())
    with pytest.raises(ValueError, match="heads"):
        w8a8.rotary(x, pos, freq, k=torch.zeros((5, 2, 16)))
    with pytest.raises(ValueError, match="without k"):
        w8a8.rotary(x, pos, freq, out_k=x)
    with pytest.raises(ValueError, match="out"):
        w8a8.rotary(x, pos, freq, out=torch.zeros((4, 3, 16)))
    with pytest.raises(ValueError, match="stride"):
        w8a8.rotary(x.transpose(1, 2), pos, torch.ones(1, dtype=torch.float64))
    with pytest.raises(ValueError, match="heads"):
        w8a8.rotary(x[0], pos, freq)


def test_rotary_frequencies():
    f, s = w8a8.rotary_frequencies(64, 10000.0)
    assert s == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    assert f[0] == 1.0 and math.isclose(f[31].item(), 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = w8a8.rotary_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.allclose(lin * 4, f, rtol=1e-14)
    wide, _ = w8a8.rotary_frequencies(64, 10000.0, "base", 4.0)   # fastest kept, slowest divided
    assert wide[0] == 1.0 and math.isclose((f[31] / wide[31]).item(), 4.0, rel_tol=1e-12)
    ramp, s = w8a8.rotary_frequencies(64, 10000.0, "ramp", 4.0, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(4.0) + 1.0)
    assert torch.equal(ramp[turns > 64], f[turns > 64])           # many turns: kept
    assert torch.allclose(ramp[turns < 0.5] * 4, f[turns < 0.5], rtol=1e-14)
    assert ((ramp <= f) & (ramp >= f / 4 * (1 - 1e-14))).all()
    for bad in ((63,), (0,), (64, 1.0), (64, 10000.0, "linear", 0.5), (64, 10000.0, "other"), (2, 10.0, "base", 2.0),
                (64, 10000.0, "ramp", 2.0)):
        with pytest.raises(ValueError):
            w8a8.rotary_frequencies(*bad)


@pytest.mark.parametrize("rot,base,factor,trained,fast,slow", [
    (128, 10000.0, 4.0, 131072, 32.0, 1.0), (128, 100.0, 4.0, 4096, 32.0, 1.0), (64, 10000.0, 40.0, 4096, 32.0, 1.0),
    (64, 1e6, 32.0, 32768, 32.0, 1.0), (2, 10.0, 2.0, 1000, 32.0, 1.0), (32, 2.0, 8.0, 10 ** 9, 32.0, 1.0),
    (64, 10000.0, 4.0, 100, 32.0, 1.0), (64, 10000.0, 4.0, 5, 32.0, 1.0), (64, 10000.0, 4.0, 1, 32.0, 1.0),
])
def test_rotary_frequencies_ramp_whole_range(rot, base, factor, trained, fast, slow):
    # pair j turns trained * base^(-2j / rot) / 2 pi times; solved for j, and
    # the part divided grows linearly from there to there
    f, _ = w8a8.rotary_frequencies(rot, base)
    ramp, _ = w8a8.rotary_frequencies(rot, base, "ramp", factor, trained, fast, slow)
    at = lambda turns: rot / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)  # noqa: E731
    low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    for j in range(rot // 2):
        turns = trained * f[j].item() / (2 * math.pi)
        part = 1.0 - (ramp[j] / f[j]).item()
        if turns <= slow and high <= j:
            want = 1.0 - 1.0 / factor
        elif j <= low:
            want = 0.0
        else:
            want = (1.0 - 1.0 / factor) * min(1.0, (j - low) / (high - low))
        assert math.isclose(part, want, abs_tol=1e-12), j
        if turns > slow * base ** (2.0 / rot):   # by more than a pair: divided in part at most
            assert part < 1.0 - 1.0 / factor or j >= rot - 1
    if trained == 131072:  # the slowest pair turns 2.4 times
        assert math.isclose((ramp[63] / f[63]).item(), 0.46, abs_tol=1e-12)


# ----------------------------------------------------------------- group norm

def norm(kind="norm", x=P, xb=64000, xs=64, dtype=0, Bn=2, S=1000, C=64, G=8, w=P, b=P, pdt=0, eps=1e-5, act=0, y=P, yb=64000,
         ys=64, mean=None, rstd=None, ws=P, ws_bytes=BIG):
    if kind == "norm":
        return B.w8a8_group_norm(x, xb, xs, dtype, Bn, S, C, G, w, b, pdt, eps, act, y, yb, ys, mean, rstd, ws, ws_bytes, None)
    if kind == "quant":
        return B.w8a8_group_norm_quant(x, xb, xs, Bn, S, C, G, w, b, pdt, eps, act, y, P, mean, rstd, ws, ws_bytes, None)
    return B.w8a8_group_norm_backward(P, yb, ys, x, xb, xs, dtype, Bn, S, C, G, P, P, w, b, pdt, act, y, yb, ys, None,
                                      None, ws, ws_bytes, None)


@pytest.mark.parametrize("kind", ["norm", "quant", "backward"])
@pytest.mark.parametrize("change,expect", [
    ({"x": None}, INV), ({"y": None}, INV), ({"Bn": 0}, INV), ({"S": 0}, INV), ({"C": 0}, INV), ({"G": 0}, INV),
    ({"G": 7}, INV), ({"act": 2}, INV), ({"pdt": 1}, INV), ({"xs": 56}, INV), ({"xb": 56}, INV),
    ({"C": 60, "G": 6}, SHAPE), ({"C": 4104, "xs": 4104, "xb": 4104000}, SHAPE), ({"xs": 68}, SHAPE), ({"xb": 64004}, SHAPE),
    ({"S": 1 << 30}, SHAPE), ({"Bn": 1 << 31}, SHAPE),
    ({"x": 264}, ALIGN), ({"y": 258}, ALIGN), ({"w": 257}, ALIGN), ({"b": 258, "w": None, "pdt": 2}, ALIGN),
    ({"ws": None}, WS), ({"ws_bytes": 8}, WS), ({"ws": 264}, WS),
])
def test_group_norm_refusals(kind, change, expect):
    assert norm(kind, **change) == expect


def test_group_norm_more_refusals():
    assert norm(dtype=3) == INV and norm(eps=-1.0) == INV and norm(eps=math.nan) == INV
    assert norm(mean=P) == INV and norm(rstd=P) == INV and norm(mean=258, rstd=P) == ALIGN
    assert norm(ys=56) == INV and norm(yb=56) == INV and norm(yb=64004) == SHAPE
    assert norm("quant", C=72, xs=72, xb=72000) == SHAPE          # the int8 layer's K % 16
    assert norm(dtype=2, pdt=2, C=2056, G=1, xs=2056, xb=2056000, ys=2056, yb=2056000) == SHAPE


def test_group_norm_workspace():
    assert w8a8.group_norm_workspace_size(1, 1, 64, 8) == 0        # one block: nothing to exchange
    assert w8a8.group_norm_workspace_size(1, 1, 64, 8, torch.bfloat16, True) >= 64 * 8
    assert w8a8.group_norm_workspace_size(2, 4096, 512, 32) >= 2 * 32 * 16
    assert w8a8.group_norm_workspace_size(2, 4096, 512, 32, torch.bfloat16, True) > \
        w8a8.group_norm_workspace_size(2, 4096, 512, 32)
    assert B.w8a8_group_norm_workspace_size(1, 1, 60, 1, 0, 0)[0] == SHAPE


def test_group_norm_python_checks():
    x, w = torch.zeros((2, 3, 4, 16)), torch.ones(16)
    with pytest.raises(ValueError, match="CUDA"):
        w8a8.group_norm(x, 4, w, w)
    with pytest.raises(ValueError, match="activation"):
        w8a8.group_norm(x, 4, activation="gelu")
    with pytest.raises(TypeError):
        w8a8.group_norm(x.double(), 4)
    with pytest.raises(TypeError, match="weight"):
        w8a8.group_norm(x, 4, w.half())
    with pytest.raises(TypeError, match="same type"):
        w8a8.group_norm(x.half(), 4, w, w.half())
    with pytest.raises(ValueError, match="weight"):
        w8a8.group_norm(x, 4, w[:8])
    with pytest.raises(ValueError, match="channels last"):
        w8a8.group_norm(x[0, 0], 4)
    with pytest.raises(ValueError, match="unit stride"):
        w8a8.group_norm(x.permute(0, 3, 1, 2), 4)
    with pytest.raises(ValueError, match="evenly"):
        w8a8.group_norm(torch.zeros((2, 3, 8, 16))[:, :, :4], 4)
    with pytest.raises(ValueError, match="out"):
        w8a8.group_norm(x, 4, out=torch.zeros((2, 12, 16)))
    with pytest.raises(TypeError):
        w8a8.group_norm_quant(x, 4)
    stat = torch.zeros((2, 4))
    with pytest.raises(ValueError, match="mean"):
        w8a8.group_norm_backward(x, x, torch.zeros((1, 4)), stat)
    with pytest.raises(ValueError, match="rstd"):
        w8a8.group_norm_backward(x, x, stat, torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="dy"):
        w8a8.group_norm_backward(x[:, :2], x, stat, stat)
