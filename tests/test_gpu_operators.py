"""Rotary positions, group norm and the layer's input gradient on the GPU,
against plain implementations in 64 bits.

Tolerances count roundings: an output is rounded once (half a step of its
type), and the fp32 work ahead of it is off by a stated number of units of
2^-24 of the terms it adds.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import w8a8_int8_dynamic_token_b200 as w8a8
from w8a8_int8_dynamic_token_b200 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from w8a8_int8_dynamic_token_b200 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    assert w8a8.last_device_error() == B.W8A8_OK


def rounding(value64, dtype):
    """Half a step of `dtype` at a 64-bit value."""
    f = torch.finfo(dtype)
    return value64.abs().clamp_min(f.tiny) * (f.eps / 2)


def close(got, want64, slack64, what):
    """|got - want| <= slack + half a step at |want| + slack."""
    got = got.detach().cpu()
    err = (got.double() - want64).abs()
    tol = slack64 + rounding(want64.abs() + slack64, got.dtype)
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err / tol).max()):.3g} of the tolerance"


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ----------------------------------------------------------------- rotary

# cos and sin: the angle's 32 bits to fp32 (pi 2^-25), its cut at 2^-32 turns,
# one step of sincospif and the product with scale; then one product and one
# fused product, rounded: below 2^-21 of (|a| + |b|) * scale together.
ROT_SLACK = 2.0 ** -21


def rotary64(x, pos, freq, layout, axis, scale, backward):
    """x [B, T, H, D] and pos [B, T, A] on the CPU -> (y, slack), 64 bits."""
    rot = 2 * len(freq)
    ang = pos.double()[..., axis.long()] * freq           # [B, T, rot / 2]
    ang = -ang if backward else ang
    c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]
    y = x.double().clone()
    slack = torch.zeros_like(y)
    ia, ib = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
              else (slice(0, rot, 2), slice(1, rot, 2)))
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia] = scale * (a * c - b * s)
    y[..., ib] = scale * (a * s + b * c)
    slack[..., ia] = slack[..., ib] = ROT_SLACK * scale * (a.abs() + b.abs())
    return y, slack


ROT_CASES = [
    # batch, tokens, heads, kv heads, dim, rot, layout, axes, dtype, storage
    (1, 1, 1, None, 2, 2, "half", 1, torch.bfloat16, "tokens"),
    (1, 1, 32, 8, 128, 128, "half", 1, torch.bfloat16, "tokens"),
    (1, 37, 3, 3, 128, 128, "interleaved", 3, torch.bfloat16, "qkv"),
    (2, 53, 5, 1, 80, 40, "half", 1, torch.float16, "heads"),      # 16-byte units do not divide
    (2, 53, 5, 1, 80, 40, "interleaved", 1, torch.float16, "heads"),
    (3, 65, 4, 2, 256, 64, "half", 1, torch.float32, "heads"),
    (1, 700, 2, None, 64, 64, "interleaved", 1, torch.float32, "qkv"),
    (1, 19, 7, 2, 96, 32, "interleaved", 2, torch.bfloat16, "tokens"),
    (1, 5, 2, 1, 512, 512, "half", 1, torch.bfloat16, "tokens"),
    (1, 5, 2, 1, 512, 510, "half", 1, torch.float32, "tokens"),    # odd number of pairs
    (1, 11, 3, 2, 6, 4, "interleaved", 1, torch.float16, "odd"),   # rows off 16 bytes
    (1, 11, 300, 1, 16, 16, "half", 1, torch.bfloat16, "odd"),
    (4, 1, 9, 3, 128, 64, "half", 8, torch.bfloat16, "tokens"),
]


def make_heads(b, t, h, kv, d, dtype, storage, seed):
    g = gen(seed)
    kv = kv or 0
    if storage == "qkv":
        both = torch.randn((b, t, h + 2 * kv, d), generator=g).to(dtype)
        dev = both.cuda()
        return both[:, :, :h], both[:, :, h:h + kv], dev[:, :, :h], dev[:, :, h:h + kv]
    if storage == "odd":  # rows of h * d + 1 values
        both = torch.randn((b, t, (h + kv) * d + 1), generator=g).to(dtype)
        dev = both.cuda()
        cut = lambda v, lo, n: v[..., 1 + lo * d:1 + (lo + n) * d].unflatten(-1, (n, d))  # noqa: E731
        return cut(both, 0, h), cut(both, h, kv), cut(dev, 0, h), cut(dev, h, kv)
    q = torch.randn((b, t, h, d), generator=g).to(dtype)
    k = torch.randn((b, t, kv, d), generator=g).to(dtype)
    if storage == "heads":
        return q, k, q.transpose(1, 2).contiguous().cuda().transpose(1, 2), \
            k.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return q, k, q.cuda(), k.cuda()


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("b,t,h,kv,d,rot,layout,axes,dtype,storage", ROT_CASES)
def test_rotary(b, t, h, kv, d, rot, layout, axes, dtype, storage, backward):
    q, k, qd, kd = make_heads(b, t, h, kv, d, dtype, storage, 1)
    freq = torch.rand(rot // 2, generator=gen(2), dtype=torch.float64)
    axis = torch.randint(0, axes, (rot // 2,), generator=gen(3), dtype=torch.int32)
    pos = torch.randint(-5000, 100000, (b, t, axes), generator=gen(4))
    scale = 1.25
    posd = pos.cuda() if axes > 1 else pos[..., 0].cuda()
    if t % 2:  # 32-bit positions in half of the cases
        posd = posd.int()
    got = w8a8.rotary(qd, posd, freq, k=kd if kv else None, layout=layout,
                      axis=axis if axes > 1 else None, scale=scale, backward=backward)
    yq, yk = got if kv else (got, None)
    for x, y, name in ((q, yq, "q"), (k, yk, "k")):
        if y is None:
            continue
        want, slack = rotary64(x, pos, freq, layout, axis, scale, backward)
        close(y, want, slack, name)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])  # copied bit for bit


def test_rotary_far_positions_and_a_shared_row_of_them():
    # positions up to 2^31 and beyond: the fixed-point turns are off by at most
    # |pos| 2^-65 turns plus the frequency's own rounding to 53 bits, which the
    # 64-bit product below has too
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 33 + 7])
    freq = w8a8.rotary_frequencies(64, 1000000.0)[0]
    x = torch.randn((3, len(pos), 2, 64), generator=gen(5))
    y = w8a8.rotary(x.cuda(), pos.cuda(), freq, layout="half")  # [tokens], shared by the batch
    # exact turns in whole numbers
    turns = torch.tensor([[p * int(f * (2.0 ** 64 / (2 * math.pi))) % 2 ** 64 / 2.0 ** 64 for f in freq.tolist()]
                          for p in pos.tolist()], dtype=torch.float64) * (2 * math.pi)
    c, s = turns.cos()[None, :, None], turns.sin()[None, :, None]
    a, b = x[..., :32].double(), x[..., 32:].double()
    slack = ROT_SLACK * (a.abs() + b.abs())
    close(y[..., :32], a * c - b * s, slack, "a")
    close(y[..., 32:], a * s + b * c, slack, "b")


def two_pi():
    """2 pi to 200 bits: Machin's 16 atan(1/5) - 4 atan(1/239), in whole numbers."""
    one = 1 << 230

    def atan(n):
        total, power, k = 0, one // n, 1
        while power:
            total += power // k if k % 4 == 1 else -(power // k)
            power //= n * n
            k += 2
        return total
    return Fraction(2 * (16 * atan(5) - 4 * atan(239)), one)


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 33, 2 ** 36, 2 ** 38])
def test_rotary_far_positions_against_whole_numbers(far):
    # turns of pos * f from the exact product and a long 2 pi: the kernel's are
    # off by |pos| 2^-65 at most
    rng = np.random.default_rng(far)
    freq = torch.from_numpy(np.concatenate([w8a8.rotary_frequencies(64, 1000000.0)[0].numpy(), rng.random(30), [6.5, 1e5]]))
    pos = [far, -far, far - 1, far // 3, -far + 12345]
    turn = two_pi()
    ang = torch.tensor([[float(Fraction(f) * p / turn % 1) * (2 * math.pi) for f in freq.tolist()] for p in pos],
                       dtype=torch.float64)
    x = torch.randn((1, len(pos), 3, 128), generator=gen(65))
    y = w8a8.rotary(x.cuda(), torch.tensor(pos).cuda(), freq, layout="half")
    c, s = ang.cos()[None, :, None], ang.sin()[None, :, None]
    a, b = x[..., :64].double(), x[..., 64:].double()
    slack = (ROT_SLACK + far * 2.0 ** -65 * 2 * math.pi) * (a.abs() + b.abs())
    close(y[..., :64], a * c - b * s, slack, "a")
    close(y[..., 64:], a * s + b * c, slack, "b")


def test_rotary_cosines_and_sines():
    # of pairs (1, 0) and (0, 1).  The angle is off by half a step of fp32 below a
    # quarter of a half turn (pi 2^-27) and its cut at 2^-32 turns, cosine and sine
    # by a step of their own
    freq = torch.rand(64, generator=gen(66), dtype=torch.float64) * 4
    pos = torch.arange(-3000, 3000)
    x = torch.zeros((6000, 2, 128))
    x[:, 0, :64] = 1.0
    x[:, 1, 64:] = 1.0
    ang = pos.double()[:, None] * freq
    c, s = ang.cos(), ang.sin()
    slack = lambda v: math.pi * (2.0 ** -27 + 2.0 ** -31) + 2.0 ** -23 * v.abs()  # noqa: E731
    for sign, back in ((1.0, False), (-1.0, True)):
        y = w8a8.rotary(x.cuda(), pos.cuda(), freq, layout="half", backward=back).cpu().double()
        for got, want in ((y[:, 0, :64], c), (y[:, 0, 64:], sign * s), (y[:, 1, :64], -sign * s), (y[:, 1, 64:], c)):
            assert ((got - want).abs() <= slack(want)).all()


def test_rotary_in_place_partial_and_out():
    freq = w8a8.rotary_frequencies(32)[0]
    x = torch.randn((9, 4, 64), generator=gen(6)).bfloat16().cuda()
    pos = torch.arange(9, device="cuda")
    want = w8a8.rotary(x, pos, freq)
    big = torch.full((9, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 1:5]
    assert w8a8.rotary(x, pos, freq, out=out) is out
    assert torch.equal(out, want)
    assert (big[:, 0] == 7).all() and (big[:, 5] == 7).all()  # neighbours are left alone
    same = x.clone()
    assert w8a8.rotary(same, pos, freq, out=same) is same
    assert torch.equal(same, want)


def test_rotary_broadcast_input():
    freq = w8a8.rotary_frequencies(16)[0]
    x = torch.randn((7, 1, 16), generator=gen(7)).cuda().expand(7, 5, 16)
    pos = torch.arange(7, device="cuda", dtype=torch.int32)
    y = w8a8.rotary(x, pos, freq)
    assert torch.equal(y, w8a8.rotary(x.contiguous(), pos, freq))


def test_rotary_calls_one_after_another_without_a_pause():
    # each call starts while the one before it drains, and reads what that wrote
    def chain(pause):
        x, k = xs.clone(), ks.clone()
        for i in range(12):
            w8a8.rotary(x, pos, freq, k=k, layout="half", backward=i % 3 == 2, out=x, out_k=k)
            pause()
            h = w8a8.linear_input_grad(x.view(600, 512), Wq, s_w)
            pause()
            k = (k + h.view(600, 2, 128)) * 0.5
            pause()
        return x, k
    g = gen(15)
    xs, ks = (torch.randn((600, n, 128), generator=g).bfloat16().cuda() for n in (4, 2))
    Wq = torch.randint(-9, 10, (512, 256), generator=g, dtype=torch.int8).cuda()
    s_w = (torch.rand(512, generator=g) * 1e-2).cuda()
    pos, freq = torch.arange(600, device="cuda"), w8a8.rotary_frequencies(128)[0]
    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain(lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rotary_extents_of_one_have_no_stride():
    freq = w8a8.rotary_frequencies(64)[0]
    x = torch.randn((1, 9, 4, 64), generator=gen(67)).bfloat16().cuda()
    pos = torch.arange(9, device="cuda")
    want = w8a8.rotary(x, pos, freq, layout="half")
    for shape, strides, at in (((1, 9, 4, 64), (3, 256, 64, 1), pos), ((9, 1, 4, 64), (256, 5, 64, 1), pos[:, None]),
                               ((1, 36, 1, 64), (1, 64, 7, 1), pos.repeat_interleave(4))):
        out = torch.zeros_like(x)
        w8a8.rotary(torch.as_strided(x, shape, strides), at, freq, layout="half", out=torch.as_strided(out, shape, strides))
        assert torch.equal(out, want)
        same = x.clone()
        view = torch.as_strided(same, shape, strides)
        w8a8.rotary(view, at, freq, layout="half", out=view)
        assert torch.equal(same, want)


def test_rotary_gradient_is_the_transpose():
    # <u, R x> = <R^T u, x> up to the roundings of both sides
    freq = w8a8.rotary_frequencies(64, scaling="ramp", factor=8.0, trained=512)
    x, u = (torch.randn((2, 33, 3, 64), generator=gen(s)) for s in (8, 9))
    pos = torch.arange(33, device="cuda") * 37
    y = w8a8.rotary(x.cuda(), pos, freq[0], scale=freq[1]).cpu().double()
    g = w8a8.rotary(u.cuda(), pos, freq[0], scale=freq[1], backward=True).cpu().double()
    left, right = (y * u.double()).sum(), (g * x.double()).sum()
    # per value: slack of (|a| + |b|) <= 2 max and half a step
    bound = (ROT_SLACK + U) * freq[1] * 2 * (x.abs().max() * u.abs().double().sum() + u.abs().max() * x.abs().double().sum())
    assert abs(left - right) <= bound


# ----------------------------------------------------------------- group norm

def norm64(x, G, w, b, eps, silu):
    """x [B, S, C] -> (y, mean, rstd, z, xhat), 64 bits."""
    Bn, S, C = x.shape
    xg = x.double().view(Bn, S, G, C // G)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1.0 / torch.sqrt(var + eps)
    xhat = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).view(Bn, S, C)
    z = xhat
    if w is not None:
        z = z * w.double()
    if b is not None:
        z = z + b.double()
    y = z * torch.sigmoid(z) if silu else z
    return y, mean, rstd, z, xhat


def chain(S, C):
    """Roundings one after another in a statistic, at most: batches of 8 pixels
    joined one by one in a thread (no slab is longer than S pixels over 148
    blocks, or than one batch per thread), sums within a batch, the joins."""
    return math.ceil(S / 148 / 8) + 8 + 24


def norm_slack(x, y, mean, rstd, z, xhat, w, b, silu):
    """How far the fp32 z and y may be from the 64-bit ones."""
    Bn, S, C = x.shape
    G = mean.shape[1]
    n = chain(S, C)
    aw = 1.0 if w is None else w.double().abs()
    ab = 0.0 if b is None else b.double().abs()
    mr = (mean.abs() * rstd)[:, None, :, None].expand(Bn, S, G, C // G).reshape(Bn, S, C)
    one = 1.0 + xhat.abs()
    dz = U * (n * (mr + one) * aw + 4 * ab)   # mean off by n U (|mean| + sigma), rstd by n U
    if not silu:
        return dz
    # |y'| <= 1.1; exp is off by 2 + 1.16 |z| steps of 2^-23, the quotient by 4
    return 1.1 * dz + z.abs() * torch.sigmoid(z) * (6 + 1.2 * z.abs()) * 2 * U


NORM_CASES = [
    # shape [B, ..., C], groups, silu, dtype, parameters, offset
    ((1, 1, 8), 1, False, torch.bfloat16, "same", 0.0),
    ((2, 64, 1280), 32, True, torch.bfloat16, "same", 0.0),
    ((2, 9, 13, 640), 32, True, torch.float16, "float", 1.0),
    ((3, 257, 24), 3, True, torch.float32, "same", 0.0),
    ((1, 1000, 320), 32, False, torch.bfloat16, "none", 0.5),       # 10 channels a group
    ((5, 3, 128), 128, True, torch.bfloat16, "float", 0.0),         # a channel a group
    ((2, 31, 4096), 32, False, torch.float16, "same", 0.0),
    ((1, 17, 2048), 1, True, torch.float32, "same", 0.0),
    ((300, 5, 64), 8, True, torch.bfloat16, "same", 0.0),           # more samples than blocks
    ((1, 70000, 16), 2, True, torch.bfloat16, "same", 0.0),
    ((1, 5000, 128), 32, False, torch.float32, "same", 1000.0),     # a mean far from zero
    ((2, 4, 3, 5, 2, 48), 6, True, torch.float16, "same", 0.0),
    ((1, 2500, 256), 256, True, torch.bfloat16, "same", 2.0),       # many groups, many blocks
    ((1, 1300, 1024), 512, False, torch.float16, "same", 0.0),
    ((1, 700, 2048), 2048, True, torch.float32, "same", -3.0),
    ((1, 30000, 64), 64, True, torch.bfloat16, "same", 0.0),
]


def make_norm(shape, dtype, params, offset, seed=11):
    g = gen(seed)
    C = shape[-1]
    x = (torch.randn(shape, generator=g) * (0.5 + torch.rand(C, generator=g)) + 0.3 * torch.randn(C, generator=g) + offset).to(dtype)
    w = b = None
    if params != "none":
        pt = torch.float32 if params == "float" else dtype
        w = (1.0 + 0.3 * torch.randn(C, generator=g)).to(pt)
        b = (0.3 * torch.randn(C, generator=g)).to(pt)
    dev = [None if t is None else t.cuda() for t in (x, w, b)]
    return x, w, b, dev


@pytest.mark.parametrize("shape,groups,silu,dtype,params,offset", NORM_CASES)
def test_group_norm(shape, groups, silu, dtype, params, offset):
    x, w, b, (xd, wd, bd) = make_norm(shape, dtype, params, offset)
    y, mean, rstd = w8a8.group_norm(xd, groups, wd, bd, eps=1e-5, activation="silu" if silu else None,
                                    return_stats=True)
    x3 = x.view(shape[0], -1, shape[-1])
    y64, m64, r64, z64, xh64 = norm64(x3, groups, w, b, 1e-5, silu)
    n = chain(x3.shape[1], shape[-1])
    close(mean, m64, n * U * (m64.abs() + 1 / r64), "mean")
    close(rstd, r64, n * U * r64 * (1 + 0 * m64), "rstd")
    assert y.shape == xd.shape and y.dtype == dtype
    close(y.view(x3.shape), y64, norm_slack(x3, y64, m64, r64, z64, xh64, w, b, silu), "y")
    plain = w8a8.group_norm(xd, groups, wd, bd, eps=1e-5, activation="silu" if silu else None)
    assert torch.equal(plain, y)


def test_group_norm_strided_out_and_in_place():
    x, w, b, (xd, wd, bd) = make_norm((2, 30, 64), torch.bfloat16, "same", 0.0)
    want = w8a8.group_norm(xd, 8, wd, bd, activation="silu")
    wide = torch.full((2, 32, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    src = wide[:, 1:31, 16:80]
    src.copy_(xd)
    out = torch.full((2, 33, 80), 5.0, dtype=torch.bfloat16, device="cuda")
    dst = out[:, 2:32, 8:72]
    assert torch.equal(w8a8.group_norm(src, 8, wd, bd, activation="silu", out=dst), want)
    assert (out[:, :2] == 5).all() and (out[:, 32:] == 5).all() and (out[..., :8] == 5).all() and (out[..., 72:] == 5).all()
    same = xd.clone()
    w8a8.group_norm(same, 8, wd, bd, activation="silu", out=same)
    assert torch.equal(same, want)


def test_group_norm_takes_channels_last_images():
    img = torch.randn((2, 32, 6, 7), generator=gen(12)).half().cuda().contiguous(memory_format=torch.channels_last)
    x = img.permute(0, 2, 3, 1)
    y = w8a8.group_norm(x, 4)
    assert torch.equal(y, w8a8.group_norm(x.reshape(2, 42, 32).contiguous(), 4).view(2, 6, 7, 32))


def test_group_norm_constant_groups():
    # no variance: rstd = 1 / sqrt(eps), y = bias
    x = torch.full((2, 40, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    w, b = torch.full((16,), 2.0, device="cuda"), torch.arange(16.0, device="cuda")
    y, mean, rstd = w8a8.group_norm(x, 4, w, b, eps=1e-6, return_stats=True)
    assert torch.equal(y, b.bfloat16().expand_as(y)) and (mean == 3).all()
    close(rstd, torch.full((2, 4), 1e3, dtype=torch.float64), torch.tensor(4 * U * 1e3), "rstd")


@pytest.mark.parametrize("shape,groups,silu,params", [
    ((1, 1, 16), 2, False, "same"), ((2, 100, 1280), 32, False, "same"), ((2, 37, 320), 32, True, "float"),
    ((1, 3000, 48), 6, True, "none"), ((3, 5, 4096), 32, False, "same"), ((1, 130, 2064), 1, True, "same"),
])
def test_group_norm_quant(shape, groups, silu, params):
    x, w, b, (xd, wd, bd) = make_norm(shape, torch.bfloat16, params, 0.2)
    q, s, mean, rstd = w8a8.group_norm_quant(xd, groups, wd, bd, activation="silu" if silu else None, return_stats=True)
    y64, m64, r64, z64, xh64 = norm64(x, groups, w, b, 1e-5, silu)
    slack = norm_slack(x, y64, m64, r64, z64, xh64, w, b, silu).reshape(-1, shape[-1])
    y64 = y64.view(-1, shape[-1])
    amax = y64.abs().amax(1)
    close(s, amax / 127, slack.amax(1) / 127 + 2 * U * amax / 127, "scales")
    assert q.shape == y64.shape and s.shape == amax.shape
    qs = q.cpu().double() * s.cpu().double()[:, None]
    # half a code, and what the quotient's rounding moves
    tol = s.cpu().double()[:, None] * (0.5 + 127 * 2 * U) + slack
    assert ((qs - y64).abs() <= tol).all()
    assert (q.cpu().abs().amax(1) == 127).logical_or(s.cpu() == 0).all()
    ys, m2, r2 = w8a8.group_norm(xd, groups, wd, bd, activation="silu" if silu else None, return_stats=True)
    assert torch.equal(m2, mean) and torch.equal(r2, rstd)


def test_group_norm_quant_zero_rows():
    # no variance and no bias: rows of zeros have scale 0 and codes 0
    x = torch.full((2, 5, 32), -1.5, dtype=torch.bfloat16, device="cuda")
    q, s = w8a8.group_norm_quant(x, 4)
    assert (q == 0).all() and (s == 0).all()


@pytest.mark.parametrize("size", [6e37, 2e37, 5e36, 1e-29, 1e-32])
def test_group_norm_quant_rows_at_the_ends_of_fp32(size):
    # weights that put a row's maximum near fp32's largest or smallest values
    x = make_norm((1, 20, 32), torch.bfloat16, "none", 0.0)[0]
    w = torch.full((32,), size)
    q, s, mean, rstd = w8a8.group_norm_quant(x.cuda(), 4, w.cuda(), return_stats=True)
    y64, m64, r64, z64, xh64 = norm64(x, 4, w, None, 1e-5, False)
    slack = norm_slack(x, y64, m64, r64, z64, xh64, w, None, False)[0]
    y64 = y64[0]
    amax = y64.abs().amax(1)
    close(s, amax / 127, slack.amax(1) / 127 + 2 * U * amax / 127, "scales")
    s64 = s.cpu().double()[:, None]
    # half a code, and what the quotient's rounding moves
    assert ((q.cpu().double() * s64 - y64).abs() <= s64 * (0.5 + 127 * 2 * U) + slack).all()


# z of every size, as the bias under a weight of zero
TAILS = [-0.5, -5.0, -20.0, -40.0, -43.5, -44.0, -50.0, -60.0, -75.0, -87.0, -88.0, -100.0, -1e3, -1e10, -1e20, -3e38,
         0.0, 0.5, 5.0, 20.0, 44.0, 60.0, 90.0, 1e3, 1e20, 3e38, -30.0, -63.0, -64.0, -70.0, -80.0, -86.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_group_norm_silu_of_every_size(dtype):
    z = torch.tensor(TAILS)
    x = torch.randn((2, 3, 32), generator=gen(60)).to(dtype).cuda()
    w = torch.zeros(32, device="cuda")
    y = w8a8.group_norm(x, 4, w, z.cuda(), activation="silu")
    z64 = z.double()
    gate = torch.sigmoid(z64)
    # the power's exponent is rounded (1.25 |z| U with its constant), the power
    # itself is off by 4 U, 1 + e, its product, reciprocal (2) and three products
    # by 8; below 2^-119 the gate is 0
    slack = (z64 * gate).abs() * (1.25 * z64.abs() + 12) * U + 2.0 ** -119
    close(y, (z64 * gate).expand_as(y), slack, "y")
    # the gradient: of one pixel dbias is dz, s + z s (1 - s) times dy
    one = x[:1, :1].contiguous()
    _, mean, rstd = w8a8.group_norm(one, 4, w, z.cuda(), return_stats=True)
    dy = torch.randn((1, 1, 32), generator=gen(61)).to(dtype)
    _, _, db = w8a8.group_norm_backward(dy.cuda(), one, mean, rstd, w, z.cuda(), activation="silu")
    d = gate * (1 + z64 * (1 - gate))
    dslack = gate * (1 + z64.abs()) * (1.25 * z64.abs().clamp_max(1e3) + 16) * U
    dslack[z64 > 100] = 16 * U  # 1 - s and with it z s (1 - s) is 0
    close(db, dy[0, 0].double() * d, dy[0, 0].double().abs() * (dslack + U * d.abs() + 2.0 ** -118), "dbias")


def test_group_norm_silu_of_large_negative_values_is_nothing():
    x = torch.randn((1, 40, 32), generator=gen(62)).cuda()
    w = torch.full((32,), 1e20, device="cuda")
    z = w8a8.group_norm(x, 4, w)
    y = w8a8.group_norm(x, 4, w, activation="silu")
    assert (z < -1e10).any() and (y[z < -1e10] == 0).all() and torch.equal(y[z > 1e10], z[z > 1e10])


def test_group_norm_quant_silu_of_negative_rows():
    # every value of a row far below zero: the scale comes from gates near 2^-80
    z = -50.0 - 0.5 * torch.arange(32.0)
    x = torch.randn((1, 20, 32), generator=gen(63)).bfloat16().cuda()
    q, s = w8a8.group_norm_quant(x, 4, torch.zeros(32, device="cuda"), z.cuda(), activation="silu")
    y = z.double() * torch.sigmoid(z.double())
    slack = y.abs() * (1.25 * z.double().abs() + 12) * U
    amax = y.abs().max().expand(20)
    close(s, amax / 127, slack.max() / 127 + 2 * U * amax / 127, "scales")
    s64 = s.cpu().double()[:, None]
    assert ((q.cpu().double() * s64 - y).abs() <= s64 * (0.5 + 127 * 2 * U) + slack).all()


def test_group_norm_quant_scales_and_codes_bit_for_bit():
    # values known exactly (the bias under a weight of zero), at ties of the
    # quotient and up to two steps beside them
    rng = np.random.default_rng(64)
    x = torch.randn((1, 3, 4096), generator=gen(64)).bfloat16().cuda()
    w = torch.zeros(4096, device="cuda")
    for size in [*np.exp2(rng.uniform(-20, 20, 30)), 1e-37, 1e-33, 3e36, 2e38, 127.0, 63.5]:
        amax = np.float32(size)
        s = np.float32(amax / np.float32(127))
        y = ((rng.integers(-127, 127, 4096) + 0.5) * np.float64(s)).astype(np.float32)
        for _ in range(2):
            y = np.where(rng.random(4096) < 0.4, np.nextafter(y, np.float32(rng.choice([-1, 1]) * np.inf)), y)
        y = np.clip(y, -amax, amax)
        y[rng.integers(4096)] = amax
        if 1e-30 <= amax <= 1e37:  # the exact product of y with the rounded factor (48 bits: exact in 64)
            want = np.rint(y.astype(np.float64) * np.float64(np.float32(127) / amax)).astype(np.int8)
        else:
            want = np.clip(np.rint(y / s), -127, 127).astype(np.int8)
        q, s_a = w8a8.group_norm_quant(x, 32, w, torch.from_numpy(y).cuda())
        assert (s_a.cpu().numpy() == s).all()
        assert np.array_equal(q.cpu().numpy(), np.broadcast_to(want, (3, 4096))), size
        # the quotient's codes are the same but next to ties: s is off by 2^-24
        # of itself, f and the quotient as much
        quotient = y.astype(np.float64) / np.float64(s)
        far = np.abs(np.abs(quotient - np.trunc(quotient)) - 0.5) > 127 * 2.0 ** -23
        assert (np.rint(quotient) == want)[far].all() and (np.abs(np.rint(quotient) - want) <= 1).all()


@pytest.mark.parametrize("C", [16, 64, 320, 1280, 4096])  # one row, two and several a warp
def test_group_norm_quant_shows_what_is_not_finite(C):
    x, w, b, (xd, wd, bd) = make_norm((2, 37, C), torch.bfloat16, "float", 0.0)
    q, s = w8a8.group_norm_quant(xd, 2, wd, bd, activation="silu")
    bad = xd.clone()
    bad[1, 5, C // 2 + 3] = math.nan  # one value spoils its sample's group, and so a part of every row
    qb, sb = w8a8.group_norm_quant(bad, 2, wd, bd, activation="silu")
    assert torch.isnan(sb[37:]).all() and torch.equal(sb[:37], s[:37]) and torch.equal(qb[:37], q[:37])
    for value, silu in ((math.nan, None), (math.nan, "silu"), (math.inf, None), (-math.inf, None), (math.inf, "silu")):
        odd = bd.clone()
        odd[C - 1] = value
        sb = w8a8.group_norm_quant(xd, 2, wd, odd, activation=silu)[1]
        assert (torch.isnan(sb) if math.isnan(value) else torch.isinf(sb)).all()


def test_group_norm_extents_of_one_have_no_stride():
    x = torch.randn((1, 9, 16), generator=gen(13)).bfloat16().cuda()
    want = w8a8.group_norm(x, 2)
    odd = torch.as_strided(x, (1, 9, 16), (149, 16, 1))
    assert torch.equal(w8a8.group_norm(odd, 2, out=torch.as_strided(torch.empty_like(x), (1, 9, 16), (3, 16, 1))), want)
    one = torch.as_strided(x, (9, 1, 16), (16, 5, 1))
    assert torch.equal(w8a8.group_norm(one, 2), w8a8.group_norm(x.view(9, 1, 16).contiguous(), 2))


def grads64(dy, x, G, w, b, mean, rstd, silu):
    Bn, S, C = x.shape
    sh = (Bn, S, G, C // G)
    xh = ((x.double().view(sh) - mean.double()[:, None, :, None]) * rstd.double()[:, None, :, None]).view(Bn, S, C)
    w64 = torch.ones(C, dtype=torch.float64) if w is None else w.double()
    z = xh * w64 + (0.0 if b is None else b.double())
    sig = torch.sigmoid(z)
    d = sig * (1 + z * (1 - sig)) if silu else torch.ones_like(z)
    dz = dy.double() * d
    wdz = (dz * w64).view(sh)
    xg = xh.view(sh)
    c1, c2 = wdz.mean((1, 3), keepdim=True), (wdz * xg).mean((1, 3), keepdim=True)
    r = rstd.double()[:, None, :, None]
    dx = (r * (wdz - c1 - xg * c2)).view(Bn, S, C)
    # fp32 slack.  xh: U (|xh| 3 + |mean| rstd); z and the derivative from it
    # (|y''| <= 0.5), the derivative's own quotient and exponential
    n = chain(S, C)
    mr = (mean.double().abs() * rstd.double())[:, None, :, None].expand(sh).reshape(Bn, S, C)
    exh = U * (3 * xh.abs() + 2 * mr)
    ez = exh * w64.abs() + 2 * U * z.abs()
    ed = (0.5 * ez + (8 + 1.2 * z.abs()) * (1 + z.abs()) * 2 * U) if silu else 0 * z
    edz = dy.double().abs() * ed + 2 * U * dz.abs()
    adz, axh = dz.abs(), xh.abs()
    sl_db = (edz + n * U * adz).sum((0, 1))
    sl_dw = (edz * axh + adz * exh + n * U * adz * axh).sum((0, 1))
    ew = (edz * w64.abs()).view(sh)
    awdz = wdz.abs()
    e1 = (ew + (n + 4) * U * awdz).mean((1, 3), keepdim=True)
    e2 = (ew * xg.abs() + awdz * exh.view(sh) + (n + 4) * U * awdz * xg.abs()).mean((1, 3), keepdim=True)
    sl_dx = r * (ew + e1 + xg.abs() * e2 + exh.view(sh) * c2.abs() + 4 * U * (awdz + c1.abs() + (xg * c2).abs()))
    return (dx, sl_dx.reshape(Bn, S, C)), ((dz * xh).sum((0, 1)), sl_dw), (dz.sum((0, 1)), sl_db)


@pytest.mark.parametrize("shape,groups,silu,dtype,params,offset", NORM_CASES)
def test_group_norm_backward(shape, groups, silu, dtype, params, offset):
    x, w, b, (xd, wd, bd) = make_norm(shape, dtype, params, offset)
    act = "silu" if silu else None
    _, mean, rstd = w8a8.group_norm(xd, groups, wd, bd, activation=act, return_stats=True)
    dy = torch.randn(shape, generator=gen(13)).to(dtype)
    dx, dw, db = w8a8.group_norm_backward(dy.cuda(), xd, mean, rstd, wd, bd, activation=act)
    x3, dy3 = x.view(shape[0], -1, shape[-1]), dy.view(shape[0], -1, shape[-1])
    wx, ww, wb = grads64(dy3, x3, groups, w, b, mean.cpu(), rstd.cpu(), silu)
    close(dx.view(x3.shape), wx[0], wx[1], "dx")
    if w is None:
        assert dw is None and db is None
    else:
        close(dw, *ww, "dweight")
        close(db, *wb, "dbias")
    again = w8a8.group_norm_backward(dy.cuda(), xd, mean, rstd, wd, bd, activation=act)
    assert torch.equal(again[0], dx) and (w is None or (torch.equal(again[1], dw) and torch.equal(again[2], db)))
    same = dy.cuda()
    assert torch.equal(w8a8.group_norm_backward(same, xd, mean, rstd, wd, bd, activation=act, out=same)[0], dx)


@pytest.mark.parametrize("silu", [False, True])
def test_group_norm_gradient_against_differences(silu):
    # the 64-bit forward's central differences along random directions
    x, w, b, (xd, wd, bd) = make_norm((2, 21, 24), torch.float32, "same", 0.0)
    act = "silu" if silu else None
    _, mean, rstd = w8a8.group_norm(xd, 3, wd, bd, activation=act, return_stats=True)
    dy = torch.randn(x.shape, generator=gen(14))
    dx, dw, db = w8a8.group_norm_backward(dy.cuda(), xd, mean, rstd, wd, bd, activation=act)
    f = lambda xx, ww, bb: (norm64(xx, 3, ww, bb, 1e-5, silu)[0] * dy.double()).sum()  # noqa: E731
    h = 1e-4
    for i, g in enumerate((dx, dw, db)):
        args = [x.double(), w.double(), b.double()]
        v = torch.randn(args[i].shape, generator=gen(15 + i), dtype=torch.float64)
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + h * v, args[i] - h * v
        diff = (f(*plus) - f(*minus)) / (2 * h)
        got = (g.cpu().double() * v).sum()
        # fp32 gradients: some 100 U of every term; third derivatives of order
        # rstd^3 |dy| |v|^3 leave h^2 of them
        scale = (g.cpu().double().abs() * v.abs()).sum() + (dy.abs().double().sum() * v.abs().max())
        assert abs(got - diff) <= scale * (100 * U + 10 * h * h)


# Slabs longer than a block's ring: the second pass reads chunks again, in
# place too, adjacent rows and strided ones.
@pytest.mark.parametrize("shape,groups,dtype,pad", [
    ((1, 130001, 128), 32, torch.bfloat16, 0), ((1, 130001, 128), 32, torch.bfloat16, 16),
    ((3, 20011, 320), 32, torch.float32, 0), ((2, 3001, 4096), 32, torch.float16, 0),
    ((1, 300007, 128), 32, torch.bfloat16, 0), ((148, 1500, 256), 8, torch.bfloat16, 0),  # several rings
])
def test_group_norm_longer_than_the_ring(shape, groups, dtype, pad):
    Bn, S, C = shape
    wide = torch.zeros((Bn, S, C + pad), dtype=dtype, device="cuda")
    x = wide[..., :C]
    x.copy_(torch.randn(shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda") + 1.5)
    w, b = (1 + 0.2 * torch.randn(C, generator=gen(4))).cuda(), (0.2 * torch.randn(C, generator=gen(5))).cuda()
    xg = x.double().reshape(Bn, S, groups, C // groups)
    m64 = xg.mean((1, 3))
    r64 = 1 / torch.sqrt(((xg - m64[:, None, :, None]) ** 2).mean((1, 3)) + 1e-5)
    xh = ((xg - m64[:, None, :, None]) * r64[:, None, :, None]).reshape(shape)
    z = xh * w.double() + b.double()
    gate = torch.sigmoid(z)
    n = chain(S, C)
    slack = 1.1 * U * (n * (1 + xh.abs() + (m64.abs() * r64).max()) * w.double().abs() + 4 * b.double().abs()) + \
        z.abs() * gate * (6 + 1.2 * z.abs()) * 2 * U
    y, mean, rstd = w8a8.group_norm(x, groups, w, b, activation="silu", return_stats=True)
    close(y, (z * gate).cpu(), slack.cpu(), "y")
    close(mean, m64.cpu(), (n * U * (m64.abs() + 1 / r64)).cpu(), "mean")
    if dtype == torch.bfloat16:
        q, s = w8a8.group_norm_quant(x, groups, w, b, activation="silu")
        qs = q.double() * s.double()[:, None]
        y64 = (z * gate).view(-1, C)
        assert ((qs - y64).abs() <= s.double()[:, None] * (0.5 + 127 * 2 * U) + slack.view(-1, C)).all()
    # gradient, against the formula on the device in 64 bits
    dy = torch.randn(shape, generator=torch.Generator("cuda").manual_seed(6), device="cuda").to(dtype)
    dx, dw, db = w8a8.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu")
    dz = dy.double() * gate * (1 + z * (1 - gate))
    wdz = (dz * w.double()).view(xg.shape)
    xhg = xh.view(xg.shape)
    c1, c2 = wdz.mean((1, 3), keepdim=True), (wdz * xhg).mean((1, 3), keepdim=True)
    want = (r64[:, None, :, None] * (wdz - c1 - xhg * c2)).reshape(shape)
    # every term's fp32 roundings: the statistics' n U, the derivative's some
    # 30 (1 + |z|), on |w dz|, its means and their products
    part = r64[:, None, :, None] * (wdz.abs() + wdz.abs().mean((1, 3), keepdim=True) * (1 + xhg.abs()))
    zz = (1 + z.abs().view(xg.shape)) * (1 + (m64.abs() * r64)[:, None, :, None])
    tol = (part * (n + 60 * zz) * U + r64[:, None, :, None] * dy.double().view(xg.shape).abs() * 60 * zz * U).reshape(shape)
    close(dx, want.cpu(), tol.cpu(), "dx")
    sw = (dz * xh).abs().sum((0, 1)) + (dy.double().abs() * xh.abs() + dz.abs()).sum((0, 1))
    close(dw, (dz * xh).sum((0, 1)).cpu(), ((n + 200) * U * sw).cpu(), "dweight")
    close(db, dz.sum((0, 1)).cpu(), ((n + 200) * U * (dz.abs() + dy.double().abs()).sum((0, 1))).cpu(), "dbias")
    again = x.clone() if pad == 0 else x
    out = w8a8.group_norm(again, groups, w, b, activation="silu", out=again)
    assert out is again and torch.equal(out, y)
    if pad:
        assert (wide[..., C:] == 0).all()


def joins(B, S, C, G, dtype):
    """Roundings one after another in a statistic, from the kernel's own cut: a
    sample has 148 / B blocks (one at least), a block 512 threads on vectors of 16
    bytes, a thread batches of 4 rows that join one by one; then the threads' and
    the blocks' values join over 32 lanes."""
    row_threads = C * dtype.itemsize // 16
    rows = min(512 // row_threads, S)
    blocks = min(max(148 // B, 1), math.ceil(S / (4 * rows)))
    return math.ceil(math.ceil(S / blocks) / (4 * rows)) + 4 + math.ceil(rows * (C // G) / 32) + 5 + math.ceil(blocks / 32) + 5


@pytest.mark.parametrize("shape,groups,dtype,offset", [
    ((148, 6000, 64), 8, torch.float32, 0.5), ((160, 3000, 32), 4, torch.bfloat16, 0.0), ((75, 9000, 64), 8, torch.float32, 30.0),
    ((149, 2001, 128), 32, torch.float16, 2.0), ((148, 700, 8), 2, torch.float32, 1000.0),
])
def test_group_norm_many_samples(shape, groups, dtype, offset):
    Bn, S, C = shape
    x = (torch.randn(shape, generator=torch.Generator("cuda").manual_seed(68), device="cuda") + offset).to(dtype)
    w, b = (1 + 0.2 * torch.randn(C, generator=gen(69))).cuda(), (0.2 * torch.randn(C, generator=gen(70))).cuda()
    y, mean, rstd = w8a8.group_norm(x, groups, w, b, return_stats=True)
    n = joins(Bn, S, C, groups, dtype)
    for lo in range(0, Bn, 40):
        part = slice(lo, lo + 40)
        xg = x[part].double().view(-1, S, groups, C // groups)
        m64 = xg.mean((1, 3))
        r64 = 1 / torch.sqrt(((xg - m64[:, None, :, None]) ** 2).mean((1, 3)) + 1e-5)
        off = m64.abs() + 1 / r64
        close(mean[part], m64.cpu(), (n * U * off).cpu(), "mean")
        # deviations are off by U of the mean each and once per join
        close(rstd[part], r64.cpu(), (n * U * r64 * (1 + n * U * (off * r64) ** 2)).cpu(), "rstd")
        xh = ((xg - m64[:, None, :, None]) * r64[:, None, :, None])
        slack = U * (n * (1 + xh.abs() + (off * r64)[:, None, :, None])).reshape(-1, S, C) * w.double() + 4 * U * b.double().abs()
        close(y[part], (xh.reshape(-1, S, C) * w.double() + b.double()).cpu(), slack.cpu(), "y")


@pytest.mark.parametrize("fill", [0x00, 0xFF, 0x5A])
def test_group_norm_workspace_contents_do_not_matter(fill):
    x, w, b, (xd, wd, bd) = make_norm((2, 3000, 64), torch.bfloat16, "same", 0.0)
    want = w8a8.group_norm(xd, 8, wd, bd)
    need = max(w8a8.group_norm_workspace_size(2, 3000, 64, 8), w8a8.group_norm_workspace_size(2, 3000, 64, 8, torch.bfloat16, True),
               w8a8.group_norm_workspace_size(1, 900, 64, 16))
    ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
    for _ in range(3):  # one workspace, other shapes and forms in between
        assert torch.equal(w8a8.group_norm(xd, 8, wd, bd, workspace=ws), want)
        w8a8.group_norm(xd[:1, :900], 16, wd, bd, workspace=ws)
        q, s, mean, rstd = w8a8.group_norm_quant(xd, 8, wd, bd, return_stats=True, workspace=ws)
        w8a8.group_norm_backward(xd, xd, mean, rstd, wd, bd, workspace=ws)


def test_group_norm_on_two_streams_at_once():
    jobs = []
    for i, shape in enumerate([(1, 4096, 320), (2, 2000, 512)]):
        x, w, b, dev = make_norm(shape, torch.bfloat16, "same", 0.0, seed=40 + i)
        jobs.append((dev, w8a8.group_norm(dev[0], 32, dev[1], dev[2], activation="silu"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, ((x, w, b), _, s) in enumerate(jobs):
            got[i].append(w8a8.group_norm(x, 32, w, b, activation="silu", stream=s))
    torch.cuda.synchronize()
    for (_, want, _), ys in zip(jobs, got):
        assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("shape,groups", [((2, 600, 64), 8), ((1, 9000, 48), 6), ((300, 5, 64), 8)])
def test_group_norm_gradient_of_one_parameter_or_none(shape, groups):
    x, w, b, (xd, wd, bd) = make_norm(shape, torch.bfloat16, "float", 0.0)
    dy = torch.randn(shape, generator=gen(14)).bfloat16().cuda()
    for wi, bi in ((wd, None), (None, bd), (None, None)):
        _, mean, rstd = w8a8.group_norm(xd, groups, wi, bi, activation="silu", return_stats=True)
        dx, dw, db = w8a8.group_norm_backward(dy, xd, mean, rstd, wi, bi, activation="silu")
        x3, dy3 = x.view(shape), dy.cpu()
        wx, ww, wb = grads64(dy3, x3, groups, None if wi is None else w, None if bi is None else b, mean.cpu(), rstd.cpu(), True)
        close(dx, wx[0], wx[1], "dx")
        assert (dw is None) == (wi is None) and (db is None) == (bi is None)
        if dw is not None:
            close(dw, *ww, "dweight")
        if db is not None:
            close(db, *wb, "dbias")


def norm_calls(ws, x, dy, w, b):
    y, mean, rstd = w8a8.group_norm(x, 8, w, b, activation="silu", return_stats=True, workspace=ws)
    q, s = w8a8.group_norm_quant(x, 8, w, b, workspace=ws)
    return (y, q, s, *w8a8.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu", workspace=ws))


def test_group_norm_graphs_that_share_a_workspace():
    jobs, graphs = [], []
    need = w8a8.group_norm_workspace_size(2, 3000, 64, 8, torch.bfloat16, True)
    ws = torch.full((need,), 0x77, dtype=torch.uint8, device="cuda")
    for i, shape in enumerate([(2, 3000, 64), (1, 2500, 64)]):
        x, w, b, (xd, wd, bd) = make_norm(shape, torch.bfloat16, "same", 0.0, seed=50 + i)
        dy = torch.randn(shape, generator=gen(52 + i)).bfloat16().cuda()
        want = norm_calls(ws, xd, dy, wd, bd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = norm_calls(ws, xd, dy, wd, bd)
        jobs.append((want, got, (xd, wd, bd, dy)))  # the graph reads them: they have to live
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        want, got, _ = jobs[i]
        for t in got:
            t.zero_()
        graphs[i].replay()
        for a, c in zip(want, got):
            assert torch.equal(a, c)


def test_group_norm_on_branches_of_a_graph_and_streams_of_two_priorities():
    # launches that may run at once, each with blocks that wait for one another
    x, w, b, (xd, wd, bd) = make_norm((1, 30000, 64), torch.bfloat16, "same", 0.0)
    dy = torch.randn((1, 30000, 64), generator=gen(54)).bfloat16().cuda()
    want = norm_calls(None, xd, dy, wd, bd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0)]
    for _ in range(10):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(norm_calls(None, xd, dy, wd, bd))
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for one in got for a, c in zip(want, one))
    main = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        got = []
        for s in streams:
            s.wait_stream(main)
            with torch.cuda.stream(s):
                got.append(norm_calls(None, xd, dy, wd, bd))
        for s in streams:
            main.wait_stream(s)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert w8a8.last_device_error() == B.W8A8_OK
    assert all(torch.equal(a, c) for one in got for a, c in zip(want, one))


# ----------------------------------------------------------------- input gradient

def input_grad_ref(dy, Wq, s_w):
    """The definition, in numpy: fp32 rows and codes, exact sums."""
    g = dy.float().numpy() * s_w.numpy()
    s = (np.abs(g).max(1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[:, None] > 0, np.clip(np.rint(g / s[:, None]), -127, 127), 0).astype(np.float64)
    acc = c @ Wq.numpy().astype(np.float64)        # |acc| < 2^31: exact in 64-bit floats
    y = acc.astype(np.float32) * s[:, None]
    return torch.from_numpy(y).bfloat16(), torch.from_numpy(c), torch.from_numpy(s)


def make_grad(M, N, K, seed):
    g = gen(seed)
    dy = (torch.randn((M, N), generator=g) * 1e-3).bfloat16()
    if M > 2:
        dy[M // 2] = 0  # a row of zeros
    Wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    s_w = (0.5 + torch.rand(N, generator=g)) * 1e-3
    return dy, Wq, s_w


GRAD_SHAPES = [
    (1, 8, 16), (1, 136, 128), (3, 4096, 4096), (16, 1000, 528), (17, 264, 144), (33, 520, 1040), (64, 256, 128),
    (129, 2056, 272), (300, 264, 256), (511, 1032, 2064), (700, 4096, 1024), (5, 13000, 256), (260, 24, 16),
    (1300, 520, 4112), (297, 8, 32), (600, 40, 64), (900, 5000, 128), (310, 12288, 32), (333, 9000, 16),
    (2500, 2064, 256), (890, 12288, 32), (889, 8, 32), (1200, 40, 64), (1000, 9000, 16),
]


@pytest.mark.parametrize("M,N,K", GRAD_SHAPES)
def test_linear_input_grad_is_exact(M, N, K):
    dy, Wq, s_w = make_grad(M, N, K, M + N)
    want = input_grad_ref(dy, Wq, s_w)[0]
    got = w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda())
    assert got.shape == (M, K)
    assert torch.equal(got.cpu(), want), f"{int((got.cpu() != want).sum())} of {want.numel()} differ"


@pytest.mark.parametrize("variant", [B.VARIANT_GEMM_BN128, B.VARIANT_GEMM_BN256, B.VARIANT_GEMM_PAIR, B.VARIANT_GEMV_TC])
@pytest.mark.parametrize("M,N,K", [(1, 24, 16), (37, 1000, 528), (128, 392, 2048), (300, 5128, 272), (2600, 264, 2320)])
def test_linear_input_grad_variants_agree(M, N, K, variant):
    dy, Wq, s_w = make_grad(M, N, K, 21)
    if variant == B.VARIANT_GEMV_TC and M > 128:
        with pytest.raises(w8a8.W8A8Error):
            w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda(), variant=variant)
        return
    got = w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda(), variant=variant)
    assert torch.equal(got.cpu(), input_grad_ref(dy, Wq, s_w)[0])


def test_linear_input_grad_strides_and_out():
    dy, Wq, s_w = make_grad(70, 200, 96, 22)
    wide = torch.zeros((70, 224), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:208] = dy.cuda()
    big = torch.full((72, 112), 9.0, dtype=torch.bfloat16, device="cuda")
    out = big[1:71, 8:104]
    w8a8.linear_input_grad(wide[:, 8:208], Wq.cuda(), s_w.cuda(), out=out)
    assert torch.equal(out.cpu(), input_grad_ref(dy, Wq, s_w)[0])
    big[1:71, 8:104] = 9.0
    assert (big == 9).all()


def test_linear_input_grad_one_row_has_no_stride():
    dy, Wq, s_w = make_grad(1, 64, 48, 30)
    want = input_grad_ref(dy, Wq, s_w)[0]
    column = dy.cuda().view(64, 1).t()  # [1, 64] with strides (1, 1)
    assert column.stride(0) == 1
    assert torch.equal(w8a8.linear_input_grad(column, Wq.cuda(), s_w.cuda()).cpu(), want)
    out = torch.as_strided(torch.empty(64, dtype=torch.bfloat16, device="cuda"), (1, 48), (3, 1))
    for odd in (0, 7, 64):
        row = torch.as_strided(dy.cuda(), (1, 64), (odd, 1))
        assert torch.equal(w8a8.linear_input_grad(row, Wq.cuda(), s_w.cuda(), out=out).cpu(), want)


def test_linear_input_grad_against_the_unrounded_product():
    # every code stands within half a step of its value: the product is off by
    # at most s_g / 2 * sum |Wq| and its own rounding
    dy, Wq, s_w = make_grad(40, 520, 256, 23)
    got = w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda())
    full = (dy.double() * s_w.double()) @ Wq.double()
    s = (dy.double() * s_w.double()).abs().amax(1, keepdim=True) / 127
    slack = s * (0.5 + 127 * 4 * U) * Wq.double().abs().sum(0) + 4 * U * full.abs()
    close(got, full, slack, "dx")
    # and against differences of the layer: <dx, v> = d/dh <dy, (x + h v) W^T>
    v = torch.randn((40, 256), generator=gen(24), dtype=torch.float64)
    w64 = Wq.double() * s_w.double()[:, None]
    fwd = lambda x: ((x @ w64.T) * dy.double()).sum()  # noqa: E731
    diff = (fwd(v) - fwd(-v)) / 2
    tol = ((slack + rounding(full.abs() + slack, torch.bfloat16)) * v.abs()).sum()
    assert abs((got.cpu().double() * v).sum() - diff) <= tol


@pytest.mark.parametrize("M,N,K", [(600, 12288, 2064), (40, 264, 512), (320, 4096, 256)])
def test_linear_input_grad_workspace_contents_do_not_matter(M, N, K):
    dy, Wq, s_w = make_grad(M, N, K, 25)
    want = input_grad_ref(dy, Wq, s_w)[0]
    dyd, Wd, sd = dy.cuda(), Wq.cuda(), s_w.cuda()
    need = w8a8.input_grad_workspace_size(M, N, K)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [w8a8.linear_input_grad(dyd, Wd, sd, workspace=ws) for _ in range(3)]
    outs.append(w8a8.linear_input_grad(dyd, Wd, sd, workspace=ws[:((M * ((N + 15) // 16 * 16) + 255) // 256 + (4 * M + 255) // 256) * 256]))
    for o in outs:  # the last one without the K split's region
        assert torch.equal(o.cpu(), want)


def test_linear_input_grad_right_after_quantize_weights():
    # the channel scales and codes are written by the launch just before
    g = gen(26)
    dy = (torch.randn((48, 1024), generator=g) * 1e-3).bfloat16().cuda()
    for i in range(8):
        W = (torch.randn((1024, 2048), generator=g) * (i + 1)).bfloat16().cuda()
        torch.cuda.synchronize()
        Wq, s_w = w8a8.quantize_weights(W)
        got = w8a8.linear_input_grad(dy, Wq, s_w)
        assert torch.equal(got.cpu(), input_grad_ref(dy.cpu(), Wq.cpu(), s_w.cpu())[0])


def test_linear_input_grad_extreme_scales():
    # products next to the subnormals and next to the largest numbers: the
    # codes take the dividing path
    dy, Wq, s_w = make_grad(300, 64, 48, 27)
    scale = torch.ones(300)
    scale[::3], scale[1::3] = 1e-36, 1e36
    dy = (dy.float() * scale[:, None]).bfloat16()
    got = w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda())
    assert torch.equal(got.cpu(), input_grad_ref(dy, Wq, s_w)[0])
    few = w8a8.linear_input_grad(dy[:30].cuda(), Wq.cuda(), s_w.cuda())
    assert torch.equal(few.cpu(), got[:30].cpu())
    many = w8a8.linear_input_grad(dy.repeat(4, 1).cuda(), Wq.cuda(), s_w.cuda())
    assert torch.equal(many, got.repeat(4, 1))


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (20, 4096, 64), (20, 8192, 64), (300, 12288, 32), (20, 13000, 64),
                                   (1000, 12288, 32), (900, 5000, 256), (900, 24, 16)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_linear_input_grad_shows_what_is_not_finite(M, N, K, what):
    # anywhere in a row, in any number of rows: all of that row, and no other
    dy, Wq, s_w = make_grad(M, N, K, 29)
    want = input_grad_ref(dy, Wq, s_w)[0]
    rows = sorted({0, M // 3, M - 1})
    for i, r in enumerate(rows):
        dy[r, (i * N) // 3 + N // 4] = what
    got = w8a8.linear_input_grad(dy.cuda(), Wq.cuda(), s_w.cuda()).cpu()
    hit = torch.zeros(M, dtype=torch.bool)
    hit[rows] = True
    assert not torch.isfinite(got[hit].float()).any()
    if math.isnan(what):
        assert torch.isnan(got[hit].float()).all()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("M,N,K", [(3000, 12288, 32), (2400, 10240, 16), (2000, 9000, 64), (4000, 6144, 16), (5000, 2960, 16)])
def test_linear_input_grad_rows_of_a_shared_ring(M, N, K):
    # many rows per block in rings of 7, 9, 10 and 16 slots for 4, 8 and 16
    # groups, against calls of few rows, which take a block per row
    dy, Wq, s_w = (t.cuda() for t in make_grad(M, N, K, 28))
    want = torch.cat([w8a8.linear_input_grad(dy[i:i + 500], Wq, s_w) for i in range(0, M, 500)])
    for _ in range(10):
        assert torch.equal(w8a8.linear_input_grad(dy, Wq, s_w), want)


# ----------------------------------------------------------------- together

def block(x, p, act_rows):
    """One attention input: norm -> int8 projection -> rotary on q and k."""
    q8, s_a, mean, rstd = w8a8.group_norm_quant(x, p["groups"], p["w"], p["b"], return_stats=True)
    y = w8a8.linear(q8, s_a, p["Wq"], p["s_w"], p["bias"]).view(x.shape[0], act_rows, 3 * p["heads"], p["dim"])
    H = p["heads"]
    q, k = w8a8.rotary(y[:, :, :H], p["pos"], p["freq"], k=y[:, :, H:2 * H], out=y[:, :, :H], out_k=y[:, :, H:2 * H])
    return y, mean, rstd


def block_grad(dy, x, mean, rstd, p):
    H = p["heads"]
    w8a8.rotary(dy[:, :, :H], p["pos"], p["freq"], k=dy[:, :, H:2 * H], backward=True, out=dy[:, :, :H],
                out_k=dy[:, :, H:2 * H])
    dh = w8a8.linear_input_grad(dy.view(-1, 3 * H * p["dim"]), p["Wq"], p["s_w"])
    return w8a8.group_norm_backward(dh.view(x.shape), x, mean, rstd, p["w"], p["b"])


def make_block(Bn, S, C, heads, dim):
    g = gen(31)
    x = (torch.randn((Bn, S, C), generator=g) + 0.3).bfloat16().cuda()
    W = (torch.randn((3 * heads * dim, C), generator=g) * 0.05).bfloat16().cuda()
    Wq, s_w = w8a8.quantize_weights(W)
    p = {"groups": 8, "w": (1 + 0.1 * torch.randn(C, generator=g)).bfloat16().cuda(),
         "b": (0.1 * torch.randn(C, generator=g)).bfloat16().cuda(), "Wq": Wq, "s_w": s_w,
         "bias": (0.1 * torch.randn(3 * heads * dim, generator=g)).bfloat16().cuda(), "heads": heads, "dim": dim,
         "pos": torch.arange(S).cuda(), "freq": w8a8.rotary_frequencies(dim)[0]}
    return x, p


@pytest.mark.parametrize("Bn,S,C,heads,dim", [(2, 40, 64, 3, 16), (1, 300, 256, 4, 64)])
def test_block_forward_and_backward(Bn, S, C, heads, dim):
    x, p = make_block(Bn, S, C, heads, dim)
    y, mean, rstd = block(x, p, S)
    # the same steps in 64 bits, from the device's own int8 rows (their
    # rounding is checked above)
    q8, s_a = w8a8.group_norm_quant(x, p["groups"], p["w"], p["b"])
    lin = (q8.cpu().double() * s_a.cpu().double()[:, None]) @ (p["Wq"].cpu().double() * p["s_w"].cpu().double()[:, None]).T
    lin = (lin + p["bias"].cpu().double()).view(Bn, S, 3 * heads, dim)
    # the layer's bf16 result feeds the rotation: each of its values may be
    # half a bf16 step off (2^-8 of itself)
    pos = torch.arange(S).expand(Bn, S)[..., None]
    want, slack = rotary64(lin[:, :, :2 * heads], pos, p["freq"], "interleaved", torch.zeros(dim // 2), 1.0, False)
    a, b = lin[:, :, :2 * heads, 0::2].abs(), lin[:, :, :2 * heads, 1::2].abs()
    slack = slack + (2.0 ** -8 + 8 * U) * (a + b).repeat_interleave(2, -1)
    close(y[:, :, :2 * heads], want, slack, "q and k")
    close(y[:, :, 2 * heads:], lin[:, :, 2 * heads:], 8 * U * lin[:, :, 2 * heads:].abs(), "v")
    # backward, step by step against the definitions on the device's own inputs
    dy = torch.randn(y.shape, generator=gen(32)).bfloat16()
    turned = dy.cuda()
    dx, dw, db = block_grad(turned, x, mean, rstd, p)
    tw, ts = rotary64(dy[:, :, :2 * heads], pos, p["freq"], "interleaved", torch.zeros(dim // 2), 1.0, True)
    close(turned[:, :, :2 * heads], tw, ts, "turned")
    dh = input_grad_ref(turned.cpu().reshape(-1, 3 * heads * dim), p["Wq"].cpu(), p["s_w"].cpu())[0].view(x.shape)
    wx, ww, wb = grads64(dh, x.cpu(), 8, p["w"].cpu(), p["b"].cpu(), mean.cpu(), rstd.cpu(), False)
    close(dx, *wx, "dx")
    close(dw, *ww, "dweight")
    close(db, *wb, "dbias")


def test_block_in_a_graph_on_another_stream_and_twice():
    x, p = make_block(2, 300, 256, 4, 64)
    dy0 = torch.randn((2, 300, 12, 64), generator=gen(33)).bfloat16().cuda()
    y_ref, mean, rstd = block(x, p, 300)
    ref = block_grad(dy0.clone(), x, mean, rstd, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xin, dyin = x.clone(), dy0.clone()
    with torch.cuda.stream(side):
        block_grad(dy0.clone(), x, *block(x, p, 300)[1:], p)  # warm up
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, m, r = block(xin, p, 300)
        dyc = dyin.clone()
        dx, dw, db = block_grad(dyc, xin, m, r, p)
    # other inputs first, then the first ones again: a replay keeps nothing
    xin.copy_(x.flip(1))
    dyin.copy_(dy0.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    other = (y.clone(), dx.clone())
    xin.copy_(x)
    dyin.copy_(dy0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y_ref)
    for a, b in zip((dx, dw, db), ref):
        assert torch.equal(a, b)
    yo, mo, ro = block(x.flip(1).contiguous(), p, 300)
    assert torch.equal(other[0], yo)
    assert torch.equal(other[1], block_grad(dy0.flip(2).contiguous(), x.flip(1).contiguous(), mo, ro, p)[0])


def test_operators_on_a_given_stream():
    x, p = make_block(1, 64, 128, 2, 32)
    y_ref = block(x, p, 64)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q8, s_a = w8a8.group_norm_quant(x, 8, p["w"], p["b"], stream=s)
    y = w8a8.linear(q8, s_a, p["Wq"], p["s_w"], p["bias"], stream=s).view(1, 64, 6, 32)
    q = w8a8.rotary(y[:, :, :4], p["pos"], p["freq"], stream=s)
    s.synchronize()
    assert torch.equal(q, y_ref[:, :, :4]) and torch.equal(y[:, :, 4:], y_ref[:, :, 4:])
