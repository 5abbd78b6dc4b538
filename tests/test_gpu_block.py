"""The operators around the layer on the GPU against plain 64-bit
computations: layer norm, the dense gated feed-forward block and products
with 8-bit integer weights (through the tensor front ends), and a run of them
together with the layer itself.

Tolerances, as the 2-norm of the difference over the 2-norm of the result
unless a test says otherwise. u is half a rounding step of the storage type
(bf16 2^-8, fp32 2^-24); each rounding of a result adds at most u, each
rounding of an operand inside a product at most u too (a sum's error is at
most the largest relative error of its terms when these are independent of
sign, which the 2-norm over a whole matrix of random sums respects with room).

* norm: y and dx are rounded once from fp32: u + 64 * 2^-24 (sums of up to
  16384 terms in a tree of at most 64 sequential additions a thread).
* ffn: hidden values rounded (1 u), output rounded (1 u): 2 u forward.
  Backward: the 20 bits kept of act(a) and b act'(a) (2^-12 each, far under
  1 u), da and db (1 u), result (1 u); 5 u has room over that, and
  test_gpu_block_forms.py holds the roundings themselves.
  fp32: sums of n products by MFMA in sequence add at most n 2^-24 in the
  worst case and about sqrt(n) 2^-24 in the 2-norm; 1e-5 covers n = 2^14.
* int8: the integers and their sums are exact; scaling rounds three times in
  fp32 (gated: SiLU adds 2^-21) and the result once: u + 2^-20.
"""

import math

import numpy as np
import pytest

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from gpu_util import Case, note

pytestmark = pytest.mark.gpu

U = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


def types():
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, std=1.0, dtype="fp32": (
        torch.randn(*shape, generator=g, device="cuda") * std).to(types()[dtype])


def off(got, want):
    got, want = got.double(), want.double()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float((got - want).norm())


def near(name, got, want, tol):
    import torch
    assert got.shape == want.shape, name
    assert bool(torch.isfinite(got.float()).all()), name
    e = off(got, want)
    assert e <= tol, f"{name}: {e:.3g} > {tol:.3g}"


# ---------------------------------------------------------------- layer norm

def norm64(x, w, b, eps, dy=None):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    xh = (x - mean) * rstd
    wd = 1.0 if w is None else w.double()
    y = xh * wd + (0.0 if b is None else b.double())
    if dy is None:
        return y, mean[:, 0], rstd[:, 0]
    g = dy.double() * wd
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return y, mean[:, 0], rstd[:, 0], dx, (dy.double() * xh).sum(0), dy.double().sum(0)


@pytest.mark.parametrize("rows,width,dtype", [
    (1, 1, "fp32"), (3, 1, "bf16"), (5, 2, "bf16"), (1, 7, "fp32"), (2, 511, "bf16"), (9, 512, "bf16"),
    (7, 513, "bf16"), (1000, 512, "bf16"), (33, 1024, "bf16"), (33, 1025, "bf16"), (6, 4096, "bf16"),
    (5, 4097, "bf16"), (5, 8192, "bf16"), (3, 8193, "bf16"), (2, 16384, "bf16"), (4, 255, "fp32"),
    (4, 257, "fp32"), (11, 1155, "fp32"), (3, 2049, "fp32"), (2, 4096, "fp32"), (2, 8191, "fp32"),
    (3, 8193, "fp32"), (2, 16383, "fp32"), (70001, 64, "bf16"), (5001, 130, "fp32"),
    (17, 200, "bf16"), (19, 100, "fp32"), (13, 700, "fp32"), (11, 900, "fp32"), (9, 2000, "bf16"), (7, 1500, "fp32"),
    (5, 5000, "bf16"), (4, 9000, "bf16"), (6, 2300, "fp32"), (3, 5000, "fp32")])
def test_norm(rows, width, dtype):
    note(f"norm {rows} {width} {dtype}")
    r = gen(rows + width)
    x = r(rows, width, dtype=dtype, std=2.0) + 1.5
    dy, w, b = r(rows, width, dtype=dtype), 1 + r(width, std=0.2), r(width, std=0.3)
    buf = K.allocate_norm(rows, width, dtype, training=True)
    K.layer_norm(x, w, b, 1e-5, buf)
    K.layer_norm_backward(x, w, dy, buf)
    y, mean, rstd, dx, dw, db = norm64(x, w, b, 1e-5, dy)
    acc = 64 * 2.0 ** -24
    near("y", buf.y, y, U[dtype] + acc)
    near("mean", buf.mean, mean, acc)
    near("rstd", buf.rstd, rstd, acc)
    if width > 1:
        # width 2: xh is +-1 and the two terms of dx cancel: hold dx to its terms' size
        scale = float((rstd[:, None] * dy.double() * w.double()).norm())
        assert float((buf.grad_x.double() - dx).norm()) <= U[dtype] * float(dx.norm()) + 2 * acc * scale
    # a column sums `rows` products: each thread's and the partials' sequential
    # additions stay under 1024, and the sum may cancel: hold it to its terms
    terms = float((dy.double().abs() * ((x.double() - mean[:, None]) * rstd[:, None]).abs()).sum(0).norm())
    assert float((buf.grad_weight.double() - dw).norm()) <= 1024 * 2.0 ** -24 * terms
    assert float((buf.grad_bias.double() - db).norm()) <= 1024 * 2.0 ** -24 * float(dy.double().abs().sum(0).norm())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("width", [96, 333, 2050])
def test_norm_strided_and_in_place(width, dtype):
    import torch
    r = gen(width)
    wide = r(21, 2 * width + 7, dtype=dtype)
    x = wide[:, 3:3 + width]  # rows at odd offsets
    w = 1 + r(width, std=0.2)
    buf = K.allocate_norm(21, width, dtype, training=True)
    K.layer_norm(x.contiguous(), w, None, 1e-5, buf)
    want = buf.y.clone()
    before = wide.clone()
    buf.y = torch.full((21, width + 5), 7.0, device="cuda").to(wide.dtype)[:, :width]
    K.layer_norm(x, w, None, 1e-5, buf)
    assert torch.equal(buf.y, want)
    assert bool((buf.y._base[:, width:] == 7).all()), "columns behind the rows were written"
    assert torch.equal(wide, before)
    dy = r(21, width + 1, dtype=dtype)[:, 1:]
    K.layer_norm_backward(x.contiguous(), w, dy.contiguous(), buf)
    gx, gw = buf.grad_x.clone(), buf.grad_weight.clone()
    # grad_x over grad_out, then y over x
    d2 = r(21, width + 1, dtype=dtype)[:, 1:]
    d2.copy_(dy)
    buf.grad_x = d2
    K.layer_norm_backward(x, w, d2, buf)
    assert torch.equal(d2, gx) and torch.equal(buf.grad_weight, gw)
    buf.y = x
    K.layer_norm(x, w, None, 1e-5, buf)
    assert torch.equal(x, want)
    assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, 3 + width:], before[:, 3 + width:])


def test_norm_optional_arguments_and_odd_values():
    import torch
    r = gen(3)
    x = r(40, 200) * 1e-3 + 1000.0  # a mean that a difference of squares would lose
    buf = K.allocate_norm(40, 200, "fp32", training=True)
    K.layer_norm(x, None, None, 0.0, buf)
    y, mean, rstd = norm64(x, None, None, 0.0)
    # x is spaced 2^-14 around 1000 and so is the mean: (x - mean) is off by up to
    # 2^-15 + 64 sequential roundings of the sum, against a deviation of 1e-3
    assert float((buf.y.double() - y).abs().max()) < (2.0 ** -14 * 4) / 1e-3
    x = r(6, 300, dtype="bf16")
    x[1, 7], x[2, 0], x[3] = float("nan"), float("inf"), 0.25
    K.layer_norm(x, None, None, 1e-5, buf := K.allocate_norm(6, 300, "bf16", training=True))
    fin = torch.isfinite(buf.y.float()).all(1).tolist()
    assert fin == [True, False, False, True, True, True]
    assert bool((buf.y[3] == 0).all())  # a constant row
    # gradients that are not wanted
    c = K.moe_norm(6, 300, 1, 0.0, 0, 0, 0, 0)
    K.moe_layer_norm_bwd(c, x, None, buf.mean, buf.rstd, x, buf.grad_x, None, None, None)
    gx = buf.grad_x.clone()
    buf.grad_bias.fill_(5)
    K.moe_layer_norm_bwd(c, x, None, buf.mean, buf.rstd, x, buf.grad_x, buf.grad_weight, None, buf.workspace)
    assert torch.equal(gx[3:], buf.grad_x[3:]) and bool((buf.grad_bias == 5).all())
    # no rows: gradients of zero
    b0 = K.allocate_norm(0, 300, "bf16", training=True)
    b0.grad_weight.fill_(1), b0.grad_bias.fill_(1)
    K.layer_norm(x[:0], None, None, 1e-5, b0)
    K.layer_norm_backward(x[:0], None, x[:0], b0)
    assert not b0.grad_weight.any() and not b0.grad_bias.any()


# -------------------------------------------------- gated feed-forward block

def act64(a, act):
    import torch
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "relu":
        return a.clamp(min=0)
    if act == "gelu":
        return a * 0.5 * torch.erfc(-a / math.sqrt(2))
    return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))


def ffn_case(t, d, h, dtype, act="silu", grad="fp32", seed=0, training=True):
    import torch
    r = gen(t * 7 + d + h + seed)
    f = K.GatedFfn(t, d, h, dtype, act, grad)
    x = r(t, d, dtype=dtype)
    w = dict(w_gate=r(d, h, std=d ** -0.5, dtype=dtype), w_up=r(d, h, std=d ** -0.5, dtype=dtype),
             w_down=r(h, d, std=h ** -0.5, dtype=dtype))
    dy = r(t, d, dtype=dtype)
    return f, x, w, dy, K.allocate_ffn(f, training=training)


def ffn64(x, w, dy, act):
    import torch
    leaves = [v.double().requires_grad_() for v in (x, w["w_gate"], w["w_up"], w["w_down"])]
    xd, wg, wu, wd = leaves
    y = (act64(xd @ wg, act) * (xd @ wu)) @ wd
    return y.detach(), torch.autograd.grad(y, leaves, dy.double())


FFN = [(1, 1, 1), (1, 128, 256), (2, 8, 24), (3, 65, 131), (5, 256, 128), (16, 512, 1024), (17, 100, 333),
       (31, 128, 128), (32, 192, 320), (33, 130, 257), (64, 512, 512), (65, 640, 129), (127, 256, 1000),
       (130, 512, 1024), (300, 333, 1001), (513, 1024, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,d,h", FFN)
def test_ffn(t, d, h, dtype):
    note(f"ffn {t} {d} {h} {dtype}")
    f, x, w, dy, buf = ffn_case(t, d, h, dtype)
    K.gated_ffn(f, x, w, buf)
    infer = buf.out.clone()
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    y, grads = ffn64(x, w, dy, "silu")
    u = U[dtype] if dtype == "bf16" else 1e-5
    near("inference", infer, y, 2 * u)
    near("out", buf.out, y, 2 * u)
    near("grad_x", buf.grad_x, grads[0], 5 * u)
    for name, g in zip(("w_gate", "w_up", "w_down"), grads[1:]):
        near(name, buf.grads[name], g, 5 * u)


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("t,d,h", [(17, 64, 64), (40, 2048, 512), (129, 64, 192), (200, 192, 320), (257, 1024, 4096),
                                   (300, 512, 64), (1000, 128, 512), (384, 1088, 576),
                                   (100, 64, 16384), (33, 128, 16448), (1300, 576, 2112), (515, 2048, 8192),
                                   (8200, 64, 192), (9000, 832, 64)])
def test_ffn_weights_in_place(t, d, h, act):
    """More tokens than the serving form is for, in widths that are multiples
    of 64 but not all of 128: the forward multiplies by the weights where they are."""
    note(f"ffn in place {t} {d} {h} {act}")
    f, x, w, dy, buf = ffn_case(t, d, h, "bf16", act)
    before = [v.clone() for v in w.values()]
    K.gated_ffn(f, x, w, buf)
    infer = buf.out.clone()
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    y, grads = ffn64(x, w, dy, act)
    u = U["bf16"]
    near("inference", infer, y, 2 * u)
    near("out", buf.out, y, 2 * u)
    near("grad_x", buf.grad_x, grads[0], 5 * u)
    for name, g in zip(("w_gate", "w_up", "w_down"), grads[1:]):
        near(name, buf.grads[name], g, 5 * u)
    assert all(bool((a == b).all()) for a, b in zip(before, w.values()))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("t,d,h,dtype,grad", [(7, 128, 256, "bf16", "bf16"), (300, 256, 385, "bf16", "bf16"),
                                              (150, 100, 200, "fp32", "fp32")])
def test_ffn_activations(t, d, h, dtype, grad, act):
    f, x, w, dy, buf = ffn_case(t, d, h, dtype, act, grad)
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    y, grads = ffn64(x, w, dy, act)
    u = U[dtype] if dtype == "bf16" else 1e-5
    near("out", buf.out, y, 2 * u)
    near("grad_x", buf.grad_x, grads[0], 5 * u)
    for name, g in zip(("w_gate", "w_up", "w_down"), grads[1:]):
        assert buf.grads[name].dtype == types()[grad]
        near(name, buf.grads[name], g, 6 * u)  # one more rounding into grad_dtype


@pytest.mark.parametrize("t,d,h,dtype", [(8200, 512, 1024, "bf16"), (16400, 1024, 1000, "bf16"),
                                         (8200, 512, 515, "fp32"), (200, 1024, 1400, "fp32")])
def test_ffn_large_and_ragged(t, d, h, dtype):
    """Sizes that take the larger tiles, with ragged last ones."""
    note(f"ffn large {t} {d} {h} {dtype}")
    f, x, w, dy, buf = ffn_case(t, d, h, dtype, grad=dtype)
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    y, grads = ffn64(x, w, dy, "silu")
    u = U[dtype] if dtype == "bf16" else 1e-5
    near("out", buf.out, y, 2 * u)
    for got, want in zip((buf.grad_x, *buf.grads.values()), grads):
        near("gradient", got, want, 6 * u)
    K.gated_ffn(f, x, w, buf)
    near("inference", buf.out, y, 2 * u)


def test_ffn_gradient_against_differences():
    """fp32 gradients against central differences of the 64-bit block."""
    f, x, w, dy, buf = ffn_case(9, 24, 40, "fp32", "gelu_tanh")
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    v = {n: t.double().cpu() for n, t in dict(w, x=x).items()}
    dyd = dy.double().cpu()

    def loss(v):
        return float(((act64(v["x"] @ v["w_gate"], "gelu_tanh") * (v["x"] @ v["w_up"])) @ v["w_down"] * dyd).sum())

    rng = np.random.default_rng(0)
    for name, g in dict(buf.grads, x=buf.grad_x).items():
        for _ in range(6):
            i = tuple(int(rng.integers(n)) for n in g.shape)
            step = 1e-5
            up, down = {n: t.clone() for n, t in v.items()}, {n: t.clone() for n, t in v.items()}
            up[name][i] += step
            down[name][i] -= step
            want = (loss(up) - loss(down)) / (2 * step)
            # differences: step^2 times a third derivative of order 1, rounding 2^-53 / step; kernel: 1e-5 of the largest
            assert abs(float(g[i]) - want) < 1e-7 + 2e-5 * float(g.abs().max()), (name, i)


@pytest.mark.parametrize("t", [1, 20, 200])
def test_ffn_odd_values_and_zero_tokens(t):
    """A token that is not finite spoils its own row only; no token at all
    gives weight gradients of zero; rows behind the last one stay."""
    import torch
    f, x, w, dy, buf = ffn_case(t, 96, 160, "bf16", grad="bf16")
    K.gated_ffn(f, x, w, buf)
    clean = buf.out.clone()
    x[t // 2, 5] = float("nan")
    room = torch.full((t + 3, 96), 9.0, device="cuda").bfloat16()
    buf.out = room[:t]
    K.gated_ffn(f, x, w, buf)
    keep = [i for i in range(t) if i != t // 2]
    assert torch.equal(room[:t][keep], clean[keep]) and bool(room[t // 2].isnan().all())
    assert bool((room[t:] == 9).all())
    # every activation keeps a NaN and the sizes that overflow inside its formula
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        fa = K.GatedFfn(t, 96, 160, "bf16", act, "bf16")
        K.gated_ffn(fa, x, w, buf)
        assert bool(room[t // 2].isnan().all()), act
        ba = K.allocate_ffn(fa, training=True)
        big = torch.where(x.isnan(), torch.zeros_like(x), x) * 1e18
        K.gated_ffn(fa, big, {n: v * (1e-19 if n == "w_up" else 1.0) for n, v in w.items()}, ba, training=True)
        K.gated_ffn_backward(fa, big, w, dy * 1e-12, ba)
        assert bool(torch.isfinite(ba.out.float()).all()) and bool(torch.isfinite(ba.grad_x.float()).all()), act
    f0 = K.GatedFfn(0, 96, 160, "bf16", grad_dtype="bf16")
    b0 = K.allocate_ffn(f0, training=True)
    for g in b0.grads.values():
        g.fill_(1)
    K.gated_ffn(f0, x[:0], w, b0, training=True)
    K.gated_ffn_backward(f0, x[:0], w, dy[:0], b0)
    assert not any(bool(g.any()) for g in b0.grads.values())


# ------------------------------------------------- products in 8-bit integers

def quantized(x):
    """The definition in numpy's fp32: (q int64, scale fp32)."""
    x = x.float().cpu().numpy()
    bad = ~np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        scale = np.abs(x).max(1) * np.float32(1 / 127)
        q = np.clip(np.round(x / np.where(scale > 0, scale, 1).astype(np.float32)[:, None]), -127, 127)
    q[bad] = 0
    scale[bad] = np.nan
    q[~(scale > 0)] = 0
    return q.astype(np.int64), scale


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 5), (7, 127), (5, 512), (2, 513), (9, 1024), (4, 2047),
                                        (3, 4096), (2, 8200), (2, 20001), (3000, 65)])
def test_quantize_rows(rows, width, dtype):
    import torch
    note(f"quantize {rows} {width} {dtype}")
    r = gen(rows + width)
    x = r(rows, width, dtype=dtype) * torch.exp(3 * r(rows, 1)).to(types()[dtype])
    if rows >= 3:
        x[0] = 0
        x[1, width // 2] = float("nan")
        x[2, 0] = float("-inf")
    q, s = K.quantize_rows(x)
    qw, sw = quantized(x)
    assert np.array_equal(s.cpu().numpy(), sw, equal_nan=True)
    assert np.array_equal(q[:, :width].cpu().numpy(), qw)
    assert not q[:, width:].any()
    ts = x.float().abs().amax(1) / 127.0  # the same expression in torch
    assert torch.equal(s[3:], ts[3:])
    if rows > 3:
        assert torch.equal(q[3:, :width].float(), torch.round(x[3:].float() / ts[3:, None]))
    # rows that lie apart
    wide = torch.cat([x, x], 1)[:, 1:1 + width]
    q2, s2 = K.quantize_rows(wide)
    assert np.array_equal(q2[:, :width].cpu().numpy(), quantized(wide)[0])


def test_quantize_ties_and_small_numbers():
    """Halves go to the even number; rows of subnormal numbers stay in range."""
    import torch
    x = torch.zeros(3, 260, device="cuda")
    x[0, :255] = torch.arange(-127, 128, device="cuda") / 2
    x[0, 255] = 127.0
    x[1, :4] = torch.tensor([1e-44, -3e-44, 2.8e-45, 0.0])
    x[2, :3] = torch.tensor([3.4e38, -3.4e38, 1e30])
    q, s = K.quantize_rows(x)
    qw, sw = quantized(x)
    assert float(s[0]) == 1.0
    assert np.array_equal(q[:, :260].cpu().numpy(), qw) and np.array_equal(s.cpu().numpy(), sw)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_quantize_weights(dtype):
    r = gen(5)
    g, u = r(3, 77, 130, dtype=dtype), r(3, 77, 130, dtype=dtype)
    q, s = K.quantize_weights(g, u)
    assert q.shape == (3, 260, 128)
    for e in range(3):
        for i, w in enumerate((g, u)):
            qw, sw = quantized(w[e].t())
            rows = slice(130 * i, 130 * (i + 1))
            assert np.array_equal(q[e, rows, :77].cpu().numpy(), qw)
            assert np.array_equal(s[e, rows].cpu().numpy(), sw)
    assert not q[:, :, 77:].any()


def dequantized(x):
    import torch
    q, s = quantized(x)
    return torch.from_numpy(q).cuda().double() * torch.from_numpy(s).cuda().double()[:, None]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 512, 512), (2, 100, 300), (4, 4096, 4096), (7, 130, 33),
                                   (16, 1024, 256), (17, 640, 129), (32, 128, 128), (33, 257, 1001),
                                   (100, 1111, 515), (128, 512, 512), (129, 8200, 64), (400, 333, 2049),
                                   (700, 65, 7), (2100, 384, 8200), (2100, 300, 2100),
                                   (4200, 1100, 4100), (8, 900, 300), (9, 1000, 40), (16, 1024, 8193),
                                   (3, 200, 8209), (16, 2000, 520), (60, 256, 16500), (120, 200, 33000)])
def test_linear_i8(t, k, n, dtype):
    note(f"linear_i8 {t} {k} {n} {dtype}")
    r = gen(t + k + n)
    x, bias = r(t, k, dtype=dtype), r(n)
    wq, ws = K.quantize_weights(r(k, n))
    l = K.LinearI8(t, k, n, dtype)
    buf = K.allocate_linear_i8(l)
    want = dequantized(x) @ (wq[0, :, :k].double() * ws[0].double()[:, None]).t()
    tol = U[dtype] + 2.0 ** -20
    near("y", K.linear_i8(l, x, wq, ws, buf), want, tol)
    first = buf.y.clone()
    near("with bias", K.linear_i8(l, x, wq, ws, buf, bias=bias), want + bias.double(), tol)
    # an input that is already quantised gives the same bits
    q, s = K.quantize_rows(x)
    K.linear_i8(l, q, wq, ws, buf, x_scale=s)
    import torch
    assert torch.equal(buf.y, first)


def test_linear_i8_odd_rows():
    """Zero rows give the bias, rows that are not finite give NaN, and only
    they do; the sums of extreme integers are exact."""
    import torch
    for t in (5, 40, 300):
        k, n = 20001, 70
        x = torch.ones(t, k, device="cuda")
        x[1] = 0
        x[2, 3] = float("nan")
        x[3, 0] = float("inf")
        wq = torch.full((1, n, K.moe_i8_pitch(k)), 127, dtype=torch.int8, device="cuda")
        wq[:, :, k:] = 0
        wq[0, 1] = -wq[0, 1]
        ws = torch.ones(1, n, device="cuda")
        l = K.LinearI8(t, k, n, "fp32")
        y = K.linear_i8(l, x, wq, ws, K.allocate_linear_i8(l), bias=torch.full((n,), 3.0, device="cuda"))
        one = float(np.float32(1) / np.float32(127))
        sums = np.float32(np.float32(127 * 127 * k) * np.float32(one)) + np.float32(3)
        assert bool((y[1] == 3).all()) and bool(y[2:4].isnan().all())
        assert bool((y[4:, 2:] == float(sums)).all()) and bool((y[0, 2:] == float(sums)).all())
        assert bool((y[4:, 1] < 0).all())


def routing_of(t, e, top, seed, skew=0.0):
    import torch
    r = gen(seed)
    logits = r(t, e) - skew * torch.arange(e, device="cuda")
    idx = torch.topk(logits, top, 1).indices.reshape(-1)
    perm = torch.sort(idx, stable=True).indices.to(torch.int32)
    counts = torch.bincount(idx, minlength=e)
    ends = torch.cumsum(counts, 0)
    return {"perm": perm, "expert_offsets": torch.cat([ends.new_zeros(1), ends]).to(torch.int32)}, counts.tolist()


@pytest.mark.parametrize("t,k,n,e,top,gated,dtype", [
    (1, 128, 256, 8, 2, True, "bf16"), (3, 100, 66, 5, 3, False, "fp32"), (40, 512, 512, 64, 8, True, "bf16"),
    (200, 130, 70, 4, 1, True, "fp32"), (500, 256, 258, 33, 4, False, "bf16"), (2000, 512, 256, 8, 2, True, "bf16"),
    (2500, 128, 130, 3, 3, False, "bf16"), (3000, 512, 512, 2, 1, True, "bf16"),
    (1, 130, 70, 64, 3, False, "fp32"), (7, 640, 512, 64, 1, True, "bf16"), (2, 100, 4200, 8, 2, False, "bf16"),
    (9000, 128, 258, 8, 2, True, "bf16"), (4000, 1100, 2100, 2, 2, False, "fp32"), (4000, 1100, 2200, 3, 2, True, "bf16")])
def test_linear_i8_routed(t, k, n, e, top, gated, dtype):
    import torch
    note(f"linear_i8 routed {t} {k} {n} {e} {top} {gated} {dtype}")
    r = gen(t + n)
    x, w = r(t, k, dtype=dtype), r(e, k, n, std=k ** -0.5)
    wq, ws = K.quantize_weights(w)
    routing, counts = routing_of(t, e, top, t, skew=0.3)
    cap = max(1, max(counts) // 2)
    token = (routing["perm"].long() // top).cpu()
    xd, wd = dequantized(x), wq[:, :, :k].double() * ws.double()[:, :, None]
    want = torch.cat([xd[token[sum(counts[:g]):sum(counts[:g + 1])]] @ wd[g].t() for g in range(e)])
    if gated:
        a, b = want.chunk(2, 1)
        want = a * torch.sigmoid(a) * b
    tol = U[dtype] + 2.0 ** -20
    l = K.LinearI8(t, k, n, dtype, groups=e, top_k=top, gated=gated)
    buf = K.allocate_linear_i8(l)
    near("gathered", K.linear_i8(l, x, wq, ws, buf, routing=routing), want, tol)
    first = buf.y.clone()
    q, qs = K.quantize_rows(x)
    assert torch.equal(K.linear_i8(l, q, wq, ws, buf, routing=routing, x_scale=qs), first)
    ls = K.LinearI8(t, k, n, dtype, groups=e, top_k=top, gated=gated, sorted_input=True)
    K.linear_i8(ls, x[token.cuda()].contiguous(), wq, ws, buf2 := K.allocate_linear_i8(ls), routing=routing)
    assert torch.equal(buf2.y, first)
    lc = K.LinearI8(t, k, n, dtype, groups=e, top_k=top, gated=gated, capacity=cap)
    buf.y.fill_(11.0)
    K.linear_i8(lc, x, wq, ws, buf, routing=routing)
    at = 0
    for c in counts:
        kept = min(c, cap)
        assert torch.equal(buf.y[at:at + kept], first[at:at + kept])
        assert bool((buf.y[at + kept:at + c] == 11).all()), "rows past the capacity were written"
        at += c


def test_linear_i8_one_expert():
    """A routing over a single expert is the dense product in perm's order."""
    import torch
    r = gen(8)
    for t in (9, 150):
        x, (wq, ws) = r(t, 200, dtype="bf16"), K.quantize_weights(r(200, 130))
        l = K.LinearI8(t, 200, 130, "bf16")
        want = K.linear_i8(l, x, wq, ws, K.allocate_linear_i8(l))
        perm = torch.arange(t, device="cuda", dtype=torch.int32).flip(0).contiguous()
        routing = {"perm": perm, "expert_offsets": torch.tensor([0, t], dtype=torch.int32, device="cuda")}
        got = K.linear_i8(l, x, wq, ws, K.allocate_linear_i8(l), routing=routing)
        assert torch.equal(got, want.flip(0))


# ----------------------------------------------------------------- long ones

def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes and 2^31 elements: the last rows come
    out as a small call makes them."""
    import torch
    note("large norm and int8")
    rows, width, last = 1_100_000, 2048, 300
    x = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = 1 + gen(2)(width, std=0.1)
    big = K.allocate_norm(rows, width, "bf16", training=True)
    small = K.allocate_norm(last, width, "bf16", training=True)
    tail = x[-last:].contiguous()
    assert torch.equal(K.layer_norm(x, w, None, 1e-5, big)[-last:], K.layer_norm(tail, w, None, 1e-5, small))
    K.layer_norm_backward(x, w, big.y, big)
    K.layer_norm_backward(tail, w, small.y, small)
    assert torch.equal(big.grad_x[-last:], small.grad_x)
    del big
    wide = x.view(rows // 2, 2 * width)
    q, s = K.quantize_rows(wide)
    wq, ws = K.quantize_weights(gen(3)(2 * width, 130))
    l = K.LinearI8(rows // 2, 2 * width, 130, "bf16")
    got = K.linear_i8(l, q, wq, ws, K.allocate_linear_i8(l), x_scale=s)
    ls = K.LinearI8(last, 2 * width, 130, "bf16")
    assert torch.equal(got[-last:], K.linear_i8(ls, wide[-last:].contiguous(), wq, ws, K.allocate_linear_i8(ls)))
    del x, wide, q
    note("large ffn")
    f, x, w, dy, buf = ffn_case(280_000, 64, 8000, "bf16", training=False)
    K.gated_ffn(f, x, w, buf)
    fs = K.GatedFfn(300, 64, 8000, "bf16")
    bs = K.allocate_ffn(fs)
    K.gated_ffn(fs, x[-300:].contiguous(), w, bs)
    near("last rows", buf.out[-300:], bs.out.double(), 2 * U["bf16"])


def test_many_rows():
    """More rows than a launch has workgroups for."""
    import torch
    n = 17_000_000
    x = torch.ones(n, 3, device="cuda")
    x[-1] = torch.tensor([1.0, -2.0, 0.5])
    q, s = K.quantize_rows(x)
    assert q[-1, :3].tolist() == [64, -127, 32] and float(s[-1]) == float(np.float32(2) / np.float32(127))
    assert bool((q[:-1, :3] == 127).all()) and not q[:, 3:].any()


# ------------------------------------------------------------- used together

def test_streams_and_graphs():
    """Calls on a side stream, two at once with their own buffers, and a
    captured run replayed between eager work."""
    import torch
    f, x, w, dy, buf = ffn_case(200, 192, 256, "bf16", grad="bf16")
    nb = K.allocate_norm(200, 192, "bf16", training=True)
    nw = 1 + gen(1)(192, std=0.1)
    wq, ws = K.quantize_weights(w["w_gate"].float())
    l = K.LinearI8(200, 192, 256, "bf16")
    lb = K.allocate_linear_i8(l)

    def step(buf, nb, lb, x):
        h = K.layer_norm(x, nw, None, 1e-5, nb)
        K.gated_ffn(f, h, w, buf, training=True)
        gx, _ = K.gated_ffn_backward(f, h, w, dy, buf)
        K.layer_norm_backward(x, nw, gx, nb)
        K.linear_i8(l, h, wq, ws, lb)

    def outs(buf, nb, lb):
        return [t.clone() for t in (buf.out, nb.grad_x, nb.grad_weight, nb.grad_bias, lb.y, *buf.grads.values())]

    step(buf, nb, lb, x)
    want = outs(buf, nb, lb)
    others = [(K.allocate_ffn(f, training=True), K.allocate_norm(200, 192, "bf16", training=True),
               K.allocate_linear_i8(l)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(streams, others):
        with torch.cuda.stream(s):
            step(*o, x)
    torch.cuda.synchronize()
    for o in others:
        assert all(torch.equal(a, b) for a, b in zip(outs(*o), want))
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(buf, nb, lb, xs)
    for i in range(4):
        xs.copy_(x * (1 + 0.5 * i))
        graph.replay()
        torch.cuda.synchronize()
        got = outs(buf, nb, lb)
        step(*others[0], xs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs(*others[0]))), i


def test_answering_in_a_graph():
    """One step of answering four sequences, captured and replayed: norm,
    gated block and a product in their serving forms, and the layer with 8-bit
    experts."""
    import torch
    p = Problem(4, 16, 4, 256, 128, 0, "bf16", 64)
    c = Case(p, seed=5)
    wt = c.weights()
    gu, dn = K.quantize_weights(wt["w_gate"], wt["w_up"]), K.quantize_weights(wt["w_down"])
    f, x, w, _, _ = ffn_case(4, 256, 500, "bf16", training=False)
    wq, ws = K.quantize_weights(gen(4)(256, 300))
    l = K.LinearI8(4, 256, 300, "bf16")
    nw = 1 + gen(1)(256, std=0.1)

    def make():
        return (K.allocate_norm(4, 256, "bf16"), K.allocate_ffn(f), K.allocate_experts_i8(p),
                B.allocate(p, "cuda"), K.allocate_linear_i8(l))

    def step(x, bufs):
        nb, fb, eb, mb, lb = bufs
        h = K.layer_norm(x, nw, None, 1e-5, nb)
        y = K.gated_ffn(f, h, w, fb)
        z = K.forward_i8(p, y, wt["w_router"], gu, dn, mb, eb)
        return K.linear_i8(l, z, wq, ws, lb)

    one, two, xs = make(), make(), x.clone()
    step(xs, one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(xs, one)
    for i in range(4):
        xs.copy_(x * (i + 1) + i)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step(xs, two)), i
        torch.cuda.synchronize()


def test_linear_i8_routing_changes_between_replays():
    """The tiles are counted on the device: a captured product follows rows
    that gather in one expert, spread over all, or leave most without any."""
    import torch
    note("linear_i8 replays")
    t, k, n, e = 130, 200, 192, 16
    r = gen(3)
    x, w = r(t, k, dtype="bf16"), r(e, k, n, std=k ** -0.5)
    wq, ws = K.quantize_weights(w)
    l = K.LinearI8(t, k, n, "bf16", groups=e)
    buf = K.allocate_linear_i8(l)
    routing = {"perm": torch.arange(t, dtype=torch.int32, device="cuda"),
               "expert_offsets": torch.zeros(e + 1, dtype=torch.int32, device="cuda")}
    routing["expert_offsets"][1:] = t
    K.linear_i8(l, x, wq, ws, buf, routing=routing)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.linear_i8(l, x, wq, ws, buf, routing=routing)
    xd = dequantized(x)
    for chosen in ([15], list(range(16)), [0], [3, 9], [0, 15]):
        idx = torch.tensor([chosen[i * 7 % len(chosen)] for i in range(t)], device="cuda")
        routing["perm"].copy_(torch.sort(idx, stable=True).indices)
        routing["expert_offsets"][1:] = torch.cumsum(torch.bincount(idx, minlength=e), 0)
        buf.y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        order = routing["perm"].long()
        wd = wq[:, :, :k].double() * ws.double()[:, :, None]
        want = torch.stack([xd[i] @ wd[idx[i]].t() for i in order.tolist()])
        near(f"experts {chosen}", buf.y, want, U["bf16"] + 2.0 ** -20)


def test_int8_experts_in_the_layer():
    """Serving with 8-bit experts: route, permute, gated product, product,
    combine, against the layer with the experts' weights as they were rounded."""
    import torch
    p = Problem(700, 16, 4, 256, 128, 0, "bf16", 64)
    c = Case(p, seed=3)
    x, wt = c.dev["x"], c.weights()
    gu, gus = K.quantize_weights(wt["w_gate"], wt["w_up"])
    dn, dns = K.quantize_weights(wt["w_down"])
    got = K.forward_i8(p, x, wt["w_router"], (gu, gus), (dn, dns), c.buf,
                       K.allocate_experts_i8(p, "cuda"))
    rounded = dict(wt)
    deq = (gu[:, :, :256].float() * gus[:, :, None]).transpose(1, 2)
    rounded["w_gate"], rounded["w_up"] = deq[:, :, :128].bfloat16().contiguous(), deq[:, :, 128:].bfloat16().contiguous()
    rounded["w_down"] = (dn[:, :, :128].float() * dns[:, :, None]).transpose(1, 2).bfloat16().contiguous()
    c2 = Case(p, seed=3)
    want = B.forward(p, x, rounded, c2.buf)
    assert torch.equal(c.buf.routing["perm"], c2.buf.routing["perm"])
    # two quantisations of activations, each a uniform error of a step: amax / 127 / sqrt(12) against
    # a deviation of amax / 3.5 or less: 1 % each, and bf16 roundings of the reference's weights
    near("layer", got, want, 0.03)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prenorm_layer(dtype):
    """The layer behind its norm, forward and backward, against the two run
    one after the other."""
    import torch
    p = Problem(300, 8, 2, 256, 128, 128, dtype, 64)
    c = Case(p, seed=1, training=True)
    w = c.weights()
    r = gen(9)
    w["norm_weight"], w["norm_bias"] = 1 + r(256, std=0.2), r(256, std=0.2)
    x, g = c.dev["x"], c.dev["grad_out"]
    nb = K.allocate_norm(300, 256, dtype, training=True)
    out = K.prenorm_forward(p, x, w, c.buf, nb, training=True).clone()
    gx, grads = K.prenorm_backward(p, x, w, g, c.buf, nb)
    d = Case(p, seed=1, training=True)
    nb2 = K.allocate_norm(300, 256, dtype, training=True)
    h = K.layer_norm(x, w["norm_weight"], w["norm_bias"], 1e-5, nb2)
    want = B.forward(p, h, d.weights(), d.buf, training=True)
    gh, gw = B.backward(p, h, d.weights(), g, d.buf)
    gx2, dw, db = K.layer_norm_backward(x, w["norm_weight"], gh, nb2)
    assert torch.equal(out, want) and torch.equal(gx, gx2)
    assert torch.equal(grads["norm_weight"], dw) and torch.equal(grads["norm_bias"], db)
    for n in gw:
        assert torch.equal(grads[n], gw[n]), n
