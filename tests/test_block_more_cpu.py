"""The product with its epilogue, the step between two blocks and the balance
loss on the host, no GPU: sizes, and every argument check, all of which run
before any HIP call."""

import pytest
import torch

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from test_block_cpu import INV, ODD2, ODD4, ODD16, UNS, WS, A, At, C, D, E, F, G, H, refused


def each(args, bad, skip=()):
    """Argument lists with one argument after the other replaced by `bad`."""
    for i in range(len(args)):
        if i not in skip:
            yield args[:i] + [bad] + args[i + 1:]


# -------------------------------------------------------------------- linear

def lin(tokens=10, k=256, n=512, dtype=1, act=0, grad=0):
    return K.moe_linear(tokens, k, n, dtype, act, grad)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(k=0), INV), (dict(n=0), INV), (dict(dtype=2), INV), (dict(act=-1), INV),
    (dict(act=5), INV), (dict(dtype=0, grad=1), INV), (dict(grad=2), INV), (dict(k=65537), UNS), (dict(n=65537), UNS),
    (dict(tokens=1 << 31), UNS), (dict(tokens=1 << 20, n=65536), UNS), (dict(tokens=1 << 20, k=65536), UNS)])
def test_linear_problem_refusals(kw, code):
    l = lin(**kw)
    refused(code, K.moe_linear_fwd, l, A, C, D, E, F, G, H, stream=0)
    refused(code, K.moe_linear_bwd, l, A, C, D, E, F, G, H, A, stream=0)
    assert K.moe_linear_workspace_bytes(l) == K.moe_linear_workspace_bytes(l, True) == 0
    assert K.moe_linear_saved_bytes(l) == 0


def test_linear_argument_refusals():
    fwd, bwd = [A, C, D, E, F, G, H], [A, C, D, E, F, G, H, A]
    for args in each(fwd, None, skip=(2, 3, 4)):
        refused(INV, K.moe_linear_fwd, lin(), *args, workspace_bytes=1 << 30, stream=0)
    for args in each(fwd, ODD4):
        refused(INV, K.moe_linear_fwd, lin(), *args, workspace_bytes=1 << 30, stream=0)
    for args in each(bwd, None, skip=(6,)):
        refused(INV, K.moe_linear_bwd, lin(), *args, workspace_bytes=1 << 30, stream=0)
    for args in each(bwd, ODD4):
        refused(INV, K.moe_linear_bwd, lin(), *args, workspace_bytes=1 << 30, stream=0)
    refused(INV, K.moe_linear_fwd, lin(), A, C, D, E, ODD16, G, H, stream=0)
    refused(INV, K.moe_linear_fwd, lin(), A, C, D, E, F, G, ODD16, stream=0)
    for t in (10, 300):
        need = K.moe_linear_workspace_bytes(lin(t))
        refused(WS, K.moe_linear_fwd, lin(t), A, C, D, E, F, G, H, workspace_bytes=need - 1, stream=0)
        need = K.moe_linear_workspace_bytes(lin(t), True)
        refused(WS, K.moe_linear_bwd, lin(t), A, C, D, E, F, G, H, A, workspace_bytes=need - 1, stream=0)
    K.moe_linear_fwd(lin(0), None, None, None, None, None, None, None, stream=0)
    assert K.moe_linear_saved_bytes(lin(300, act=4)) == 0
    assert K.moe_linear_saved_bytes(lin(300, n=9)) >= 300 * 16 * 5 // 2
    assert K.moe_linear_saved_bytes(lin(300, n=9, dtype=0)) >= 300 * 16 * 4


def test_linear_tensor_refusals():
    l = K.Linear(6, 64, 96, "bf16", "silu")
    x, w, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((6, 64), (64, 96), (6, 96)))
    ws, bias = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(96)
    buf = K.LinearBuffers(y, ws, ws, x.clone(), torch.zeros(64, 96), bias.clone())
    cases = [dict(x=x[:5]), dict(x=x.float()), dict(x=torch.zeros(64, 6, dtype=x.dtype).t()), dict(w=w.t()),
             dict(w=w.float()), dict(bias=bias[:9]), dict(bias=bias.bfloat16()), dict(residual=y.float()),
             dict(residual=y[:, :5]), dict(x=x)]  # the last: not on a GPU
    for c in cases:
        a = dict(dict(x=x, w=w, bias=bias, residual=y), **c)
        with pytest.raises(ValueError):
            K.linear(l, a["x"], a["w"], buf, bias=a["bias"], residual=a["residual"])
    for name, t in (("y", y[:3]), ("workspace", ws[::2]), ("saved", ws[:5]), ("saved", None)):
        other = K.LinearBuffers(**dict(vars(buf), **{name: t}))
        with pytest.raises(ValueError):
            K.linear(l, x, w, other, training=True)
    for name, t in (("grad_x", y), ("grad_w", w), ("grad_bias", bias[:4]), ("saved", ws[:7]), ("workspace", bias)):
        other = K.LinearBuffers(**dict(vars(buf), **{name: t}))
        with pytest.raises(ValueError):
            K.linear_backward(l, x, w, y, other)
    with pytest.raises(ValueError):
        K.linear_backward(l, x, w, y[:2], buf)
    with pytest.raises(ValueError, match="GPU"):
        K.linear_backward(l, x, w, y, buf)
    with pytest.raises(ValueError, match="True or False"):
        K.linear_backward(l, x, w, y, buf, bias=bias)
    with pytest.raises(ValueError):
        K.allocate_linear(K.Linear(1, 70000, 5), "cpu")
    l.struct().tokens = 99  # the caller's own
    assert l.struct().tokens == 6


# ------------------------------------------------------------- residual step

def step(rows=10, width=512, dtype=1, kind=0, post=1, pre=1, eps=1e-5, scale=1.0, ld=(0,) * 8):
    return K.moe_residual_norm(rows, width, dtype, kind, post, pre, eps, scale, *ld)


P = dict(post_weight=A, post_bias=C, gate=D, pre_weight=E, pre_bias=F)


def lds(i, v):
    return tuple(v if j == i else 0 for j in range(8))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(width=0), INV), (dict(dtype=2), INV), (dict(kind=2), INV), (dict(kind=-1), INV),
    (dict(post=2), INV), (dict(pre=-1), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(width=16385), UNS), (dict(rows=1 << 31), UNS)]
    + [(dict(ld=lds(i, 511)), INV) for i in range(8)] + [(dict(ld=lds(i, 1 << 31)), UNS) for i in range(8)])
def test_step_problem_refusals(kw, code):
    n = step(**kw)
    refused(code, K.moe_residual_norm_fwd, n, A, C, P, D, E, F, stream=0)
    refused(code, K.moe_residual_norm_bwd, n, A, C, P, D, E, F, G, H, P, A, stream=0)
    assert K.moe_residual_norm_workspace_bytes(n) == 0


def test_step_argument_refusals():
    fwd, bwd = K.moe_residual_norm_fwd, K.moe_residual_norm_bwd
    for i in (0, 1, 3, 4):
        args = [A, C, P, D, E, F]
        args[i] = None
        refused(INV, fwd, step(), *args, stream=0)
        args[i] = At(0x1001)
        refused(INV, fwd, step(), *args, stream=0)
        args[i] = ODD2
        refused(INV, fwd, step(dtype=0), *args, stream=0)
    refused(INV, fwd, step(), A, C, P, D, E, ODD2, stream=0)
    refused(INV, fwd, step(), A, C, P, D, D, F, stream=0)
    refused(INV, fwd, step(pre=0), A, C, P, D, E, F, stream=0)
    for name in P:
        refused(INV, fwd, step(), A, C, dict(P, **{name: ODD2}), D, E, F, stream=0)
        refused(INV, bwd, step(), A, C, P, D, E, F, G, H, dict(P, **{name: ODD2}), A, stream=0)
    for i in (0, 1, 3, 5, 6, 7):
        args = [A, C, P, D, E, F, G, H, P, A]
        args[i] = None
        refused(INV, bwd, step(), *args, stream=0)
        args[i] = At(0x1001)
        refused(INV, bwd, step(), *args, stream=0)
    refused(INV, bwd, step(), A, C, P, D, E, F, G, G, P, A, stream=0)
    refused(INV, bwd, step(pre=0), A, C, P, D, E, F, G, H, P, A, stream=0)
    need = K.moe_residual_norm_workspace_bytes(step())
    assert need >= 4 * 512 * 4
    refused(WS, bwd, step(), A, C, P, D, E, F, G, H, P, A, workspace_bytes=need - 1, stream=0)
    refused(INV, bwd, step(), A, C, P, D, E, F, G, H, P, ODD16, workspace_bytes=need, stream=0)
    fwd(step(rows=0), None, None, {}, None, None, None, stream=0)
    bwd(step(rows=0), None, None, {}, None, None, None, None, None, {}, None, stream=0)


def test_step_tensor_refusals():
    n = K.ResidualNorm(6, 64, "bf16")
    z = torch.zeros(6, 64, dtype=torch.bfloat16)
    buf = K.allocate_residual_norm(n, "cpu", training=True)
    for c in (dict(z=z[:5]), dict(z=z.float()), dict(res=torch.zeros(64, 6, dtype=z.dtype).t()), dict(res=z[:1].expand(6, 64)),
              dict(gate=torch.zeros(63)), dict(post_bias=torch.zeros(64).bfloat16()), dict(z=z)):
        a = dict(dict(z=z, res=z, gate=None, post_bias=None), **c)
        with pytest.raises(ValueError):
            K.residual_norm(n, a["z"], a["res"], a, buf)
    for name in ("out", "y", "stats"):
        with pytest.raises(ValueError):
            K.residual_norm(n, z, z, {}, K.ResidualNormBuffers(**dict(vars(buf), **{name: z[:, :3]})))
    without = K.allocate_residual_norm(K.ResidualNorm(6, 64, "bf16", pre=False), "cpu")
    assert without.y is None
    with pytest.raises(ValueError, match="norm before"):
        K.residual_norm(n, z, z, {}, without)
    with pytest.raises(ValueError, match="training"):
        K.residual_norm_backward(n, z, z, {}, z, z, without)
    for go, gy in ((z, None), (z[:3], z), (z, z.float())):
        with pytest.raises(ValueError):
            K.residual_norm_backward(n, z, z, {}, go, gy, buf)
    for name, t in (("grad_z", z[:, :9]), ("grad_res", z.float()), ("grads", dict(buf.grads, gate=z)),
                    ("workspace", z), ("stats", z)):
        with pytest.raises(ValueError):
            K.residual_norm_backward(n, z, z, dict(gate=buf.grads["gate"]), z, z, K.ResidualNormBuffers(**dict(vars(buf), **{name: t})))
    with pytest.raises(ValueError, match="GPU"):
        K.residual_norm_backward(n, z, z, {}, z, z, buf)
    with pytest.raises(ValueError):
        K.allocate_residual_norm(K.ResidualNorm(1, 20000), "cpu")


# -------------------------------------------------------------- balance loss

def bal(tokens=100, experts=8, top_k=2, d=512, dtype=1, balance=0.01, z=0.001):
    return K.moe_balance(tokens, experts, top_k, d, dtype, balance, z)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(experts=0), INV), (dict(top_k=0), INV), (dict(top_k=9), INV), (dict(d=0), INV),
    (dict(dtype=2), INV), (dict(balance=float("nan")), INV), (dict(z=float("inf")), INV), (dict(experts=65), UNS),
    (dict(d=500), UNS), (dict(d=8320), UNS), (dict(tokens=1 << 30), UNS)])
def test_balance_problem_refusals(kw, code):
    b = bal(**kw)
    refused(code, K.moe_balance_loss, b, A, C, D, E, F, G, H, A, C, stream=0)
    refused(code, K.moe_balance_loss_bwd, b, A, C, D, E, False, G, H, A, stream=0)
    assert K.moe_balance_workspace_bytes(b) == K.moe_balance_saved_bytes(b) == 0


def test_balance_argument_refusals():
    fwd, bwd, big = K.moe_balance_loss, K.moe_balance_loss_bwd, 1 << 30
    args = [A, C, D, E, F, G, H, A, C]
    for a in each(args, None, skip=(3, 7)):
        refused(INV, fwd, bal(), *a, workspace_bytes=big, stream=0)
    for a in each(args, ODD2, skip=(3,)):
        refused(INV, fwd, bal(), *a, workspace_bytes=big, stream=0)
    refused(INV, fwd, bal(), A, C, D, E, F, G, H, ODD16, C, workspace_bytes=big, stream=0)
    need = K.moe_balance_workspace_bytes(bal())
    refused(WS, fwd, bal(), *args, workspace_bytes=need - 1, stream=0)
    args = [A, C, D, E, False, F, G, H]
    for a in each(args, None, skip=(1, 3, 4)):
        refused(INV, bwd, bal(), *a, workspace_bytes=big, stream=0)
    for a in each(args, ODD2, skip=(1, 4)):
        refused(INV, bwd, bal(), *a, workspace_bytes=big, stream=0)
    refused(INV, bwd, bal(), A, C, D, E, 2, F, G, H, workspace_bytes=big, stream=0)
    refused(WS, bwd, bal(), *args, workspace_bytes=need - 1, stream=0)
    assert K.moe_balance_saved_bytes(bal()) >= 100 * 32 * 4
    assert K.moe_balance_saved_bytes(bal(experts=33)) >= 100 * 64 * 4


def test_balance_tensor_refusals():
    b = K.BalanceLoss(10, 8, 2, 128, "bf16")
    x, w = torch.zeros(10, 128, dtype=torch.bfloat16), torch.zeros(128, 8)
    idx, mask = torch.zeros(10, 2, dtype=torch.int32), torch.ones(10, dtype=torch.bool)
    buf = K.allocate_balance_loss(b, "cpu", training=True)
    for c in (dict(x=x[:9]), dict(x=x.float()), dict(w=w.t()), dict(w=w.bfloat16()), dict(idx=idx.long()),
              dict(idx=idx[:, :1]), dict(mask=mask[:4]), dict(mask=mask.float()), dict(mask=mask.to(torch.uint8)[:3]),
              dict(x=x)):
        a = dict(dict(x=x, w=w, idx=idx, mask=mask), **c)
        with pytest.raises(ValueError):
            K.balance_loss(b, a["x"], a["w"], a["idx"], buf, mask=a["mask"])
    for name in ("loss", "mean_prob", "counts", "workspace", "saved"):
        with pytest.raises(ValueError):
            K.balance_loss(b, x, w, idx, K.BalanceBuffers(**dict(vars(buf), **{name: w[:3, :3]})), training=True)
    with pytest.raises(ValueError, match="training"):
        K.balance_loss(b, x, w, idx, K.allocate_balance_loss(b, "cpu"), training=True)
    for name in ("saved", "workspace", "grad_x", "grad_router"):
        with pytest.raises(ValueError):
            K.balance_loss_backward(b, x, w, K.BalanceBuffers(**dict(vars(buf), **{name: idx})))
    for kw in (dict(grad_loss=w), dict(grad_loss=torch.ones(1, dtype=torch.float64)), dict(mask=mask[1:]),
               dict(add_to=(x, x)), dict(add_to=(w, w)), {}):
        with pytest.raises(ValueError):
            K.balance_loss_backward(b, x, w, buf, **kw)
    with pytest.raises(ValueError):
        K.allocate_balance_loss(K.BalanceLoss(1, 8, 2, 100), "cpu")


def test_residual_layer_refusals():
    p = Problem(10, 8, 2, 128, 128, 0, "bf16", 32)
    x = torch.zeros(10, 128, dtype=torch.bfloat16)
    w = dict(w_router=torch.zeros(128, 8), w_gate=torch.zeros(8, 128, 128).bfloat16(),
             w_up=torch.zeros(8, 128, 128).bfloat16(), w_down=torch.zeros(8, 128, 128).bfloat16())
    n = K.ResidualNorm(10, 128, "bf16")
    buf, step = B.allocate(p, "cpu", training=True), K.allocate_residual_norm(n, "cpu", training=True)
    other = K.BalanceLoss(10, 4, 2, 128, "bf16")
    loss = (other, K.allocate_balance_loss(other, "cpu", training=True))
    with pytest.raises(ValueError):
        K.residual_layer_forward(p, x[:5], x, w, buf, n, step)
    with pytest.raises(ValueError, match="GPU"):
        K.residual_layer_forward(p, x, x, w, buf, n, step)
    with pytest.raises(ValueError, match="loss"):
        K.residual_layer_backward(p, x, x, w, x, x, buf, n, step, loss)
    with pytest.raises(ValueError, match="training"):
        K.residual_layer_backward(p, x, x, w, x, x, B.allocate(p, "cpu"), n, step)
