"""Forms of the product, the residual step and the balance loss that need a look
of their own. Tolerances are derived at each test; u as in test_gpu_block.py is half
a rounding step of the storage type (bf16 2^-8, fp32 2^-24)."""

import pytest

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from gpu_util import Case, note
from test_gpu_block import U, act64, gen, off
from test_gpu_block_forms import slope64
from test_gpu_block_more import balance64, balance_case, linear_case, step_params
from test_gpu_block_more import test_step_strided_and_in_place as strided_and_in_place

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- product

def products64(x, w, b, dy, act):
    """da and the gradients (dx, dw, dbias) in 64 bits, and the sizes of their
    terms; with the sizes of the terms that the slopes' errors make, dy for da."""
    x, w, dy = x.double(), w.double(), dy.double()
    a = x @ w + b.double()
    da = dy * slope64(a, act)

    def back(da, x, w):
        return da @ w.t(), x.t() @ da, da.sum(0)

    return da, back(da, x, w), back(da.abs(), x.abs(), w.abs()), back(dy.abs(), x.abs(), w.abs())


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k,n", [(1, 130, 70), (7, 2048, 4096), (16, 2048, 2048),   # on one side of the limits
                                   (1, 64, 4104), (2, 9001, 33), (7, 8200, 40), (16, 2056, 2048), (9, 70, 6001),
                                   (1, 4096, 8192), (16, 65536, 8)])                   # and on the other
def test_linear_few_rows_round_the_result_only(t, k, n, grad):
    """Every gradient of up to 16 bf16 rows, element by element: half a step of
    its type; da as two bf16 numbers, which leave 2^-17 of it; fp32 sums, sqrt(terms)
    2^-24 four times over; and slopes off by 2^-20, as they are kept and GELU's
    distribution is fitted, and by the error of a, four sqrt(k) 2^-24 of its deviation of
    about one, times the slope's own slope, below 0.8. (da rounded to bf16 would be 2^-9 off
    in every term of a column of dw.)"""
    note(f"linear few rows {t} {k} {n} {grad}")
    l, x, w, b, _, dy, buf = linear_case(t, k, n, "bf16", "gelu", grad, res=False)
    for m in (buf.grad_x, buf.grad_w, buf.grad_bias):
        m.fill_(float("nan"))
    K.linear(l, x, w, buf, bias=b, training=True)
    buf.workspace.fill_(255)
    got = K.linear_backward(l, x, w, dy, buf)
    _, want, terms, slopes = products64(x, w, b, dy, "gelu")
    u = 2.0 ** -24
    slope = 2.0 ** -20 + 0.8 * 4 * k ** 0.5 * u
    for name, g, v, size, dsize, half, long in zip(("dx", "dw", "dbias"), got, want, terms, slopes,
                                                   (U["bf16"], U[grad], 0.0), (n, t, t)):
        bound = half * v.abs() + ((0.0 if name == "dbias" else 2.0 ** -17) + 4 * long ** 0.5 * u) * size + slope * dsize
        assert bool(((g.double() - v).abs() <= bound).all()), name


@pytest.mark.parametrize("t,k,n", [(3, 64, 96), (3, 64, 4104), (16, 8200, 65)])
def test_linear_few_rows_infinities(t, k, n):
    """Infinite gradients, inputs and weights give what they give in da and its
    products, whatever the second half of a number is."""
    import torch
    note(f"linear few rows infinities {t} {k} {n}")
    l, x, w, b, _, dy, buf = linear_case(t, k, n, "bf16", "gelu", "fp32", res=False)

    def run(x, w, dy):
        # the forward's slopes are those of finite numbers
        return [g.clone() for g in K.linear_backward(l, x, w, dy, buf)]

    K.linear(l, x, w, buf, bias=b, training=True)
    plain = run(x, w, dy)
    da, want, _, _ = products64(x, w, b, dy, "gelu")
    inf = float("inf")
    dys, xs, ws = dy.clone(), x.clone(), w.clone()
    dys[1, 3], xs[2, 5], ws[7, 2] = inf, -inf, inf
    gx, gw, gb = run(x, w, dys)
    sign = (dys[1, 3].double() * (da[1, 3] / dy[1, 3].double())).sign()
    assert bool((gx[1].double() == inf * sign * w[:, 3].double().sign()).all())
    assert bool((gw[:, 3].double() == inf * sign * x[1].double().sign()).all()) and float(gb[3]) == float(inf * sign)
    others = torch.arange(n, device="cuda") != 3
    assert torch.equal(gw[:, others], plain[1][:, others]) and torch.equal(gx[[0, 2]], plain[0][[0, 2]])
    gx, gw, gb = run(xs, w, dy)
    assert torch.equal(gx, plain[0]) and torch.equal(gb, plain[2])
    assert bool((gw[5].double() == -inf * da[2].sign()).all())
    others = torch.arange(k, device="cuda") != 5
    assert torch.equal(gw[others], plain[1][others])
    gx, gw, gb = run(x, ws, dy)
    assert bool((gx[:, 7].double() == inf * da[:, 2].sign()).all())
    others = torch.arange(k, device="cuda") != 7
    assert torch.equal(gx[:, others], plain[0][:, others]) and torch.equal(gw, plain[1])


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k,n,act", [(17, 300, 200, "gelu"), (33, 512, 1000, "silu"), (300, 1024, 512, "gelu_tanh"),
                                       (2000, 256, 512, "silu"), (2000, 2048, 640, "gelu"), (5000, 640, 1155, "silu")])
def test_linear_roundings(t, k, n, act, grad):
    """From 17 bf16 rows on the results are rounded, and da before its products, and
    nothing else that counts. These roundings are made here in 64 bits, and a kernel may
    be off the unrounded result by at most 1.08 times what they are, in the 2-norm: slopes
    are off by 2^-20, sums in fp32 by less than 2^-18, beside errors of 2^-10 and more, and
    the roundings of thousands of elements average to a few per cent at most. Every call
    repeats bit for bit, whatever its buffers held."""
    import torch
    note(f"linear roundings {t} {k} {n} {act} {grad}")
    l, x, w, b, add, dy, buf = linear_case(t, k, n, "bf16", act, grad)
    da, (dx, dw, _), _, _ = products64(x, w, b, dy, act)
    y = act64(x.double() @ w.double() + b.double(), act) + add.double()
    da = da.bfloat16().double()
    rx, rw = (da @ w.double().t()).bfloat16(), (x.double().t() @ da).to(buf.grad_w.dtype)
    once = None
    for fill in (255, 0):
        for m in (buf.workspace, buf.saved):
            m.fill_(fill)
        K.linear(l, x, w, buf, bias=b, residual=add, training=True)
        buf.workspace.fill_(fill)
        got = [buf.y.clone(), *(g.clone() for g in K.linear_backward(l, x, w, dy, buf))]
        for name, g, r, want in zip(("y", "dx", "dw"), got, (y.bfloat16(), rx, rw), (y, dx, dw)):
            assert off(g, want) <= 1.08 * off(r, want), name
        assert once is None or all(torch.equal(a, c) for a, c in zip(got, once))
        once = got


# ------------------------------------------------------------- residual step

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 1), (9, 65), (700, 512), (300, 1155), (5, 6200), (4, 16384)])
def test_step_gradients_of_an_absent_norm(rows, width, dtype):
    """A norm that is not there has gradients of zero, whatever the streams hold,
    and the other parameters' are what they are without its parameters."""
    import torch
    for post, pre, kind in ((False, True, "layer"), (True, False, "rms"), (False, False, "layer")):
        note(f"absent norm {rows} {width} {dtype} post {post} pre {pre}")
        n = K.ResidualNorm(rows, width, dtype, kind, scale=0.75, post=post, pre=pre)
        r = gen(rows + width)
        z, res, go = (r(rows, width, dtype=dtype) for _ in range(3))
        gy = r(rows, width, dtype=dtype) if pre else None
        p = step_params(r, width, K.NORM_PARAMS)
        absent = [k for k in K.NORM_PARAMS if k.startswith("post") and not post or k.startswith("pre") and not pre]
        for odd in (False, True):
            if odd:
                z[0, 0], res[-1, -1] = float("inf"), float("nan")
            buf = K.allocate_residual_norm(n, "cuda", training=True)
            for t in buf.grads.values():
                t.fill_(float("nan"))
            buf.workspace.fill_(255)
            K.residual_norm(n, z, res, p, buf)
            g = K.residual_norm_backward(n, z, res, p, go, gy, buf)[2]
            assert set(g) == set(K.NORM_PARAMS)
            for k in absent:
                assert torch.equal(g[k], torch.zeros_like(g[k])), k
            only = {k: v for k, v in p.items() if k not in absent}
            want = K.allocate_residual_norm(n, "cuda", training=True)
            K.residual_norm(n, z, res, only, want)
            w = K.residual_norm_backward(n, z, res, only, go, gy, want)[2]
            assert set(w) == set(only)
            for k in only:
                assert torch.equal(g[k].view(torch.int32), w[k].view(torch.int32)), k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [257, 4100, 6200, 8191, 8200, 16383])
def test_wide_step_strided_and_in_place(width, dtype):
    # rows of several waves, and workgroups of 1024 threads that read the parameters
    # for every row
    note(f"step strided {width} {dtype}")
    strided_and_in_place(width, dtype)


# -------------------------------------------------------------- balance loss

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,e,k,d", [(31, 5, 2, 256), (200, 8, 2, 512), (1000, 47, 6, 1152), (5000, 64, 8, 512),
                                     (8193, 40, 2, 256), (66000, 20, 2, 128)])
def test_balance_each_loss(t, e, k, d, dtype):
    """Each of the three against its own size. A logit is off by sqrt(d) 2^-24 of
    |x| |w|, under 2^-20, p by that and an exponential's 2^-21 of itself and lse by as
    much: 2^-18 of each loss, whose terms are of one sign, holds both. The weighted sum
    is held to its two terms."""
    import torch
    note(f"balance losses {t} {e} {k} {d} {dtype}")
    for kw in ({}, dict(balance=1.0, z=0.1), dict(balance=0.5, z=-0.02)):
        b, x, w, idx, m, buf = balance_case(t, e, k, d, dtype, mask=0.8, **kw)
        want = balance64(b, x, w, idx, m)[0].tolist()
        c1, c2 = (float(torch.tensor(c, dtype=torch.float32)) for c in (b.balance, b.z))
        for training in (False, True):
            got = K.balance_loss(b, x, w, idx, buf, mask=m, training=training).tolist()
            for i in (1, 2):
                assert abs(got[i] - want[i]) <= 2.0 ** -18 * want[i], i
            assert abs(got[0] - (c1 * want[1] + c2 * want[2])) <= 2.0 ** -18 * (abs(c1) * want[1] + abs(c2) * want[2])


@pytest.mark.parametrize("t,e,k,d", [(300, 8, 2, 512), (4999, 33, 3, 1152), (16384, 64, 8, 512)])
def test_balance_gradient_is_rounded_once(t, e, k, d):
    """dx in bf16, element by element: half a step; dl and the router as two bf16
    numbers each, which leave 2^-17 of either and, of the product of their second ones,
    2^-16; and dl itself, whose p, lse and shares are 2^-18 off, from the size of its
    terms. In the 2-norm that is nothing beside the rounding. Calls repeat bit for bit."""
    import torch
    note(f"balance dx {t} {e} {k} {d}")
    b, x, w, idx, m, buf = balance_case(t, e, k, d, "bf16", mask=0.9)
    _, p, counts, dx, _ = balance64(b, x, w, idx, m)
    n, l, w64 = int(m.sum()), x.double() @ w.double(), w.double().abs()
    p, lse, f = torch.softmax(l, 1), torch.logsumexp(l, 1, keepdim=True), counts.double() / (int(m.sum()) * k)
    inner = (p * f).sum(1, keepdim=True)
    dl = p * (b.balance * e * (f - inner) + 2 * b.z * lse) / n
    terms = p * (b.balance * e * (f + inner) + 2 * b.z * lse.abs()) / n
    bound = U["bf16"] * dx.abs() + 2.0 ** -15 * dl.abs() @ w64.t() + 2.0 ** -18 * terms @ w64.t()
    once = None
    for fill in (255, 0):
        for t in (buf.workspace, buf.saved):
            t.fill_(fill)
        K.balance_loss(b, x, w, idx, buf, mask=m, training=True)
        buf.workspace.fill_(fill)
        gx, gw = (g.clone() for g in K.balance_loss_backward(b, x, w, buf, mask=m))
        assert bool(((gx.double() - dx).abs() <= bound).all())
        assert off(gx, dx) <= 1.01 * off(dx.bfloat16(), dx)
        assert once is None or torch.equal(gx, once[0]) and torch.equal(gw, once[1])
        once = gx, gw


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_residual_layer_of_a_problem_struct(dtype):
    # the layer's C problem, whose type is a number, gives what the named one gives
    import torch
    p = Problem(70, 8, 2, 128, 128, 0, dtype, 64)
    c, r = Case(p, seed=3, training=True), gen(11)
    n, b = K.ResidualNorm(70, 128, dtype), K.BalanceLoss(70, 8, 2, 128, dtype, 1.0, 0.1)
    step, loss = K.allocate_residual_norm(n, "cuda", training=True), K.allocate_balance_loss(b, "cuda", training=True)
    h, w, res, go, gy = c.dev["x"], c.weights(), *(r(70, 128, dtype=dtype) for _ in range(3))
    got = []
    for problem in (p, B.problem_struct(p)):
        out, y = K.residual_layer_forward(problem, h, res, w, c.buf, n, step, (b, loss), training=True)
        gh, gs, grads = K.residual_layer_backward(problem, h, res, w, go, gy, c.buf, n, step, (b, loss))
        got.append([t.clone() for t in (out, y, loss.loss, gh, gs, *(grads[k] for k in sorted(grads)))])
    assert all(torch.equal(a, c) for a, c in zip(*got))


def test_residual_layer_refuses_before_it_launches():
    """A part that does not fit leaves every buffer as it was."""
    import torch
    p = Problem(70, 8, 2, 128, 128, 0, "bf16", 64)
    c, r = Case(p, seed=4, training=True), gen(12)
    n, b = K.ResidualNorm(70, 128, "bf16"), K.BalanceLoss(70, 8, 2, 128, "bf16")
    step, loss = K.allocate_residual_norm(n, "cuda", training=True), K.allocate_balance_loss(b, "cuda", training=True)
    h, w, res, go, gy = c.dev["x"], c.weights(), *(r(70, 128, dtype="bf16") for _ in range(3))
    mask = torch.ones(70, dtype=torch.bool, device="cuda")
    kept = [c.buf.out, c.buf.saved, c.buf.grad_x, *c.buf.grads.values(), *c.buf.routing.values(), step.out, step.y,
            step.stats, step.grad_z, step.grad_res, loss.loss, loss.counts, loss.saved]
    for t in kept:
        t.fill_(7)
    bad = [dict(res=res[:69]), dict(res=res.float()), dict(mask=mask[:69]), dict(mask=mask.float()),
           dict(w=dict(w, gate=r(127))), dict(loss=(K.BalanceLoss(70, 8, 2, 128, "fp32"), loss))]
    for kw in bad:
        a = dict(dict(res=res, mask=mask, w=w, loss=(b, loss)), **kw)
        with pytest.raises(ValueError):
            K.residual_layer_forward(p, h, a["res"], a["w"], c.buf, n, step, a["loss"], a["mask"], training=True)
        with pytest.raises(ValueError):
            K.residual_layer_backward(p, h, a["res"], a["w"], go, gy, c.buf, n, step, a["loss"], mask=a["mask"])
    for go2, gy2, gl in ((go[:9], gy, None), (go, None, None), (go, gy, r(2))):
        with pytest.raises(ValueError):
            K.residual_layer_backward(p, h, res, w, go2, gy2, c.buf, n, step, (b, loss), gl, mask)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in kept)
