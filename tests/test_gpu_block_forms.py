"""Forms of the operators around the layer that need a look of their own: what
the gated block's roundings leave, that its calls repeat bit for bit whatever
their buffers held, the dense gated 8-bit product, and every buffer of the
layer with 8-bit experts.

The gated block in bf16 rounds: the hidden values (in the serving form to a
sum of two bf16 numbers, 2^-17, which does not count), act(a) and b act'(a)
to 20 bits (2^-12), da and db, and every result of that type. These roundings
are made here in 64 bits, and a kernel may be off the unrounded result by at
most 1.08 times what they are, in the 2-norm: the 20 bits add 2^-12 / sqrt(3)
to errors of 2^-9 and more, under 1 %, sums in fp32 less, and the rounding
errors of thousands of elements average to a few per cent at most. Values
kept to 16 bits instead of 20 would give 1.35 times and more, swapped low bits
1.3, a serving form that rounds its hidden values 1.4.
"""

import pytest

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from gpu_util import Case, note
from test_gpu_block import U, act64, ffn64, ffn_case, gen, near, off, quantized

pytestmark = pytest.mark.gpu


def slope64(a, act):
    import torch
    a = a.detach().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(act64(a, act).sum(), a)[0]


def rounded64(x, w, dy, act, hidden=True):
    """The block and its gradients in 64 bits with bf16 roundings of the hidden
    values (``hidden``), da and db; the results are not rounded."""
    r = lambda v: v.bfloat16().double()
    x, wg, wu, wd, dy = (v.double() for v in (x, w["w_gate"], w["w_up"], w["w_down"], dy))
    a, b = x @ wg, x @ wu
    f, h = act64(a, act), act64(a, act) * b
    dh = dy @ wd.t()
    da, db = r(dh * b * slope64(a, act)), r(dh * f)
    return ((r(h) if hidden else h) @ wd,
            (da @ wg.t() + db @ wu.t(), x.t() @ da, x.t() @ db, r(h).t() @ dy))


def along(got, want):
    """How much longer ``got`` is than ``want`` in its direction."""
    got, want = got.double(), want.double()
    return float((got * want).sum() / (want * want).sum()) - 1


ROUNDINGS = [(4, 512, 1024, "silu"), (16, 500, 1001, "gelu"), (17, 512, 1024, "silu"), (130, 333, 1001, "gelu_tanh"),
             (200, 512, 1024, "silu"), (2000, 256, 512, "silu"), (4100, 640, 1152, "gelu")]


@pytest.mark.parametrize("t,d,h,act", ROUNDINGS)
def test_ffn_roundings(t, d, h, act):
    note(f"ffn roundings {t} {d} {h} {act}")
    f, x, w, dy, buf = ffn_case(t, d, h, "bf16", act)
    y, grads = ffn64(x, w, dy, act)
    ry, rgrads = rounded64(x, w, dy, act, hidden=t > 16)
    K.gated_ffn(f, x, w, buf)
    limit = 1.08 * off(ry.bfloat16(), y)
    assert off(buf.out, y) <= limit, "inference"
    K.gated_ffn(f, x, w, buf, training=True)
    assert off(buf.out, y) <= limit, "training"
    K.gated_ffn_backward(f, x, w, dy, buf)
    got = (buf.grad_x, buf.grads["w_gate"], buf.grads["w_up"], buf.grads["w_down"])
    for name, g, rg, want in zip(("x", "w_gate", "w_up", "w_down"), got, rgrads, grads):
        limit = 1.08 * off(rg.bfloat16() if name == "x" else rg, want)
        assert off(g, want) <= limit, name


@pytest.mark.parametrize("t,d,h,act", [(2000, 256, 512, "silu"), (3000, 200, 400, "gelu")])
def test_ffn_gradients_are_not_short(t, d, h, act):
    """What the forward keeps is rounded to nearest, not cut: cutting to 20 bits
    shortens every value by 1.8e-4 on average, and so the gradients, over
    however many tokens. Beside the roundings of da and db, which are made here
    as well, rounding what is kept changes da and db by 2^-12 at most, which
    moves one in 16 of them to the next bf16 number: 2^-8 / sqrt(16) = 1e-3 in
    the 2-norm, at random, so 1e-3 / sqrt(d h) along the gradient: 3.5e-6 at
    most here, and 3e-5 is more than eight times that."""
    note(f"ffn gradients {t} {d} {h} {act}")
    f, x, w, dy, buf = ffn_case(t, d, h, "bf16", act)
    K.gated_ffn(f, x, w, buf, training=True)
    K.gated_ffn_backward(f, x, w, dy, buf)
    _, grads = ffn64(x, w, dy, act)
    _, rgrads = rounded64(x, w, dy, act)
    for name, rg, want in zip(("w_gate", "w_up"), rgrads[1:], grads[1:]):
        assert abs(along(buf.grads[name], want) - along(rg, want)) < 3e-5, name


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("t,d,h", [(1, 130, 200), (16, 64, 128), (17, 130, 200), (40, 64, 192), (300, 128, 256)])
def test_ffn_kept_activations(t, d, h, act):
    """act(a) and b act'(a) as they are kept, element by element: [t][h padded
    to 128] of the hidden values, then the high 16 bits of both, then a byte
    with the next four bits of each. Rounding them to 20 bits costs 2^-12; a
    and b are sums of d products, each at most d 2^-24 of its terms' sum off,
    act and act' have slopes under 1.2, and are themselves evaluated to 2^-20."""
    import torch
    note(f"ffn kept {t} {d} {h} {act}")
    f, x, w, dy, buf = ffn_case(t, d, h, "bf16", act)
    K.gated_ffn(f, x, w, buf, training=True)
    hp = (h + 127) // 128 * 128
    cells = t * hp
    n = (2 * cells + 255) // 256 * 256
    high = [buf.saved[i * n:i * n + 2 * cells].view(torch.int16).view(t, hp).int() << 16 for i in (1, 2)]
    low = buf.saved[3 * n:3 * n + cells].view(t, hp).int()
    got = [(hi | (bits << 12)).view(torch.float32).double()[:, :h]
           for hi, bits in zip(high, (low & 15, low >> 4))]
    x64, wg, wu = x.double(), w["w_gate"].double(), w["w_up"].double()
    a, b = x64 @ wg, x64 @ wu
    want = act64(a, act), b * slope64(a, act)
    ea, eb = (d * 2.0 ** -24 * (x64.abs() @ v.abs()) for v in (wg, wu))
    clear = a.abs() > ea if act == "relu" else torch.ones_like(a, dtype=torch.bool)  # on one side of the kink
    for name, g, v, more in (("act", got[0], want[0], 1.2 * ea + 2.0 ** -20 * a.abs()),
                             ("slope", got[1], want[1], 1.2 * eb + b.abs() * (1.2 * ea + 2.0 ** -20))):
        over = ((g - v).abs() - 2.0 ** -12 * v.abs() - more)[clear]
        assert float(over.max()) <= 0, (name, float(over.max()))


def test_ffn_kept_activations_that_are_not_finite():
    """Rounding what is kept takes no infinity or NaN for anything else."""
    import torch
    for t in (5, 60):
        f, x, w, dy, buf = ffn_case(t, 64, 128, "bf16", "relu")
        x[1, 3], x[2, 4], x[3, 5] = float("inf"), float("nan"), float("-inf")
        x.view(torch.int16)[4, 6] = -1  # a NaN with every bit set
        K.gated_ffn(f, x, w, buf, training=True)
        n = t * 128
        high = [buf.saved[i * 2 * n:(i + 1) * 2 * n].view(torch.int16).view(t, 128).int() << 16 for i in (1, 2)]
        low = buf.saved[6 * n:7 * n].view(t, 128).int()
        kept = [(hi | (bits << 12)).view(torch.float32) for hi, bits in zip(high, (low & 15, low >> 4))]
        a, b = x.double() @ w["w_gate"].double(), x.double() @ w["w_up"].double()
        act = torch.where(a < 0, torch.zeros_like(a), a)
        slope = b * (a > 0)
        for got, want in zip(kept, (act, slope)):
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())


@pytest.mark.parametrize("t,d,h,dtype", [(1, 2048, 512, "bf16"), (300, 1024, 4096, "bf16"), (130, 333, 1001, "bf16"),
                                         (8200, 512, 1024, "bf16"), (20, 100, 333, "fp32"), (300, 500, 1001, "fp32")])
def test_ffn_repeats_whatever_its_buffers_held(t, d, h, dtype):
    """The same bits from every call, over workspaces, kept activations and
    results that hold NaN or large numbers before it."""
    import torch
    note(f"ffn repeats {t} {d} {h} {dtype}")
    f, x, w, dy, buf = ffn_case(t, d, h, dtype)
    first = None
    for fill in (0, 255, 127, 255):
        buf.workspace.fill_(fill), buf.saved.fill_(fill)
        for v in (buf.out, buf.grad_x, *buf.grads.values()):
            v.fill_(float("nan"))
        outs = [K.gated_ffn(f, x, w, buf).clone()]
        buf.workspace.fill_(fill)
        outs.append(K.gated_ffn(f, x, w, buf, training=True).clone())
        buf.workspace.fill_(fill)
        gx, g = K.gated_ffn_backward(f, x, w, dy, buf)
        outs += [v.clone() for v in (gx, *g.values())]
        first = first or outs
        assert all(torch.equal(a, b) for a, b in zip(first, outs)), fill
    assert all(bool(torch.isfinite(v.float()).all()) for v in first)


# ------------------------------------------- the dense gated product in 8 bits

def product64(q, s, wq, ws):
    """The product of integers, exact in 64 bits (a sum that is 0 is 0), by the
    rows' and the weights' scales."""
    k = q.shape[1]
    return (q.double() @ wq[:, :k].double().t()) * s.double()[:, None] * ws.double()


def integers(x):
    """The definition's (integers, scales) of the rows of x, on the device."""
    import torch
    return [torch.from_numpy(v).cuda() for v in quantized(x)]


def each(name, got, gate, up, dtype):
    """Every element: the result's rounding (and 2^-20 of the scalings), and the
    SiLU: the gate is 2^-22 off after three roundings, which its slope of at most
    1.1 passes on, the logistic function another 2^-22: 2^-20 of the gate,
    2^-19 of gate times up with the up value's own."""
    import torch
    want = gate * torch.sigmoid(gate) * up
    over = (got.double() - want).abs() - (U[dtype] + 2.0 ** -20) * want.abs() - 2.0 ** -19 * (gate * up).abs()
    assert got.shape == want.shape and bool(torch.isfinite(got.float()).all()), name
    assert float(over.max()) <= 0, (name, float(over.max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k,h", [
    (1, 1, 1), (1, 512, 33), (4, 4096, 256), (7, 130, 17), (8, 1000, 257), (2, 5000, 65), (8, 2000, 515),  # few rows
    (9, 1100, 129), (16, 2000, 515), (16, 1152, 8191),
    (9, 1000, 257), (17, 640, 65), (3, 200, 8200), (64, 333, 1001), (100, 1111, 515),  # 64 x 64 tiles
    (1100, 200, 2001), (2100, 300, 2101), (4200, 1100, 2051)])  # 128 x 128, 256 x 128, 256 x 256
def test_linear_i8_dense_gated(t, k, h, dtype):
    import torch
    note(f"linear_i8 dense gated {t} {k} {h} {dtype}")
    r = gen(t + k + h)
    x, g, u = r(t, k, dtype=dtype), r(k, h, std=k ** -0.5), r(k, h, std=k ** -0.5)
    wq, ws = K.quantize_weights(g, u)
    l = K.LinearI8(t, k, 2 * h, dtype, gated=True)
    buf = K.allocate_linear_i8(l)
    assert buf.y.shape == (t, h)
    gate, up = product64(*integers(x), wq[0], ws[0]).chunk(2, 1)
    each("y", K.linear_i8(l, x, wq, ws, buf), gate, up, dtype)
    first = buf.y.clone()
    # rows that are already in 8 bits give the same bits, into either type
    q, s = K.quantize_rows(x)
    assert torch.equal(K.linear_i8(l, q, wq, ws, buf, x_scale=s), first)
    other = "fp32" if dtype == "bf16" else "bf16"
    lo = K.LinearI8(t, k, 2 * h, other, gated=True)
    each("other type", K.linear_i8(lo, x, wq, ws, K.allocate_linear_i8(lo)), gate, up, other)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("t", [1, 8, 16])
def test_linear_i8_few_rows_of_every_length(t, gated):
    """The serving form shares the 64-byte steps of a row among eight waves, four
    at a time: every number of steps up to past two rounds of that, in rows that
    are already in 8 bits and, where they are short enough, quantised on the way."""
    import torch
    note(f"linear_i8 lengths {t} {gated}")
    r, n = gen(t), 20
    for k in range(128, 84 * 64, 128):
        x, w = r(t, k - 3), r(k - 3, 2 * n, std=k ** -0.5)
        q, s = K.quantize_rows(x)
        wq, ws = K.quantize_weights(w)
        l = K.LinearI8(t, k - 3, 2 * n, "fp32", gated=gated)
        buf = K.allocate_linear_i8(l)
        want = product64(q[:, :k - 3], s, wq[0], ws[0])
        for got in (K.linear_i8(l, q, wq, ws, buf, x_scale=s).clone(), K.linear_i8(l, x, wq, ws, buf)):
            if gated:
                each(f"{k - 3}", got, *want.chunk(2, 1), "fp32")
            else:
                # a sum of integers, exact, rounded by its conversion and two scalings: 3 u
                assert bool(((got.double() - want).abs() <= 3.01 * U["fp32"] * want.abs()).all()), k - 3


# ---------------------------------------------- the layer with 8-bit experts

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,e,top,d,h,cap,shared", [
    (1, 8, 2, 128, 64, 0, False), (4, 16, 4, 256, 128, 0, True), (4, 64, 8, 512, 128, 0, False),
    (9, 1, 1, 128, 64, 0, True), (60, 4, 2, 128, 192, 11, False), (700, 16, 4, 256, 128, 100, True),
    (3000, 8, 2, 512, 320, 0, True), (3000, 3, 1, 384, 64, 700, False)])
def test_layer_with_8_bit_experts(t, e, top, d, h, cap, shared, dtype):
    """Every buffer of the path against 64 bits of what went into it: the hidden
    values, the experts' outputs and the sum, with and without a capacity and a
    shared expert's output. Rows past a capacity stay as they were."""
    import torch
    note(f"layer in 8 bits {t} {e} {top} {d} {h} {cap} {shared} {dtype}")
    p = Problem(t, e, top, d, h, 0, dtype, 64, skew=0.5 if cap else 0.0, capacity=cap)
    c = Case(p, seed=4)
    x, wt = c.dev["x"], c.weights()
    gu, dn = K.quantize_weights(wt["w_gate"], wt["w_up"]), K.quantize_weights(wt["w_down"])
    more = gen(6)(t, d, dtype=dtype) if shared else None
    ex = K.allocate_experts_i8(p)
    ex.hidden.y.fill_(7.0), ex.sorted.y.fill_(7.0)
    out = K.forward_i8(p, x, wt["w_router"], gu, dn, c.buf, ex, shared_out=more)
    assert out is c.buf.out
    B.moe_route(p, x, wt["w_router"], (r := B.allocate(p, "cuda")).routing)
    for name in ("topk_idx", "topk_w"):
        assert torch.equal(c.buf.routing[name], r.routing[name])
    ends = c.buf.routing["expert_offsets"].tolist()
    assert ends[-1] == t * top
    token = c.buf.routing["perm"].long() // top
    q, s = integers(x)
    kept = torch.zeros(t * top, dtype=torch.bool, device="cuda")
    for g in range(e):
        i, j = ends[g], min(ends[g + 1], ends[g] + cap) if cap else ends[g + 1]
        if i < j:
            both = product64(q[token[i:j]], s[token[i:j]], gu[0][g], gu[1][g])
            each(f"hidden {g}", ex.hidden.y[i:j], *both.chunk(2, 1), dtype)
            want = product64(*integers(ex.hidden.y[i:j]), dn[0][g], dn[1][g])
            near(f"sorted {g}", ex.sorted.y[i:j], want, U[dtype] + 2.0 ** -20)
        kept[i:j] = True
    assert bool(kept.all()) == (not cap or max(b - a for a, b in zip(ends, ends[1:])) <= cap)
    assert bool((ex.hidden.y[~kept] == 7).all() and (ex.sorted.y[~kept] == 7).all())
    if cap:
        assert not bool(kept.all()), "the capacity drops nothing here"
    at = c.buf.routing["inv_perm"].view(t, top).long()
    assert torch.equal((at >= 0).sum(), kept.sum())
    w = torch.where(at >= 0, c.buf.routing["topk_w"], 0.0).double()
    want = (w[:, :, None] * ex.sorted.y.double()[at.clamp(min=0)]).sum(1) + (more.double() if shared else 0.0)
    near("out", out, want, U[dtype] + top * 2.0 ** -24)
