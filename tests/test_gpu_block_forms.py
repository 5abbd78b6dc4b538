"""Forms of the operators around the layer that need a look of their own: what
the gated block keeps of its activations."""

import pytest

from dropless_grouped_gemm_router_amd import block as K

from gpu_util import note
from test_gpu_block import act64, ffn64, ffn_case

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
