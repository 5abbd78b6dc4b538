"""The operators around the layer on the host, no GPU: the library exports
every symbol include/moe_block.h declares, sizes, and every argument check,
all of which run before any HIP call."""

import ctypes
import os
import re

import pytest

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS = B.MOE_ERR_INVALID, B.MOE_ERR_UNSUPPORTED, -3


class At:
    """Host stand-in for a tensor: an address that is never dereferenced."""

    def __init__(self, addr, nbytes=1 << 40):
        self.addr, self.nbytes = addr, nbytes

    def data_ptr(self):
        return self.addr

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1


A, C, D, E, F, G, H = (At((i + 1) << 28) for i in range(7))
ODD2, ODD4, ODD16 = At((1 << 28) + 2), At((1 << 28) + 4), At((1 << 28) + 16)


def refused(code, fn, *a, **k):
    with pytest.raises(B.MoeError) as e:
        fn(*a, **k)
    assert e.value.status == code


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "moe_block.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src)))
    assert sorted(K.EXPORTED) == names
    lib = K.load()
    for n in names:
        assert hasattr(lib, n), n


def norm(rows=10, width=512, dtype=1, eps=1e-5, ld=(0, 0, 0, 0)):
    return K.moe_norm(rows, width, dtype, eps, *ld)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(width=0), INV), (dict(dtype=2), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(ld=(511, 0, 0, 0)), INV),
    (dict(ld=(0, 511, 0, 0)), INV), (dict(ld=(0, 0, 1, 0)), INV), (dict(ld=(0, 0, 0, -5)), INV),
    (dict(width=16385), UNS), (dict(rows=1 << 31), UNS), (dict(ld=(1 << 31, 0, 0, 0)), UNS)])
def test_norm_problem_refusals(kw, code):
    refused(code, K.moe_layer_norm, norm(**kw), A, C, D, E, None, None, stream=0)
    refused(code, K.moe_layer_norm_bwd, norm(**kw), A, C, D, E, F, G, H, H, A, stream=0)
    assert K.moe_layer_norm_workspace_bytes(norm(**kw)) == 0


def test_norm_argument_refusals():
    fwd, bwd = K.moe_layer_norm, K.moe_layer_norm_bwd
    refused(INV, fwd, norm(), None, C, D, E, None, None, stream=0)
    refused(INV, fwd, norm(), At(0x1001), C, D, E, None, None, stream=0)
    refused(INV, fwd, norm(dtype=0), ODD2, C, D, E, None, None, stream=0)
    refused(INV, fwd, norm(), A, ODD2, D, E, None, None, stream=0)
    refused(INV, fwd, norm(), A, C, D, None, None, None, stream=0)
    refused(INV, fwd, norm(), A, C, D, E, F, None, stream=0)
    refused(INV, fwd, norm(), A, C, D, E, None, F, stream=0)
    need = K.moe_layer_norm_workspace_bytes(norm())
    assert need >= 2 * 512 * 4
    refused(WS, bwd, norm(), A, C, D, E, F, G, H, H, A, workspace_bytes=need - 1, stream=0)
    refused(INV, bwd, norm(), A, C, D, E, F, G, H, H, ODD16, workspace_bytes=need, stream=0)
    refused(INV, bwd, norm(), A, C, None, E, F, G, H, H, A, stream=0)
    refused(INV, bwd, norm(), A, C, D, E, F, None, H, H, A, stream=0)
    refused(INV, bwd, norm(), A, C, D, E, F, G, ODD2, H, A, stream=0)
    fwd(norm(rows=0), None, None, None, None, None, None, stream=0)
    bwd(norm(rows=0), None, None, None, None, None, None, None, None, None, stream=0)


def ffn(tokens=10, d=256, h=512, dtype=1, act=0, grad=0):
    return K.moe_ffn(tokens, d, h, dtype, act, grad)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(d=0), INV), (dict(h=0), INV), (dict(dtype=2), INV),
    (dict(act=-1), INV), (dict(act=4), INV), (dict(dtype=0, grad=1), INV), (dict(grad=2), INV),
    (dict(d=32769), UNS), (dict(h=32769), UNS), (dict(tokens=1 << 31), UNS),
    (dict(tokens=1 << 20, h=32768), UNS)])
def test_ffn_problem_refusals(kw, code):
    f = ffn(**kw)
    refused(code, K.moe_gated_ffn, f, A, C, D, E, None, F, G, stream=0)
    refused(code, K.moe_gated_ffn_bwd, f, A, C, D, E, F, G, H, H, H, H, A, stream=0)
    assert K.moe_gated_ffn_workspace_bytes(f) == K.moe_gated_ffn_saved_bytes(f) == 0


def test_ffn_argument_refusals():
    fwd, bwd, f = K.moe_gated_ffn, K.moe_gated_ffn_bwd, ffn()
    for i in range(4):
        args = [A, C, D, E]
        args[i] = None
        refused(INV, fwd, f, *args, None, F, G, stream=0)
        args[i] = ODD4
        refused(INV, fwd, f, *args, None, F, G, stream=0)
    refused(INV, fwd, f, A, C, D, E, ODD16, F, G, stream=0)
    refused(INV, fwd, f, A, C, D, E, None, None, G, stream=0)
    refused(INV, fwd, f, A, C, D, E, None, F, ODD16, stream=0)
    for training in (False, True):
        need = K.moe_gated_ffn_workspace_bytes(f, training)
        refused(WS, fwd, f, A, C, D, E, H if training else None, F, G, workspace_bytes=need - 1, stream=0)
    refused(WS, bwd, f, A, C, D, E, F, G, H, H, H, H, A, workspace_bytes=need - 1, stream=0)
    for i in range(11):
        args = [A, C, D, E, F, G, H, H, H, H, A]
        args[i] = None
        refused(INV, bwd, f, *args, workspace_bytes=need, stream=0)
    fwd(ffn(tokens=0), None, None, None, None, None, None, None, stream=0)
    refused(INV, bwd, ffn(tokens=0), None, None, None, None, None, None, None, None, None, None, None, stream=0)


def test_size_queries_over_the_range():
    """Sizes exist, and grow with training, from no token to the largest."""
    for t in (0, 1, 16, 17, 128, 129, 5000, 1 << 19):
        for d, h in ((1, 1), (128, 256), (500, 1001), (8192, 32768)):
            for dtype in (0, 1):
                f = ffn(t, d, h, dtype)
                few, more = (K.moe_gated_ffn_workspace_bytes(f, training) for training in (False, True))
                assert 0 < few <= more and few % 256 == 0
                assert K.moe_gated_ffn_saved_bytes(f) >= 3 * t * h * (4 if dtype == 0 else 2)
                assert K.moe_layer_norm_workspace_bytes(norm(t, min(d, 16384), dtype)) > 0
                assert K.moe_linear_i8_workspace_bytes(i8(t, d, h)) >= t * (d + 4)


def i8(tokens=10, inputs=512, outputs=256, x=1, y=1, groups=1, top_k=1, gather=0, gated=0, cap=0):
    return K.moe_i8_linear(tokens, inputs, outputs, x, y, groups, top_k, gather, gated, cap)


ROUTING = {"expert_offsets": A, "perm": C}


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INV), (dict(inputs=0), INV), (dict(outputs=0), INV), (dict(groups=0), INV),
    (dict(top_k=0), INV), (dict(cap=-1), INV), (dict(x=3), INV), (dict(y=2), INV),
    (dict(gather=2), INV), (dict(gated=-1), INV), (dict(gated=1, outputs=255), INV),
    (dict(groups=4, top_k=5), INV), (dict(groups=65, top_k=2), UNS), (dict(inputs=65537), UNS),
    (dict(outputs=65537), UNS), (dict(groups=8, tokens=1 << 30, top_k=2), UNS),
    (dict(tokens=1 << 20, outputs=65536), UNS)])
def test_i8_problem_refusals(kw, code):
    l = i8(**kw)
    refused(code, K.moe_linear_i8, l, A, None, C, D, None, ROUTING, E, F, stream=0)
    assert K.moe_linear_i8_workspace_bytes(l) == 0


def test_i8_argument_refusals():
    fn, l = K.moe_linear_i8, i8()
    for i, name in enumerate("x wq ws y".split()):
        args = dict(x=A, wq=C, ws=D, y=E)
        args[name] = None
        refused(INV, fn, l, args["x"], None, args["wq"], args["ws"], None, None, args["y"], F, stream=0)
    refused(INV, fn, l, ODD4, None, C, D, None, None, E, F, stream=0)
    refused(INV, fn, l, A, None, C, D, ODD2, None, E, F, stream=0)
    refused(INV, fn, l, A, None, C, D, None, None, E, None, stream=0)
    refused(WS, fn, l, A, None, C, D, None, None, E, F,
            workspace_bytes=K.moe_linear_i8_workspace_bytes(l) - 1, stream=0)
    refused(INV, fn, i8(x=K.MOE_I8), A, None, C, D, None, None, E, None, stream=0)
    refused(UNS, fn, i8(gated=1), A, None, C, D, G, None, E, F, stream=0)
    # routed arguments need a routing
    for kw in (dict(groups=4), dict(gather=1), dict(cap=3)):
        refused(INV, fn, i8(**kw), A, None, C, D, None, None, E, F, stream=0)
    r = i8(groups=4, top_k=2, gather=1)
    refused(INV, fn, r, A, None, C, D, None, {"expert_offsets": A, "perm": None}, E, F, stream=0)
    refused(INV, fn, r, A, None, C, D, None, {"expert_offsets": None, "perm": A}, E, F, stream=0)
    fn(i8(tokens=0), None, None, None, None, None, None, None, None, stream=0)


def test_quantize_refusals():
    rows, weight = K.moe_quantize_rows, K.moe_quantize_weight
    assert [K.moe_i8_pitch(w) for w in (-1, 0, 1, 128, 129)] == [0, 0, 128, 128, 256]
    for a, code in (((-1, 8, 0, A, 0), INV), ((1, 0, 0, A, 0), INV), ((1, 8, 2, A, 0), INV),
                    ((1, 8, 0, A, 7), INV), ((1, 65537, 0, A, 0), UNS), ((1 << 31, 8, 0, A, 0), UNS),
                    ((1, 8, 0, None, 0), INV), ((1, 8, 0, ODD2, 0), INV)):
        refused(code, rows, *a, C, D, stream=0)
    refused(INV, rows, 1, 8, 0, A, 0, ODD4, D, stream=0)
    rows(0, 8, 0, None, 0, None, None, stream=0)
    for a, code in (((0, 8, 8, 0, A, 0), INV), ((1, 0, 8, 0, A, 0), INV), ((1, 8, 0, 0, A, 0), INV),
                    ((1, 8, 8, 5, A, 0), INV), ((1, 8, 8, 0, A, 7), INV), ((65, 8, 8, 0, A, 0), UNS),
                    ((1, 65537, 8, 0, A, 0), UNS), ((1, 8, 8, 0, None, 0), INV)):
        refused(code, weight, *a, C, D, stream=0)


def test_tensor_checks():
    """The tensor front ends refuse CPU tensors and wrong shapes or types
    before anything reaches the library."""
    import torch
    x = torch.zeros(4, 8)
    buf = K.NormBuffers(y=torch.zeros(4, 8), mean=torch.zeros(4), rstd=torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        K.layer_norm(x, None, None, 1e-5, buf)
    with pytest.raises(ValueError, match="weight"):
        K.layer_norm(x, torch.zeros(9), None, 1e-5, buf)
    with pytest.raises(ValueError, match="y: "):
        K.layer_norm(x.bfloat16(), None, None, 1e-5, buf)
    with pytest.raises(ValueError, match="contiguous"):
        K.layer_norm(torch.zeros(8, 4).t(), None, None, 1e-5, buf)
    f = K.GatedFfn(4, 8, 16, "fp32")
    w = dict(w_gate=torch.zeros(8, 16), w_up=torch.zeros(8, 16), w_down=torch.zeros(8, 16))
    with pytest.raises(ValueError, match="w_down"):
        K.gated_ffn(f, x, w, K.FfnBuffers(out=x, workspace=x))
    l = K.LinearI8(4, 8, 16, "fp32")
    with pytest.raises(ValueError, match="weights"):
        K.linear_i8(l, x, torch.zeros(1, 16, 8, dtype=torch.int8), torch.zeros(1, 16),
                    K.I8Buffers(y=torch.zeros(4, 16), workspace=x))
    with pytest.raises(ValueError, match="x_scale"):
        K.linear_i8(l, torch.zeros(4, 128, dtype=torch.int8), torch.zeros(1, 16, 128, dtype=torch.int8),
                    torch.zeros(1, 16), K.I8Buffers(y=torch.zeros(4, 16), workspace=x))


def ffn_tensors(t, d, h):
    import torch
    make = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
    return make(t, d), dict(w_gate=make(d, h), w_up=make(d, h), w_down=make(h, d)), make(t, d)


# A workspace is not larger for every larger d_hidden (widths that are no
# multiple of 128 or 64 take copies of the weights), so its size, which the
# library checks, does not stand for that of `saved`.
@pytest.mark.parametrize("t,d,small,large", [(8, 512, 1000, 1152), (300, 2048, 64, 4096)])
def test_ffn_buffers_of_another_block(t, d, small, large):
    made = K.allocate_ffn(K.GatedFfn(t, d, small), "cpu", training=True)
    f = K.GatedFfn(t, d, large)
    assert made.workspace.numel() >= K.moe_gated_ffn_workspace_bytes(f.struct(), True)
    assert made.saved.numel() < K.moe_gated_ffn_saved_bytes(f.struct())
    x, w, dy = ffn_tensors(t, d, large)
    with pytest.raises(ValueError, match="saved: .* bytes"):
        K.gated_ffn(f, x, w, made, training=True)
    made.grads = K.allocate_ffn(f, "cpu", training=True).grads
    with pytest.raises(ValueError, match="saved: .* bytes"):
        K.gated_ffn_backward(f, x, w, dy, made)


@pytest.mark.parametrize("what", ["saved", "workspace"])
def test_byte_buffers_of_another_device_or_type(what):
    """`saved` and workspaces are bytes on the tensors' device."""
    import torch
    f, (x, w, dy) = K.GatedFfn(20, 64, 128), ffn_tensors(20, 64, 128)
    l, n = K.LinearI8(20, 64, 128), K.allocate_norm(20, 64, "bf16", "cpu", training=True)
    wq, ws = torch.zeros(1, 128, 128, dtype=torch.int8), torch.zeros(1, 128)
    b, i = K.allocate_ffn(f, "cpu", training=True), K.allocate_linear_i8(l, "cpu")
    size = getattr(b, what).numel()
    for wrong in (torch.empty(size, dtype=torch.uint8, device="meta"), torch.empty(size, dtype=torch.float32),
                  torch.empty(2 * size, dtype=torch.uint8)[::2]):
        setattr(b, what, wrong)
        i.workspace = n.workspace = wrong
        with pytest.raises(ValueError, match=what):
            K.gated_ffn(f, x, w, b, training=True)
        with pytest.raises(ValueError, match=what):
            K.gated_ffn_backward(f, x, w, dy, b)
        with pytest.raises(ValueError, match="workspace"):
            K.linear_i8(l, x, wq, ws, i)
        with pytest.raises(ValueError, match="workspace"):
            K.layer_norm_backward(x, None, dy, n)


def test_problem_structs_are_the_callers_own():
    """What a caller changes in a problem's struct reaches no other call."""
    f, l = K.GatedFfn(300, 192, 320), K.LinearI8(300, 192, 320)
    ffn_size = K.allocate_ffn(f, "cpu", training=True).workspace.numel()
    i8_size = K.allocate_linear_i8(l, "cpu").workspace.numel()
    f.struct().d_hidden = 64
    l.struct(B.MOE_FP32, False).tokens = 1
    assert f.struct().d_hidden == 320 and l.struct(B.MOE_FP32, False).tokens == 300
    assert K.allocate_ffn(f, "cpu", training=True).workspace.numel() == ffn_size
    assert K.allocate_linear_i8(l, "cpu").workspace.numel() == i8_size
    # the structs that calls take are kept by value: none was handed out
    assert K._ffn(*f._fields)[0].d_hidden == 320 and K._i8(l, B.MOE_FP32, False)[0].tokens == 300


def layer_case(dtype="bf16", **kw):
    """A layer's problem, input, weights, output gradient, its buffers and its norm's."""
    import torch
    from dropless_grouped_gemm_router_amd.inputs import Problem
    p = Problem(**{**dict(tokens=12, experts=4, top_k=2, d_model=128, d_hidden=128, d_shared=128, dtype=dtype,
                          block_m=32), **kw})
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    E, d, h, hs = p.experts, p.d_model, p.d_hidden, p.d_shared
    w = dict(w_router=torch.zeros(d, E), w_gate=torch.zeros(E, d, h, dtype=dt), w_up=torch.zeros(E, d, h, dtype=dt),
             w_down=torch.zeros(E, h, d, dtype=dt), ws_gate=torch.zeros(d, hs, dtype=dt),
             ws_up=torch.zeros(d, hs, dtype=dt), ws_down=torch.zeros(hs, d, dtype=dt))
    return (p, torch.zeros(p.tokens, d, dtype=dt), w, torch.zeros(p.tokens, d, dtype=dt),
            B.allocate(p, "cpu", training=True), K.allocate_norm(p.tokens, d, dtype, "cpu", training=True))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_behind_its_norm_refusals(dtype):
    """The layer's stages only pass pointers on: inputs, weights, gradients and
    buffers that are not the problem's are refused before any of them runs."""
    import torch
    p, x, w, dy, buf, nb = layer_case(dtype)
    for fn in (lambda: K.prenorm_forward(p, x, w, buf, nb, training=True),
               lambda: K.prenorm_backward(p, x, w, dy, buf, nb)):
        with pytest.raises(ValueError, match="GPU"):
            fn()
    # an output gradient as sum().backward() makes it: one element, expanded
    with pytest.raises(ValueError, match="grad_out"):
        K.prenorm_backward(p, x, w, dy[:1, :1].expand(12, 128), buf, nb)
    with pytest.raises(ValueError, match="grad_out"):
        K.prenorm_backward(p, x, w, dy.half(), buf, nb)
    for name in w:
        for wrong in (w[name].transpose(-1, -2), w[name][..., :-1].contiguous(), w[name].half()):
            with pytest.raises(ValueError, match=name):
                K.prenorm_forward(p, x, {**w, name: wrong}, buf, nb)
            with pytest.raises(ValueError, match=name):
                K.prenorm_backward(p, x, {**w, name: wrong}, dy, buf, nb)
    # buffers of the layer with fewer tokens, fewer experts, or another width
    for kw in (dict(tokens=11), dict(experts=3), dict(top_k=1), dict(d_hidden=64), dict(d_shared=64)):
        q, qx, qw, qdy, qbuf, qnb = layer_case(dtype, **kw)
        with pytest.raises(ValueError, match="shape|bytes"):
            K.prenorm_forward(p, x, w, qbuf, nb, training=True)
        buf2 = B.allocate(p, "cpu", training=True)
        buf2.saved = qbuf.saved
        if qbuf.saved.numel() < buf.saved.numel():
            with pytest.raises(ValueError, match="saved"):
                K.prenorm_forward(p, x, w, buf2, nb, training=True)
            with pytest.raises(ValueError, match="saved"):
                K.prenorm_backward(p, x, w, dy, buf2, nb)
    # normalised rows that lie apart
    nb.y = torch.zeros(12, 256, dtype=x.dtype)[:, :128]
    with pytest.raises(ValueError, match="y of the norm"):
        K.prenorm_forward(p, x, w, buf, nb)
    with pytest.raises(ValueError, match="training"):
        K.prenorm_backward(p, x, w, dy, B.allocate(p, "cpu"), nb)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_with_8_bit_experts_refusals(dtype):
    import torch
    p, x, w, _, buf, _ = layer_case(dtype)
    q8 = lambda rows, width: (torch.zeros(4, rows, width, dtype=torch.int8), torch.zeros(4, rows))
    gu, dn, ex = q8(256, 128), q8(128, 128), K.allocate_experts_i8(p, "cpu")
    with pytest.raises(ValueError, match="GPU"):
        K.forward_i8(p, x, w["w_router"], gu, dn, buf, ex)
    for wrong in (x[:11], x.t().contiguous().t(), x.half(), x[:1].expand(12, 128)):
        with pytest.raises(ValueError, match="x: "):
            K.forward_i8(p, wrong, w["w_router"], gu, dn, buf, ex)
    with pytest.raises(ValueError, match="w_router"):
        K.forward_i8(p, x, w["w_router"].t(), gu, dn, buf, ex)
    with pytest.raises(ValueError, match="shared_out"):
        K.forward_i8(p, x, w["w_router"], gu, dn, buf, ex, shared_out=x[:11])
    for kw in (dict(tokens=11), dict(experts=3), dict(top_k=1), dict(d_hidden=64)):
        q, *_, qbuf, _ = layer_case(dtype, **kw)
        with pytest.raises(ValueError, match="experts"):
            K.forward_i8(p, x, w["w_router"], gu, dn, buf, K.allocate_experts_i8(q, "cpu"))
        if "d_hidden" not in kw:  # nothing that this path uses of the buffers knows it
            with pytest.raises(ValueError, match="shape"):
                K.forward_i8(p, x, w["w_router"], gu, dn, qbuf, ex)
