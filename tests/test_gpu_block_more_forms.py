"""Forms of the product, the residual step and the balance loss that need a look
of their own. Tolerances are derived at each test; u as in test_gpu_block.py is half
a rounding step of the storage type (bf16 2^-8, fp32 2^-24)."""

import pytest

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from gpu_util import Case, note
from test_gpu_block import gen
from test_gpu_block_more import step_params, test_step_strided_and_in_place as strided_and_in_place

pytestmark = pytest.mark.gpu


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
