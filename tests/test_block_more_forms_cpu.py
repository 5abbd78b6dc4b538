"""The product with its epilogue, the step between two blocks and the balance
loss on the host, no GPU: problems as values, and refusals of calls whose
arguments fit one by one but not together."""

import copy
import pickle

import pytest
import torch

from dropless_grouped_gemm_router_amd import binding as B
from dropless_grouped_gemm_router_amd import block as K
from dropless_grouped_gemm_router_amd.inputs import Problem

from test_block_cpu import INV, A, At, C, D, E, F, G, H, refused


@pytest.mark.parametrize("problem", [K.Linear(4, 64, 96, "bf16", "gelu"), K.ResidualNorm(3, 65, "fp32", "rms", pre=False),
                                     K.BalanceLoss(5, 4, 2, 128, "bf16", 0.5, 0.25)])
def test_problems_are_copied_and_pickled(problem):
    # before and after a call has kept its plan
    for _ in range(2):
        for again in (copy.copy(problem), copy.deepcopy(problem), pickle.loads(pickle.dumps(problem)),
                      copy.deepcopy([problem, problem])[1]):
            assert type(again) is type(problem) and again == problem and hash(again) == hash(problem)
            assert again._plan[1:-1] == problem._plan[1:-1]
            assert again._plan is not problem._plan
        assert "_plan" in vars(problem)


@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_refuses_shared_memory(dtype):
    """An output over an input would be stored while other tiles still read it."""
    l = K.moe_linear(300, 256, 512, dtype, 0, dtype)
    e = 2 if dtype else 4
    nx, ny, nw = 300 * 256 * e, 300 * 512 * e, 256 * 512 * e
    room = dict(workspace_bytes=1 << 40, stream=0)
    fwd = [A, C, D, E, F, G, H]  # x, w, bias, residual, saved, y, workspace
    for i, n in ((0, nx), (1, nw), (3, ny)):
        # the same address, the output's last bytes over the input's first, and the reverse
        for at in (0, 16 - ny, n - 16):
            args = list(fwd)
            args[5] = At(args[i].addr + at)
            refused(INV, K.moe_linear_fwd, l, *args, **room)
    bwd = [A, C, D, E, F, G, H, At(9 << 28)]  # x, w, saved, grad_out, grad_x, grad_w, grad_bias, workspace
    for o, no in ((4, nx), (5, nw)):
        for i, n in ((0, nx), (1, nw), (3, ny)):
            for at in (0, 16 - no, n - 16):
                args = list(bwd)
                args[o] = At(args[i].addr + at)
                refused(INV, K.moe_linear_bwd, l, *args, **room)
    args = list(bwd)
    args[5] = At(args[4].addr + nx - 16)
    refused(INV, K.moe_linear_bwd, l, *args, **room)


def test_linear_refuses_its_output_as_residual():
    l = K.Linear(6, 64, 96, "bf16")
    x, w, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((6, 64), (64, 96), (6, 96)))
    buf = K.LinearBuffers(y, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="residual"):
        K.linear(l, x, w, buf, residual=y)
    with pytest.raises(ValueError, match="GPU"):
        K.linear(l, x, w, buf, residual=y.clone())


def test_step_refuses_other_strides_in_place():
    """An output over an input has to have its rows."""
    def step(**ld):
        names = ("z", "res", "out", "y", "grad_out", "grad_y", "grad_z", "grad_res")
        return K.moe_residual_norm(10, 512, 1, 0, 1, 1, 1e-5, 1.0, *[ld.get(n, 0) for n in names])

    p = dict(post_weight=A)
    for out in ("out", "y"):
        for given in ("z", "res"):
            at = dict(z=A, res=C, out=D, y=E)
            at[out] = at[given]
            for ld in ({out: 520}, {given: 520}, {out: 520, given: 528}):
                refused(INV, K.moe_residual_norm_fwd, step(**ld), at["z"], at["res"], p, at["out"], at["y"], F, stream=0)
    for out in ("grad_z", "grad_res"):
        for given in ("z", "res", "grad_out", "grad_y"):
            at = dict(z=A, res=C, grad_out=D, grad_y=E, grad_z=F, grad_res=G)
            at[out] = at[given]
            for ld in ({out: 520}, {given: 520}, {out: 520, given: 528}):
                refused(INV, K.moe_residual_norm_bwd, step(**ld), at["z"], at["res"], p, H, at["grad_out"], at["grad_y"],
                        at["grad_z"], at["grad_res"], p, At(9 << 28), stream=0)


def test_loss_of_a_problem_struct():
    """The layer takes any object with its fields, the type a name or a number."""
    for p in (Problem(12, 4, 2, 128, 64, 0, "bf16", 64), B.problem_struct(Problem(12, 4, 2, 128, 64, 0, "bf16", 64))):
        K._want_loss(p, (K.BalanceLoss(12, 4, 2, 128, "bf16"), None))
        for b in (K.BalanceLoss(12, 4, 2, 128, "fp32"), K.BalanceLoss(13, 4, 2, 128, "bf16"), K.BalanceLoss(12, 4, 1, 128)):
            with pytest.raises(ValueError, match="loss"):
                K._want_loss(p, (b, None))
