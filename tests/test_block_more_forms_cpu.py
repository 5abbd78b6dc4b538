"""The product with its epilogue, the step between two blocks and the balance
loss on the host, no GPU: problems as values, and refusals of calls whose
arguments fit one by one but not together."""

import copy
import pickle

import pytest

from dropless_grouped_gemm_router_amd import block as K


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
