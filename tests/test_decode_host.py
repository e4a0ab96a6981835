"""The host side of the decode path on the CPU: budgets, argument checks and the build of the binding."""

import pytest
import torch

from block_sparse_causal_pooling_b200 import decode as D
from block_sparse_causal_pooling_b200 import stem as S


@pytest.mark.parametrize("k_start,mu,k_min", [(20.0, 0.25, 2), (7.5, 0.9, 3), (300.0, 1.0, 1),
                                              (1.0, 0.01, 1)])
def test_the_linear_schedule_is_that_of_a_context_which_ends_here(k_start, mu, k_min):
    """A token in block i is in the last of i + 1 blocks, whatever the width of the table."""
    m = S.make_method("linear", k_start=k_start, mu=mu, k_min=k_min)
    for width in (1, 2, 3, 50, 400):
        budget, kcap = D.stem_decode_budget(width, m, "cpu")
        want = [int(S.stem_budget_m(i + 1, m)[0][i]) for i in range(width)]
        assert budget.tolist() == want and budget.dtype == torch.int32
        assert kcap == max(want)
