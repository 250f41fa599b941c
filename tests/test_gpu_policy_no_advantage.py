"""The policy loss and its gradient where a token's ratio lies past the largest
binary32 number."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.test_gpu_policy_terms import SHAPES, loss_of
from tests.test_gpu_rows import DEV
from tests.test_gpu_train import f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("each", (True, False))
def test_tokens_of_no_advantage_add_nothing(rows, cols, each):
    """exp(logp - old_logp) past the largest number, and its advantage 0: the
    gain is 0, and so is its slope."""
    logp, old = torch.zeros(rows, cols, device=DEV), torch.zeros(rows, cols, device=DEV)
    logp[:, 1::4], old[:, 1::4] = 0.0, -100.0
    logp[:, 2::4], old[:, 2::4] = 3.4e38, -3.4e38
    a = torch.zeros(rows, cols, device=DEV)
    if each:
        a[:, ::4] = 2.0                        # their ratio is 1
    want = -2.0 * rows * cols / 4 if each else 0.0
    loss, stats, weights = loss_of(logp, old, a if each else a[:, 0].contiguous())
    assert float(loss) == want and float(stats[0]) == want and float(stats[2]) == 0.0
    dlogp = f32(rows, cols)
    ew.ew_policy_loss_grad_f32(logp, old, a if each else a[:, 0].contiguous(), weights, dlogp)
    assert torch.equal(dlogp, -a)
    # a NaN is one still, and an advantage below 0 pays for the whole ratio
    if each:
        a[0, 1] = -1e-3
        loss, _, _ = loss_of(logp, old, a)
        assert float(loss) == math.inf
        a[0, 1] = 0.0
    old[0, 0] = math.nan
    loss, _, _ = loss_of(logp, old, a)
    assert math.isnan(float(loss))
