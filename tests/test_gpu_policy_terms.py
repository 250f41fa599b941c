"""The policy loss where neighbouring tokens' terms are of very different size, or
a token's ratio lies past the largest binary32 number."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.rows_ref import U, close
from tests.test_gpu_rows import DEV
from tests.test_gpu_train import f32, space

pytestmark = pytest.mark.gpu

# one block, sequences below a wave's, a wave's, a block's, parts of long ones
SHAPES = ((1, 4), (8, 512), (300, 1028), (3, 20004), (20000, 4), (700, 64), (6000, 12), (5000, 1300),
          (1, 300004))


def loss_of(logp, old, advantage, mean="none", **kw):
    rows, cols = logp.shape
    loss, stats, weights = f32(1), f32(4), f32(rows)
    ew.ew_policy_loss_f32(logp, old, advantage, loss, weights=weights, stats=stats, mean=mean,
                          workspace=space(ew.ew_policy_loss_workspace(rows, cols)), **kw)
    return loss, stats, weights


def repeated(four, rows, cols):
    return torch.tensor(four, device=DEV).repeat(rows, cols // 4)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_terms_of_different_size_are_added_in_binary64(rows, cols):
    """At ratio 1 the loss is minus the advantages' sum; each is exact, as is
    every partial sum in binary64."""
    zero, fours = torch.zeros(rows, cols, device=DEV), rows * cols // 4
    for four, want in (((1e8, 1.0, -1e8, 1.0), -2.0), ((2.0 ** 127, 2.0 ** 127, -2.0 ** 127, -2.0 ** 127), 0.0),
                       ((2.0 ** 100, 3.0, 5.0, -2.0 ** 100), None)):
        loss, stats, _ = loss_of(zero, zero, repeated(four, rows, cols))
        if want is not None:
            close(loss, torch.tensor([want * fours]), abs(want) * fours * U, "loss")
            close(stats[:1], torch.tensor([want * fours]), abs(want) * fours * U, "policy")
        else:                      # the sum is not exact in binary64; it is finite
            assert bool(torch.isfinite(loss).all())
    # a mean of terms whose sum is past binary32
    loss, _, _ = loss_of(zero, zero, repeated((2.0 ** 127,) * 4, rows, cols), mean="tokens")
    close(loss, torch.tensor([-(2.0 ** 127)]), 2.0 ** 127 * U * 2, "loss")
    # old_logp - logp
    x = repeated((1e8, -1.0, -1e8, -1.0), rows, cols)
    _, stats, _ = loss_of(x, zero, torch.zeros(rows, cols, device=DEV), mean="tokens")
    close(stats[3:], torch.tensor([0.5]), U, "fall")


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_divergences_whose_sum_is_past_binary32(rows, cols):
    d = torch.tensor(88.5)
    k = math.exp(88.5) - 89.5                  # 2.7e38
    zero = torch.zeros(rows, cols, device=DEV)
    loss, stats, _ = loss_of(zero, zero, zero, mean="tokens", ref_logp=zero + d, kl=0.25)
    # the exponent is rounded twice at its size, and the result
    close(stats[1:2], torch.tensor([k], dtype=torch.float64), k * (2 * 88.5 + 4) * U, "kl")
    close(loss, torch.tensor([k / 4], dtype=torch.float64), k / 4 * (2 * 88.5 + 5) * U, "loss")


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
