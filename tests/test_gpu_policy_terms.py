"""The policy loss where neighbouring tokens' terms are of very different size, or
their sum past binary32."""
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
