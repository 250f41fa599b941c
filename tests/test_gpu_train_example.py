"""The example that runs layer norm, experts and policy loss together, against
autograd."""
import importlib.util
import os

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location(
        "_expert_step", os.path.join(ROOT, "examples", "expert_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("hidden,experts,top", ((512, 8, 2), (1000, 17, 5)))
def test_expert_step_matches_autograd(hidden, experts, top):
    """bfloat16 buffers between the operators: some twelve of them are each
    rounded (at most 2^-8 of a value) on the way from x to its gradient, which
    add up at random to less than four roundings; the roundings before the
    logits change the probability ratios, of the order of the gradients
    themselves, by as much again."""
    off, (alone, batched, ids, ids_batched) = _example().main(
        ["--sequences", "6", "--length", "30", "--hidden", str(hidden), "--vocab", "5003",
         "--experts", str(experts), "--top", str(top)])
    assert all(v < 8 * 2.0 ** -8 for v in off.values()), off
    # a product of one row may add up in another order: roundings of y2 and of
    # the logit, a few at random
    assert ids == ids_batched and abs(alone - batched) < 8 * 2.0 ** -8
