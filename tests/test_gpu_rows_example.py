"""The example that runs every row operator together, against autograd."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location(
        "_policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_policy_step_matches_autograd():
    """bfloat16 buffers between the operators: y, the logits and their
    gradients are each rounded (2^-8 of a value), the products of a row add
    up such roundings at random, and the policy's gradient is a difference
    of terms of its own size: a few roundings in all."""
    off, (q, scales, logp, top_logp, top_ids) = _example().main(
        ["--rows", "96", "--hidden", "512", "--vocab", "5003", "--kept", "9"])
    assert all(v < 4 * 2.0 ** -8 for v in off.values()), off
    assert torch.equal(logp, top_logp[:, 0])
    assert bool((top_logp[:, :-1] >= top_logp[:, 1:]).all())
    assert len(set(top_ids[0].tolist())) == top_ids.shape[1]
    assert bool(torch.isfinite(q.float()).all()) and bool((scales > 0).all())
