"""The row operators' binding and C entry points without a GPU: arguments that
contradict each other are refused."""
import pytest
import torch

import memory_bound_elementwise_amd as ew

BASE = 0x7F0000000000          # a made-up, 256-byte aligned device address


def test_rows_or_cols_given_alone_count():
    """One of them given with a tensor is not dropped for the tensor's own."""
    x, y, w, r = torch.zeros(8, 16), torch.zeros(8, 16), torch.zeros(16), torch.zeros(8)
    ids = torch.zeros(8, dtype=torch.int64)
    for sizes, says in (({"rows": 3}, "covers 3 rows of 16"), ({"cols": 8}, "covers 8 rows of 8")):
        with pytest.raises(ValueError, match=says):
            ew.ew_rmsnorm_f32(x, w, y, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_rmsnorm_e4m3_f32(x, w, torch.zeros(8, 16, dtype=torch.uint8), r, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_rmsnorm_grad_f32(x, x, w, r, y, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_logprobs_f32(x, ids, r, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_logprobs_grad_f32(x, ids, r, r, y, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_distill_f32(x, r, ids.view(8, 1), r, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_distill_grad_f32(x, r, ids.view(8, 1), r, r, y, **sizes)
    # the tensor's own sizes, and those of more dimensions, are what they were
    with pytest.raises(ValueError, match="not on a GPU"):
        ew.ew_rmsnorm_f32(x, w, y, rows=8)
    with pytest.raises(ValueError, match="not on a GPU"):
        ew.ew_rmsnorm_f32(x.view(2, 4, 16), w, y, cols=16)
    with pytest.raises(ValueError, match="covers 7 rows of 16"):
        ew.ew_rmsnorm_f32(x.view(2, 4, 16), w, y, rows=7)
