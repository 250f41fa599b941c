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


@pytest.mark.parametrize("t", ("f32", "f16", "bf16"))
def test_top_logp_and_top_ids_come_together(t):
    """One without the other would be left unwritten."""
    def call(top_logp, top_ids, top):
        return ew._c["ew_logprobs_" + t](BASE, 64, BASE + (1 << 20), BASE + (2 << 20), None, None,
                                         top_logp, top_ids, top, 1.0, None, 0, 8, 64, 0)

    for top in (0, 5):
        assert call(BASE + (3 << 20), None, top) == -1
        assert call(None, BASE + (4 << 20), top) == -1
    ids = torch.zeros(8, 5, dtype=torch.int64)
    fn = getattr(ew, "ew_logprobs_" + t)
    for more in ({"top_logp": torch.zeros(8, 5)}, {"top_ids": ids}, {"top_ids": ids, "top": 5},
                 {"top_logp": BASE, "top": 5}):
        with pytest.raises(ValueError, match="both or neither"):
            fn(BASE, BASE, BASE, rows=8, cols=64, stream=0, **more)


def test_tables_of_other_widths():
    """teacher, ids, top_logp, top_ids and scales hold a row of values per row
    of the matrix: a wider tensor's rows are not taken for narrower ones."""
    x, r, targets = torch.zeros(4, 64), torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    narrow, wide = (torch.zeros(4, k, dtype=torch.int64) for k in (3, 6))
    for teacher, ids, kept, role in ((torch.zeros(4, 6), narrow, None, "teacher"),
                                     (torch.zeros(4, 3), wide, 3, "ids"),
                                     (torch.zeros(2, 4, 6), narrow, None, "teacher")):
        with pytest.raises(ValueError, match=f"{role}: shape .* covers 4 rows of 3"):
            ew.ew_distill_f32(x, teacher, ids, r, kept=kept)
        with pytest.raises(ValueError, match=f"{role}: shape .* covers 4 rows of 3"):
            ew.ew_distill_grad_f32(x, teacher, ids, r, r, x, kept=kept)
    with pytest.raises(ValueError, match="top_logp: shape .* covers 4 rows of 3"):
        ew.ew_logprobs_f32(x, targets, r, top_logp=torch.zeros(4, 6), top_ids=narrow)
    with pytest.raises(ValueError, match="top_ids: shape .* covers 4 rows of 3"):
        ew.ew_logprobs_f32(x, targets, r, top_logp=torch.zeros(4, 3), top_ids=wide, top=3)
    with pytest.raises(ValueError, match="scales: shape .* covers 4 rows of 2"):
        ew.ew_rmsnorm_e4m3_f32(BASE, BASE, BASE, torch.zeros(4, 4), group=32, rows=4, cols=64,
                               stream=0)
    with pytest.raises(ValueError, match="ids: a scalar"):
        ew.ew_distill_f32(x, r, torch.zeros((), dtype=torch.int64), r)
    # as many values in another arrangement of the rows, and flat buffers
    flat = torch.zeros(64, dtype=torch.int64)
    for teacher, ids, kept in ((torch.zeros(2, 2, 3), narrow, None), (torch.zeros(64), flat, 3),
                               (torch.zeros(4, 1), torch.zeros(4, 1, 1, dtype=torch.int64), None),
                               (torch.zeros(2, 2), torch.zeros(2, 2, 1, dtype=torch.int64), None)):
        with pytest.raises(ValueError, match="logits: .* not on a GPU"):
            ew.ew_distill_f32(x, teacher, ids, r, kept=kept)
