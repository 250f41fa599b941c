"""The layer norm's gradient without dweight and dbias: the same dx, whatever the
number of rows, with which a call with sums takes other blocks."""
import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.rows_ref import TYPES
from tests.test_gpu_train import f32, grad_inputs, space

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,cols", ((1, 9), (4, 4096), (32, 512), (33, 100), (161, 8200), (250, 4100),
                                       (300, 2600), (384, 16384), (1030, 700), (2100, 3)))
def test_dx_does_not_depend_on_the_sums(t, rows, cols):
    dy, x, w, mean, rstd, dto = grad_inputs(t, rows, cols, 3, 1, rows)
    fn = getattr(ew, "ew_layernorm_grad_" + t)
    ws = space(ew.ew_layernorm_grad_workspace(rows, cols))
    out = [torch.empty(rows, cols, dtype=TYPES[t], device=x.device) for _ in range(4)]
    dw, db = f32(cols), f32(cols)
    fn(dy, x, w, mean, rstd, out[0], dw, db, ws, dtotal=dto)
    fn(dy, x, w, mean, rstd, out[1], dtotal=dto)
    fn(dy, x, w, mean, rstd, out[2], dweight=dw, workspace=ws, dtotal=dto)
    fn(dy, x, w, mean, rstd, out[3], dbias=db, workspace=ws, dtotal=dto)
    for other in out[1:]:
        assert torch.equal(other, out[0])
