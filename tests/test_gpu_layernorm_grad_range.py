"""The layer norm's gradient of rows whose differences, or their products with a
gradient, leave binary32: against its definition by the given statistics."""
import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.rows_ref import TYPES
from tests.test_gpu_rows import DEV, gen, randn
from tests.test_gpu_train import check_grad, f32, space

pytestmark = pytest.mark.gpu

COLS = (7, 64, 300, 1000, 1281, 4100, 8200, 16384, 20000, 40000)


@pytest.mark.parametrize("t", ("f32", "bf16"))
@pytest.mark.parametrize("cols", COLS)
def test_gradients_of_large_and_small_numbers(t, cols):
    g, dt = gen(5 + cols), TYPES[t]
    x = randn(g, 9, cols)
    at = torch.arange(cols, device=DEV)
    x[0] *= 1e30
    x[1] = torch.where(at % 2 == 0, 1e37, -1e37)
    x[2] = torch.where(at % 3 == 0, -3e38, 3e38)
    x[3, 0] = 3e38
    x[4] *= 1e19
    x[5] *= 2.0 ** -60
    x[6] *= 2.0 ** -110
    x[7] *= 1e36
    x = x.to(dt)
    h = x.double()
    mean = h.mean(1)
    rstd = (h - mean[:, None]).square().mean(1).rsqrt().float()
    mean = mean.float()
    w, dto = (1 + 0.2 * randn(g, cols)).to(dt), torch.zeros_like(x)
    ws = space(ew.ew_layernorm_grad_workspace(9, cols))
    for size in (1.0, 1e10, 1e-6):
        dy = (size * randn(g, 9, cols)).to(dt)
        # (a gradient past the type's largest is not asked for)
        dy[6] = (dy[6].float() * 1e-6).to(dt)
        dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
        getattr(ew, "ew_layernorm_grad_" + t)(dy, x, w, mean, rstd, dx, dw, db, ws, dtotal=dto)
        check_grad(t, dy, x, w, mean, rstd, dto, dx, dw, db)
