"""The layer norm's gradient, forward and backward as they are called, of rows
far from 0: against the gradient of the norm's definition in 64 bits, whose
mean is not rounded."""
import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.rows_ref import TYPES, U, adds, close
from tests.test_gpu_rows import DEV, gen, randn
from tests.test_gpu_train import f32, space
from tests import train_ref as ref

pytestmark = pytest.mark.gpu

every_type = pytest.mark.parametrize("t", TYPES)
COLS = (7, 64, 300, 1000, 1281, 4100, 8200, 16384, 20000, 40000)


def definition(x, dy, w, eps, mean, rstd):
    """(dx, dweight, dbias and their tolerances) of the norm of x.

    The statistics that the kernel is given are binary32.  rstd is off by its
    own rounding and the forward call's (rel, measured against the definition
    here).  The place h = (x - mean) * rstd takes the difference from the given
    mean, one rounding, less what the mean's rounding lost, a mean of
    differences of that size: a row's additions and some roundings, at the size
    of h and of the lost part both."""
    n = x.shape[1]
    x, dy = x.double(), dy.double()
    m = x.mean(1, keepdim=True)
    d = x - m
    r = (d.square().mean(1, keepdim=True) + eps).rsqrt()
    h, g = d * r, dy * (1.0 if w is None else w.double())
    first, second = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = r * (g - first - h * second)
    rel = (rstd.double()[:, None] / r - 1).abs() + 2 * U
    lost = (mean.double()[:, None] - m).abs() * r
    # rows whose mean is within 2^12 deviations of 0 keep what its rounding lost
    kept = torch.where(m.abs() * r <= 4200.0, lost, 0.0)
    size = h.abs() + h.abs().mean(1, keepdim=True) + 2 * lost
    eh = (adds(n) + 10) * U * size + rel * h.abs() + kept
    off_second = (g.abs() * eh).mean(1, keepdim=True) + \
        (adds(n) + 6) * U * ((g * h).abs() + g.abs() * lost).mean(1, keepdim=True)
    off_first = (adds(n) + 6) * U * g.abs().mean(1, keepdim=True)
    tol = r * (6 * U * (g.abs() + first.abs() + (h * second).abs() + lost * second.abs()) + off_first
               + h.abs() * off_second + eh * second.abs()) + rel * dx.abs() + 3 * U * dx.abs()
    rows = x.shape[0] + 8
    return (dx, (dy * h).sum(0), dy.sum(0), tol,
            (dy.abs() * (eh + rows * U * (h.abs() + lost))).sum(0), dy.abs().sum(0) * rows * U)


def far_rows(t, cols, g):
    """Values a few last places apart, as far from 0 as they come."""
    dt = TYPES[t]
    top = 3e4 if t == "f16" else 1e30
    base = torch.tensor([0.0, 1.0, 1 / 3, -1e4, top, 1e6 / 16, -77.7, 1.0], device=DEV)
    apart = torch.randint(0, 4, (len(base), cols), generator=g, device=DEV)
    x = base[:, None] * (1 + torch.finfo(dt).eps * apart)
    x[7] = 1.0
    x[7, cols // 3] += 1.0                                # one value beside equal ones
    return torch.cat([x, randn(g, 2, cols)]).to(dt)


@every_type
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("copies", (1, 37))
def test_rows_far_from_zero(t, cols, copies):
    """copies: one round of rows, several a block."""
    g, dt, eps = gen(cols), TYPES[t], 2.0 ** -80
    x = far_rows(t, cols, g)
    x[0] = randn(g, cols).to(dt)
    x = x.repeat(copies, 1)
    rows = x.shape[0]
    w, dy = (1 + 0.2 * randn(g, cols)).to(dt), randn(g, rows, cols).to(dt)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    getattr(ew, "ew_layernorm_" + t)(x, w, None, y, mean=mean, rstd=rstd, eps=eps)
    grad = getattr(ew, "ew_layernorm_grad_" + t)
    dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
    ws = space(ew.ew_layernorm_grad_workspace(rows, cols))
    grad(dy, x, w, mean, rstd, dx, dw, db, ws)
    want, want_w, want_b, tol, tol_w, tol_b = definition(x, dy, w, eps, mean, rstd)
    close(dw, want_w, tol_w + 2.0 ** -126, "dweight")
    close(db, want_b, tol_b + 2.0 ** -126, "dbias")
    close(dx, want, ref.rounded(want, tol, dt), "dx")
    alone = torch.empty_like(x)
    grad(dy, x, w, mean, rstd, alone)                     # without the sums
    assert torch.equal(alone, dx)
    for k in range(2):                                    # in place
        args = [dy.clone(), x.clone()]
        grad(args[0], args[1], w, mean, rstd, args[k], dw, db, ws)
        assert torch.equal(args[k], dx)
        close(dw, want_w, tol_w + 2.0 ** -126, "dweight")
