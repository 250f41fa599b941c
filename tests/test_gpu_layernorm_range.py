"""The layer norm of rows whose numbers are so large, or with eps = 0 so small,
that the squares of their differences (or the differences themselves) lie
outside binary32, against its definition in 64 bits with the tolerances of
tests/train_ref.py, which count roundings at any size of the numbers."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests import train_ref as ref
from tests.rows_ref import TYPES, U, close
from tests.test_gpu_rows import DEV, gen, randn
from tests.test_gpu_train import check_norm, f32

pytestmark = pytest.mark.gpu

# rows of one wave, of several, of the most registers, of three passes
COLS = (5, 300, 1000, 4096, 5003, 12289, 16384, 24576, 40000)


def large_rows(t, cols, seed):
    g = gen(seed)
    x = randn(g, 12, cols)
    at = torch.arange(cols, device=DEV)
    x[0] = torch.where(at < 8, 0.0, 1e37)                # far from the first numbers
    x[1] = torch.where(at % 2 == 0, 1e37, -1e37)
    x[2] *= 1e30
    x[3] = torch.where(at % 3 == 0, -3e38, 3e38)         # the differences overflow
    x[4, cols // 2] = 3e38                               # one number above all others
    x[5] = 1e37 * (1 + 1e-3 * x[5])
    x[6] *= 1e19                                         # the squares are near the border
    x[7] *= 1e20
    x[8] = torch.where(at >= cols - 3, 3e38, 1.0)        # another wave's numbers are small
    x[9] = 3e38                                          # equal numbers: exactly the bias
    x[10, 0] = -3e38
    x[11] *= 1e25                                        # beside an ordinary row of its block
    return torch.cat([x, randn(g, 3, cols)]).to(TYPES[t])


@pytest.mark.parametrize("t", ("f32", "bf16"))
@pytest.mark.parametrize("cols", COLS)
def test_rows_of_large_numbers(t, cols):
    x = large_rows(t, cols, cols)
    rows = x.shape[0]
    g, fn = gen(1 + cols), getattr(ew, "ew_layernorm_" + t)
    w, b = (1 + 0.2 * randn(g, cols)).to(x.dtype), randn(g, cols).to(x.dtype)
    for eps in (1e-5, 0.5, 1e38):
        y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
        fn(x, w, b, y, mean=mean, rstd=rstd, eps=eps)
        # (the mean of equal numbers is exact; the definition's in 64 bits is not)
        assert torch.equal(y[9], b) and torch.equal(mean[9], x[9, 0].float())
        close(rstd[9], torch.tensor(ref.f32(eps)) ** -0.5, 3 * U * ref.f32(eps) ** -0.5, "rstd")
        on = [k for k in range(rows) if k != 9]
        check_norm(t, x[on], None, w, b, y[on], None, mean[on], rstd[on], ref.f32(eps))
    # with the residual's addition, whose sum stays finite, in place
    res = torch.where(x.float().abs() > 1e38, 0.0, x.float() * 0.25).to(x.dtype)
    total = res.clone()
    fn(x, w, b, y, residual=total, total=total, mean=mean, rstd=rstd)
    assert torch.equal(y[9], b)
    check_norm(t, x[on], res[on], w, b, y[on], total[on], mean[on], rstd[on])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("eps", (0.0, 2.0 ** -140, 2.0 ** -70))
def test_rows_of_small_numbers(t, cols, eps):
    """eps that does not cover them.  (Standard deviations of 2^-126 and more:
    rstd is binary32.)"""
    g = gen(2 + cols)
    x = randn(g, 6, cols)
    if t == "f16":
        x[0], x[1], x[2] = x[0] * 2.0 ** -10, x[1] * 2.0 ** -14, 1 + x[2] * 2.0 ** -9
    else:
        x[0], x[1], x[2], x[3] = (x[k] * 2.0 ** -e for k, e in enumerate((40, 70, 100, 120)))
        x[5] = 1 + x[5] * 2.0 ** -7
    x = x.to(TYPES[t])
    # (some differences in each row)
    assert bool((x.double().std(1) > 2.0 ** -126).all()) and ref.f32(eps) == eps
    y, mean, rstd = torch.empty_like(x), f32(6), f32(6)
    fn = getattr(ew, "ew_layernorm_" + t)
    fn(x, None, None, y, mean=mean, rstd=rstd, eps=eps)
    check_norm(t, x, None, None, None, y, None, mean, rstd, eps)
    # equal numbers of any size
    x = torch.tensor([0.0, 2.0 ** -14, 0.75, 1.5, 6e4, 6e4 if t == "f16" else 3e38], device=DEV)
    x = x.to(TYPES[t])[:, None].expand(6, cols).contiguous()
    fn(x, None, None, y, mean=mean, rstd=rstd, eps=eps)
    assert torch.equal(mean, x[:, 0].float())
    if eps:
        assert not bool(y.any())
        close(rstd, torch.full((6,), eps ** -0.5), 3 * U * eps ** -0.5, "rstd")
    else:
        assert bool(torch.isnan(y).all()) and bool((rstd == math.inf).all())


@pytest.mark.parametrize("t", ("f32", "bf16"))
@pytest.mark.parametrize("cols", (300, 4096, 40000))
def test_rows_of_infinities_stay_nan(t, cols):
    x = large_rows(t, cols, 3)
    x[0, 17], x[1, cols - 1], x[2, 0], x[12, 200] = math.inf, -math.inf, math.inf, math.nan
    y, mean, rstd = torch.empty_like(x), f32(15), f32(15)
    getattr(ew, "ew_layernorm_" + t)(x, None, None, y, mean=mean, rstd=rstd)
    odd = torch.tensor([0, 1, 2, 12], device=DEV)
    fine = torch.tensor([k for k in range(15) if k not in (0, 1, 2, 9, 12)], device=DEV)
    for v in (y, mean, rstd):
        assert bool(torch.isnan(v[odd]).all())
    check_norm(t, x[fine], None, None, None, y[fine], None, mean[fine], rstd[fine])


@pytest.mark.parametrize("t", ("f32", "bf16"))
@pytest.mark.parametrize("cols", COLS[1:])
def test_first_numbers_at_the_other_end(t, cols):
    """A row, or a wave's part of it, whose first numbers are farther from its mean
    than the largest binary32 number."""
    at = torch.arange(cols, device=DEV)
    x = torch.where(at < 8, -3e38, 3e38).expand(4, cols).clone()
    x[1] = -x[1]
    x[2] = torch.where(at % 512 < 8, -3.3e38, 3.3e38)
    x[3, 8:] *= 1 - 2.0 ** -6 * (at[8:] % 5)
    x = x.to(TYPES[t])
    y, mean, rstd = torch.empty_like(x), f32(4), f32(4)
    getattr(ew, "ew_layernorm_" + t)(x, None, None, y, mean=mean, rstd=rstd)
    check_norm(t, x, None, None, None, y, None, mean, rstd)
