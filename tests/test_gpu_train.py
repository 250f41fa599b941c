"""Layer norm, policy loss and the movement of rows to experts on the GPU,
against their definitions in 64 bits (tests/train_ref.py, which derives the
tolerances)."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests import train_ref as ref
from tests.rows_ref import TYPES, U, close, norm_total
from tests.test_gpu_rows import DEV, GUARD, gen, guards_kept, matrix, randn

pytestmark = pytest.mark.gpu

every_type = pytest.mark.parametrize("t", TYPES)

# one column, below a vector, around vectors, waves and blocks, odd, large
COLS = (1, 2, 3, 5, 7, 8, 9, 15, 63, 64, 65, 255, 257, 260, 511, 513, 1000, 1025, 2048, 2056,
        2561, 4095, 4096, 4097, 5003, 8192, 10007, 12289, 16384)
LAYOUTS = ((0, 0), (8, 0), (1, 0), (0, 1), (13, 3))      # (pad, offset)


def f32(*shape):
    return torch.full(shape, GUARD, device=DEV)


def space(n):
    return torch.full((max(n, 1),), 0xAB, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def norm_inputs(t, rows, cols, pad, off, seed):
    g, dt = gen(seed), TYPES[t]
    x = matrix(rows, cols, dt, pad, off, randn(g, rows, cols) + 3 * randn(g, rows, 1))[0]
    res = matrix(rows, cols, dt, pad, off, 2 * randn(g, rows, cols))[0]
    w, b = (1 + 0.2 * randn(g, cols)).to(dt), randn(g, cols).to(dt)
    return x, res, w, b


def check_norm(t, x, res, w, b, y, total, mean, rstd, eps=1e-5):
    dt = TYPES[t]
    h = norm_total(x, res)
    if total is not None:
        assert torch.equal(total, h)
    want, m, r, tol, tol_m, tol_r = ref.layernorm(h, w, b, eps)
    if mean is not None:
        close(mean, m, tol_m, "mean")
    if rstd is not None:
        close(rstd, r, tol_r, "rstd")
    close(y, want, ref.rounded(want, tol, dt), "y")


@every_type
@pytest.mark.parametrize("cols", COLS)
def test_layernorm_columns(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows = (1, 2, 5, 9, 33)[k]
        x, res, w, b = norm_inputs(t, rows, cols, pad, off, 100 + cols + k)
        (y, ya), (total, ta) = (matrix(rows, cols, TYPES[t], pad, off) for _ in range(2))
        mean, rstd = f32(rows + 1), f32(rows + 1)
        getattr(ew, "ew_layernorm_" + t)(x, w, b, y, residual=res, total=total, mean=mean[:rows],
                                         rstd=rstd[:rows])
        check_norm(t, x, res, w, b, y, total, mean[:rows], rstd[:rows])
        guards_kept(y, ya)
        guards_kept(total, ta)
        assert float(mean[rows]) == GUARD and float(rstd[rows]) == GUARD


@every_type
@pytest.mark.parametrize("rows,cols", [(1, 65536), (3, 40001), (2, 24577), (2, 24576), (1100, 100),
                                       (5000, 64), (300, 4096), (700, 1281)])
def test_layernorm_long_rows_and_many_rows(t, rows, cols):
    x, res, w, b = norm_inputs(t, rows, cols, 0, 0, 7)
    y, total = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = f32(rows), f32(rows)
    getattr(ew, "ew_layernorm_" + t)(x, w, b, y, residual=res, total=total, mean=mean, rstd=rstd)
    check_norm(t, x, res, w, b, y, total, mean, rstd)


@every_type
@pytest.mark.parametrize("cols", (5, 1024, 4100, 40000))
def test_layernorm_options_and_aliases(t, cols):
    rows = 6
    fn = getattr(ew, "ew_layernorm_" + t)
    x, res, w, b = norm_inputs(t, rows, cols, 3, 1, 11)
    y = torch.empty(rows, cols, dtype=TYPES[t], device=DEV)
    fn(x, None, None, y)                             # the plain norm
    check_norm(t, x, None, None, None, y, None, None, None)
    fn(x, w, None, y, eps=0.5)
    check_norm(t, x, None, w, None, y, None, None, None, 0.5)
    fn(x, None, b, y, residual=res)                  # a residual, no total
    check_norm(t, x, res, None, b, y, None, None, None)
    a = x.clone()
    fn(a, w, b, a)                                   # y is x
    check_norm(t, x, None, w, b, a, None, None, None)
    c = res.clone()
    fn(x, w, b, y, residual=c, total=c)              # the residual stream in place
    check_norm(t, x, res, w, b, y, c, None, None)
    a, c = x.clone(), res.clone()
    fn(a, w, b, c, residual=c, total=a)              # both in place
    check_norm(t, x, res, w, b, c, a, None, None)
    a, c = x.clone(), res.clone()
    fn(a, w, b, a, residual=c)                       # y is x, the residual only read
    check_norm(t, x, res, w, b, a, None, None, None)
    # the two halves of one buffer; three dimensions
    both = torch.empty(rows, 2 * cols, dtype=TYPES[t], device=DEV)
    both[:, :cols].copy_(x)
    fn(both[:, :cols], w, b, both[:, cols:])
    check_norm(t, x, None, w, b, both[:, cols:], None, None, None)
    assert torch.equal(both[:, :cols], x)
    three = x.contiguous().view(2, 3, cols)
    out = torch.empty_like(three)
    fn(three, w, b, out)
    check_norm(t, x, None, w, b, out.view(rows, cols), None, None, None)


@every_type
@pytest.mark.parametrize("cols", (1, 3, 64, 1000, 4097, 40000))
def test_layernorm_of_rows_far_from_zero(t, cols):
    """Equal values give the bias exactly; differences survive a large mean."""
    g, dt = gen(3 * cols), TYPES[t]
    top = 6e4 if t == "f16" else 1e30
    base = torch.tensor([0.0, 1.0, 1 / 3, -1e4, top], device=DEV).to(dt)
    x = base[:, None].expand(5, cols).contiguous()
    b = randn(g, cols).to(dt)
    y, mean, rstd = torch.empty_like(x), f32(5), f32(5)
    fn = getattr(ew, "ew_layernorm_" + t)
    fn(x, (1 + randn(g, cols)).to(dt), b, y, mean=mean, rstd=rstd)
    assert torch.equal(y, b.expand(5, cols))
    assert torch.equal(mean, base.float())
    close(rstd, torch.full((5,), ref.f32(1e-5) ** -0.5), 316.0 * 3 * U, "rstd")
    # a few last places apart
    x = (base[:, None].float() * (1 + torch.finfo(dt).eps * torch.randint(0, 4, (5, cols), generator=g,
                                                                        device=DEV))).to(dt)
    x[4].clamp_(max=6e4)          # (f16: finite)
    if t != "f16":
        x[4] /= 1e15              # (its squares: finite)
    fn(x, None, None, y, mean=mean, rstd=rstd)
    check_norm(t, x, None, None, None, y, None, mean, rstd)


@every_type
@pytest.mark.parametrize("cols", (300, 4096, 40000))
def test_layernorm_of_nan_and_infinities(t, cols):
    x = torch.zeros(4, cols, device=DEV)
    x[1] = torch.arange(cols, device=DEV) % 7
    x[2, 17], x[3, 5] = math.nan, math.inf
    x = x.to(TYPES[t])
    y, mean, rstd = torch.empty_like(x), f32(4), f32(4)
    getattr(ew, "ew_layernorm_" + t)(x, None, None, y, mean=mean, rstd=rstd)
    assert bool(torch.isnan(y[2:]).all()) and bool(torch.isnan(rstd[2:]).all())
    assert bool(torch.isnan(mean[2:]).all())
    check_norm(t, x[:2], None, None, None, y[:2], None, mean[:2], rstd[:2])


def grad_inputs(t, rows, cols, pad, off, seed, dtotal=True):
    g, dt = gen(seed), TYPES[t]
    x, _, w, _ = norm_inputs(t, rows, cols, pad, off, seed)
    dy = matrix(rows, cols, dt, pad, off, randn(g, rows, cols))[0]
    dto = matrix(rows, cols, dt, pad, off, randn(g, rows, cols))[0] if dtotal else None
    h = x.double()
    mean = h.mean(1)
    rstd = ((h - mean[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    return dy, x, w, mean.float(), rstd, dto


def check_grad(t, dy, x, w, mean, rstd, dto, dx, dw, db):
    want, want_w, want_b, tol, tol_w, tol_b = ref.layernorm_grad(dy, x, w, mean, rstd, dto)
    close(dx, want, ref.rounded(want, tol, TYPES[t]), "dx")
    if dw is not None:
        close(dw, want_w, tol_w + 2.0 ** -126, "dweight")
    if db is not None:
        close(db, want_b, tol_b + 2.0 ** -126, "dbias")


@every_type
@pytest.mark.parametrize("cols", COLS + (33000,))
def test_layernorm_grad_columns(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows = (1, 2, 5, 9, 33)[k]
        dy, x, w, mean, rstd, dto = grad_inputs(t, rows, cols, pad, off, 200 + cols + k, k % 2 == 0)
        dx, da = matrix(rows, cols, TYPES[t], pad, off)
        dw, db = f32(cols + 1), f32(cols + 1)
        getattr(ew, "ew_layernorm_grad_" + t)(dy, x, w, mean, rstd, dx, dw[:cols], db[:cols],
                                              space(ew.ew_layernorm_grad_workspace(rows, cols)),
                                              dtotal=dto)
        check_grad(t, dy, x, w, mean, rstd, dto, dx, dw[:cols], db[:cols])
        guards_kept(dx, da)
        assert float(dw[cols]) == GUARD and float(db[cols]) == GUARD


@every_type
@pytest.mark.parametrize("rows,cols", [(4000, 64), (1500, 1000), (700, 4096), (513, 257),
                                       (600, 8200), (2100, 12), (300, 20000)])
def test_layernorm_grad_many_rows(t, rows, cols):
    dy, x, w, mean, rstd, dto = grad_inputs(t, rows, cols, 0, 0, 31)
    dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
    ws = space(ew.ew_layernorm_grad_workspace(rows, cols))
    getattr(ew, "ew_layernorm_grad_" + t)(dy, x, w, mean, rstd, dx, dw, db, ws, dtotal=dto)
    check_grad(t, dy, x, w, mean, rstd, dto, dx, dw, db)


@every_type
@pytest.mark.parametrize("cols", (64, 1001, 8191, 40000))
def test_layernorm_grad_options_and_aliases(t, cols):
    rows = 21
    fn = getattr(ew, "ew_layernorm_grad_" + t)
    dy, x, w, mean, rstd, dto = grad_inputs(t, rows, cols, 0, 0, 41)
    ws = space(ew.ew_layernorm_grad_workspace(rows, cols))
    dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
    fn(dy, x, None, mean, rstd, dx)                  # neither weight, sums nor workspace
    check_grad(t, dy, x, None, mean, rstd, None, dx, None, None)
    fn(dy, x, w, mean, rstd, dx, dweight=dw, workspace=ws)
    check_grad(t, dy, x, w, mean, rstd, None, dx, dw, None)
    fn(dy, x, w, mean, rstd, dx, dbias=db, workspace=ws)
    check_grad(t, dy, x, w, mean, rstd, None, dx, None, db)
    for k in range(3):                               # dx is dy, x or dtotal
        args = [dy.clone(), x.clone(), dto.clone()]
        fn(args[0], args[1], w, mean, rstd, args[k], dw, db, ws, dtotal=args[2])
        check_grad(t, dy, x, w, mean, rstd, dto, args[k], dw, db)


@every_type
def test_layernorm_grad_of_no_rows_clears_the_sums(t):
    dw, db = f32(100), f32(100)
    x = torch.empty(0, 100, dtype=TYPES[t], device=DEV)
    none = torch.empty(0, device=DEV)
    getattr(ew, "ew_layernorm_grad_" + t)(x, x, None, none, none, x, dw, db)
    assert not bool(dw.any()) and not bool(db.any())


def test_layernorm_grad_against_differences():
    """The gradient of sum(c * y) by x, the weight and the bias against central
    differences of the forward kernel in binary32: y is off by about 1e-6, so
    a difference over 2h by 1e-6 / h; its own error is of the order of h^2."""
    g, rows, cols, h = gen(5), 3, 37, 1e-2
    x, w, b, c = randn(g, rows, cols), 1 + 0.2 * randn(g, cols), randn(g, cols), randn(g, rows, cols)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)

    def loss(x, w, b):
        ew.ew_layernorm_f32(x, w, b, y, mean=mean, rstd=rstd)
        return float((c.double() * y.double()).sum())

    loss(x, w, b)
    dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
    ew.ew_layernorm_grad_f32(c, x, w, mean, rstd, dx, dw, db,
                             space(ew.ew_layernorm_grad_workspace(rows, cols)))
    for k, (v, d) in enumerate(((x, dx), (w, dw), (b, db))):
        for i in range(0, v.numel(), 7):
            args = [x, w, b]
            sides = []
            for sign in (1, -1):
                args[k] = v.clone()
                args[k].view(-1)[i] += sign * h
                sides.append(loss(*args))
            assert abs((sides[0] - sides[1]) / (2 * h) - float(d.view(-1)[i])) < 5e-3


# ---------------------------------------------------------------------------
# Policy loss
# ---------------------------------------------------------------------------

class Batch:
    """A batch of sequences with what lies around it."""

    def __init__(self, rows, cols, pad=0, off=0, seed=0, ref_logp=True, each=True, mask=True):
        g = gen(seed + 7 * rows + cols)
        old = -torch.rand(rows, cols, generator=g, device=DEV) * 4
        self.old = matrix(rows, cols, torch.float32, pad, off, old)[0]
        self.logp = matrix(rows, cols, torch.float32, pad, off, old + 0.3 * randn(g, rows, cols))[0]
        # far and near references: both sides of the series
        far = torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 0.2, 3.0, 0.05)
        self.ref = matrix(rows, cols, torch.float32, pad, off,
                          self.logp + far * randn(g, rows, cols))[0] if ref_logp else None
        self.advantage = (matrix(rows, cols, torch.float32, pad, off, randn(g, rows, cols))[0]
                          if each else randn(g, rows))
        self.mask = None
        if mask:
            length = torch.randint(0, cols + 1, (rows, 1), generator=g, device=DEV)
            live = torch.arange(cols, device=DEV) < length
            live &= torch.rand(rows, cols, generator=g, device=DEV) < 0.9     # gaps too
            whole = torch.full((rows, cols + pad + off,), 1, dtype=torch.uint8, device=DEV)
            self.mask = whole[:, off:off + cols]
            self.mask.copy_(live.to(torch.uint8) * 3)
        self.rows, self.cols, self.pad, self.off = rows, cols, pad, off

    def check(self, low=0.2, high=0.3, kl=0.1, mean="tokens", scale=1.0, dloss=None):
        rows, cols = self.rows, self.cols
        a = self.advantage if self.advantage.dim() == 2 else self.advantage[:, None]
        want = ref.Policy(self.logp, self.old, a, self.ref, self.mask, low, high, kl, mean, scale)
        loss, stats, weights = f32(2), f32(5), f32(rows + 1)
        ew.ew_policy_loss_f32(self.logp, self.old, self.advantage, loss[:1],
                              weights=weights[:rows], ref_logp=self.ref, mask=self.mask,
                              stats=stats[:4], clip_low=low, clip_high=high, kl=kl, mean=mean,
                              scale=scale, workspace=space(ew.ew_policy_loss_workspace(rows, cols)))
        close(weights[:rows], want.weights, want.weights.abs() * U * 1.01, "weights")
        close(loss[:1], want.loss[None], want.tol_loss + 2.0 ** -126, "loss")
        close(stats[:1], want.policy[None], want.tol_loss + want.tol_policy + 2.0 ** -126, "policy")
        close(stats[1:2], want.kl[None], want.tol_kl + 2.0 ** -126, "kl")
        close(stats[2:3], want.fraction[None], U, "fraction")
        close(stats[3:4], want.fall[None], want.tol_fall + 2.0 ** -126, "fall")
        for v in (loss, stats, weights):
            assert float(v[-1]) == GUARD
        dlogp, whole = matrix(rows, cols, torch.float32, self.pad, self.off)
        d = None if dloss is None else torch.tensor([dloss], device=DEV)
        ew.ew_policy_loss_grad_f32(self.logp, self.old, self.advantage, weights[:rows], dlogp,
                                   ref_logp=self.ref, mask=self.mask, dloss=d, clip_low=low,
                                   clip_high=high, kl=kl)
        g, tol = want.grad(weights[:rows], 1.0 if dloss is None else ref.f32(dloss))
        close(dlogp, g, tol, "dlogp")
        guards_kept(dlogp, whole)
        return loss[0], weights[:rows], dlogp


# one block, whole sequences, parts of long ones
SHAPES = ((1, 1), (1, 2), (1, 3), (1, 4), (2, 5), (7, 7), (3, 63), (8, 512), (9, 1025), (16, 1024),
          (1, 16385), (3, 20001), (1, 300001), (40, 5000), (255, 1030), (256, 1031), (300, 257),
          (1500, 65), (5000, 7), (20000, 1), (70000, 3))


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("mean", ("tokens", "sequences", "none"))
def test_policy_shapes(rows, cols, mean):
    for k, (pad, off) in enumerate(LAYOUTS[:1] + LAYOUTS[2:]):
        batch = Batch(rows, cols, pad, off, k, ref_logp=k != 1, each=k != 2, mask=k != 3)
        batch.check(mean=mean, scale=(1.0, -0.5, 3.0, 1e-3)[k], dloss=(None, 0.25, -2.0, 1.0)[k],
                    kl=(0.1, 0.1, 0.0, 0.02)[k])


@pytest.mark.parametrize("rows,cols", ((4, 300), (6, 9000), (700, 64)))
@pytest.mark.parametrize("low,high", ((0.0, 0.0), (0.2, 0.2), (1.0, 0.5), (7.0, math.inf),
                                      (math.inf, 0.1)))
def test_policy_borders(rows, cols, low, high):
    Batch(rows, cols, seed=9).check(low=low, high=high)


@pytest.mark.parametrize("low,high", ((0.2, 0.2), (0.1, 0.28)))
def test_policy_sides_of_a_border_are_decided_exactly(low, high):
    """Log ratios one last place around the borders, at every size of log
    probability: the reference decides in 64 bits."""
    old, logp = [], []
    for border in (math.log1p(ref.f32(high)), math.log1p(-ref.f32(low))):
        for base in (0.0, -0.1, -1.0, -3.7, -20.0, -300.0):
            o = torch.tensor(base, dtype=torch.float32)
            p = (o.double() + border).float()
            for step in range(-3, 4):
                q = p.clone()
                for _ in range(abs(step)):
                    q = torch.nextafter(q, torch.tensor(math.inf if step > 0 else -math.inf))
                old.append(float(o))
                logp.append(float(q))
    n = len(old)
    batch = Batch(2, n, ref_logp=False, mask=False, each=False)
    batch.old.copy_(torch.tensor(old).expand(2, n))
    batch.logp.copy_(torch.tensor(logp).expand(2, n))
    batch.advantage.copy_(torch.tensor([1.0, -1.0]))
    _, _, dlogp = batch.check(low=low, high=high)
    want = ref.Policy(batch.logp, batch.old, batch.advantage[:, None], low=low, high=high)
    assert torch.equal(dlogp == 0, want.clipped) and 0 < int(want.clipped.sum()) < 2 * n


def test_policy_at_the_first_step_and_of_equal_references():
    """logp, old_logp and ref_logp the same tensor: ratio 1, no divergence."""
    batch = Batch(5, 700, seed=2)
    batch.old = batch.ref = batch.logp
    loss, weights, dlogp = batch.check(low=0.0, high=0.0)
    a = torch.where(batch.mask != 0, batch.advantage, 0.0)
    close(dlogp, -a.double() * weights.double()[:, None], a.abs() * weights[:, None] * 4 * U, "grad")


@pytest.mark.parametrize("rows,cols", ((5, 70), (4, 6000), (600, 40), (1, 40000)))
@pytest.mark.parametrize("mean", ("tokens", "sequences", "none"))
def test_policy_masked_places_hold_anything(rows, cols, mean):
    batch = Batch(rows, cols, seed=4)
    batch.mask[rows // 2] = 0                    # a sequence of no counted tokens
    loss, weights, dlogp = batch.check(mean=mean)
    out = batch.mask == 0
    for bad in (math.nan, math.inf, -math.inf):
        for v in (batch.logp, batch.old, batch.ref, batch.advantage):
            v[out] = bad
        again = batch.check(mean=mean)
        for one, other in zip((loss, weights, dlogp), again):
            assert torch.equal(one, other)
    assert not bool(dlogp[out].any()) and float(weights[rows // 2]) == 0.0
    batch.mask.zero_()                           # nothing counts at all
    loss, weights, dlogp = batch.check(mean=mean)
    assert float(loss) == 0.0 and not bool(weights.any()) and not bool(dlogp.any())


def test_policy_without_tokens():
    for rows, cols in ((0, 8), (5, 0), (0, 0), (40000, 0)):
        for each in (True, False):
            z = torch.empty(rows, cols, device=DEV)
            a = z if each else torch.empty(rows, device=DEV)
            loss, stats, weights = f32(1), f32(4), f32(rows + 1)
            ew.ew_policy_loss_f32(z, z, a, loss, weights=weights, stats=stats, per_token=each,
                                  workspace=space(ew.ew_policy_loss_workspace(rows, cols)))
            assert float(loss) == 0.0 and not bool(stats.any()) and not bool(weights[:rows].any())
            assert float(weights[rows]) == GUARD
            ew.ew_policy_loss_grad_f32(z, z, a, weights, z, per_token=each)


def test_policy_far_references_and_infinities():
    """k = exp(d) - d - 1 over the whole range; a term of weight 0 may be infinite."""
    d = torch.tensor([0.0, 1e-8, -1e-8, 1e-4, -3e-3, 0.5, -0.999, 0.9999, 1.0, -1.0, 1.1, -5.0, 20.0,
                      80.0, -80.0, -1e6], device=DEV)
    n = d.numel()
    batch = Batch(2, n, mask=False)
    batch.logp.zero_()
    batch.ref.copy_(d.expand(2, n))
    batch.check(kl=0.5)
    for one in range(n):                         # each by itself: no larger one covers it
        single = Batch(1, 1, mask=False)
        single.logp.zero_()
        single.ref.fill_(float(d[one]))
        single.check(kl=0.5)
    for bad in (math.inf, -math.inf):
        batch.ref[0, 3] = bad
        loss, stats, weights = f32(1), f32(4), f32(2)
        dlogp = f32(2, n)
        for kl in (0.0, 0.5):
            ew.ew_policy_loss_f32(batch.logp, batch.old, batch.advantage, loss, weights=weights,
                                  ref_logp=batch.ref, stats=stats, kl=kl,
                                  workspace=space(ew.ew_policy_loss_workspace(2, n)))
            ew.ew_policy_loss_grad_f32(batch.logp, batch.old, batch.advantage, weights, dlogp,
                                       ref_logp=batch.ref, kl=kl)
            assert float(stats[1]) == math.inf
            assert math.isfinite(float(loss)) == (kl == 0.0)
            if kl == 0.0 or bad < 0:             # the slope far below is finite
                assert bool(torch.isfinite(dlogp).all())
            else:
                assert float(dlogp[0, 3]) == -math.inf
    batch.logp[1, 2] = math.nan
    ew.ew_policy_loss_f32(batch.logp, batch.old, batch.advantage, loss,
                          workspace=space(ew.ew_policy_loss_workspace(2, n)))
    assert math.isnan(float(loss))


@pytest.mark.parametrize("rows,cols", ((3, 37), (2, 5001), (400, 130)))
def test_policy_grad_in_place(rows, cols):
    batch = Batch(rows, cols, 1, 1, seed=6)
    _, weights, want = batch.check()
    for name in ("logp", "old", "ref", "advantage"):
        args = {k: getattr(batch, k).clone() for k in ("logp", "old", "ref", "advantage")}
        ew.ew_policy_loss_grad_f32(args["logp"], args["old"], args["advantage"], weights, args[name],
                                   ref_logp=args["ref"], mask=batch.mask, clip_high=0.3, kl=0.1)
        assert torch.equal(args[name], want), name


def test_policy_grad_against_differences():
    """Central differences of the definition in 64 bits, away from the borders:
    their error is of the order of h^2, the kernel's about 1e-6 of a slope."""
    batch, h = Batch(3, 21, seed=8), 1e-4
    x = (batch.logp - batch.old).double()
    far = ((x - math.log1p(ref.f32(0.3))).abs() > 1e-3) & ((x - math.log1p(-ref.f32(0.2))).abs() > 1e-3)
    _, _, dlogp = batch.check(mean="sequences", kl=0.1)
    for i in range(63):
        if not bool(far.view(-1)[i]):
            continue
        sides = []
        for sign in (1, -1):
            logp = batch.logp.double().clone()
            logp.view(-1)[i] += sign * h
            sides.append(ref.Policy(logp, batch.old, batch.advantage, batch.ref, batch.mask, 0.2,
                                    0.3, 0.1, "sequences").loss)
        assert abs(float(sides[0] - sides[1]) / (2 * h) - float(dlogp.view(-1)[i])) < 1e-5


# ---------------------------------------------------------------------------
# Tokens and experts
# ---------------------------------------------------------------------------

def i32(*shape):
    return torch.full(shape, 123, dtype=torch.int32, device=DEV)


def sort(ids, experts, align):
    """slot, offsets, counts, source of the kernel, checked entry by entry."""
    n = ids.numel()
    rows = ew.ew_experts_rows(n, experts, align)
    slot, offsets, counts, source = i32(n + 1), i32(experts + 2), i32(experts + 1), i32(rows + 1)
    ew.ew_experts_sort(ids, experts, slot[:n], offsets[:-1], counts=counts[:-1], source=source[:-1],
                       align=align, workspace=space(ew.ew_experts_sort_workspace(n, experts)))
    got = slot[:n], offsets[:-1], counts[:-1], source[:-1]
    for name, v, w in zip(("slot", "offsets", "counts", "source"), got,
                          ref.sort(ids, experts, align, rows)):
        assert torch.equal(v.cpu(), w), name
    for v in (slot, offsets, counts, source):
        assert int(v[-1]) == 123
    return got


@pytest.mark.parametrize("entries", (0, 1, 2, 63, 64, 65, 100, 1000, 1025, 8191, 8192, 8193, 30001,
                                     200000, 600001))
@pytest.mark.parametrize("experts", (1, 2, 3, 8, 100, 256, 512, 513, 1000, 1024))
def test_sort(entries, experts):
    g = gen(entries + experts)
    for align in (1, 16, 100):
        ids = torch.randint(-2, experts + 2, (entries,), generator=g, device=DEV)
        sort(ids, experts, align)


@pytest.mark.parametrize("entries", (70, 3000, 40000))
def test_sort_of_uneven_choices(entries):
    at = torch.arange(entries, device=DEV)
    far = torch.tensor([1 << 40, -(1 << 40), (1 << 32) + 1, (1 << 63) - 1, -(1 << 63)], device=DEV)
    for experts, align in ((7, 1), (300, 1024), (1024, 64)):
        for ids in (torch.zeros_like(at), torch.full_like(at, experts - 1), -1 - at,
                    at * experts // entries, (entries - 1 - at) * experts // entries, far[at % 5],
                    torch.where(at % 3 == 0, 1, -1)):
            sort(ids.long(), experts, align)


def test_sort_without_options():
    ids = torch.randint(0, 9, (500, 4), generator=gen(1), device=DEV)
    slot, offsets = i32(500, 4), i32(10)
    ew.ew_experts_sort(ids, 9, slot, offsets, align=8)
    want = ref.sort(ids, 9, 8, ew.ew_experts_rows(2000, 9, 8))
    assert torch.equal(slot.cpu().view(-1), want[0]) and torch.equal(offsets.cpu(), want[1])


class Routed:
    """Tokens with their choices sorted, and a matrix of the experts' rows."""

    def __init__(self, t, tokens, cols, top, experts=8, align=16, pad=0, off=0, seed=0, drop=0.2):
        g, self.dt = gen(seed + tokens + cols), TYPES[t]
        self.t, self.tokens, self.cols, self.top, self.experts = t, tokens, cols, top, experts
        self.pad, self.off = pad, off
        ids = torch.randint(0, experts, (tokens, top), generator=g, device=DEV)
        ids[torch.rand(tokens, top, generator=g, device=DEV) < drop] = -1
        self.slot, self.offsets, self.counts, self.source = sort(ids, experts, align)
        self.slot = self.slot.view(tokens, top)
        self.places = self.source.numel()
        self.x = self.matrix(tokens, randn(g, tokens, cols))[0]
        self.res = self.matrix(tokens, randn(g, tokens, cols))[0]
        self.z = self.matrix(self.places, randn(g, self.places, cols))[0]
        self.w = torch.rand(tokens, top, generator=g, device=DEV)

    def matrix(self, rows, fill=None):
        return matrix(rows, self.cols, self.dt, self.pad, self.off, fill)

    def call(self, name, *args, **kw):
        getattr(ew, f"ew_experts_{name}_{self.t}")(*args, **kw)

    def expected(self, rows_and_values, cleared=True):
        """What a matrix of the experts' rows holds: values, zeros in the
        padding, the guard elsewhere."""
        at, values = rows_and_values
        want = torch.full((self.places, self.cols), GUARD, dtype=torch.float64, device=DEV)
        if cleared:
            lo, n, hi = (v.long() for v in (self.offsets[:-1], self.counts, self.offsets[1:]))
            r = torch.arange(self.places, device=DEV)
            pad = ((r >= (lo + n)[:, None]) & (r < hi[:, None])).any(0)
            want[pad] = 0.0
        want[at] = values
        return want

    def check_gather(self):
        kept = self.slot >= 0
        values = self.x.double()[:, None].expand(-1, self.top, -1)[kept]
        for cleared in (True, False):
            out, whole = self.matrix(self.places)
            pads = {"offsets": self.offsets, "counts": self.counts} if cleared else {}
            self.call("gather", self.x, self.slot, out, **pads)
            assert torch.equal(out.double(), self.expected((self.slot.long()[kept], values), cleared))
            guards_kept(out, whole)

    def check_combine(self):
        for w, res in ((self.w, self.res), (None, None), (self.w, None), (None, self.res)):
            y, whole = self.matrix(self.tokens)
            self.call("combine", self.z, self.slot, y, weights=w, residual=res)
            want, tol = ref.combine(self.z, self.slot, w, res)
            close(y, want, ref.rounded(want, tol, self.dt), "y")
            guards_kept(y, whole)
        y = self.res.clone()
        self.call("combine", self.z, self.slot, y, weights=self.w, residual=y)
        want, tol = ref.combine(self.z, self.slot, self.w, self.res)
        close(y, want, ref.rounded(want, tol, self.dt), "y in place")

    def check_grad(self):
        at, values, dots, tol = ref.combine_grad(self.x, self.z, self.slot, self.w)
        for cleared in (True, False):
            dz, whole = self.matrix(self.places)
            dw = f32(self.tokens + 1, self.top)
            pads = {"offsets": self.offsets, "counts": self.counts} if cleared else {}
            self.call("combine_grad", self.x, self.z, self.slot, self.w, dz, dw[:-1], **pads)
            want = self.expected((at, values), cleared)
            close(dz, want, ref.rounded(want, want.abs() * U, self.dt), "dz")
            close(dw[:-1], dots, tol, "dweights")
            guards_kept(dz, whole)
            assert bool((dw[-1] == GUARD).all())
        z = self.z.clone()                           # in place
        dw2 = f32(self.tokens, self.top)
        self.call("combine_grad", self.x, z, self.slot, self.w, z, dw2)
        assert torch.equal(dw2, dw[:-1])
        kept = torch.zeros(self.places, dtype=torch.bool, device=DEV)
        kept[at] = True
        assert torch.equal(z[kept], dz[kept]) and torch.equal(z[~kept], self.z[~kept])


@every_type
@pytest.mark.parametrize("cols", (1, 2, 3, 7, 8, 9, 63, 64, 65, 128, 257, 512, 1000, 2048, 4097, 9000))
def test_rows_to_experts_and_back(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        r = Routed(t, (1, 5, 16, 33, 70)[k], cols, (1, 2, 4, 8, 3)[k], pad=pad, off=off, seed=k,
                   align=(1, 16, 4, 16, 7)[k], experts=(1, 8, 32, 5, 8)[k])
        r.check_gather()
        r.check_combine()
        r.check_grad()


@every_type
@pytest.mark.parametrize("tokens,cols,top", [(3000, 64, 2), (2100, 24, 8), (700, 2048, 6),
                                             (5, 100, 64), (300, 700, 17), (1, 30000, 9)])
def test_many_tokens_and_choices(t, tokens, cols, top):
    r = Routed(t, tokens, cols, top, experts=40, align=32)
    r.check_gather()
    r.check_combine()
    r.check_grad()


@every_type
def test_all_and_no_choices_kept(t):
    for drop in (0.0, 1.0):
        r = Routed(t, 50, 200, 4, drop=drop)
        r.check_gather()
        r.check_combine()
        r.check_grad()


@every_type
def test_slots_and_offsets_outside_the_matrix(t):
    """Slots that name no row are dropped, offsets past the end are not followed."""
    r = Routed(t, 30, 100, 3)
    for bad in (-1, -(1 << 31), r.places, (1 << 31) - 1):
        r.slot[::4, 1] = bad
        r.slot[3] = bad
        kept = (r.slot >= 0) & (r.slot < r.places)
        out, whole = r.matrix(r.places)
        r.call("gather", r.x, r.slot, out)
        values = r.x.double()[:, None].expand(-1, 3, -1)[kept]
        assert torch.equal(out.double(), r.expected((r.slot.long()[kept], values), False))
        guards_kept(out, whole)
        r.check_combine()
        at, values, dots, tol = ref.combine_grad(r.x, r.z, r.slot, r.w)
        dz, whole = r.matrix(r.places)
        dw = f32(30, 3)
        r.call("combine_grad", r.x, r.z, r.slot, r.w, dz, dw)
        want = r.expected((at, values), False)
        close(dz, want, ref.rounded(want, want.abs() * U, r.dt), "dz")
        close(dw, dots, tol, "dweights")
        guards_kept(dz, whole)
    slot = torch.full_like(r.slot, -1)
    for lo, n, hi in ((-50, 10, 5), (0, 0, r.places + 1000), (r.places - 2, 0, (1 << 31) - 1),
                      (-(1 << 31), 0, -5), ((1 << 31) - 1, (1 << 31) - 1, 3)):
        out, whole = r.matrix(r.places)
        r.call("gather", r.x, slot, out,
               offsets=torch.tensor([lo, hi], dtype=torch.int32, device=DEV),
               counts=torch.tensor([n], dtype=torch.int32, device=DEV))
        guards_kept(out, whole)
        cleared = (torch.arange(r.places, device=DEV) >= lo + n) & \
                  (torch.arange(r.places, device=DEV) < hi)
        assert not bool(out[cleared].any()) and bool((out[~cleared].float() == GUARD).all())


@every_type
def test_masked_choices_hold_anything(t):
    """NaN weights and rows behind dropped choices do not reach the results."""
    r = Routed(t, 40, 300, 4, drop=0.5)
    some = (r.source >= 0)
    r.w[r.slot < 0] = math.nan
    r.z[~some] = math.nan
    want, tol = ref.combine(r.z, r.slot, torch.where(r.slot < 0, 0.0, r.w), r.res)
    y = torch.empty(40, 300, dtype=r.dt, device=DEV)
    r.call("combine", r.z, r.slot, y, weights=r.w, residual=r.res)
    close(y, want, ref.rounded(want, tol, r.dt), "y")
    dz, dw = r.z.clone(), f32(40, 4)
    r.call("combine_grad", r.x, r.z, r.slot, r.w, dz, dw, offsets=r.offsets, counts=r.counts)
    assert bool(torch.isfinite(dw).all()) and not bool(dw[r.slot < 0].any())
    assert bool(torch.isfinite(dz[:int(r.offsets[-1])].float()).all())


def test_no_rows_of_experts():
    """No place for any choice: the residual alone, gradients of 0."""
    x, none = torch.ones(4, 8, device=DEV), torch.empty(0, 8, device=DEV)
    slot, w, dw = i32(4, 2), torch.ones(4, 2, device=DEV), f32(4, 2)
    y = torch.empty_like(x)
    ew.ew_experts_gather_f32(x, slot, none)
    ew.ew_experts_combine_f32(none, slot, y, weights=w, residual=x)
    assert torch.equal(y, x)
    ew.ew_experts_combine_f32(none, slot, y)
    assert not bool(y.any())
    ew.ew_experts_combine_grad_f32(x, none, slot, w, none, dw)
    assert not bool(dw.any())
    # no columns: the dot products are 0
    none, dw = torch.empty(4, 0, device=DEV), f32(4, 2)
    ew.ew_experts_combine_grad_f32(none, none, slot, w, none, dw)
    assert not bool(dw.any())


def test_combine_gradients_against_differences():
    """sum(c * y) is linear in z and in the weights: differences are exact but
    for the roundings of y, about 1e-6 over a step of 1."""
    r = Routed("f32", 6, 33, 3, experts=4, align=4)
    c = randn(gen(77), 6, 33)
    y, dz, dw = torch.empty_like(c), torch.zeros_like(r.z), f32(6, 3)

    def loss(z, w):
        ew.ew_experts_combine_f32(z, r.slot, y, weights=w, residual=r.res)
        return float((c.double() * y.double()).sum())

    ew.ew_experts_combine_grad_f32(c, r.z, r.slot, r.w, dz, dw)
    for i in range(18):
        w = [r.w.clone(), r.w.clone()]
        w[0].view(-1)[i] += 1
        assert abs(loss(r.z, w[0]) - loss(r.z, w[1]) - float(dw.view(-1)[i])) < 1e-4
    for i in range(0, r.z.numel(), 11):
        z = r.z.clone()
        z.view(-1)[i] += 1
        assert abs(loss(z, r.w) - loss(r.z, r.w) - float(dz.view(-1)[i])) < 1e-4


def test_gather_gradient_is_combine_without_weights():
    r = Routed("f32", 9, 20, 4)
    dout, out, dx = randn(gen(78), r.places, 20), torch.zeros(r.places, 20, device=DEV), \
        torch.empty(9, 20, device=DEV)
    ew.ew_experts_combine_f32(dout, r.slot, dx)
    v = randn(gen(79), 9, 20)
    ew.ew_experts_gather_f32(v, r.slot, out)
    # <dout, gather(v)> = <combine(dout), v>
    a, b = (dout.double() * out.double()).sum(), (dx.double() * v.double()).sum()
    assert abs(float(a - b)) < 1e-4
