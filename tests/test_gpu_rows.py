"""The row operators on the GPU against their definitions in 64 bits
(tests/rows_ref.py, which derives the tolerances)."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests import rows_ref as ref
from tests.rows_ref import TYPES, close

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 7.0          # what lies around the outputs and must stay

every_type = pytest.mark.parametrize("t", TYPES)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def matrix(rows, cols, dt, pad=0, off=0, fill=None):
    """rows x cols view whose rows lie cols + pad apart, `off` elements into
    its allocation, guard values around it: (view, allocation)."""
    whole = torch.full((off + rows * (cols + pad) + 16,), GUARD, device=DEV).to(dt)
    view = whole[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if fill is not None:
        view.copy_(fill)
    return view, whole


def guards_kept(view, whole):
    """Everything of the allocation outside the view still holds the guard."""
    w = whole.clone()
    torch.as_strided(w, view.shape, view.stride(), view.storage_offset()).fill_(GUARD)
    assert bool((w.float() == GUARD).all()), "written outside the output"


# one column, below a vector, around vectors, waves and blocks, odd, large
NORM_COLS = (1, 2, 3, 7, 8, 9, 63, 64, 65, 127, 255, 256, 260, 511, 513, 1000, 1024, 2048, 2056,
             4095, 4096, 4097, 5003, 8192, 10007, 16384)
LAYOUTS = ((0, 0), (8, 0), (1, 0), (0, 1), (13, 3))      # (pad, offset)


def norm_inputs(t, rows, cols, pad, off, seed, residual=True):
    g, dt = gen(seed), TYPES[t]
    x = matrix(rows, cols, dt, pad, off, randn(g, rows, cols))[0]
    res = matrix(rows, cols, dt, pad, off, 2 * randn(g, rows, cols))[0] if residual else None
    w = (1 + 0.2 * randn(g, cols)).to(dt)
    return x, res, w


def check_norm(t, x, res, w, y, total, rstd, eps):
    dt = TYPES[t]
    h = ref.norm_total(x, res)
    if total is not None:
        assert torch.equal(total, h)
    want, want_r, tol, tol_r = ref.norm(h, w, eps)
    if rstd is not None:
        close(rstd, want_r, tol_r, "rstd")
    if y is not None:
        close(y, want, tol + (want.abs() + tol) * ref.half_ulp(dt) + ref.tiny(dt), "y")
    return want, tol


@every_type
@pytest.mark.parametrize("cols", NORM_COLS)
def test_norm_columns(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows = (1, 2, 5, 9, 33)[k]
        x, res, w = norm_inputs(t, rows, cols, pad, off, 100 + cols + k)
        (y, ya), (total, ta) = (matrix(rows, cols, TYPES[t], pad, off) for _ in range(2))
        rstd = torch.empty(rows, device=DEV)
        getattr(ew, "ew_rmsnorm_" + t)(x, w, y, residual=res, total=total, rstd=rstd, eps=1e-5)
        check_norm(t, x, res, w, y, total, rstd, 1e-5)
        guards_kept(y, ya)
        guards_kept(total, ta)


@every_type
@pytest.mark.parametrize("rows,cols", [(1, 65536), (3, 40001), (2, 33000), (1100, 100), (5000, 64),
                                       (300, 4096)])
def test_norm_long_rows_and_many_rows(t, rows, cols):
    x, res, w = norm_inputs(t, rows, cols, 0, 0, 7)
    y, total, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV)
    getattr(ew, "ew_rmsnorm_" + t)(x, w, y, residual=res, total=total, rstd=rstd)
    check_norm(t, x, res, w, y, total, rstd, 1e-5)
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(rows, 1, device=DEV)
    getattr(ew, "ew_rmsnorm_e4m3_" + t)(x, w, q, scales, group=0, residual=res, total=total,
                                        rstd=rstd)
    check_norm8(t, x, res, w, q, scales, 0, total, rstd)


@every_type
@pytest.mark.parametrize("cols", (5, 1024, 4100, 40000))
def test_norm_options_and_aliases(t, cols):
    rows = 6
    fn = getattr(ew, "ew_rmsnorm_" + t)
    x, res, w = norm_inputs(t, rows, cols, 3, 1, 11)
    y = torch.empty(rows, cols, dtype=TYPES[t], device=DEV)
    fn(x, w, y)                                   # neither residual, total nor rstd
    check_norm(t, x, None, w, y, None, None, 1e-5)
    fn(x, w, y, residual=res)                     # a residual, no total
    check_norm(t, x, res, w, y, None, None, 1e-5)
    a, b = x.clone(), res.clone()
    fn(a, w, a)                                   # y is x
    check_norm(t, x, None, w, a, None, None, 1e-5)
    a = x.clone()
    fn(a, w, y, residual=b, total=b)              # the residual stream in place
    check_norm(t, x, res, w, y, b, None, 1e-5)
    a, b = x.clone(), res.clone()
    fn(a, w, b, residual=b, total=a)              # both in place
    check_norm(t, x, res, w, b, a, None, 1e-5)
    a, b = x.clone(), res.clone()
    fn(a, w, a, residual=b)                       # y is x, the residual only read
    check_norm(t, x, res, w, a, None, None, 1e-5)
    # the two halves of one buffer
    both = torch.empty(rows, 2 * cols, dtype=TYPES[t], device=DEV)
    both[:, :cols].copy_(x)
    fn(both[:, :cols], w, both[:, cols:])
    check_norm(t, x, None, w, both[:, cols:], None, None, 1e-5)
    assert torch.equal(both[:, :cols], x)


@every_type
def test_norm_of_zeros_large_values_and_nan(t):
    rows, cols = 4, 300
    x = torch.zeros(rows, cols, device=DEV)
    x[1] = 100.0
    x[2, 17] = math.nan
    x[3, 5] = math.inf
    x, w = x.to(TYPES[t]), torch.ones(cols, dtype=TYPES[t], device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    getattr(ew, "ew_rmsnorm_" + t)(x, w, y, rstd=rstd, eps=1e-6)
    assert bool((y[0] == 0).all())
    check_norm(t, x[:2], None, w, y[:2], None, rstd[:2], 1e-6)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(rstd[2]))
    assert float(rstd[3]) == 0.0 and bool(torch.isnan(y[3, 5])) and float(y[3, 6]) == 0.0
    getattr(ew, "ew_rmsnorm_" + t)(x[:1], w, y[:1], rstd=rstd[:1], eps=0.0)
    assert math.isinf(float(rstd[0])) and bool(torch.isnan(y[0]).all())    # 0 * inf


def check_norm8(t, x, res, w, q, scales, group, total, rstd, eps=1e-5):
    want, tol = check_norm(t, x, res, w, None, total, rstd, eps)
    s, each = ref.group_scales(want, group)
    _, tol_s = ref.group_scales(tol, group)
    rel = (ref.adds(x.shape[1]) / 2 + 10) * ref.U
    close(scales, s, s * rel, "scales")
    # q rounds y / scale: half a step of e4m3, or of its subnormals (2^-10)
    got = q.double() * scales.double().repeat_interleave(group or x.shape[1], 1)[:, :x.shape[1]]
    close(got, want, want.abs() * (2.0 ** -4 * (1 + rel) + 4 * rel)
          + each * 2.0 ** -10 * (1 + 4 * rel) + tol, "q * scale")


@every_type
@pytest.mark.parametrize("group", (0, 16, 32, 64, 128, 256))
@pytest.mark.parametrize("cols", (1, 15, 64, 100, 1000, 2048, 4097, 8192, 16384))
def test_norm_e4m3(t, group, cols):
    for k, (pad, off) in enumerate(((0, 0), (13, 1))):
        rows = (3, 10)[k]
        x, res, w = norm_inputs(t, rows, cols, pad, off, 300 + cols + group + k)
        x[:, :cols // 2] *= 0.01                       # groups of different sizes
        total, _ = matrix(rows, cols, TYPES[t], pad, off)
        qw = torch.full((rows, cols + pad), GUARD, device=DEV).to(torch.float8_e4m3fn)
        q = qw[:, :cols]
        groups = -(-cols // group) if group else 1
        scales = torch.empty(rows, groups, device=DEV)
        rstd = torch.empty(rows, device=DEV)
        getattr(ew, "ew_rmsnorm_e4m3_" + t)(x, w, q, scales, group=group, residual=res,
                                            total=total, rstd=rstd)
        check_norm8(t, x, res, w, q, scales, group, total, rstd)
        assert bool((qw[:, cols:].float() == GUARD).all())


@every_type
def test_norm_e4m3_zero_rows_and_nan_weights(t):
    rows, cols = 3, 256
    x = torch.zeros(rows, cols, device=DEV, dtype=TYPES[t])
    x[1] = 1.0
    x[2] = 1.0
    w = torch.ones(cols, dtype=TYPES[t], device=DEV)
    w[70] = math.nan
    w[200] = 0.0
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(rows, 4, device=DEV)
    getattr(ew, "ew_rmsnorm_e4m3_" + t)(x, w, q, s, group=64)
    assert bool((s[0, [0, 2, 3]] == ref.SCALE_MIN).all()) and bool((q[0, :64].float() == 0).all())
    assert bool(torch.isnan(s[:, 1]).all())
    assert bool(torch.isnan(q[1, 64:128].float()).all())
    assert not bool(torch.isnan(q[1:, 128:].float()).any())
    assert bool((q[1, 0:64].float() == 448).all()) and float(q[1, 200].float()) == 0.0


def check_norm_grad(t, dy, x, w, rstd, dt_, dx, dw, inputs=None):
    dy0, x0, dt0 = inputs or (dy, x, dt_)
    want, want_w, tol, tol_w = ref.norm_grad(dy0, x0, w, rstd, dt0)
    dt = TYPES[t]
    close(dx, want, tol + (want.abs() + tol) * ref.half_ulp(dt) + ref.tiny(dt), "dx")
    if dw is not None:
        close(dw, want_w, tol_w, "dweight")


def grad_space(rows, cols):
    return torch.empty(ew.ew_rmsnorm_grad_workspace(rows, cols), dtype=torch.uint8, device=DEV)


@every_type
@pytest.mark.parametrize("cols", NORM_COLS + (33000,))
def test_norm_grad_columns(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows = (1, 2, 5, 9, 33)[k]
        g = gen(500 + cols + k)
        x, _, w = norm_inputs(t, rows, cols, pad, off, 600 + cols + k, residual=False)
        dy = matrix(rows, cols, TYPES[t], pad, off, 0.1 * randn(g, rows, cols))[0]
        dtotal = matrix(rows, cols, TYPES[t], pad, off, 0.1 * randn(g, rows, cols))[0]
        rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
        dx, dxa = matrix(rows, cols, TYPES[t], pad, off)
        dw = torch.full((cols + 2,), GUARD, device=DEV)
        getattr(ew, "ew_rmsnorm_grad_" + t)(dy, x, w, rstd, dx, dw[1:-1], grad_space(rows, cols),
                                            dtotal=dtotal)
        check_norm_grad(t, dy, x, w, rstd, dtotal, dx, dw[1:-1])
        guards_kept(dx, dxa)
        assert float(dw[0]) == GUARD and float(dw[-1]) == GUARD


@every_type
@pytest.mark.parametrize("rows,cols", [(4000, 64), (1500, 1000), (700, 4096), (513, 257), (600, 8200)])
def test_norm_grad_many_rows(t, rows, cols):
    g = gen(rows + cols)
    x, _, w = norm_inputs(t, rows, cols, 0, 0, 9, residual=False)
    dy = (0.1 * randn(g, rows, cols)).to(TYPES[t])
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
    fn, space = getattr(ew, "ew_rmsnorm_grad_" + t), grad_space(rows, cols)
    fn(dy, x, w, rstd, dx, dw, space)
    check_norm_grad(t, dy, x, w, rstd, None, dx, dw)
    again, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    fn(dy, x, w, rstd, again, dw2, torch.full_like(space, 0xff))    # what the space held is nothing
    assert torch.equal(dx, again) and torch.equal(dw, dw2)          # and the same bits


@every_type
@pytest.mark.parametrize("cols", (64, 1001, 40000))
def test_norm_grad_in_place_and_without_dweight(t, cols):
    rows = 40
    g = gen(cols)
    x, _, w = norm_inputs(t, rows, cols, 0, 0, 10, residual=False)
    dy, dtotal = ((0.1 * randn(g, rows, cols)).to(TYPES[t]) for _ in range(2))
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    fn = getattr(ew, "ew_rmsnorm_grad_" + t)
    dx = torch.empty_like(x)
    fn(dy, x, w, rstd, dx, dtotal=dtotal)
    check_norm_grad(t, dy, x, w, rstd, dtotal, dx, None)
    for which in range(3):
        a = [dy.clone(), x.clone(), dtotal.clone()]
        dw = torch.empty(cols, device=DEV)
        fn(a[0], a[1], w, rstd, a[which], dw, grad_space(rows, cols), dtotal=a[2])
        check_norm_grad(t, None, None, w, rstd, None, a[which], dw, inputs=(dy, x, dtotal))


@every_type
def test_norm_grad_of_no_rows_clears_dweight(t):
    x = torch.empty(0, 100, dtype=TYPES[t], device=DEV)
    w = torch.ones(100, dtype=TYPES[t], device=DEV)
    dw = torch.full((100,), GUARD, device=DEV)
    getattr(ew, "ew_rmsnorm_grad_" + t)(x, x, w, torch.empty(0, device=DEV), torch.empty_like(x), dw,
                                        grad_space(0, 100))
    assert bool((dw == 0).all())


def test_norm_grad_against_differences():
    """The loss <c, y> + <e, total> changes along a direction as the gradient
    says: central differences of the 64-bit norm."""
    rows, cols = 3, 130
    g = gen(3)
    x, dy, dtotal, v = (randn(g, rows, cols) for _ in range(4))
    w, u = 1 + 0.2 * randn(g, cols), randn(g, cols)

    def loss(x, w):
        y = x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w
        return float((y * dy.double()).sum() + (x * dtotal.double()).sum())

    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ew.ew_rmsnorm_grad_f32(dy, x, w, rstd, dx, dw, grad_space(rows, cols), dtotal=dtotal)
    x, w, v, u, h = x.double(), w.double(), v.double(), u.double(), 1e-5
    # third derivatives times h^2 are ~1e-10 of the slopes, whose terms sum to ~30
    assert abs((loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h) - float((dx * v).sum())) < 1e-3
    assert abs((loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h) - float((dw * u).sum())) < 1e-3


# ---------------------------------------------------------------------------
# Log probabilities
# ---------------------------------------------------------------------------

def logits_of(t, rows, cols, pad, off, seed, masked=0.0):
    g = gen(seed)
    x = 3 * randn(g, rows, cols)
    hot = torch.randint(cols, (rows, 3), generator=g, device=DEV)
    x.scatter_(1, hot, 9 + 2 * randn(g, rows, 3))
    if masked:
        x.masked_fill_(torch.rand(rows, cols, generator=g, device=DEV) < masked, -math.inf)
    targets = hot[:, 0].clone()
    targets[::5] = -100
    targets[3::7] = cols                                     # outside as well
    targets[2::6] = torch.randint(cols, targets[2::6].shape, generator=g, device=DEV)
    return matrix(rows, cols, TYPES[t], pad, off, x)[0], targets


def run_logprobs(t, x, targets, top, scale, entropy=True, lse=True):
    rows, cols = x.shape
    out = {"logp": torch.full((rows + 1,), GUARD, device=DEV),
           "entropy": torch.full((rows + 1,), GUARD, device=DEV) if entropy else None,
           "lse": torch.full((rows + 1,), GUARD, device=DEV) if lse else None,
           "top_logp": torch.full((rows + 1, top), GUARD, device=DEV),
           "top_ids": torch.full((rows + 1, top), -7, dtype=torch.int64, device=DEV)}
    ws = torch.full((ew.ew_logprobs_workspace(rows, cols, top) + 16,), 0xff, dtype=torch.uint8,
                    device=DEV)
    body = {k: v[:rows] if v is not None else None for k, v in out.items()}
    getattr(ew, "ew_logprobs_" + t)(x, targets, body["logp"], entropy=body["entropy"],
                                    lse=body["lse"], top_logp=body["top_logp"],
                                    top_ids=body["top_ids"], scale=scale, workspace=ws)
    for k, v in out.items():
        if v is not None:
            assert bool((v[rows:] == (-7 if k == "top_ids" else GUARD)).all()), k
    assert bool((ws[-16:] == 0xff).all())
    return body


def check_logprobs(t, x, targets, top, scale, **options):
    got = run_logprobs(t, x, targets, top, scale, **options)
    want = ref.logprobs(x, targets, scale)
    if got["lse"] is not None:
        close(got["lse"], want.lse, want.lse_tol, "lse")
    if got["entropy"] is not None:
        close(got["entropy"], want.entropy, want.entropy_tol, "entropy")
    close(got["logp"], want.target_logp, want.target_tol, "logp")
    if top:
        assert torch.equal(got["top_ids"], want.top(top))
        v, tol = want.logp(got["top_ids"])
        close(got["top_logp"], v, tol, "top_logp")
    return got


VOCAB_COLS = (1, 2, 3, 7, 8, 15, 16, 17, 63, 64, 65, 100, 255, 257, 511, 1000, 1024, 2047, 4096, 5003,
              8191, 16384, 32001, 50257, 131072, 151936)


@every_type
@pytest.mark.parametrize("cols", VOCAB_COLS)
def test_logprobs_columns(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows = (1, 3, 8, 5, 17)[k]
        top = min(cols, (20, 0, 5, 64, 1)[k])
        x, targets = logits_of(t, rows, cols, pad, off, 1000 + cols + k, (0, 0, 0.875, 0, 0.3)[k])
        check_logprobs(t, x, targets, top, (1.0, 1.25, 0.5, 1.0, 2.0)[k])


@every_type
@pytest.mark.parametrize("rows,cols,top", [(300, 5000, 5), (1500, 1000, 20), (2100, 257, 3),
                                           (700, 32001, 0), (129, 9001, 64), (1030, 8192, 10)])
def test_logprobs_many_rows(t, rows, cols, top):
    x, targets = logits_of(t, rows, cols, 1, 0, rows + cols)
    a = check_logprobs(t, x, targets, top, 1.0)
    b = run_logprobs(t, x, targets, top, 1.0)
    assert all(torch.equal(a[k], b[k]) for k in a)          # the same bits


@every_type
@pytest.mark.parametrize("rows,cols", [(2, 131072), (2, 5003), (600, 9000), (9, 65)])
def test_logprobs_order_and_ties(t, rows, cols):
    """Rising, falling, constant and few-valued rows: the ranking must not
    depend on where the large logits lie; ties go to the lowest column."""
    n = torch.arange(cols, device=DEV, dtype=torch.float32)
    kinds = [n / cols * 8 - 4, 4 - n / cols * 8, torch.zeros_like(n), (n * 7919 % 5) - 2,
             torch.where(n < cols - 3, -1.0, 1.0), (n % 2) * 0.0 - 0.0 * (n % 3)]
    kinds[5][::3] = -0.0                                    # -0 and +0 tie
    g = gen(5)
    for x in kinds:
        x = x.expand(rows, cols).to(TYPES[t]).contiguous()
        targets = torch.randint(cols, (rows,), generator=g, device=DEV)
        for top in (1, 20, 64):
            check_logprobs(t, x, targets, min(top, cols), 1.0)


@every_type
@pytest.mark.parametrize("rows,cols", [(8, 70), (8, 3000), (8, 60000), (1200, 4000)])
def test_logprobs_masks(t, rows, cols):
    """Rows whose mask leaves nothing, one or a few columns, in every place,
    with -inf and with the type's lowest value; a target that is masked."""
    x, targets = logits_of(t, rows, cols, 0, 0, 77)
    low = torch.finfo(TYPES[t]).min
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, cols - 1] = 2.0
    x[2, :] = -math.inf
    x[2, 0] = -3.0
    x[3, 1:cols - 1] = -math.inf
    x[4] = low
    x[5, ::2] = low
    x[6, 5:] = low
    x[7, targets[7].clamp(0, cols - 1)] = -math.inf
    targets[:4] = torch.tensor([1, cols - 1, cols - 1, 0], device=DEV)
    for scale in (1.0, 0.75, 1.25):
        got = check_logprobs(t, x, targets, min(20, cols), scale)
        assert float(got["lse"][0]) == -math.inf and float(got["entropy"][0]) == 0.0
        assert float(got["logp"][0]) == -math.inf
        assert float(got["logp"][1]) == 0.0 and float(got["logp"][2]) == -math.inf


@every_type
@pytest.mark.parametrize("cols", (70, 3000, 60000))
def test_logprobs_nan_and_infinities(t, cols):
    rows, top = 6, 20
    x, targets = logits_of(t, rows, cols, 0, 0, 78, 0.5)
    targets[:] = torch.arange(rows, device=DEV)
    targets[5] = -1
    x[0, cols // 2] = math.nan
    x[1, 3] = math.inf
    x[2] = math.nan
    x[3, cols - 1] = math.nan
    x[3, 0] = math.inf
    x[5, 2] = math.nan
    got = run_logprobs(t, x, targets, top, 1.0)
    for r in (0, 1, 2, 3, 5):
        for k in ("lse", "entropy", "top_logp"):
            assert bool(torch.isnan(got[k][r]).all()), (k, r)
        assert r == 5 or math.isnan(float(got["logp"][r]))
    assert float(got["logp"][5]) == 0.0                     # no target
    assert torch.equal(got["top_ids"], ref.Rows(x, 1.0).top(top))
    want = ref.logprobs(x[4:5], targets[4:5], 1.0)
    close(got["lse"][4:5], want.lse, want.lse_tol, "lse beside such rows")


@every_type
def test_logprobs_without_options_and_without_columns(t):
    x, targets = logits_of(t, 5, 1000, 0, 0, 79)
    check_logprobs(t, x, targets, 0, 1.0, entropy=False, lse=False)
    check_logprobs(t, x, targets, 3, 1.0, entropy=False)
    none = torch.empty(3, 0, dtype=TYPES[t], device=DEV)
    got = run_logprobs(t, none, torch.tensor([0, -1, 5], device=DEV), 0, 1.0)
    assert got["logp"].tolist() == [0, 0, 0] and got["entropy"].tolist() == [0, 0, 0]
    assert got["lse"].tolist() == [-math.inf] * 3


@every_type
@pytest.mark.parametrize("cols", (1, 2, 7, 8, 9, 64, 65, 1000, 4097, 8192, 16385, 50257, 131072))
def test_logprobs_grad(t, cols):
    for k, (pad, off) in enumerate(LAYOUTS):
        rows, scale = (1, 3, 8, 40, 17)[k], (1.0, 1.25, 0.5, 1.0, 2.0)[k]
        x, targets = logits_of(t, rows, cols, pad, off, 2000 + cols + k, (0, 0.3, 0.875, 0, 0)[k])
        x[rows - 1] = -math.inf
        rows_ = ref.logprobs(x, targets, scale)
        lse, ent = rows_.lse.float(), rows_.entropy.float()
        g = gen(k)
        dlogp, dent = randn(g, rows), 0.1 * randn(g, rows)
        for entropy in (False, True):
            dx, dxa = matrix(rows, cols, TYPES[t], pad, off)
            more = {"entropy": ent, "dentropy": dent} if entropy else {}
            fn = getattr(ew, "ew_logprobs_grad_" + t)
            fn(x, targets, lse, dlogp, dx, scale=scale, **more)
            want, tol = ref.logprobs_grad(x, targets, lse, dlogp, scale, **more)
            dt = TYPES[t]
            tol = tol + (want.abs() + tol) * ref.half_ulp(dt) + ref.tiny(dt)
            close(dx, want, tol, "dlogits")
            guards_kept(dx, dxa)
        y = x.clone()
        fn(y, targets, lse, dlogp, y, scale=scale, **more)              # in place
        close(y, want, tol, "dlogits in place")


@every_type
def test_logprobs_grad_masks_and_nan(t):
    rows, cols = 5, 3000
    x, targets = logits_of(t, rows, cols, 0, 0, 80)
    x[0] = torch.finfo(TYPES[t]).min
    x[1, 100:] = torch.finfo(TYPES[t]).min
    x[2, 4] = math.nan
    x[3, targets[3].clamp(0, cols - 1)] = -math.inf
    targets[2:4] = 7
    x[3, 7] = -math.inf
    got = run_logprobs(t, x, targets, 0, 0.9)
    dlogp, dent = torch.ones(rows, device=DEV), torch.full((rows,), 0.1, device=DEV)
    dx = torch.empty_like(x)
    getattr(ew, "ew_logprobs_grad_" + t)(x, targets, got["lse"], dlogp, dx, entropy=got["entropy"],
                                         dentropy=dent, scale=0.9)
    assert bool(torch.isfinite(dx[[0, 1, 3, 4]].float()).all())
    assert bool(torch.isnan(dx[2].float()).all())
    assert float(dx[3, 7]) == 0.0


def test_logprobs_grad_against_differences():
    rows, cols, scale = 4, 90, 1.25
    g = gen(4)
    x, v = randn(g, rows, cols), randn(g, rows, cols).double()
    targets = torch.tensor([3, 89, -100, 0], device=DEV)
    dlogp, dent = randn(g, rows), randn(g, rows)
    got = run_logprobs("f32", x, targets, 0, scale)
    dx = torch.empty_like(x)
    ew.ew_logprobs_grad_f32(x, targets, got["lse"], dlogp, dx, entropy=got["entropy"],
                            dentropy=dent, scale=scale)

    def loss(x):
        logq = torch.log_softmax(x * scale, 1)
        lp = logq.gather(1, targets.clamp_min(0)[:, None])[:, 0] * (targets >= 0)
        h = -(logq.exp() * logq).sum(1)
        return float((lp * dlogp.double() + h * dent.double()).sum())

    h, xd = 1e-5, x.double()
    assert abs((loss(xd + h * v) - loss(xd - h * v)) / (2 * h) - float((dx * v).sum())) < 1e-3


# ---------------------------------------------------------------------------
# Distillation
# ---------------------------------------------------------------------------

def teacher_of(rows, cols, kept, seed):
    g = gen(seed)
    ids = torch.randint(cols, (rows, kept), generator=g, device=DEV)
    z = 6 + 3 * randn(g, rows, kept)
    ids[1::4, kept // 2:] = -1                                # fewer kept
    ids[2::5] = cols                                          # none kept
    z[3::5, :1] = -math.inf                                   # a masked teacher logit
    if kept > 2:
        ids[:, 1] = ids[:, 0]                                 # a column named twice
    return z, ids


def run_distill(t, x, z, ids, scale, lse=True):
    rows, cols = x.shape
    loss = torch.full((rows + 1,), GUARD, device=DEV)
    out = torch.full((rows + 1,), GUARD, device=DEV)
    ws = torch.full((ew.ew_distill_workspace(rows, cols) + 16,), 0xff, dtype=torch.uint8, device=DEV)
    getattr(ew, "ew_distill_" + t)(x, z, ids, loss[:rows], lse=out[:rows] if lse else None,
                                   scale=scale, workspace=ws)
    assert float(loss[rows]) == GUARD and float(out[rows]) == GUARD
    assert bool((ws[-16:] == 0xff).all())
    return loss[:rows], out[:rows]


@every_type
@pytest.mark.parametrize("cols", (1, 2, 7, 9, 64, 65, 1000, 4097, 16385, 32001, 131072))
@pytest.mark.parametrize("kept", (1, 10, 64, 100, 700))
def test_distill_and_its_gradient(t, cols, kept):
    for k, (pad, off) in enumerate(LAYOUTS[::2]):
        rows, scale = (7, 1, 21)[k], (0.5, 1.0, 0.3)[k]
        x, _ = logits_of(t, rows, cols, pad, off, 3000 + cols + k)
        z, ids = teacher_of(rows, cols, kept, 4000 + cols + kept + k)
        loss, lse = run_distill(t, x, z, ids, scale)
        want, tol, rows_ = ref.distill(x, z, ids, scale)
        close(loss, want, tol, "loss")
        close(lse, rows_.lse, rows_.lse_tol, "lse")
        dloss = torch.rand(rows, generator=gen(k), device=DEV)
        dx, dxa = matrix(rows, cols, TYPES[t], pad, off)
        fn, dt = getattr(ew, "ew_distill_grad_" + t), TYPES[t]
        fn(x, z, ids, lse, dloss, dx, scale=scale)
        want, tol = ref.distill_grad(x, z, ids, lse, dloss, scale)
        tol = tol + (want.abs() + tol) * ref.half_ulp(dt) + ref.tiny(dt)
        close(dx, want, tol, "dlogits")
        guards_kept(dx, dxa)
        y = x.clone()
        fn(y, z, ids, lse, dloss, y, scale=scale)             # in place
        close(y, want, tol, "dlogits in place")


@every_type
@pytest.mark.parametrize("rows,cols", [(1300, 2000), (2100, 513), (520, 20001)])
def test_distill_many_rows(t, rows, cols):
    x, _ = logits_of(t, rows, cols, 0, 0, 81)
    z, ids = teacher_of(rows, cols, 20, 82)
    loss, lse = run_distill(t, x, z, ids, 0.5)
    want, tol, rows_ = ref.distill(x, z, ids, 0.5)
    close(loss, want, tol, "loss")
    close(lse, rows_.lse, rows_.lse_tol, "lse")
    again, _ = run_distill(t, x, z, ids, 0.5, lse=False)
    assert torch.equal(loss, again)


@every_type
@pytest.mark.parametrize("cols", (70, 3000, 40000))
def test_distill_masks(t, cols):
    rows, kept = 6, 12
    x, _ = logits_of(t, rows, cols, 0, 0, 83)
    z, ids = teacher_of(rows, cols, kept, 84)
    ids.copy_(torch.arange(kept, device=DEV) * 5)
    z.clamp_(-50, 50)
    x[0] = -math.inf                       # a student that allows nothing
    x[1, 10] = -math.inf                   # and one that forbids a kept column
    ids[2] = -1                            # nothing kept, a student that allows nothing
    x[2] = -math.inf
    z[3] = -math.inf                       # a teacher that allows nothing
    x[4, cols // 2] = math.nan
    z[5, 0] = 200.0
    z[5, 1:] = -200.0                      # one certain entry: the others' t is 0
    x[5, 5] = -math.inf                    # among them a forbidden column
    loss, lse = run_distill(t, x, z, ids, 1.0)
    assert loss[:2].tolist() == [math.inf, math.inf]
    assert loss[2:4].tolist() == [0.0, 0.0]
    assert math.isnan(float(loss[4])) and math.isfinite(float(loss[5]))
    want, tol, _ = ref.distill(x[5:], z[5:], ids[5:], 1.0)
    close(loss[5:], want, tol, "loss")
    dx, dloss = torch.full_like(x, GUARD), torch.ones(rows, device=DEV)
    getattr(ew, "ew_distill_grad_" + t)(x, z, ids, lse, dloss, dx)
    assert bool((dx[[0, 2, 3]] == 0).all()) and float(dx[1, 10]) == 0.0
    want, tol = ref.distill_grad(x, z, ids, lse, dloss, 1.0)
    dt = TYPES[t]
    tol = tol + (want.abs() + tol) * ref.half_ulp(dt) + ref.tiny(dt)
    keep = [0, 1, 2, 3, 5]
    close(dx[keep], want[keep], tol[keep], "dlogits")
    # no entries at all
    loss, _ = run_distill(t, x[5:], z[5:, :0], ids[5:, :0], 1.0)
    assert loss.tolist() == [0.0]
    none = torch.empty(2, 0, dtype=dt, device=DEV)
    loss, lse = run_distill(t, none, z[:2], ids[:2], 1.0)
    assert loss.tolist() == [0.0, 0.0] and lse.tolist() == [-math.inf] * 2


def test_distill_grad_against_differences():
    rows, cols, kept, scale = 3, 80, 9, 0.5
    g = gen(6)
    x, v = randn(g, rows, cols), randn(g, rows, cols).double()
    ids = torch.randperm(cols, generator=g, device=DEV)[:kept].expand(rows, kept).contiguous()
    z, dloss = 3 * randn(g, rows, kept), randn(g, rows)
    _, lse = run_distill("f32", x, z, ids, scale)
    dx = torch.empty_like(x)
    ew.ew_distill_grad_f32(x, z, ids, lse, dloss, dx, scale=scale)

    def loss(x):
        t = torch.softmax(z.double() * scale, 1)
        logq = torch.log_softmax(x * scale, 1).gather(1, ids)
        return float(((t * (t.log() - logq)).sum(1) * dloss.double()).sum())

    h, xd = 1e-5, x.double()
    assert abs((loss(xd + h * v) - loss(xd - h * v)) / (2 * h) - float((dx * v).sum())) < 1e-3


# ---------------------------------------------------------------------------
# Streams, graphs, large offsets
# ---------------------------------------------------------------------------

def test_calls_follow_the_current_stream():
    x, res, w = norm_inputs("bf16", 64, 4096, 0, 0, 90)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(4):
            big = big @ big * 0.01
        h = x + 0                                   # ready only on the side stream
        ew.ew_rmsnorm_bf16(h, w, y, residual=res)
    side.synchronize()
    check_norm("bf16", x, res, w, y, None, None, 1e-5)


def test_a_graph_of_every_operator_replays():
    """One capture of a training step's calls, replayed on changing inputs
    with eager work between, against eager calls."""
    rows, cols, vocab, kept = 24, 512, 33000, 8
    x, res, w = norm_inputs("bf16", rows, cols, 0, 0, 91)
    logits, targets = logits_of("bf16", rows, vocab, 0, 0, 92)
    z, ids = teacher_of(rows, vocab, kept, 93)
    one = torch.ones(rows, device=DEV)

    def outputs():
        f = dict(device=DEV)
        return {"y": torch.zeros_like(x), "total": torch.zeros_like(x),
                "rstd": torch.zeros(rows, **f), "logp": torch.zeros(rows, **f),
                "q": torch.zeros(rows, cols, dtype=torch.uint8, **f),
                "scales": torch.zeros(rows, 4, **f),
                "entropy": torch.zeros(rows, **f), "lse": torch.zeros(rows, **f),
                "top_logp": torch.zeros(rows, 5, **f),
                "top_ids": torch.zeros(rows, 5, dtype=torch.int64, **f),
                "dlogits": torch.zeros_like(logits), "loss": torch.zeros(rows, **f),
                "lse2": torch.zeros(rows, **f), "ddistill": torch.zeros_like(logits),
                "dx": torch.zeros_like(x), "dw": torch.zeros(cols, **f)}

    ws = torch.empty(max(ew.ew_logprobs_workspace(rows, vocab, 5), ew.ew_distill_workspace(rows, vocab),
                         ew.ew_rmsnorm_grad_workspace(rows, cols)), dtype=torch.uint8, device=DEV)

    def step(o):
        ew.ew_rmsnorm_bf16(x, w, o["y"], residual=res, total=o["total"], rstd=o["rstd"])
        ew.ew_rmsnorm_e4m3_bf16(x, w, o["q"], o["scales"], residual=res)
        ew.ew_logprobs_bf16(logits, targets, o["logp"], entropy=o["entropy"], lse=o["lse"],
                            top_logp=o["top_logp"], top_ids=o["top_ids"], workspace=ws)
        ew.ew_logprobs_grad_bf16(logits, targets, o["lse"], one, o["dlogits"], entropy=o["entropy"],
                                 dentropy=one)
        ew.ew_distill_bf16(logits, z, ids, o["loss"], lse=o["lse2"], workspace=ws)
        ew.ew_distill_grad_bf16(logits, z, ids, o["lse2"], one, o["ddistill"])
        ew.ew_rmsnorm_grad_bf16(o["y"], o["total"], w, o["rstd"], o["dx"], o["dw"], ws)

    got, want = outputs(), outputs()
    step(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got)
    for k in range(4):
        x.copy_(randn(gen(k), rows, cols))
        logits.copy_(randn(gen(10 + k), rows, vocab))
        step(want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)


def test_offsets_past_32_bits():
    """The last rows of matrices of more than 2^32 elements."""
    rows, cols = 33000, 131080                     # 4.3e9 elements, 8.7 GB in bf16
    whole = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x = whole[:, :131072]
    tail = 3
    data, targets = logits_of("bf16", tail, 131072, 0, 0, 94)
    whole.zero_()
    x[-tail:].copy_(data)
    t = torch.zeros(rows, dtype=torch.int64, device=DEV)
    t[-tail:] = targets
    got = run_logprobs("bf16", x, t, 3, 1.0)
    want = ref.logprobs(data, targets, 1.0)
    close(got["lse"][-tail:], want.lse, want.lse_tol, "lse")
    close(got["logp"][-tail:], want.target_logp, want.target_tol, "logp")
    assert torch.equal(got["top_ids"][-tail:], want.top(3))
    assert bool((got["top_ids"][:-tail] == torch.arange(3, device=DEV)).all())
    dlogp = torch.ones(rows, device=DEV)
    ew.ew_logprobs_grad_bf16(x, t, got["lse"], dlogp, x)
    g, tol = ref.logprobs_grad(data, targets, got["lse"][-tail:], dlogp[-tail:], 1.0)
    close(x[-tail:], g, tol + (g.abs() + tol) * 2.0 ** -8 + ref.tiny(torch.bfloat16), "dlogits")


def test_norm_offsets_past_32_bits():
    """The last rows of matrices of more than 2^32 elements, and dweight, to
    which only they contribute."""
    rows, cols, tail = 263000, 16400, 3            # 4.3e9 elements, 8.6 GB in bf16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(x)
    data, res, w = norm_inputs("bf16", tail, cols, 0, 0, 95)
    x[-tail:].copy_(data)
    rstd = torch.empty(rows, device=DEV)
    ew.ew_rmsnorm_bf16(x, w, y, rstd=rstd)
    check_norm("bf16", x[-tail:], None, w, y[-tail:], None, rstd[-tail:], 1e-5)
    assert bool((y[:-tail].view(torch.int16) == 0).all())
    y[-tail:].copy_(res)                           # as dy
    dw = torch.empty(cols, device=DEV)
    ew.ew_rmsnorm_grad_bf16(y, x, w, rstd, y, dw, grad_space(rows, cols))
    want, want_w, tol, tol_w = ref.norm_grad(res, data, w, rstd[-tail:], None)
    close(y[-tail:], want, tol + (want.abs() + tol) * 2.0 ** -8 + ref.tiny(torch.bfloat16), "dx")
    close(dw, want_w, tol_w, "dweight")            # every other row adds an exact 0
