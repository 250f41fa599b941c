"""The row operators in 64 bits, from their definitions, and how far a
binary32 computation may be from them.

Every bound counts roundings: u = 2^-24 is one binary32 rounding, a type's
own rounding is half its eps.  A sum of n terms in any order of at most `adds`
additions a term is off by at most adds * u times the sum of magnitudes; ADDS
is what the kernels stay under (a lane adds up at most cols / 64 terms, then a
tree joins the lanes, waves and blocks).  Where masked logits or dropped
entries make a term infinite it is left out of the sum, as the definition
says.
"""
import math

import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -126


def adds(cols):
    return cols / 64 + 24


def half_ulp(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the spacing of a type's subnormals."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def close(got, ref, tol, what):
    """Every element of got within tol of ref; infinities and NaNs in the same places."""
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaNs differ"
    odd = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[odd], ref[odd]), f"{what}: infinities differ"
    off = torch.where(fine, (got - ref).abs(), 0.0)
    bad = off > torch.where(fine, tol, 1.0)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()!r} instead of {ref[i].item()!r}, "
                             f"tolerance {tol[i].item():.3e}")


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

def norm_total(x, residual):
    """round(x + residual): the binary32 sum rounded to the type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(total, weight, eps):
    """(y, rstd, tolerance of y before its rounding, tolerance of rstd)."""
    h, w = total.double(), weight.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    y = h * rstd[:, None] * w
    rel = (adds(total.shape[1]) / 2 + 5) * U
    return y, rstd, y.abs() * (rel + 2 * U), rstd * rel


def group_scales(y, group):
    r, c = y.shape
    size = group or c
    groups = -(-c // size)
    a = torch.zeros(r, groups * size, dtype=y.dtype, device=y.device)
    a[:, :c] = y.abs()
    scales = (a.view(r, groups, size).amax(2) / E4M3_MAX).clamp_min(SCALE_MIN)
    return scales, scales.repeat_interleave(size, 1)[:, :c]


def norm_grad(dy, x, weight, rstd, dtotal):
    """(dx, dweight, tolerances before dx's rounding and of dweight)."""
    n = x.shape[1]
    dy, h, w, r = dy.double(), x.double(), weight.double(), rstd.double()[:, None]
    wdy = dy * w
    dot, mag = (h * wdy).sum(1, keepdim=True), (h * wdy).abs().sum(1, keepdim=True)
    first, second = r * wdy, h * (dot * r ** 3 / n)
    dx = first - second
    tol = 4 * first.abs() + (h * r ** 3 / n).abs() * mag * (adds(n) + 10)
    if dtotal is not None:
        dx = dx + dtotal.double()
        tol = tol + 2 * dtotal.double().abs()
    terms = dy * h * r
    return (dx, terms.sum(0), (tol + 3 * dx.abs()) * U,
            terms.abs().sum(0) * (x.shape[0] + 4) * U)


# ---------------------------------------------------------------------------
# Logits
# ---------------------------------------------------------------------------

class Rows:
    """Softmax statistics of scale * logits in 64 bits, with their tolerances."""

    def __init__(self, logits, scale):
        self.x, self.scale, self.cols = logits.double(), scale, logits.shape[1]
        # a product beyond binary32 is an infinity there
        s = self.x * scale
        s = torch.where(s.abs() > torch.finfo(torch.float32).max * (1 + U), s.sign() * math.inf, s)
        self.s = s
        r = s.shape[0]
        top = s.amax(1) if self.cols else s.new_full((r,), -math.inf)
        self.empty = top == -math.inf
        self.nan = torch.isnan(self.x).any(1) | (top == math.inf)
        base = torch.where(self.empty | self.nan, 0.0, top)
        d = s - base[:, None]
        e = torch.where(d > -math.inf, d.exp(), 0.0)
        z = e.sum(1)
        log_z = z.log()
        self.lse = torch.where(self.nan, math.nan, torch.where(self.empty, -math.inf, base + log_z))
        self.p = e / z[:, None]
        far = torch.where(e > 0, d.abs(), 0.0)
        mean_far = (self.p * far).nan_to_num().sum(1)
        self.entropy = torch.where(self.nan, math.nan, torch.where(
            self.empty, 0.0, log_z + mean_far))
        self.base, self.log_z = base, log_z
        # z: each term's exponent is rounded four times at its size
        z_rel = 4 * mean_far + adds(self.cols)
        self.z_tol = z_rel * U
        self.lse_tol = (z_rel + 2 * base.abs() + 4 * log_z.abs() + 2 * self.lse.abs()) * U
        square = (self.p * far * far).nan_to_num().sum(1)
        self.entropy_tol = (z_rel * (1 + mean_far) + 4 * log_z.abs() + 4 * square
                            + mean_far * adds(self.cols) + 2 * self.entropy.abs() + 4) * U

    def logp(self, cols):
        """log probability at (rows, k) columns, and its tolerance."""
        d = self.s.gather(1, cols) - self.base[:, None]
        got = d - self.log_z[:, None]
        got = torch.where(self.empty[:, None], -math.inf, got)
        got = torch.where(self.nan[:, None], math.nan, got)
        tol = self.z_tol[:, None] + (4 * d.abs() + 4 * self.log_z.abs()[:, None]
                                     + 2 * got.abs()) * U
        return got, tol

    def top(self, k):
        """The k best columns: a NaN counts as -inf, ties to the lowest column."""
        x = torch.where(torch.isnan(self.x), -math.inf, self.x)
        return torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]


def logprobs(logits, targets, scale):
    """Rows, with .target_logp and .target_tol."""
    rows = Rows(logits, scale)
    given = (targets >= 0) & (targets < rows.cols)
    if rows.cols:
        v, tol = rows.logp(targets.clamp(0, rows.cols - 1)[:, None])
        rows.target_logp = torch.where(given, v[:, 0], 0.0)
        rows.target_tol = tol[:, 0]
    else:
        rows.target_logp = torch.zeros_like(rows.lse)
        rows.target_tol = torch.zeros_like(rows.lse)
    return rows


def logprobs_grad(logits, targets, lse, dlogp, scale, entropy=None, dentropy=None):
    """(dlogits, tolerance before its rounding), from lse and entropy as given."""
    x, n = logits.double(), logits.shape[1]
    s = (logits.float() * scale).double()          # masked where binary32 says -inf
    live = (s > -math.inf) | torch.isnan(s)
    live &= (lse != -math.inf)[:, None]
    log_p = torch.where(live, x * scale - lse.double()[:, None], 0.0).clamp_max(0.0)
    p = torch.where(live, log_p.exp(), 0.0)
    given = (targets >= 0) & (targets < n)
    dl = torch.where(given, dlogp.double(), 0.0)[:, None]
    hot = torch.zeros_like(p).scatter_(1, targets.clamp(0, n - 1)[:, None], 1.0)
    g = dl * (hot - p)
    mag = dl.abs() * (p * (3 * log_p.abs() + 8) + 4 * hot)
    if dentropy is not None:
        de, h = dentropy.double()[:, None], entropy.double()[:, None]
        g = g - de * p * (log_p + h)
        mag = mag + de.abs() * p * (log_p.abs() + h.abs()) * (3 * log_p.abs() + 12)
    return (torch.where(live, scale * g, 0.0), torch.where(live, scale * mag, 0.0) * U)


class Teacher:
    """The teacher's distribution over its kept entries."""

    def __init__(self, teacher, ids, cols, scale):
        z = teacher.double() * scale
        self.kept = (ids >= 0) & (ids < cols) & ~(z == -math.inf)
        z = torch.where(self.kept, z, -math.inf)
        top = z.amax(1, keepdim=True) if z.shape[1] else z.new_full((z.shape[0], 1), -math.inf)
        self.some = top > -math.inf
        base = torch.where(self.some, top, 0.0)
        d = z - base
        e = torch.where(self.kept, d.exp(), 0.0)
        total = torch.where(self.some, e.sum(1, keepdim=True), 1.0)
        self.p = e / total
        self.log_p = torch.where(self.kept, d - total.log(), 0.0)
        self.at = ids.clamp(0, max(cols - 1, 0))
        # of p, relative: its exponent, the sum, the division
        self.rel = torch.where(self.kept, (4 * d.abs() + z.shape[1] + 12) * U, 0.0)


def distill(logits, teacher, ids, scale):
    """(loss, tolerance, Rows)."""
    rows = Rows(logits, scale)
    t = Teacher(teacher, ids, rows.cols, scale)
    if not rows.cols or not teacher.shape[1]:
        zero = rows.lse.new_zeros(rows.lse.shape)
        return zero, zero, rows
    log_q, q_tol = rows.logp(t.at)
    live = t.p >= torch.finfo(torch.float32).smallest_normal      # below it t is 0
    term = torch.where(live, t.p * (t.log_p - log_q), 0.0)
    size = torch.where(live & torch.isfinite(log_q), t.log_p.abs() + log_q.abs() + 1, 0.0)
    tol = t.p * (size * (t.rel + 6 * U) + torch.where(torch.isfinite(q_tol), q_tol, 0.0))
    tol = tol.sum(1) + term.abs().nan_to_num(posinf=0.0).sum(1) * (teacher.shape[1] + 8) * U
    return term.sum(1), tol, rows


def distill_grad(logits, teacher, ids, lse, dloss, scale):
    """(dlogits, tolerance before its rounding), from lse as given."""
    x, n = logits.double(), logits.shape[1]
    t = Teacher(teacher, ids, n, scale)
    s = (logits.float() * scale).double()
    live = (s > -math.inf) | torch.isnan(s)
    live &= (lse != -math.inf)[:, None] & t.some
    log_p = torch.where(live, x * scale - lse.double()[:, None], 0.0).clamp_max(0.0)
    p = torch.where(live, log_p.exp(), 0.0)
    weight, slack = torch.zeros_like(p), torch.zeros_like(p)
    weight.scatter_add_(1, t.at, torch.where(t.kept, t.p, 0.0))
    slack.scatter_add_(1, t.at, torch.where(t.kept, t.p * (t.rel + 4 * U), 0.0))
    g = dloss.double()[:, None] * scale
    tol = g.abs() * (p * (3 * log_p.abs() + 8) * U + slack + 4 * U * weight)
    return torch.where(live, g * (p - weight), 0.0), torch.where(live, tol, 0.0)
