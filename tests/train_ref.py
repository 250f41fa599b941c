"""Layer norm, policy loss and the movement of rows to experts in 64 bits, from
their definitions, and how far a binary32 computation may be from them.

Bounds count roundings as in tests/rows_ref.py: U = 2^-24 is one binary32
rounding, adds(cols) the longest chain of additions over a row.
"""
import math

import torch

from tests.rows_ref import U, adds, half_ulp, tiny


def rounded(want, tol, dt):
    """Tolerance of a value that is off by tol before its rounding to dt."""
    if dt is torch.float32:
        return tol + want.abs() * U + tiny(dt)
    return tol + (want.abs() + tol) * half_ulp(dt) + tiny(dt)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def norm_adds(cols):
    """The longest chain of additions of a row's sums: 32 elements a lane and
    the joins, or a long row's 1024th part of it."""
    return 48 + cols / 1024


def layernorm(total, weight, bias, eps):
    """(y, mean, rstd, tolerances of y before its rounding, of mean, of rstd).

    The mean is that of numbers near the row's parts (exact) and of the
    differences from them: their sum is off by its additions, at most twice
    the mean difference in size.  d = (h - hi) - lo is off by two roundings, by
    that of lo (U^2 of the mean), and with the mean; the sum of squares by
    four roundings a term, its additions and four of the join; rstd by half of
    that, the mean's division, eps's addition, the root and the division."""
    h = total.double()
    n = h.shape[1]
    one = torch.ones(n, dtype=torch.float64, device=h.device)
    w = one if weight is None else weight.double()
    b = 0 * one if bias is None else bias.double()
    mean = h.sum(1) / n
    d = h - mean[:, None]
    var = d.square().sum(1) / n
    rstd = (var + eps).rsqrt()
    y = d * rstd[:, None] * w + b
    off = 2 * (norm_adds(n) + 3) * d.abs().mean(1) * U
    lost = U * U * mean.abs() + off
    rel = ((norm_adds(n) + 12) / 2 + 3) * U + (lost * var.sqrt() / (var + eps)).nan_to_num()
    tol_mean = mean.abs() * U + off + h.abs().mean(1) * n * 2.0 ** -52 + 2.0 ** -149
    tol = (d * rstd[:, None] * w).abs() * (rel[:, None] + 4 * U) + y.abs() * U
    tol = tol + (w.abs() * (lost * rstd)[:, None])
    return y, mean, rstd, tol, tol_mean, rstd * rel


def layernorm_grad(dy, x, weight, mean, rstd, dtotal):
    """(dx, dweight, dbias, tolerances: dx before its rounding, the sums)."""
    n = x.shape[1]
    dy, r = dy.double(), rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * r
    g = dy if weight is None else dy * weight.double()
    first, second = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = r * (g - first - h * second)
    off_first = g.abs().mean(1, keepdim=True) * (adds(n) + 3)
    off_second = (g * h).abs().mean(1, keepdim=True) * (adds(n) + 6)
    tol = r * (4 * g.abs() + 4 * first.abs() + off_first + 6 * (h * second).abs()
               + h.abs() * off_second)
    if dtotal is not None:
        dx = dx + dtotal.double()
        tol = tol + 2 * dtotal.double().abs()
    rows = x.shape[0] + 6
    return (dx, (dy * h).sum(0), dy.sum(0), (tol + 3 * dx.abs()) * U,
            (dy * h).abs().sum(0) * rows * U, dy.abs().sum(0) * rows * U)


# ---------------------------------------------------------------------------
# Policy loss
# ---------------------------------------------------------------------------

def f32(x):
    """x as binary32 holds it."""
    return float(torch.tensor(x, dtype=torch.float32))


class Policy:
    """The loss of counted tokens by its definition.  advantage: a value a
    token, or a column of one a sequence."""

    def __init__(self, logp, old, advantage, ref=None, mask=None, low=0.2, high=0.2, kl=0.0,
                 mean="tokens", scale=1.0):
        low, high, kl, scale = f32(low), f32(high), f32(kl), f32(scale)
        live = torch.ones_like(logp, dtype=torch.bool) if mask is None else mask != 0
        zero = torch.zeros_like(logp, dtype=torch.float64)
        pick = lambda v: torch.where(live, v.double().expand_as(zero), zero)   # noqa: E731
        logp, old, a = pick(logp), pick(old), pick(advantage)
        x = logp - old
        r = x.exp()
        inner = r.clamp(1.0 - low, 1.0 + high) * a
        clipped = live & (r * a > inner)
        gain = torch.where(clipped, inner, r * a)       # the lesser of the two
        self.live, self.clipped = live, clipped
        k = one = torch.zeros_like(gain)
        tol_k = tol_one = torch.zeros_like(gain)
        if ref is not None:
            d = pick(ref) - logp
            one, near = d.expm1(), d.abs() < 1
            k = torch.where(near, self._line(d), one - d)
            k = torch.where(d == math.inf, d, k)
            # d, its square, the series (its sum at least three quarters of
            # its largest term's half): ten roundings; beyond 1 the exp's
            # exponent is rounded twice at its size
            wide = d.exp() * (2 * d.abs() + 4)
            tol_k = torch.where(near, 10 * k, 10 * k.abs() + wide).nan_to_num(posinf=0.0)
            tol_one = torch.where(near, 3 * d.abs() + 10 * k, wide + 1).nan_to_num(posinf=0.0)
        if not kl:
            k_loss, one_loss = 0 * torch.zeros_like(k), torch.zeros_like(one)
        else:
            k_loss, one_loss = kl * k, kl * one
        tol_gain = gain.abs() * (torch.where(clipped, 0 * x, 2 * x.abs()) + 5)
        count = live.sum(1).double()
        n, s = count.sum(), (count > 0).sum().double()
        if mean == "tokens":
            w = scale / n.clamp_min(1) * torch.ones_like(count)
        elif mean == "sequences":
            w = scale / (count * s).clamp_min(1)
        else:
            w = scale * torch.ones_like(count)
        self.weights = torch.where(count > 0, w, 0.0)
        w = self.weights[:, None]

        def total(v):
            return torch.where(live, w * v, 0.0).sum()

        zero = torch.where(live, 0 * k, 0.0)
        self.policy, self.kl = -total(gain), total(k if ref is not None else zero)
        self.loss = self.policy + (kl * self.kl if kl else 0.0)
        # four tokens are added in binary32 before they meet the binary64 sum
        self.tol_policy = total(tol_gain + 4 * gain.abs()).abs() * U + self.policy.abs() * U
        self.tol_kl = total(tol_k + 4 * k.abs()).abs() * U + self.kl.abs() * U
        aw = self.weights.abs()[:, None]
        self.tol_loss = (torch.where(live, aw * (tol_gain + 4 * gain.abs()
                                                 + kl * (tol_k + 4 * k.abs())), 0.0).sum()
                         + self.loss.abs()) * U
        self.fraction = clipped.sum() / n.clamp_min(1)
        self.fall = torch.where(live, -x, 0.0).sum() / n.clamp_min(1)
        self.tol_fall = (torch.where(live, 5 * x.abs(), 0.0).sum() / n.clamp_min(1)
                         + self.fall.abs()) * U
        self.slope = torch.where(clipped, 0.0, -(a * r)) - one_loss
        self.tol_slope = (torch.where(clipped, 0.0, (a * r).abs() * (2 * x.abs() + 5))
                          + kl * (tol_one + one.abs().nan_to_num(posinf=0.0) * 2)
                          + self.slope.abs().nan_to_num(posinf=0.0)) * U

    @staticmethod
    def _line(d):
        """exp(d) - 1 - d for |d| < 1, whose difference loses up to 52 bits."""
        term, total = d * d / 2, torch.zeros_like(d)
        for i in range(3, 24):
            total, term = total + term, term * d / i
        return total

    def grad(self, weights, dloss):
        """(dlogp, tolerance) from the weights and dloss as given."""
        w = (weights.double() * dloss)[:, None]
        g = torch.where(self.live, w * self.slope, 0.0)
        tol = torch.where(self.live, w.abs() * (self.tol_slope
                                                + 3 * U * self.slope.abs().nan_to_num(posinf=0.0)),
                          0.0)
        return g, tol + 2.0 ** -126


# ---------------------------------------------------------------------------
# Tokens and experts
# ---------------------------------------------------------------------------

def sort(ids, experts, align, rows):
    """slot, offsets, counts, source, entry by entry."""
    ids = ids.reshape(-1).tolist()
    counts = [0] * experts
    for e in ids:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + -(-n // align) * align)
    following, slot, source = offsets[:-1], [], [-1] * rows
    for i, e in enumerate(ids):
        row = -1
        if 0 <= e < experts:
            row = following[e]
            following[e] += 1
            source[row] = i
        slot.append(row)
    return tuple(torch.tensor(v, dtype=torch.int32) for v in (slot, offsets, counts, source))


def combine(z, slot, weights, residual):
    """(y, tolerance before its rounding): one rounding a choice at the size
    of what has been added."""
    kept = (slot >= 0) & (slot < z.shape[0])
    w = torch.ones(slot.shape, dtype=torch.float64, device=z.device) if weights is None \
        else weights.double()
    y = 0.0 if residual is None else residual.double()
    mag = 0.0 if residual is None else residual.double().abs()
    for j in range(slot.shape[1]):
        if not z.shape[0]:
            break
        v = z[slot[:, j].long().clamp(0, z.shape[0] - 1)].double()
        part = torch.where(kept[:, j, None], w[:, j, None] * v, 0.0)
        y, mag = y + part, mag + part.abs()
    return y, mag * (slot.shape[1] + 1) * U


def combine_grad(dy, z, slot, weights):
    """({row of dz: value}, dweights, tolerance of dweights)."""
    kept = (slot >= 0) & (slot < z.shape[0])
    at = slot.long().clamp(0, max(z.shape[0] - 1, 0))
    rows = z.double()[at] if z.shape[0] else torch.zeros(*slot.shape, z.shape[1],
                                                         dtype=torch.float64, device=z.device)
    terms = torch.where(kept[:, :, None], dy.double()[:, None] * rows, 0.0)
    dz = weights.double()[:, :, None] * dy.double()[:, None]
    return (at[kept], dz[kept], terms.sum(2),
            terms.abs().sum(2) * adds(z.shape[1]) * U + 2.0 ** -126)
