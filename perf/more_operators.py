"""Cases that time libew's layer norm (with the residual's addition, and its
gradient), its clipped policy loss with a KL term (and its gradient) and its
movement of tokens to their experts and back (sorting and gathering, combining
with weights, and the gradient).

`run` computes a case in plain torch operations in 32 bits, or, with
``own = True``, through the library's entry points; `exact` computes it in 64
bits from the definitions.  A case's "op" names the operator, "type" the
element type, "pad" the elements between the end of a row and the start of the
next.  A norm's matrix is "rows" x "cols", "add" says whether a residual (or the
gradient of one) is added; a loss covers "rows" sequences of up
to "cols" tokens; "rows" tokens of "cols" values go to "top" of "experts"
experts each, whose rows start at multiples of "align".
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
LOW, HIGH, KL = 0.1875, 0.25, 0.03125      # clipping below and above 1, weight of the KL term


def listed():
    return [
        # one token through one layer's norm while decoding: launch latency
        {"name": "layernorm decode", "op": "norm", "type": "bf16", "rows": 1, "cols": 4096,
         "pad": 0, "add": True},
        # a training batch of 8192 tokens, statistics kept for the gradient
        {"name": "layernorm train", "op": "norm", "type": "bf16", "rows": 8192, "cols": 4096,
         "pad": 0, "add": True},
        # odd width and padded rows in 32 bits, the norm alone
        {"name": "layernorm odd f32", "op": "norm", "type": "f32", "rows": 1021, "cols": 5003,
         "pad": 5, "add": False},
        # the norm's gradient for the training batch, the residual's gradient added
        {"name": "layernorm gradient", "op": "norm_grad", "type": "bf16", "rows": 8192,
         "cols": 4096, "pad": 0, "add": True},
        # the gradient over narrow odd rows of 16-bit floats
        {"name": "layernorm gradient odd f16", "op": "norm_grad", "type": "f16", "rows": 4099,
         "cols": 1281, "pad": 3, "add": False},
        # a small update: 8 answers of up to 512 tokens, one advantage each
        {"name": "policy small", "op": "policy", "rows": 8, "cols": 512, "pad": 0, "ref": True,
         "each": False, "mean": "sequences"},
        # a large batch of 4096 answers of up to 4096 tokens, an advantage a token
        {"name": "policy batch", "op": "policy", "rows": 4096, "cols": 4096, "pad": 0, "ref": True,
         "each": True, "mean": "tokens"},
        # its gradient
        {"name": "policy gradient", "op": "policy_grad", "rows": 4096, "cols": 4096, "pad": 0,
         "ref": True, "each": True, "mean": "tokens"},
        # a decoding batch of 16 tokens sorted and gathered, 4 of 32 experts each
        {"name": "experts decode", "op": "dispatch", "type": "f16", "rows": 16, "cols": 2048,
         "pad": 0, "top": 4, "experts": 32, "align": 16},
        # a training batch: 8192 tokens to 8 of 128 experts each
        {"name": "experts dispatch", "op": "dispatch", "type": "bf16", "rows": 8192, "cols": 4096,
         "pad": 0, "top": 8, "experts": 128, "align": 16},
        # the experts' answers back to their tokens, added to the residual stream
        {"name": "experts combine", "op": "combine", "type": "bf16", "rows": 8192, "cols": 4096,
         "pad": 0, "top": 8, "experts": 128, "align": 16},
        # the gradient of that for half the batch, with the weights' gradient
        {"name": "experts gradient", "op": "combine_grad", "type": "bf16", "rows": 4096,
         "cols": 4096, "pad": 0, "top": 8, "experts": 128, "align": 16},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "policy", "policy_grad", "dispatch", "combine",
                     "combine_grad"])
    case = {"op": op, "pad": rng.choice([0, 0, 1, 8, 13])}
    if op.startswith("policy"):
        case.update(rows=_log_uniform(rng, 1, 4096), cols=_log_uniform(rng, 16, 16384),
                    ref=rng.random() < 0.7, each=rng.random() < 0.5,
                    mean=rng.choice(["tokens", "sequences"]))
        while case["rows"] * case["cols"] > 1 << 24:
            case["rows"] = (case["rows"] + 1) // 2
        return case
    case["type"] = rng.choice(["f32", "f16", "bf16", "bf16"])
    case["cols"] = _log_uniform(rng, 64, 16384 if op.startswith("norm") else 8192)
    if rng.random() < 0.5:
        case["cols"] += -case["cols"] % 64
    case["rows"] = _log_uniform(rng, 1, 8192)
    if op.startswith("norm"):
        case["add"] = rng.random() < 0.6
        most, each = 1 << 25, 1
    else:
        case["experts"] = rng.choice([8, 32, 64, 128, 256])
        case["top"] = rng.choice([1, 2, 4, 8])
        case["align"] = rng.choice([1, 1, 16, 32])
        most, each = 1 << (28 if op != "combine_grad" else 27), case["top"]
    if case["type"] == "f32":
        most //= 2
    while case["rows"] * case["cols"] * each > most:
        case["rows"] = (case["rows"] + 1) // 2
    return case


def work(case):
    r, c, op = case["rows"], case["cols"], case["op"]
    if op.startswith("policy"):
        # log probabilities of now, then and the reference, advantages, mask
        read = r * c * (9 + 4 * case["ref"]) + (4 * r * c if case["each"] else 4 * r)
        return {"bytes": read + 4 * r + (4 * r * c if op == "policy_grad" else 0),
                "flops": 12 * r * c}
    es = BYTES[case["type"]]
    if op == "norm":
        return {"bytes": r * c * es * (4 if case["add"] else 2) + 2 * c * es + 8 * r,
                "flops": 8 * r * c}
    if op == "norm_grad":
        return {"bytes": r * c * es * (4 if case["add"] else 3) + c * es + 8 * r + 8 * c,
                "flops": 14 * r * c}
    n = r * case["top"]
    if op == "dispatch":
        return {"bytes": (r + n) * c * es + 16 * n, "flops": n}
    if op == "combine":
        return {"bytes": (2 * r + n) * c * es + 8 * n, "flops": 2 * n * c}
    return {"bytes": (r + 2 * n) * c * es + 12 * n, "flops": 3 * n * c}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _matrix(rows, cols, pad, dtype, fill=None):
    """A rows x cols matrix whose rows lie cols + pad elements apart."""
    whole = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")
    view = whole[:, :cols]
    if fill is None:
        view.zero_()
    else:
        view.copy_(fill)
    return view


def _capacity(case):
    """Rows that any sorting of the batch fits in."""
    n, a = case["rows"] * case["top"], case["align"]
    return n if a == 1 else -(-(n + min(n, case["experts"]) * (a - 1)) // a) * a


def _prepare_norm(case, g):
    r, c, pad, dt = case["rows"], case["cols"], case["pad"], TYPES[case["type"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"weight": (1.0 + 0.2 * randn(c)).to(dt), "bias": (0.1 * randn(c)).to(dt)}
    # a stream whose channels have grown apart, with a mean of its own in each row
    x = randn(r, c) * (1.0 + randn(c).abs()) + randn(r, 1)
    s["x"] = _matrix(r, c, pad, dt, x)
    if case["op"] == "norm":
        s["y"] = _matrix(r, c, pad, dt)
        s["mean"], s["rstd"] = torch.zeros(r, device="cuda"), torch.zeros(r, device="cuda")
        if case["add"]:
            s["residual"] = _matrix(r, c, pad, dt, 2.0 * randn(r, c))
            s["total"] = _matrix(r, c, pad, dt)
        return s
    h = s["x"].double()
    mean = h.mean(1, keepdim=True)
    s["mean"] = mean[:, 0].float()
    s["rstd"] = torch.rsqrt((h - mean).square().mean(1) + EPS).float()
    s["dy"] = _matrix(r, c, pad, dt, 0.1 * randn(r, c))
    if case["add"]:
        s["dtotal"] = _matrix(r, c, pad, dt, 0.1 * randn(r, c))
    s["dx"] = _matrix(r, c, pad, dt)
    s["dweight"], s["dbias"] = torch.zeros(c, device="cuda"), torch.zeros(c, device="cuda")
    return s


def _prepare_policy(case, g):
    r, c, pad = case["rows"], case["cols"], case["pad"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # answers of any length, one in sixteen cut away altogether
    length = torch.randint(1, c + 1, (r,), generator=g, device="cuda")
    if r > 1:
        length[torch.rand(r, generator=g, device="cuda") < 1 / 16] = 0
    mask = torch.arange(c, device="cuda") < length[:, None]
    old = 1.5 * torch.rand(r, c, generator=g, device="cuda").clamp_min(1e-6).log()
    logp = old + 0.15 * randn(r, c)
    s = {"mask": _matrix(r, c, pad, torch.bool, mask)}
    # padding positions hold 0, as the log probabilities of no token do
    s["old_logp"] = _matrix(r, c, pad, torch.float32, torch.where(mask, old, 0.0))
    s["logp"] = _matrix(r, c, pad, torch.float32, torch.where(mask, logp, 0.0))
    s["ref_logp"] = None
    if case["ref"]:
        s["ref_logp"] = _matrix(r, c, pad, torch.float32,
                                torch.where(mask, old + 0.3 * randn(r, c), 0.0))
    s["advantage"] = (_matrix(r, c, pad, torch.float32, randn(r, c)) if case["each"]
                      else randn(r))
    if case["op"] == "policy":
        for name, n in (("loss", 1), ("stats", 4), ("weights", r)):
            s[name] = torch.zeros(n, device="cuda")
        return s
    s["weights"] = _token_weights(mask, case["mean"]).float()
    s["dloss"] = torch.full((1,), 0.5, device="cuda")      # one of two batches added up
    s["dlogp"] = _matrix(r, c, pad, torch.float32)
    return s


def _token_weights(mask, mean):
    """Weight of a counted token of each row in the mean, in 64 bits."""
    count = mask.sum(1).double()
    if mean == "tokens":
        weight = 1.0 / count.sum().clamp_min(1.0)
    else:
        weight = 1.0 / ((count > 0).sum().clamp_min(1) * count.clamp_min(1.0))
    return torch.where(count > 0, weight, 0.0)


def _prepare_experts(case, g):
    r, c, pad, k, e = (case[n] for n in ("rows", "cols", "pad", "top", "experts"))
    dt, cap = TYPES[case["type"]], _capacity(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # some experts are liked better; one token in sixteen is padding
    best = (randn(r, e) + 0.7 * randn(e)).topk(k, dim=1)
    ids = best.indices
    if r > 8:
        ids[torch.rand(r, generator=g, device="cuda") < 1 / 16] = -1
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"ids": ids, "slot": torch.zeros(r, k, **i32), "offsets": torch.zeros(e + 1, **i32),
         "counts": torch.zeros(e, **i32), "source": torch.zeros(cap, **i32)}
    if case["op"] == "dispatch":
        s["x"] = _matrix(r, c, pad, dt, randn(r, c))
        s["out"] = _matrix(cap, c, pad, dt)
        return s
    slot, offsets, counts, source = _sort(ids, e, case["align"], cap)
    s["slot"].copy_(slot)
    s["offsets"].copy_(offsets)
    s["counts"].copy_(counts)
    s["source"].copy_(source)
    s["mix"] = torch.softmax(best.values, 1)
    s["z"] = _matrix(cap, c, pad, dt, torch.randn(cap, c, generator=g, device="cuda", dtype=dt))
    if case["op"] == "combine":
        s["residual"] = _matrix(r, c, pad, dt, randn(r, c))
        s["y"] = _matrix(r, c, pad, dt)
    else:
        s["dy"] = _matrix(r, c, pad, dt, 0.1 * randn(r, c))
        s["dz"] = _matrix(cap, c, pad, dt)
        s["dmix"] = torch.zeros(r, k, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("norm"):
        made = _prepare_norm(case, g)
    elif case["op"].startswith("policy"):
        made = _prepare_policy(case, g)
    else:
        made = _prepare_experts(case, g)
    return {**case, **made}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


OUTPUTS = {
    "norm": ("y", "mean", "rstd", "total"), "norm_grad": ("dx", "dweight", "dbias"),
    "policy": ("loss", "stats", "weights"), "policy_grad": ("dlogp",),
    "dispatch": ("slot", "offsets", "counts", "source", "out"), "combine": ("y",),
    "combine_grad": ("dz", "dmix"),
}


def _outputs(s):
    return {k: s[k] for k in OUTPUTS[s["op"]] if k in s}


def _workspace(s, size):
    if "workspace" not in s:
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own(s):
    import memory_bound_elementwise_amd as ew
    op, t = s["op"], s.get("type")
    if op == "norm":
        getattr(ew, "ew_layernorm_" + t)(s["x"], s["weight"], s["bias"], s["y"],
                                         residual=s.get("residual"), total=s.get("total"),
                                         mean=s["mean"], rstd=s["rstd"], eps=EPS)
    elif op == "norm_grad":
        ws = _workspace(s, ew.ew_layernorm_grad_workspace(s["rows"], s["cols"]))
        getattr(ew, "ew_layernorm_grad_" + t)(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                              s["dx"], s["dweight"], s["dbias"], ws,
                                              dtotal=s.get("dtotal"))
    elif op == "policy":
        ws = _workspace(s, ew.ew_policy_loss_workspace(s["rows"], s["cols"]))
        ew.ew_policy_loss_f32(s["logp"], s["old_logp"], s["advantage"], s["loss"],
                              weights=s["weights"], ref_logp=s["ref_logp"], mask=s["mask"],
                              stats=s["stats"], clip_low=LOW, clip_high=HIGH, kl=KL,
                              mean=s["mean"], workspace=ws)
    elif op == "policy_grad":
        ew.ew_policy_loss_grad_f32(s["logp"], s["old_logp"], s["advantage"], s["weights"],
                                   s["dlogp"], ref_logp=s["ref_logp"], mask=s["mask"],
                                   dloss=s["dloss"], clip_low=LOW, clip_high=HIGH, kl=KL)
    elif op == "dispatch":
        ws = _workspace(s, ew.ew_experts_sort_workspace(s["ids"].numel(), s["experts"]))
        ew.ew_experts_sort(s["ids"], s["experts"], s["slot"], s["offsets"], counts=s["counts"],
                           source=s["source"], align=s["align"], workspace=ws)
        getattr(ew, "ew_experts_gather_" + t)(s["x"], s["slot"], s["out"], offsets=s["offsets"],
                                              counts=s["counts"])
    elif op == "combine":
        getattr(ew, "ew_experts_combine_" + t)(s["z"], s["slot"], s["y"], weights=s["mix"],
                                               residual=s["residual"])
    else:
        getattr(ew, "ew_experts_combine_grad_" + t)(s["dy"], s["z"], s["slot"], s["mix"], s["dz"],
                                                    s["dmix"], offsets=s["offsets"],
                                                    counts=s["counts"])
    return _outputs(s)


def _sort(ids, experts, align, capacity):
    """slot of each entry, first row and number of rows of each expert, entry
    of each row: entries in their order within an expert, whose first row is a
    multiple of align; -1 for an entry of no expert and a row of no entry."""
    flat = ids.reshape(-1)
    n = flat.numel()
    given = (flat >= 0) & (flat < experts)
    key, order = torch.where(given, flat, experts).sort(stable=True)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    packed = count.cumsum(0) - count
    size = (count[:experts] + align - 1) // align * align
    offsets = torch.cat([size.new_zeros(1), size.cumsum(0)])
    place = offsets[key] + torch.arange(n, device=ids.device) - packed[key]
    place = torch.where(key < experts, place, -1)
    slot = torch.empty_like(place).scatter_(0, order, place)
    source = torch.full((capacity + 1,), -1, dtype=torch.int64, device=ids.device)
    source.scatter_(0, torch.where(place >= 0, place, capacity), order)
    return slot.view(ids.shape), offsets, count[:experts], source[:capacity]


def _plain_policy(s):
    live, a = s["mask"], s["advantage"]
    if not s["each"]:
        a = a[:, None]
    logp, old = s["logp"], s["old_logp"]
    # which side of a border the ratio is on is decided in 64 bits
    x = logp.double() - old.double()
    clipped = ((a > 0) & (x > math.log1p(HIGH))) | ((a < 0) & (x < math.log1p(-LOW)))
    ratio = torch.exp(logp - old)
    if s["ref_logp"] is not None:
        d = s["ref_logp"] - logp
        grown = torch.expm1(d.double())       # e^d - 1 - d is of the order of d^2
    if s["op"] == "policy_grad":
        slope = -torch.where(clipped, 0.0, a * ratio)
        if s["ref_logp"] is not None:
            slope = slope - KL * grown.float()
        w = (s["weights"] * s["dloss"])[:, None]
        s["dlogp"].copy_(torch.where(live, w * slope, 0.0))
        return _outputs(s)
    bound = torch.where(a > 0, 1.0 + HIGH, 1.0 - LOW)
    policy = torch.where(live, -a * torch.where(clipped, bound, ratio), 0.0)
    divergence = torch.zeros_like(policy)
    if s["ref_logp"] is not None:
        divergence = torch.where(live, (grown - d.double()).float(), 0.0)
    # sums over millions of tokens
    weights = _token_weights(live, s["mean"])
    count = live.sum().clamp_min(1).double()
    gain = (weights * policy.double().sum(1)).sum()
    kl = (weights * divergence.double().sum(1)).sum()
    s["weights"].copy_(weights)
    s["loss"].copy_((gain + KL * kl)[None])
    s["stats"].copy_(torch.stack([gain, kl, (clipped & live).sum() / count,
                                  torch.where(live, -x, 0.0).sum() / count]))
    return _outputs(s)


def _plain(s):
    op, dt = s["op"], TYPES.get(s.get("type"))
    if op.startswith("policy"):
        return _plain_policy(s)
    if op == "norm":
        if "total" in s:
            s["total"].copy_((s["x"].float() + s["residual"].float()).to(dt))
        h = (s["total"] if "total" in s else s["x"]).float()
        mean = h.mean(1, keepdim=True)
        d = h - mean
        rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        s["y"].copy_((d * rstd * s["weight"].float() + s["bias"].float()).to(dt))
        s["mean"].copy_(mean[:, 0])
        s["rstd"].copy_(rstd[:, 0])
    elif op == "norm_grad":
        r = s["rstd"][:, None]
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * r
        g = dy * s["weight"].float()
        dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if "dtotal" in s:
            dx = dx + s["dtotal"].float()
        s["dx"].copy_(dx.to(dt))
        s["dweight"].copy_((dy * xh).double().sum(0))       # sums over thousands of rows
        s["dbias"].copy_(dy.double().sum(0))
    elif op == "dispatch":
        slot, offsets, counts, source = _sort(s["ids"], s["experts"], s["align"],
                                              s["source"].numel())
        for name, v in (("slot", slot), ("offsets", offsets), ("counts", counts),
                        ("source", source)):
            s[name].copy_(v)
        # rows of padding are 0, those behind the last expert's stay
        rows = s["x"][source.clamp_min(0) // s["top"]]
        rows = torch.where((source >= 0)[:, None], rows, 0.0)
        inside = torch.arange(source.numel(), device=source.device) < offsets[-1]
        s["out"].copy_(torch.where(inside[:, None], rows, s["out"]))
    elif op == "combine":
        y = s["residual"].float()
        for j in range(s["top"]):
            at = s["slot"][:, j].long()
            w = torch.where(at >= 0, s["mix"][:, j], 0.0)
            y = y + w[:, None] * s["z"][at.clamp_min(0)].float()
        s["y"].copy_(y.to(dt))
    else:
        dy = s["dy"].float()
        slot = s["slot"].reshape(-1)
        for j in range(s["top"]):
            at = s["slot"][:, j].long()
            dot = (dy * s["z"][at.clamp_min(0)].float()).sum(1)
            s["dmix"][:, j] = torch.where(at >= 0, dot, 0.0)
        source = s["source"].long()
        some = source >= 0
        w = torch.where(some, s["mix"].reshape(-1)[source.clamp_min(0)], 0.0)
        rows = w[:, None] * dy[source.clamp_min(0) // s["top"]]
        inside = torch.arange(source.numel(), device=slot.device) < s["offsets"][-1]
        s["dz"].copy_(torch.where(inside[:, None], rows.to(dt), s["dz"]))
    return _outputs(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"].startswith("policy"):
        return _exact_policy(s)
    return _exact_experts(s)


def _exact_norm(s):
    f64 = torch.float64
    n = s["cols"]
    w = s["weight"].to(f64)
    if s["op"] == "norm":
        total = s["x"].to(f64)
        if "total" in s:
            # the total is an output in the type itself: the norm is of the rounded sum
            total = (total + s["residual"].to(f64)).float().to(s["x"].dtype).to(f64)
        mean = total.sum(1) / n
        var = (total - mean[:, None]).pow(2).sum(1) / n
        rstd = (var + EPS).pow(-0.5)
        y = torch.addcmul(s["bias"].to(f64), (total - mean[:, None]) * w, rstd[:, None])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if "total" in s:
            out["total"] = total
        return out
    dy, r = s["dy"].to(f64), s["rstd"].to(f64)[:, None]
    xh = (s["x"].to(f64) - s["mean"].to(f64)[:, None]).mul_(r)
    out = {"dx": None, "dweight": torch.einsum("ij,ij->j", dy, xh), "dbias": dy.sum(0)}
    first = (dy @ w)[:, None] / n
    second = torch.einsum("ij,ij,j->i", dy, xh, w)[:, None] / n
    dx = (dy * w).sub_(first).sub_(xh.mul_(second)).mul_(r)
    if "dtotal" in s:
        dx += s["dtotal"].to(f64)
    out["dx"] = dx
    return out


def _exact_policy(s):
    """The loss by its definition, its gradient by differentiation, some rows
    at a time."""
    r = s["rows"]
    each = s["advantage"].double()
    each = each if s["each"] else each[:, None]
    if s["op"] == "policy_grad":
        weight = s["weights"].double()
    else:
        weight = _token_weights(s["mask"], s["mean"])
    grads, sums = [], torch.zeros(4, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 22) // s["cols"])
    for i in range(0, r, step):
        part = slice(i, i + step)
        live = s["mask"][part]
        logp = s["logp"][part].double().requires_grad_()
        old, a, w = s["old_logp"][part].double(), each[part], weight[part][:, None]
        ratio = (logp - old).exp()
        inner = ratio.clamp(1.0 - LOW, 1.0 + HIGH) * a
        gain = torch.minimum(ratio * a, inner)
        kl = torch.zeros_like(gain)
        if s["ref_logp"] is not None:
            d = s["ref_logp"][part].double() - logp
            kl = d.expm1() - d
        gain, kl = gain.masked_fill(~live, 0.0), kl.masked_fill(~live, 0.0)
        total = (w * (KL * kl - gain)).sum()
        if s["op"] == "policy_grad":
            total.backward()
            grads.append(logp.grad * s["dloss"].double())
            continue
        with torch.no_grad():
            hit = live & (inner < ratio * a)
            sums += torch.stack([-(w * gain).sum(), (w * kl).sum(), hit.sum(),
                                 (old - logp).masked_fill(~live, 0.0).sum()])
    if grads:
        return {"dlogp": torch.cat(grads)}
    sums[2:] /= s["mask"].sum().clamp_min(1)
    return {"loss": sums[:1] + KL * sums[1:2], "stats": sums, "weights": weight}


def _exact_experts(s):
    k, op = s["top"], s["op"]
    if op == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        counts = [0] * s["experts"]
        for e in ids:
            if 0 <= e < s["experts"]:
                counts[e] += 1
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + -(-n // s["align"]) * s["align"])
        after, slot = offsets[:-1], []
        source = [-1] * s["source"].numel()
        for i, e in enumerate(ids):
            slot.append(-1)
            if 0 <= e < s["experts"]:
                slot[i] = after[e]
                source[after[e]] = i
                after[e] += 1

        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device="cuda")

        out = torch.zeros(len(source), s["cols"], dtype=s["x"].dtype, device="cuda")
        rows = ints([i for i in range(len(source)) if source[i] >= 0])
        out[rows] = s["x"][ints([i // k for i in source if i >= 0])]
        return {"slot": ints(slot).view(-1, k), "offsets": ints(offsets), "counts": ints(counts),
                "source": ints(source), "out": out}
    y, dz, dmix = [], None, []
    if op == "combine_grad":
        dz = torch.zeros(s["z"].shape, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // (s["cols"] * k))
    for i in range(0, s["rows"], step):
        at = s["slot"][i:i + step].long()
        kept = (at >= 0)[:, :, None]
        rows = s["z"][at.clamp_min(0)].double() * kept
        mix = s["mix"][i:i + step].double()
        if op == "combine":
            y.append(s["residual"][i:i + step].double() + (mix[:, :, None] * rows).sum(1))
            continue
        dy = s["dy"][i:i + step].double()[:, None]
        dmix.append((dy * rows).sum(2))
        keep = kept.reshape(-1).nonzero()[:, 0]
        dz[at.reshape(-1)[keep]] = (mix[:, :, None] * dy).reshape(-1, s["cols"])[keep]
    if op == "combine":
        return {"y": torch.cat(y)}
    return {"dz": dz, "dmix": torch.cat(dmix)}
