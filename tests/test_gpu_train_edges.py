"""Layer norm, policy loss and the movement of rows to experts on the GPU at the
ends of their ranges: in place with a partial vector beside another wave's,
streams and graphs, offsets past 32 bits, more rows than a grid holds,
workspaces at their documented alignment.  Against the 64-bit definitions and
tolerances of tests/train_ref.py."""
import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests import train_ref as ref
from tests.rows_ref import TYPES, U, close
from tests.test_gpu_rows import DEV, GUARD, gen, randn
from tests.test_gpu_train import (Batch, Routed, check_grad, check_norm, f32, grad_inputs, i32,
                                  norm_inputs, space)

pytestmark = pytest.mark.gpu

every_type = pytest.mark.parametrize("t", TYPES)
LANES = {"f32": 4, "f16": 8, "bf16": 8}      # elements of a vector


# ---------------------------------------------------------------------------
# In place, the last vector a part that reaches into another wave's
# ---------------------------------------------------------------------------

# vectors before the part: the border of a wave, of a round of a block's waves
# and of a row's lengths that take other kernels
BORDERS = (64, 128, 192, 256, 320, 384, 512, 768, 1024, 1280, 1536, 1600, 1792, 2048, 2560, 3584,
           4096, 5120)


@every_type
@pytest.mark.parametrize("border", BORDERS)
def test_norm_in_place_at_borders(t, border):
    n = LANES[t]
    for cols in (border * n + 1, border * n + n - 1):
        for rows in (3, 300, 1500):
            if rows * cols > 8e6:
                continue
            x, res, w, b = norm_inputs(t, rows, cols, 0, 0, 7)
            fn = getattr(ew, "ew_layernorm_" + t)
            y, total, mean, rstd = torch.empty_like(x), torch.empty_like(x), f32(rows), f32(rows)
            fn(x, w, b, y, residual=res, total=total, mean=mean, rstd=rstd)
            check_norm(t, x, res, w, b, y, total, mean, rstd)
            for k in range(2):
                a = [x.clone(), res.clone()]
                fn(a[0], w, b, a[1 - k], residual=a[1], total=a[k])
                assert torch.equal(a[k], total) and torch.equal(a[1 - k], y)
            dy = (0.5 * res.float() - b.float()).to(x.dtype)
            fn = getattr(ew, "ew_layernorm_grad_" + t)
            dx = torch.empty_like(x)
            fn(dy, total, w, mean, rstd, dx, dtotal=x)
            check_grad(t, dy, total, w, mean, rstd, x, dx, None, None)
            for k in range(3):
                a = [dy.clone(), total.clone(), x.clone()]
                fn(a[0], a[1], w, mean, rstd, a[k], dtotal=a[2])
                assert torch.equal(a[k], dx), (cols, rows, k)


@every_type
@pytest.mark.parametrize("border", (64, 128, 256, 512, 1024, 1536))
@pytest.mark.parametrize("top", (2, 3, 9))
def test_experts_in_place_at_borders(t, border, top):
    n = LANES[t]
    for cols in (border * n + 1, border * n + n - 1):
        for tokens in (50, 1100):
            if tokens * top * cols > 3e7:
                continue
            r = Routed(t, tokens, cols, top)
            r.check_combine()
            r.check_grad()


@pytest.mark.parametrize("cols", (257, 259, 1025, 1027, 2049, 4099, 262145))
def test_policy_in_place_at_borders(cols):
    batch = Batch(5, cols, seed=6)
    _, weights, want = batch.check()
    for name in ("logp", "old", "ref", "advantage"):
        args = {k: getattr(batch, k).clone() for k in ("logp", "old", "ref", "advantage")}
        ew.ew_policy_loss_grad_f32(args["logp"], args["old"], args["advantage"], weights, args[name],
                                   ref_logp=args["ref"], mask=batch.mask, clip_high=0.3, kl=0.1)
        assert torch.equal(args[name], want), name


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------

class Run:
    """The operators one after another, as a training step calls them: a norm,
    tokens to their experts and back, a norm's gradient, the loss and its
    gradient.  An output of one is an input of the next."""

    def __init__(self, t="bf16", tokens=60, cols=515, top=3, experts=9, sequences=6, seed=0):
        self.t, self.tokens, self.cols, self.experts = t, tokens, cols, experts
        self.shape = sequences, tokens // sequences
        self.ids = torch.empty(tokens, top, dtype=torch.int64, device=DEV)
        self.x, self.res = (torch.empty(tokens, cols, dtype=TYPES[t], device=DEV) for _ in range(2))
        self.w, self.b = (torch.empty(cols, dtype=TYPES[t], device=DEV) for _ in range(2))
        self.gates = f32(tokens, top)
        self.logp, self.old, self.ref = (f32(*self.shape) for _ in range(3))
        self.advantage = f32(sequences)
        self.mask = torch.empty(self.shape, dtype=torch.uint8, device=DEV)
        self.fill(seed)

    def fill(self, seed):
        g = gen(seed)
        self.ids.random_(-1, self.experts, generator=g)
        for v in (self.x, self.res, self.w, self.b, self.gates, self.logp, self.old, self.ref,
                  self.advantage):
            v.copy_(randn(g, *v.shape))
        self.mask.random_(0, 2, generator=g)

    def outputs(self):
        places = ew.ew_experts_rows(self.ids.numel(), self.experts, 16)
        z = [torch.zeros(places, self.cols, dtype=self.x.dtype, device=DEV) for _ in range(2)]
        y = [torch.zeros_like(self.x) for _ in range(4)]
        return {"y": y[0], "total": y[1], "mean": f32(self.tokens), "rstd": f32(self.tokens),
                "slot": i32(*self.ids.shape), "offsets": i32(self.experts + 1),
                "counts": i32(self.experts), "source": i32(places), "rows": z[0], "back": y[2],
                "drows": z[1], "dgates": f32(*self.gates.shape), "dx": y[3],
                "dw": f32(self.cols), "db": f32(self.cols), "loss": f32(1), "stats": f32(4),
                "weights": f32(self.shape[0]), "dlogp": f32(*self.shape)}

    def need(self):
        return max(ew.ew_layernorm_grad_workspace(self.tokens, self.cols),
                   ew.ew_policy_loss_workspace(*self.shape),
                   ew.ew_experts_sort_workspace(self.ids.numel(), self.experts))

    def __call__(self, o, ws, stream=None):
        def call(name, *args, **kw):
            getattr(ew, f"ew_{name}_{self.t}")(*args, stream=stream, **kw)

        pads = {"offsets": o["offsets"], "counts": o["counts"]}
        call("layernorm", self.x, self.w, self.b, o["y"], residual=self.res, total=o["total"],
             mean=o["mean"], rstd=o["rstd"])
        ew.ew_experts_sort(self.ids, self.experts, o["slot"], o["offsets"], counts=o["counts"],
                           source=o["source"], align=16, workspace=ws, stream=stream)
        call("experts_gather", o["y"], o["slot"], o["rows"], **pads)
        call("experts_combine", o["rows"], o["slot"], o["back"], weights=self.gates,
             residual=o["total"])
        call("experts_combine_grad", o["back"], o["rows"], o["slot"], self.gates, o["drows"],
             o["dgates"], **pads)
        call("layernorm_grad", o["back"], o["total"], self.w, o["mean"], o["rstd"], o["dx"],
             o["dw"], o["db"], ws, dtotal=o["y"])
        args = {"ref_logp": self.ref, "mask": self.mask, "kl": 0.1, "stream": stream}
        ew.ew_policy_loss_f32(self.logp, self.old, self.advantage, o["loss"], weights=o["weights"],
                              stats=o["stats"], workspace=ws, mean="sequences", **args)
        ew.ew_policy_loss_grad_f32(self.logp, self.old, self.advantage, o["weights"], o["dlogp"],
                                   **args)


RUNS = ({}, {"t": "f32", "tokens": 4100, "cols": 70, "top": 4, "experts": 40, "sequences": 5},
        {"t": "f16", "tokens": 20400, "cols": 9, "top": 2, "sequences": 300})


def equal(got, want, what):
    """Whole outputs, of the experts' rows those up to the last expert's end
    (behind it they are left as they were)."""
    end = int(want["offsets"][-1])
    for name in want:
        u, v = got[name], want[name]
        if name in ("rows", "drows"):
            u, v = u[:end], v[:end]
        assert torch.equal(u, v), (what, name)


@pytest.mark.parametrize("which", range(len(RUNS)))
def test_calls_repeated_give_the_same_bits(which):
    run = Run(**RUNS[which])
    want, ws = run.outputs(), space(run.need())
    run(want, ws)
    for k in range(3):
        ws.fill_(k * 77)                      # whatever the workspace holds
        got = run.outputs()
        run(got, ws)
        equal(got, want, k)


@pytest.mark.parametrize("which", range(len(RUNS)))
def test_calls_on_a_stream(which):
    """Inputs made and outputs read on the stream that the calls are given, or
    the current one."""
    run = Run(**RUNS[which])
    want, ws = run.outputs(), space(run.need())
    run(want, ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (True, False):
        got = run.outputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big = torch.randn(4096, 4096, device=DEV)
            for v in (run.x, run.logp, run.gates):
                v.fill_(0)
            for _ in range(4):
                big = big @ big * 0.01
            run.fill(0)                       # ready only on the side stream
            if not given:
                run(got, ws)
        if given:
            run(got, ws, stream=side)
        side.synchronize()
        equal(got, want, given)


@pytest.mark.parametrize("which", range(len(RUNS)))
def test_graphs_replay(which):
    """Two captures of the run that share a workspace, replayed in turn on
    changing inputs with eager work between, against eager calls."""
    run = Run(**RUNS[which])
    ws = space(run.need())
    got, want = [run.outputs(), run.outputs()], run.outputs()
    run(want, space(run.need()))
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in got]
    for graph, o in zip(graphs, got):
        with torch.cuda.graph(graph):
            run(o, ws)
    for k in range(4):
        run.fill(100 + k)
        run(want, space(run.need()))
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in got:
            equal(o, want, k)


def test_workspaces_16_bytes_off():
    run = Run(**RUNS[1])
    want, got = run.outputs(), run.outputs()
    run(want, space(run.need()))
    ws = space(run.need() + 48)
    run(got, ws[16:16 + run.need()])
    equal(got, want, "16 bytes off")
    assert bool((ws[:16] == 0xAB).all()) and bool((ws[16 + run.need():] == 0xAB).all())


# ---------------------------------------------------------------------------
# Offsets past 32 bits, more rows than a grid holds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", ((263000, 16400), (1050000, 4099)))
def test_norm_offsets_past_32_bits(rows, cols):
    """The last rows of matrices of more than 2^32 elements, and the sums, to
    which only they contribute."""
    tail = 3
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(x)
    data, res, w, _ = norm_inputs("bf16", tail, cols, 0, 0, 95)
    x[-tail:].copy_(data)
    mean, rstd = f32(rows), f32(rows)
    ew.ew_layernorm_bf16(x, w, None, y, mean=mean, rstd=rstd)
    check_norm("bf16", data, None, w, None, y[-tail:], None, mean[-tail:], rstd[-tail:])
    assert all(not bool(part.any()) for part in y[:-tail].split(20000))
    y[-tail:].copy_(res)                           # as dy
    dw, db = f32(cols), f32(cols)
    ew.ew_layernorm_grad_bf16(y, x, w, mean, rstd, y, dw, db,
                              space(ew.ew_layernorm_grad_workspace(rows, cols)))
    # (every other row adds exact zeros)
    check_grad("bf16", res, data, w, mean[-tail:], rstd[-tail:], None, y[-tail:], dw, db)


def test_policy_offsets_past_32_bits():
    """Matrices of more than 2^32 elements whose last rows alone count."""
    rows, cols, tail = 33000, 131080, 2
    batch = Batch(tail, cols, seed=3, ref_logp=False, each=False)
    logp = torch.zeros(rows, cols, device=DEV)
    old = torch.zeros(rows, cols, device=DEV)
    mask = torch.zeros(rows, cols, dtype=torch.uint8, device=DEV)
    advantage = torch.zeros(rows, device=DEV)
    for whole, part in ((logp, batch.logp), (old, batch.old), (mask, batch.mask),
                        (advantage, batch.advantage)):
        whole[-tail:].copy_(part)
    want_loss, want_weights, want = batch.check(mean="sequences", kl=0.0)
    loss, weights = f32(1), f32(rows)
    ew.ew_policy_loss_f32(logp, old, advantage, loss, weights=weights, mask=mask, clip_high=0.3,
                          mean="sequences",
                          workspace=space(ew.ew_policy_loss_workspace(rows, cols)))
    # both are within the same tolerance of the definition
    stat = ref.Policy(batch.logp, batch.old, batch.advantage[:, None], None, batch.mask, 0.2, 0.3,
                      0.0, "sequences")
    close(loss, stat.loss[None], stat.tol_loss + 2.0 ** -126, "loss")
    assert torch.equal(weights[-tail:], want_weights) and not bool(weights[:-tail].any())
    ew.ew_policy_loss_grad_f32(logp, old, advantage, weights, old, mask=mask, clip_high=0.3)
    assert torch.equal(old[-tail:], want)
    assert all(not bool(part.any()) for part in old[:-tail].split(1000))


def test_policy_of_one_long_sequence():
    """The most tokens of a sequence, of which the last count."""
    cols, tail = (1 << 31) - 1, 70001
    batch = Batch(1, tail, seed=4, ref_logp=False, each=False, mask=False)
    logp, old = (torch.zeros(1, cols, device=DEV) for _ in range(2))
    mask = torch.zeros(1, cols, dtype=torch.uint8, device=DEV)
    logp[:, -tail:].copy_(batch.logp)
    old[:, -tail:].copy_(batch.old)
    mask[:, -tail:] = 1
    loss, weights = f32(1), f32(1)
    ew.ew_policy_loss_f32(logp, old, batch.advantage, loss, weights=weights, mask=mask,
                          workspace=space(ew.ew_policy_loss_workspace(1, cols)))
    stat = ref.Policy(batch.logp, batch.old, batch.advantage[:, None], None, None, 0.2, 0.2, 0.0,
                      "tokens")
    close(loss, stat.loss[None], stat.tol_loss + 2.0 ** -126, "loss")
    close(weights, stat.weights, stat.weights.abs() * U * 1.01, "weights")
    ew.ew_policy_loss_grad_f32(logp, old, batch.advantage, weights, logp, mask=mask)
    g, tol = stat.grad(weights, 1.0)
    close(logp[:, -tail:], g, tol, "dlogp")
    assert not bool(logp[:, :-tail].any())


def test_experts_offsets_past_32_bits():
    """Tokens whose rows lie past 2^32 elements on both sides."""
    tokens, cols = 33000, 131080
    x = torch.zeros(tokens, cols, dtype=torch.bfloat16, device=DEV)
    tail = randn(gen(5), 4, cols).bfloat16()
    x[-4:].copy_(tail)
    ids = torch.zeros(tokens, 1, dtype=torch.int64, device=DEV)
    ids[-4:, 0] = torch.tensor([1, 0, 2, 1], device=DEV)
    rows = ew.ew_experts_rows(tokens, 3, 8)
    slot, offsets, counts = i32(tokens, 1), i32(4), i32(3)
    ew.ew_experts_sort(ids, 3, slot, offsets, counts=counts, align=8,
                       workspace=space(ew.ew_experts_sort_workspace(tokens, 3)))
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    out[32900:].fill_(7.0)
    ew.ew_experts_gather_bf16(x, slot, out, offsets=offsets, counts=counts)
    # 32997 of expert 0, padded to 33000, then two of 1, one of 2
    assert counts.tolist() == [32997, 2, 1] and offsets.tolist() == [0, 33000, 33008, 33016]
    assert slot[-4:, 0].tolist() == [33000, 32996, 33008, 33001]
    assert torch.equal(out[slot[-4:, 0].long()], tail)
    assert not bool(out[32997:33000].any()) and not bool(out[33002:33008].any())
    assert not bool(out[33009:33016].any())
    x[-4:].zero_()
    ew.ew_experts_combine_bf16(out, slot, x, residual=x)
    assert torch.equal(x[-4:], tail) and not bool(x[30000:-4].any())
    w, dw = torch.full((tokens, 1), 2.0, device=DEV), f32(tokens, 1)
    ew.ew_experts_combine_grad_bf16(x, out, slot, w, out, dw, offsets=offsets, counts=counts)
    assert torch.equal(out[slot[-4:, 0].long()], 2 * tail)
    dots = tail.double().square().sum(1)
    close(dw[-4:, 0], dots, dots * (cols / 64 + 40) * U, "dweights")


@every_type
@pytest.mark.parametrize("rows,cols", ((5203, 3), (5201, 4), (5203, 250), (5131, 512), (2565, 513),
                                       (2567, 1000), (1283, 1540), (1281, 2049), (1285, 2600),
                                       (1283, 4096), (2561, 4096), (2563, 3900), (1281, 8191),
                                       (1281, 12289), (1283, 16001)))
def test_norm_of_odd_numbers_of_rows(t, rows, cols):
    """More blocks than the chip holds at once, which then take rows in pairs
    or several a block: the last one is not full."""
    x, res, w, b = norm_inputs(t, rows, cols, 3, 1, 17)
    for residual in (res, None):
        y, mean, rstd = torch.empty(rows, cols, dtype=TYPES[t], device=DEV), f32(rows + 1), f32(rows + 1)
        total = torch.empty_like(y) if residual is not None else None
        getattr(ew, "ew_layernorm_" + t)(x, w, b, y, residual=residual, total=total,
                                         mean=mean[:rows], rstd=rstd[:rows])
        check_norm(t, x, residual, w, b, y, total, mean[:rows], rstd[:rows])
        assert float(mean[rows]) == GUARD and float(rstd[rows]) == GUARD


@every_type
@pytest.mark.parametrize("rows,cols", ((161, 12801), (200, 4100), (383, 8200), (384, 2500),
                                       (385, 6000), (511, 9000), (300, 16384)))
def test_norm_grad_of_some_long_rows(t, rows, cols):
    """Numbers of rows around those whose sums are of one or two rows a part."""
    dy, x, w, mean, rstd, dto = grad_inputs(t, rows, cols, 0, 0, 33)
    dx, dw, db = torch.empty_like(x), f32(cols), f32(cols)
    getattr(ew, "ew_layernorm_grad_" + t)(dy, x, w, mean, rstd, dx, dw, db,
                                          space(ew.ew_layernorm_grad_workspace(rows, cols)),
                                          dtotal=dto)
    check_grad(t, dy, x, w, mean, rstd, dto, dx, dw, db)


@every_type
def test_experts_of_the_longest_rows(t):
    """One token whose columns are more than the blocks that share them."""
    cols, dt = 140_000_003, TYPES[t]
    x = torch.arange(cols, device=DEV).remainder_(251).to(dt)[None]
    slot = torch.tensor([[1, -1]], dtype=torch.int32, device=DEV)
    out = torch.full((2, cols), 7.0, dtype=dt, device=DEV)
    getattr(ew, "ew_experts_gather_" + t)(x, slot, out)
    assert torch.equal(out[1:], x) and bool((out[0] == 7).all())
    y = torch.empty_like(x)
    w = torch.tensor([[0.5, 3.0]], device=DEV)
    getattr(ew, "ew_experts_combine_" + t)(out, slot, y, weights=w, residual=x)
    assert torch.equal(y, (1.5 * x.float()).to(dt))
    dw = f32(1, 2)
    getattr(ew, "ew_experts_combine_grad_" + t)(x, out, slot, w, out, dw)
    assert torch.equal(out[1:], (0.5 * x.float()).to(dt)) and float(dw[0, 1]) == 0
    dot = sum(float(p.double().square().sum()) for p in x[0].split(1 << 26))
    # a lane adds up cols / 256 terms one after another
    assert abs(float(dw[0, 0]) - dot) <= dot * (cols / 256 + 40) * U


def test_more_rows_than_a_grid_holds():
    """Norms, losses and movements of more than 2^20 blocks' rows."""
    rows = (1 << 22) + 5                           # four rows a block
    x, _, w, b = norm_inputs("f16", rows, 3, 0, 0, 8)
    y, mean, rstd = torch.empty_like(x), f32(rows), f32(rows)
    ew.ew_layernorm_f16(x, w, b, y, mean=mean, rstd=rstd)
    check_norm("f16", x, None, w, b, y, None, mean, rstd)
    slot = torch.arange(rows, dtype=torch.int32, device=DEV).flip(0)[:, None].contiguous()
    out, back = torch.empty_like(x), torch.empty_like(x)
    ew.ew_experts_gather_f16(x, slot, out)
    assert torch.equal(out, x.flip(0))
    ew.ew_experts_combine_f16(out, slot, back)
    assert torch.equal(back, x)
    weights, dw = torch.ones(rows, 1, device=DEV), f32(rows, 1)
    ew.ew_experts_combine_grad_f16(x, out, slot, weights, out, dw)
    assert torch.equal(out, x.flip(0))
    dots = x.double().square().sum(1)
    close(dw[:, 0], dots, dots * 8 * U, "dweights")

    rows = (1 << 20) + 3                           # a block each
    x, _, w, b = norm_inputs("bf16", rows, 1030, 0, 0, 9)
    y = torch.empty_like(x)
    ew.ew_layernorm_bf16(x, w, b, y, mean=mean[:rows], rstd=rstd[:rows])
    for at in (slice(0, 1000), slice(rows - 1000, rows)):
        check_norm("bf16", x[at], None, w, b, y[at], None, mean[at], rstd[at])
    ends = torch.cat([x[:5], x[-5:]])
    del y
    batch = Batch(10, 1030, seed=9, ref_logp=False, each=False)
    logp, old = (torch.zeros(rows, 1030, device=DEV) for _ in range(2))
    mask = torch.zeros(rows, 1030, dtype=torch.uint8, device=DEV)
    advantage, weights = torch.zeros(rows, device=DEV), f32(rows)
    for whole, part in ((logp, batch.logp), (old, batch.old), (mask, batch.mask),
                        (advantage, batch.advantage)):
        whole[:5].copy_(part[:5])
        whole[-5:].copy_(part[5:])
    loss = f32(1)
    ew.ew_policy_loss_f32(logp, old, advantage, loss, weights=weights, mask=mask, clip_high=0.3,
                          workspace=space(ew.ew_policy_loss_workspace(rows, 1030)))
    stat = ref.Policy(batch.logp, batch.old, batch.advantage[:, None], None, batch.mask, 0.2, 0.3,
                      0.0, "tokens")
    close(loss, stat.loss[None], stat.tol_loss + 2.0 ** -126, "loss")
    ew.ew_policy_loss_grad_f32(logp, old, advantage, weights, logp, mask=mask, clip_high=0.3)
    some = torch.cat([weights[:5], weights[-5:]])
    g, tol = stat.grad(some, 1.0)
    close(torch.cat([logp[:5], logp[-5:]]), g, tol, "dlogp")
    del old, mask
    assert not bool(logp[5:-5].any())
    del logp
    wide = torch.zeros(rows, 2056, dtype=torch.bfloat16, device=DEV)
    wide[:5, :1030], wide[-5:, :1030] = ends[:5], ends[5:]
    slot = torch.arange(rows, dtype=torch.int32, device=DEV).flip(0)[:, None].contiguous()
    out = torch.empty_like(wide)
    ew.ew_experts_gather_bf16(wide, slot, out)
    assert torch.equal(out[:5], wide[-5:].flip(0)) and torch.equal(out[-5:], wide[:5].flip(0))
    ew.ew_experts_combine_bf16(out, slot, wide, residual=wide)
    assert torch.equal(wide[:5, :1030], 2 * ends[:5]) and torch.equal(wide[-5:, :1030], 2 * ends[5:])


def test_sort_of_the_most_entries():
    n = (1 << 31) - 100
    ids = torch.empty(n, dtype=torch.int64, device=DEV)
    for at in range(0, n, 1 << 26):
        part = ids[at:at + (1 << 26)]
        torch.arange(at, at + part.numel(), out=part)
        part.remainder_(4)
    slot, offsets = torch.empty(n, dtype=torch.int32, device=DEV), i32(5)
    ew.ew_experts_sort(ids, 4, slot, offsets, workspace=space(ew.ew_experts_sort_workspace(n, 4)))
    del ids
    assert offsets.tolist() == [k * (n // 4) for k in range(5)]
    for at in list(range(0, n, 1 << 28)) + [n - (1 << 20)]:
        i = torch.arange(at, min(at + (1 << 20), n), device=DEV)
        assert torch.equal(slot[i].long(), i % 4 * (n // 4) + i // 4)
