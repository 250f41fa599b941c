"""Layer norm, policy loss and the movement of rows to experts without a GPU:
every refusal of the C entry points and of the binding comes before any HIP
call."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.conftest import _gpu_visible

OK, INVALID, MISALIGNED, OVERLAP, NO_DEVICE = 0, -1, -2, -3, -4
BASE = 0x7F0000000000          # a made-up, 256-byte aligned device address
MiB = 1 << 20
TYPES = ("f32", "f16", "bf16")
A, B, C, D, E, F, G, H, W, X = (BASE + k * 64 * MiB for k in range(10))
BIG = 1 << 20                  # workspace bytes: more than these calls need


def norm(t, x=A, xs=64, w=B, b=X, res=C, ress=64, y=D, ys=64, total=E, ts=64, mean=G, rstd=F,
         rows=8, cols=64, eps=1e-5):
    return ew._c["ew_layernorm_" + t](x, xs, w, b, res, ress, y, ys, total, ts, mean, rstd, rows,
                                      cols, eps, 0)


def norm_grad(t, dy=A, dys=64, x=B, xs=64, w=C, mean=X, rstd=D, dt=E, dts=64, dx=F, dxs=64, dw=G,
              db=H, ws=W, wsb=BIG, rows=8, cols=64):
    return ew._c["ew_layernorm_grad_" + t](dy, dys, x, xs, w, mean, rstd, dt, dts, dx, dxs, dw, db,
                                           ws, wsb, rows, cols, 0)


def policy(t, logp=A, ls=64, old=B, os=64, ref=C, rs=64, adv=D, as_=64, mask=E, ms=64, loss=F,
           stats=G, weights=H, low=0.2, high=0.2, kl=0.1, scale=1.0, mean=0, ws=W, wsb=BIG, rows=8,
           cols=64):
    return ew._c["ew_policy_loss_f32"](logp, ls, old, os, ref, rs, adv, as_, mask, ms, loss, stats,
                                       weights, low, high, kl, scale, mean, ws, wsb, rows, cols, 0)


def policy_grad(t, logp=A, ls=64, old=B, os=64, ref=C, rs=64, adv=D, as_=64, mask=E, ms=64,
                weights=F, dloss=G, dlogp=H, ds=64, low=0.2, high=0.2, kl=0.1, rows=8, cols=64):
    return ew._c["ew_policy_loss_grad_f32"](logp, ls, old, os, ref, rs, adv, as_, mask, ms,
                                            weights, dloss, dlogp, ds, low, high, kl, rows, cols,
                                            0)


def sort(t, ids=A, entries=64, experts=8, align=16, slot=B, offsets=C, counts=D, source=E, ws=W,
         wsb=BIG):
    return ew._c["ew_experts_sort"](ids, entries, experts, align, slot, offsets, counts, source,
                                    ws, wsb, 0)


def gather(t, x=A, xs=64, slot=B, top=2, offsets=C, counts=D, experts=4, out=E, outs=64,
           out_rows=16, rows=8, cols=64):
    return ew._c["ew_experts_gather_" + t](x, xs, slot, top, offsets, counts, experts, out, outs,
                                           out_rows, rows, cols, 0)


def combine(t, z=A, zs=64, z_rows=16, slot=B, top=2, weights=C, res=D, ress=64, y=E, ys=64, rows=8,
            cols=64):
    return ew._c["ew_experts_combine_" + t](z, zs, z_rows, slot, top, weights, res, ress, y, ys,
                                            rows, cols, 0)


def combine_grad(t, dy=A, dys=64, z=B, zs=64, z_rows=16, slot=C, top=2, weights=D, offsets=E,
                 counts=F, experts=4, dz=G, dzs=64, dweights=H, rows=8, cols=64):
    return ew._c["ew_experts_combine_grad_" + t](dy, dys, z, zs, z_rows, slot, top, weights,
                                                 offsets, counts, experts, dz, dzs, dweights, rows,
                                                 cols, 0)


CALLS = {"norm": norm, "norm_grad": norm_grad, "policy": policy, "policy_grad": policy_grad,
         "sort": sort, "gather": gather, "combine": combine, "combine_grad": combine_grad}
REQUIRED = {"norm": "x y", "norm_grad": "dy x mean rstd dx ws", "policy": "logp old adv loss ws",
            "policy_grad": "logp old adv weights dlogp", "sort": "ids slot offsets",
            "gather": "x slot out", "combine": "z slot y",
            "combine_grad": "dy z slot weights dz dweights"}
STRIDES = {"norm": "xs ress ys ts", "norm_grad": "dys xs dts dxs", "policy": "ls os rs as_ ms",
           "policy_grad": "ls os rs as_ ms ds", "sort": "", "gather": "xs outs",
           "combine": "zs ress ys", "combine_grad": "dys zs dzs"}
OUTPUTS = {"norm": "y total mean rstd", "norm_grad": "dx dw db ws",
           "policy": "loss stats weights ws", "policy_grad": "dlogp",
           "sort": "slot offsets counts source", "gather": "out", "combine": "y",
           "combine_grad": "dz dweights"}
INPUTS = {"norm": "x w b res", "norm_grad": "dy x w mean rstd dt",
          "policy": "logp old ref adv mask", "policy_grad": "logp old ref adv mask weights dloss",
          "sort": "ids", "gather": "x slot offsets counts", "combine": "z slot weights res",
          "combine_grad": "dy z slot weights offsets counts"}
# outputs that may be exactly an input
SAME = {"norm": "y=x y=res total=x total=res", "norm_grad": "dx=dy dx=x dx=dt", "policy": "",
        "policy_grad": "dlogp=logp dlogp=old dlogp=ref dlogp=adv", "sort": "", "gather": "",
        "combine": "y=res", "combine_grad": "dz=z"}

every = pytest.mark.parametrize("t", TYPES)
each_call = pytest.mark.parametrize("name", CALLS)
matrices = pytest.mark.parametrize("name", [n for n in CALLS if n != "sort"])


def defaults(name):
    fn = CALLS[name]
    return dict(zip(fn.__code__.co_varnames[1:], fn.__defaults__))


@pytest.mark.skipif(_gpu_visible(), reason="would launch with made-up addresses")
@every
@each_call
def test_a_valid_call_reaches_the_device_check(name, t):
    assert CALLS[name](t) == NO_DEVICE
    if name != "sort":       # a single row's stride is not used
        one = {s: 0 for s in STRIDES[name].split() if s != "as_"}
        if "out_rows" in defaults(name) or "z_rows" in defaults(name):
            one = {s: v for s, v in one.items() if s not in ("outs", "zs", "dzs")}
        assert CALLS[name](t, rows=1, **one) == NO_DEVICE


@every
@each_call
def test_null_pointers(name, t):
    for arg in REQUIRED[name].split():
        assert CALLS[name](t, **{arg: None}) == INVALID, arg


@pytest.mark.skipif(_gpu_visible(), reason="would launch with made-up addresses")
@every
def test_optional_pointers(t):
    assert norm(t, w=None, b=None, res=None, total=None, mean=None, rstd=None) == NO_DEVICE
    assert norm_grad(t, w=None, dt=None, dw=None, db=None, ws=None, wsb=0) == NO_DEVICE
    assert policy(t, ref=None, mask=None, stats=None, weights=None) == NO_DEVICE
    assert policy_grad(t, ref=None, mask=None, dloss=None) == NO_DEVICE
    assert sort(t, counts=None, source=None, ws=None, wsb=0) == NO_DEVICE
    assert gather(t, offsets=None, counts=None, experts=0) == NO_DEVICE
    assert combine(t, weights=None, res=None) == NO_DEVICE
    assert combine_grad(t, offsets=None, counts=None, experts=0) == NO_DEVICE
    # one advantage a sequence
    assert policy(t, as_=0) == NO_DEVICE and policy_grad(t, as_=0) == NO_DEVICE


@every
@matrices
def test_strides_shorter_than_a_row(name, t):
    for arg in STRIDES[name].split():
        assert CALLS[name](t, **{arg: 63}) == INVALID, arg
        assert CALLS[name](t, **{arg: 1 << 61}) == INVALID, arg


@every
@matrices
def test_sizes_past_the_limits(name, t):
    big = {s: 1 << 31 for s in STRIDES[name].split()}
    assert CALLS[name](t, rows=1 << 31) == INVALID
    assert CALLS[name](t, cols=1 << 31, **big) == INVALID
    # the address range wraps
    first = STRIDES[name].split()[0]
    rows = "z_rows" if first == "zs" else "rows"
    assert CALLS[name](t, **{rows: 1 << 29, first: 1 << 40}) == INVALID


@every
def test_sizes_of_movements(t):
    for call, places in ((gather, "out_rows"), (combine, "z_rows"), (combine_grad, "z_rows")):
        assert call(t, **{places: 1 << 31}) == INVALID
        for top in (0, 65, 1 << 63):
            assert call(t, top=top) == INVALID
        assert call(t, rows=1 << 30, top=2) == INVALID
    for call in (gather, combine_grad):
        assert call(t, offsets=None) == INVALID
        assert call(t, counts=None) == INVALID
        for experts in (0, 1025, 1 << 40):
            assert call(t, experts=experts) == INVALID


def test_sizes_of_sortings():
    for wrong in ({"entries": 1 << 31}, {"experts": 0}, {"experts": 1025}, {"align": 0},
                  {"align": 1025}, {"entries": (1 << 31) - 1, "align": 2}):
        assert sort("f32", **wrong) == INVALID, wrong
        sizes = {"entries": 64, "experts": 8, "align": 16, **wrong}
        assert ew._c["ew_experts_rows"](*sizes.values()) == (1 << 64) - 1
        with pytest.raises(ValueError, match="no call accepts"):
            ew.ew_experts_rows(**sizes)
    for n, e, a, rows in ((0, 8, 1, 0), (0, 8, 16, 0), (1, 8, 16, 16), (64, 8, 16, 192),
                          (5, 3, 4, 16), (100, 7, 1, 100), (2, 1024, 1024, 2048)):
        assert ew.ew_experts_rows(n, e, a) == rows
    with pytest.raises(ValueError):
        ew.ew_experts_rows(-1, 8)
    assert ew.ew_experts_sort_workspace(8192, 1024) == 0
    assert ew.ew_experts_sort_workspace(8193, 64) > 0


@every
@matrices
def test_no_rows_is_a_no_op_with_null_pointers(name, t):
    none = {a: None for a in REQUIRED[name].split()}
    if name == "norm_grad":
        none.update(dw=None, db=None)
    if name == "policy":
        return                   # its results are still written (below)
    assert CALLS[name](t, rows=0, **none) == OK


@every
def test_results_of_empty_calls_are_still_written(t):
    assert norm_grad(t, rows=0, ws=None, wsb=0, dx=None, dw=2 + G) == MISALIGNED
    assert policy(t, rows=0, loss=None) == INVALID
    assert policy(t, cols=0, loss=None) == INVALID
    assert policy(t, rows=0, wsb=0) == INVALID
    assert sort(t, entries=0, offsets=None) == INVALID
    if not _gpu_visible():
        assert policy(t, rows=0, logp=None, old=None, adv=None, weights=None) == NO_DEVICE
        assert policy(t, cols=0, logp=None, old=None, adv=None) == NO_DEVICE
        assert policy(t, cols=0, logp=None, old=None, adv=None, as_=0) == NO_DEVICE
        assert sort(t, entries=0, ids=None, slot=None, source=None) == NO_DEVICE
        assert norm_grad(t, rows=0, dy=None, x=None, w=None, mean=None, rstd=None, dx=None, ws=None,
                         wsb=0) == NO_DEVICE
        # the weights' gradients of rows without columns
        assert combine_grad(t, cols=0, dy=None, z=None, dz=None) == NO_DEVICE
        assert combine(t, z=None, z_rows=0) == NO_DEVICE
        assert combine_grad(t, z=None, dz=None, z_rows=0) == NO_DEVICE


@every
def test_no_columns(t):
    assert norm(t, x=None, w=None, y=None, cols=0) == OK
    assert norm_grad(t, dy=None, x=None, mean=None, rstd=None, dx=None, cols=0) == OK
    assert policy_grad(t, logp=None, dlogp=None, cols=0) == OK
    assert gather(t, x=None, out=None, cols=0) == OK
    assert gather(t, x=None, out=None, out_rows=0) == OK
    assert combine(t, z=None, y=None, cols=0) == OK


WIDTH8 = {"ids": 8}
WIDTH4 = {"mean", "rstd", "dw", "db", "logp", "old", "ref", "adv", "loss", "stats", "weights",
          "dloss", "dlogp", "slot", "offsets", "counts", "source", "dweights"}


@every
@each_call
def test_misaligned_pointers(name, t):
    at = defaults(name)
    for arg in (INPUTS[name] + " " + OUTPUTS[name]).split():
        if arg == "mask":
            continue             # bytes
        off = 8 if arg == "ws" else WIDTH8.get(arg, 4 if arg in WIDTH4 or t == "f32" else 2) // 2
        assert CALLS[name](t, **{arg: at[arg] + off}) == MISALIGNED, arg


@every
@each_call
def test_overlaps(name, t):
    at = defaults(name)
    for out in OUTPUTS[name].split():
        for arg in INPUTS[name].split():
            if f"{out}={arg}" not in SAME[name].split():
                assert CALLS[name](t, **{out: at[arg]}) == OVERLAP, (out, arg)
            if arg != "dloss":   # (one value) shifted into it
                assert CALLS[name](t, **{out: at[arg] + (16 if out == "ws" else 4)}) == OVERLAP, (out, arg)
        for other in OUTPUTS[name].split():
            if other != out:
                assert CALLS[name](t, **{out: at[other]}) == OVERLAP, (out, other)


@pytest.mark.skipif(_gpu_visible(), reason="would launch with made-up addresses")
@every
@each_call
def test_exact_aliases_are_allowed(name, t):
    at = defaults(name)
    for pair in SAME[name].split():
        out, arg = pair.split("=")
        assert CALLS[name](t, **{out: at[arg]}) == NO_DEVICE, pair
    if name == "norm":
        assert norm(t, total=C, y=C) == OVERLAP           # both the residual
        assert norm(t, total=C, y=A) == NO_DEVICE
    if name == "policy_grad":
        assert policy_grad(t, as_=0, dlogp=D) == OVERLAP  # advantages a sequence are no matrix
        # the same log probabilities now, then and of the reference
        assert policy_grad(t, old=A, ref=A) == NO_DEVICE
        assert policy_grad(t, old=A, ref=A, dlogp=A) == NO_DEVICE
    if name == "combine_grad":
        assert combine_grad(t, dz=B, dzs=65) == OVERLAP


@every
def test_values_outside_their_range(t):
    for eps in (-1e-9, math.nan, math.inf):
        assert norm(t, eps=eps) == INVALID
    assert norm(t, res=None) == INVALID                   # a total without a residual
    for call in (policy, policy_grad):
        for wrong in ({"low": -0.1}, {"low": math.nan}, {"high": -1e-9}, {"high": math.nan},
                      {"kl": -0.1}, {"kl": math.nan}, {"kl": math.inf}):
            assert call(t, **wrong) == INVALID, wrong
    for wrong in ({"scale": math.nan}, {"scale": math.inf}, {"mean": -1}, {"mean": 3}):
        assert policy(t, **wrong) == INVALID, wrong
    if not _gpu_visible():
        for fine in ({"low": math.inf}, {"high": math.inf}, {"low": 0.0, "high": 0.0},
                     {"low": 1.5}, {"kl": 0.0}):
            assert policy(t, **fine) == NO_DEVICE and policy_grad(t, **fine) == NO_DEVICE
        assert policy(t, scale=-2.0, mean=2) == NO_DEVICE


@every
def test_workspaces_too_small(t):
    need = ew.ew_layernorm_grad_workspace(8, 64)
    assert need == 8 * 2 * 64 * 4
    assert norm_grad(t, wsb=need - 1) == INVALID
    assert norm_grad(t, wsb=need - 1, dw=None) == INVALID
    assert policy(t, wsb=ew.ew_policy_loss_workspace(8, 64) - 1) == INVALID
    assert sort(t, entries=9000, wsb=ew.ew_experts_sort_workspace(9000, 8) - 1) == INVALID
    for f in (ew.ew_layernorm_grad_workspace, ew.ew_policy_loss_workspace):
        assert f(1 << 31, 8) == 0 and f(8, 1 << 31) == 0
    assert ew.ew_experts_sort_workspace(1 << 31, 8) == 0
    assert ew.ew_experts_sort_workspace(8, 1025) == 0


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------

def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_checks_the_layer_norm():
    x, w, r = torch.zeros(4, 16), torch.zeros(16), torch.zeros(4)
    with pytest.raises(TypeError, match="x: .*the operation takes 2-byte"):
        ew.ew_layernorm_bf16(x, w, w, x)
    with pytest.raises(ValueError, match="y: shape"):
        ew.ew_layernorm_f32(BASE, BASE, BASE, torch.zeros(4, 15), rows=4, cols=16)
    with pytest.raises(ValueError, match="a row's elements must be contiguous"):
        ew.ew_layernorm_f32(torch.zeros(16, 4).t(), w, w, x)
    with pytest.raises(ValueError, match="workspace: the call needs"):
        ew.ew_layernorm_grad_f32(BASE, BASE, None, BASE, BASE, BASE, dbias=BASE, rows=4, cols=16)
    with pytest.raises(ValueError, match="workspace: 4 bytes"):
        ew.ew_layernorm_grad_f32(BASE, BASE, None, BASE, BASE, BASE, dweight=BASE, rows=4, cols=16,
                                 workspace=torch.zeros(1))
    for sizes, says in (({"rows": 3}, "covers 3 rows of 16"), ({"cols": 8}, "covers 4 rows of 8")):
        with pytest.raises(ValueError, match=says):
            ew.ew_layernorm_f32(x, w, w, x, **sizes)
        with pytest.raises(ValueError, match=says):
            ew.ew_layernorm_grad_f32(x, x, w, r, r, x, **sizes)
    with pytest.raises(ValueError, match="rows and cols are required"):
        ew.ew_layernorm_f32(BASE, BASE, BASE, BASE)


def test_binding_checks_the_policy_loss():
    p, one = torch.zeros(4, 16), torch.zeros(1)
    ws = torch.zeros(ew.ew_policy_loss_workspace(4, 16), dtype=torch.uint8)
    raw = dict(rows=4, cols=16, stream=0)
    with pytest.raises(ValueError, match="mean: 'token'"):
        ew.ew_policy_loss_f32(p, p, p, one, mean="token", workspace=ws)
    with pytest.raises(ValueError, match="per_token is required"):
        ew.ew_policy_loss_f32(BASE, BASE, BASE, BASE, workspace=BASE, **raw)
    for shape in ((5,), (64,), (16,), (4, 2), (2, 16)):
        with pytest.raises(ValueError, match="advantage: shape .* covers 4 sequences of 16"):
            ew.ew_policy_loss_f32(BASE, BASE, torch.zeros(*shape), BASE, workspace=BASE, **raw)
    with pytest.raises(ValueError, match="advantage: shape"):       # said to be a value a token
        ew.ew_policy_loss_f32(BASE, BASE, torch.zeros(4), BASE, workspace=BASE, per_token=True,
                              **raw)
    for shape in ((4,), (4, 1), (4, 16), (2, 2, 16)):
        with pytest.raises(ValueError, match="advantage: the tensor is on cpu"):
            ew.ew_policy_loss_f32(BASE, BASE, torch.zeros(*shape), BASE, workspace=BASE, **raw)
    with pytest.raises(TypeError, match="mask: .*the operation takes 1-byte"):
        ew.ew_policy_loss_f32(BASE, BASE, BASE, BASE, mask=i32(4, 16), workspace=BASE,
                              per_token=True, **raw)
    with pytest.raises(TypeError, match="logp: .*the operation takes 4-byte"):
        ew.ew_policy_loss_f32(p.bfloat16(), p, p, one, workspace=ws)
    with pytest.raises(ValueError, match="workspace: the call needs"):
        ew.ew_policy_loss_f32(BASE, BASE, BASE, BASE, per_token=False, **raw)
    with pytest.raises(ValueError, match="stats: 2 elements"):
        ew.ew_policy_loss_f32(BASE, BASE, BASE, BASE, stats=torch.zeros(2), workspace=BASE,
                              per_token=False, **raw)
    with pytest.raises(ValueError, match="weights: 3 elements"):
        ew.ew_policy_loss_grad_f32(BASE, BASE, BASE, torch.zeros(3), BASE, per_token=False, **raw)


def test_binding_checks_the_experts():
    ids, x = torch.zeros(6, 2, dtype=torch.int64), torch.zeros(6, 16)
    with pytest.raises(TypeError, match="ids: torch.int32"):
        ew.ew_experts_sort(i32(6, 2), 4, i32(6, 2), i32(5))
    with pytest.raises(ValueError, match="ids: .* on cpu"):
        ew.ew_experts_sort(ids, 4, i32(6, 2), i32(5))
    sizes = dict(entries=12, stream=0)
    with pytest.raises(TypeError, match="slot: torch.int64"):
        ew.ew_experts_sort(BASE, 4, ids, BASE, **sizes)
    with pytest.raises(ValueError, match="offsets: 4 elements, the call covers 5"):
        ew.ew_experts_sort(BASE, 4, BASE, i32(4), **sizes)
    with pytest.raises(ValueError, match="counts: 3 elements, the call covers 4"):
        ew.ew_experts_sort(BASE, 4, BASE, BASE, counts=i32(3), **sizes)
    with pytest.raises(ValueError, match="source: 12 elements, the call covers 80"):
        ew.ew_experts_sort(BASE, 4, BASE, BASE, source=i32(12), align=16, **sizes)
    with pytest.raises(ValueError, match="workspace: the call needs"):
        ew.ew_experts_sort(BASE, 4, BASE, BASE, entries=9000, stream=0)
    move = dict(rows=6, cols=16, stream=0)
    with pytest.raises(ValueError, match="top is required"):
        ew.ew_experts_gather_f32(BASE, BASE, BASE, out_rows=20, **move)
    with pytest.raises(ValueError, match="out_rows is required"):
        ew.ew_experts_gather_f32(BASE, BASE, BASE, top=2, **move)
    with pytest.raises(ValueError, match="slot: shape .* covers 6 rows of 3"):
        ew.ew_experts_gather_f32(BASE, i32(6, 2), BASE, top=3, out_rows=20, **move)
    with pytest.raises(ValueError, match="slot: shape .* covers 6 rows of 2"):
        ew.ew_experts_gather_f32(BASE, i32(5, 2), BASE, out_rows=20, **move)
    with pytest.raises(ValueError, match="offsets and counts: both or neither"):
        ew.ew_experts_gather_f32(BASE, BASE, BASE, top=2, out_rows=20, counts=i32(4), **move)
    with pytest.raises(ValueError, match="experts is required"):
        ew.ew_experts_gather_f32(BASE, BASE, BASE, top=2, out_rows=20, counts=BASE, offsets=BASE,
                                 **move)
    with pytest.raises(ValueError, match="offsets: 4 elements, the call covers 5"):
        ew.ew_experts_gather_f32(BASE, BASE, BASE, top=2, out_rows=20, counts=BASE,
                                 offsets=i32(4), experts=4, **move)
    with pytest.raises(ValueError, match="out: .* the tensor is on cpu|out: the tensor is on cpu"):
        ew.ew_experts_gather_f32(BASE, BASE, torch.zeros(20, 16), top=2, **move)
    with pytest.raises(ValueError, match="z_rows is required"):
        ew.ew_experts_combine_f32(BASE, BASE, BASE, top=2, **move)
    with pytest.raises(ValueError, match="weights: shape .* covers 6 rows of 2"):
        ew.ew_experts_combine_f32(BASE, BASE, BASE, weights=torch.zeros(6, 4), top=2, z_rows=20,
                                  **move)
    with pytest.raises(ValueError, match="y: shape"):
        ew.ew_experts_combine_f32(BASE, BASE, x, top=2, z_rows=20, rows=5, cols=16, stream=0)
    with pytest.raises(ValueError, match="dz: shape .* covers 20 rows of 16"):
        ew.ew_experts_combine_grad_f32(BASE, BASE, BASE, BASE, torch.zeros(19, 16), BASE, top=2,
                                       z_rows=20, **move)
    with pytest.raises(ValueError, match="dweights: shape .* covers 6 rows of 2"):
        ew.ew_experts_combine_grad_f32(BASE, BASE, BASE, BASE, BASE, torch.zeros(6, 3), top=2,
                                       z_rows=20, **move)
