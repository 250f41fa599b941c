"""The row operators' argument checks without a GPU: every refusal of the C
entry points and of the binding comes before any HIP call."""
import math

import pytest
import torch

import memory_bound_elementwise_amd as ew
from tests.conftest import _gpu_visible

OK, INVALID, MISALIGNED, OVERLAP, NO_DEVICE = 0, -1, -2, -3, -4
BASE = 0x7F0000000000          # a made-up, 256-byte aligned device address
MiB = 1 << 20
TYPES = ("f32", "f16", "bf16")
A, B, C, D, E, F, G, H, W = (BASE + k * 64 * MiB for k in range(9))
BIG = 1 << 20                  # workspace bytes: more than these calls need


def code(fn, *args):
    return ew._c[fn](*args)


def es(t):
    return 4 if t == "f32" else 2


def norm(t, x=A, xs=64, w=B, res=C, ress=64, y=D, ys=64, total=E, ts=64, rstd=F, rows=8, cols=64,
         eps=1e-5):
    return code("ew_rmsnorm_" + t, x, xs, w, res, ress, y, ys, total, ts, rstd, rows, cols, eps, 0)


def norm8(t, x=A, xs=64, w=B, res=C, ress=64, q=D, qs=64, scales=G, group=32, total=E, ts=64,
          rstd=F, rows=8, cols=64, eps=1e-5):
    return code("ew_rmsnorm_e4m3_" + t, x, xs, w, res, ress, q, qs, scales, group, total, ts, rstd,
                rows, cols, eps, 0)


def norm_grad(t, dy=A, dys=64, x=B, xs=64, w=C, rstd=D, dt=E, dts=64, dx=F, dxs=64, dw=G, ws=W,
              wsb=BIG, rows=8, cols=64):
    return code("ew_rmsnorm_grad_" + t, dy, dys, x, xs, w, rstd, dt, dts, dx, dxs, dw, ws, wsb,
                rows, cols, 0)


def logprobs(t, x=A, xs=64, targets=B, logp=C, entropy=D, lse=E, top_logp=F, top_ids=G, top=5,
             scale=1.0, ws=W, wsb=BIG, rows=8, cols=64):
    return code("ew_logprobs_" + t, x, xs, targets, logp, entropy, lse, top_logp, top_ids, top,
                scale, ws, wsb, rows, cols, 0)


def logprobs_grad(t, x=A, xs=64, targets=B, lse=C, entropy=D, dlogp=E, dentropy=F, dx=G, dxs=64,
                  scale=1.0, rows=8, cols=64):
    return code("ew_logprobs_grad_" + t, x, xs, targets, lse, entropy, dlogp, dentropy, dx, dxs,
                scale, rows, cols, 0)


def distill(t, x=A, xs=64, teacher=B, ids=C, kept=4, loss=D, lse=E, scale=1.0, ws=W, wsb=BIG,
            rows=8, cols=64):
    return code("ew_distill_" + t, x, xs, teacher, ids, kept, loss, lse, scale, ws, wsb, rows,
                cols, 0)


def distill_grad(t, x=A, xs=64, teacher=B, ids=C, kept=4, lse=D, dloss=E, dx=F, dxs=64, scale=1.0,
                 rows=8, cols=64):
    return code("ew_distill_grad_" + t, x, xs, teacher, ids, kept, lse, dloss, dx, dxs, scale,
                rows, cols, 0)


CALLS = {"norm": norm, "norm8": norm8, "norm_grad": norm_grad, "logprobs": logprobs,
         "logprobs_grad": logprobs_grad, "distill": distill, "distill_grad": distill_grad}
REQUIRED = {"norm": "x w y", "norm8": "x w q scales", "norm_grad": "dy x w rstd dx ws",
            "logprobs": "x targets logp top_logp top_ids", "logprobs_grad": "x targets lse entropy dlogp dx",
            "distill": "x teacher ids loss", "distill_grad": "x teacher ids lse dloss dx"}
STRIDES = {"norm": "xs ress ys ts", "norm8": "xs ress qs ts", "norm_grad": "dys xs dts dxs",
           "logprobs": "xs", "logprobs_grad": "xs dxs", "distill": "xs", "distill_grad": "xs dxs"}

every = pytest.mark.parametrize("t", TYPES)
each_call = pytest.mark.parametrize("name", CALLS)


@pytest.mark.skipif(_gpu_visible(), reason="would launch with made-up addresses")
@every
@each_call
def test_a_valid_call_reaches_the_device_check(name, t):
    call = CALLS[name]
    assert call(t) == NO_DEVICE
    # a single row's stride is not used
    assert call(t, rows=1, **{s: 0 for s in STRIDES[name].split()}) == NO_DEVICE


@every
@each_call
def test_null_pointers(name, t):
    for arg in REQUIRED[name].split():
        assert CALLS[name](t, **{arg: None}) == INVALID, arg


@every
@each_call
def test_strides_shorter_than_a_row(name, t):
    for arg in STRIDES[name].split():
        assert CALLS[name](t, **{arg: 63}) == INVALID, arg
        assert CALLS[name](t, **{arg: 1 << 61}) == INVALID, arg


@every
@each_call
def test_sizes_past_the_limits(name, t):
    big = {s: 1 << 31 for s in STRIDES[name].split()}
    assert CALLS[name](t, rows=1 << 31) == INVALID
    assert CALLS[name](t, cols=1 << 31, **big) == INVALID
    # the address range wraps
    first = STRIDES[name].split()[0]
    assert CALLS[name](t, rows=1 << 30, **{first: 1 << 40}) == INVALID


@every
@each_call
def test_no_rows_is_a_no_op_with_null_pointers(name, t):
    none = {a: None for a in REQUIRED[name].split()}
    if name == "norm_grad":
        none["dw"] = None
    assert CALLS[name](t, rows=0, **none) == OK


@every
def test_no_columns(t):
    assert norm(t, x=None, w=None, y=None, cols=0) == OK
    assert norm8(t, x=None, w=None, q=None, scales=None, cols=0) == OK
    assert norm_grad(t, dy=None, x=None, w=None, rstd=None, dx=None, cols=0) == OK
    assert logprobs_grad(t, x=None, dx=None, cols=0) == OK
    assert distill_grad(t, x=None, dx=None, cols=0) == OK
    # the outputs of a row of no logits are still written
    assert logprobs(t, x=None, cols=0, top=0, logp=None) == INVALID
    assert distill(t, x=None, cols=0, loss=None) == INVALID


@every
@each_call
def test_misaligned_pointers(name, t):
    odd = {"norm": {"x": 1, "w": 1, "res": 1, "y": 1, "total": 1, "rstd": 2},
           "norm8": {"x": 1, "w": 1, "res": 1, "scales": 2, "total": 1, "rstd": 2},
           "norm_grad": {"dy": 1, "x": 1, "w": 1, "rstd": 2, "dt": 1, "dx": 1, "dw": 2, "ws": 8},
           "logprobs": {"x": 1, "targets": 4, "logp": 2, "entropy": 2, "lse": 2, "top_logp": 2,
                        "top_ids": 4},
           "logprobs_grad": {"x": 1, "targets": 4, "lse": 2, "entropy": 2, "dlogp": 2,
                             "dentropy": 2, "dx": 1},
           "distill": {"x": 1, "teacher": 2, "ids": 4, "loss": 2, "lse": 2},
           "distill_grad": {"x": 1, "teacher": 2, "ids": 4, "lse": 2, "dloss": 2, "dx": 1}}[name]
    defaults = {k: v for k, v in zip(CALLS[name].__code__.co_varnames[1:],
                                     CALLS[name].__defaults__)}
    for arg, off in odd.items():
        assert CALLS[name](t, **{arg: defaults[arg] + off}) == MISALIGNED, arg


@every
def test_overlaps(t):
    e = es(t)
    row = 64 * e
    assert norm(t, y=A + row) == OVERLAP                    # y partly over x
    assert norm(t, y=E, total=E) == OVERLAP                 # y and total are one
    assert norm(t, y=B) == OVERLAP                          # y over the weight
    assert norm(t, rstd=D) == OVERLAP                       # rstd inside y
    assert norm8(t, q=A) == OVERLAP                         # bytes over x
    assert norm8(t, scales=C) == OVERLAP
    assert norm_grad(t, dx=B + e) == OVERLAP                # dx shifted against x
    assert norm_grad(t, dw=B) == OVERLAP
    assert norm_grad(t, ws=A, dx=F) == OVERLAP              # the workspace over dy
    assert logprobs(t, logp=A) == OVERLAP
    assert logprobs(t, lse=D) == OVERLAP                    # entropy and lse are one
    assert logprobs(t, top_ids=B) == OVERLAP                # over the targets
    assert logprobs_grad(t, dx=A + e) == OVERLAP
    assert logprobs_grad(t, dx=A, dxs=72) == OVERLAP        # other rows of the same buffer
    assert logprobs_grad(t, dx=C) == OVERLAP
    assert distill(t, loss=B) == OVERLAP
    assert distill_grad(t, dx=A + row) == OVERLAP
    assert distill_grad(t, dx=C) == OVERLAP


@pytest.mark.skipif(_gpu_visible(), reason="would launch with made-up addresses")
@every
def test_exact_aliases_and_interleaved_views_are_allowed(t):
    e = es(t)
    assert norm(t, total=A) == NO_DEVICE                    # the residual stream in place
    assert norm(t, total=C, y=A) == NO_DEVICE
    assert norm8(t, total=A) == NO_DEVICE
    for dx in (A, B, E):
        assert norm_grad(t, dx=dx) == NO_DEVICE
    assert logprobs_grad(t, dx=A) == NO_DEVICE
    assert distill_grad(t, dx=A) == NO_DEVICE
    # y is the right half of the buffer whose left half is x
    assert norm(t, x=A, xs=128, y=A + 64 * e, ys=128) == NO_DEVICE
    assert norm(t, x=A + 64 * e, xs=128, y=A, ys=128) == NO_DEVICE
    assert norm(t, x=A, xs=128, y=A + 63 * e, ys=128) == OVERLAP
    assert norm(t, x=A, xs=128, y=A + 65 * e, ys=128) == OVERLAP


@every
def test_values_outside_their_range(t):
    for eps in (-1e-5, math.inf, math.nan):
        assert norm(t, eps=eps) == INVALID
    assert norm(t, res=None) == INVALID                     # a total without a residual
    for group in (1, 8, 48, 100, 512):
        assert norm8(t, group=group) == INVALID
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert logprobs(t, scale=scale) == INVALID
        assert logprobs_grad(t, scale=scale) == INVALID
        assert distill(t, scale=scale) == INVALID
        assert distill_grad(t, scale=scale) == INVALID
    assert logprobs(t, top=65, cols=256, xs=256) == INVALID   # more than a call ranks
    assert logprobs(t, top=9, cols=8) == INVALID              # more than there are
    assert logprobs_grad(t, entropy=None) == INVALID          # needed with dentropy
    assert distill(t, kept=1025) == INVALID
    assert distill_grad(t, kept=1025) == INVALID


@every
def test_workspaces_too_small(t):
    need = ew.ew_rmsnorm_grad_workspace(8, 64)
    assert need > 0
    assert norm_grad(t, wsb=need - 1) == INVALID
    for rows, cols, top in ((8, 1 << 17, 0), (8, 1 << 17, 20), (1, 200000, 64), (4096, 1000, 5)):
        need = ew.ew_logprobs_workspace(rows, cols, top)
        if need:
            assert logprobs(t, rows=rows, cols=cols, xs=cols, top=top, wsb=need - 1) == INVALID
        need = ew.ew_distill_workspace(rows, cols)
        if need:
            assert distill(t, rows=rows, cols=cols, xs=cols, wsb=need - 1) == INVALID


def test_workspace_sizes_of_impossible_calls():
    assert ew.ew_rmsnorm_grad_workspace(1 << 31, 8) == 0
    assert ew.ew_logprobs_workspace(8, 1 << 31, 0) == 0
    assert ew.ew_logprobs_workspace(8, 1000, ew.TOP_MAX + 1) == 0
    assert ew.ew_distill_workspace(1 << 31, 8) == 0


def test_binding_checks_matrices():
    f, h = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float16)
    w, r = torch.zeros(8), torch.zeros(4)
    with pytest.raises(TypeError, match="x: torch.float16 has 2-byte elements"):
        ew.ew_rmsnorm_f32(h, w, f)
    with pytest.raises(TypeError, match="y: torch.float32 has 4-byte elements"):
        ew.ew_rmsnorm_bf16(BASE, BASE, f, rows=4, cols=8)
    with pytest.raises(ValueError, match="shape .* the call covers 4 rows of 8"):
        ew.ew_rmsnorm_f32(BASE, BASE, torch.zeros(4, 9), rows=4, cols=8)
    with pytest.raises(ValueError, match="contiguous"):
        ew.ew_rmsnorm_f32(torch.zeros(8, 4).t(), w, f)
    with pytest.raises(ValueError, match="rows must not overlap"):
        ew.ew_rmsnorm_f32(torch.zeros(1, 8).expand(4, 8), w, f)
    with pytest.raises(ValueError, match="not contiguous"):
        ew.ew_rmsnorm_f32(torch.zeros(2, 2, 16)[:, :, ::2], w, f)
    with pytest.raises(ValueError, match="not on a GPU"):
        ew.ew_rmsnorm_f32(f, w, f)
    with pytest.raises(ValueError, match="rows and cols are required"):
        ew.ew_rmsnorm_f32(BASE, BASE, BASE)
    with pytest.raises(ValueError, match="scalar"):
        ew.ew_rmsnorm_f32(torch.zeros(()), w, f)
    with pytest.raises(ValueError, match="weight: 7 elements, the call covers 8"):
        ew.ew_rmsnorm_f32(BASE, torch.zeros(7), BASE, rows=4, cols=8, stream=0)
    with pytest.raises(ValueError, match="scales: 4 elements, the call covers 8"):
        ew.ew_rmsnorm_e4m3_f32(BASE, BASE, BASE, r, group=16, rows=4, cols=32, stream=0)
    with pytest.raises(ValueError, match="group"):
        ew.ew_rmsnorm_e4m3_f32(BASE, BASE, BASE, r, group=-16, rows=4, cols=32, stream=0)


def test_binding_checks_vocabulary_arguments():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="targets: torch.int32"):
        ew.ew_logprobs_f32(BASE, t, BASE, rows=4, cols=8)
    with pytest.raises(TypeError, match="ids: torch.float64"):
        ew.ew_distill_f32(BASE, BASE, torch.zeros(4, 2, dtype=torch.float64), BASE, rows=4, cols=8)
    with pytest.raises(ValueError, match="targets: 3 elements"):
        ew.ew_logprobs_f32(BASE, torch.zeros(3, dtype=torch.int64), BASE, rows=4, cols=8, top=0)
    with pytest.raises(ValueError, match="top is required"):
        ew.ew_logprobs_f32(BASE, BASE, BASE, top_logp=BASE, top_ids=BASE, rows=4, cols=8)
    with pytest.raises(ValueError, match="kept is required"):
        ew.ew_distill_f32(BASE, BASE, BASE, BASE, rows=4, cols=8)
    with pytest.raises(ValueError, match="workspace: the call needs"):
        ew.ew_rmsnorm_grad_f32(BASE, BASE, BASE, BASE, BASE, BASE, rows=4, cols=8, stream=0)
    with pytest.raises(ValueError, match="workspace: 16 bytes, the call needs"):
        ew.ew_rmsnorm_grad_f32(BASE, BASE, BASE, BASE, BASE, BASE,
                               torch.zeros(16, dtype=torch.uint8), rows=4, cols=8, stream=0)
