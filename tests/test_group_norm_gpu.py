"""Gated norm over groups on the GPU against its definition in float64: every form (lanes per group, vectors per lane, groups
longer than a warp's registers), weights of each kind, odd widths, strides, infinities."""
import ctypes

import pytest
import torch

import chunkwise_gated_delta_gb300 as lib
from chunkwise_gated_delta_gb300 import _lib
import layer_ref as ref
from mixer_ref import half_step, rel

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


def make(rows, groups, C, dtype, wdt=None, shared=False, gate=True, bias=True, weight=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + rows + groups * C)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    n = C if shared else groups * C
    wdt = wdt or dtype
    return dict(x=(rn(rows, groups * C) * 1.5 + 0.5).to(dtype), weight=(1 + 0.2 * rn(n)).to(wdt) if weight else None,
                bias=(0.2 * rn(n)).to(wdt) if bias else None, gate=rn(rows, groups * C).to(dtype) if gate else None,
                dy=rn(rows, groups * C).to(dtype))


def definition(s, groups, center):
    f = {k: v.double().requires_grad_(k != "dy") for k, v in s.items() if v is not None}
    y, mean, rstd = ref.group_norm(f["x"], groups, f.get("weight"), f.get("bias"), f.get("gate"), EPS, center)
    names = [k for k in ("x", "weight", "bias", "gate") if k in f]
    grads = torch.autograd.grad((y * f["dy"]).sum(), [f[k] for k in names])
    return {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach(), **{"d" + k: v for k, v in zip(names, grads)}}


def call(s, groups, center):
    y, mean, rstd = lib.group_norm_fwd(s["x"], groups, s["weight"], s["bias"], s["gate"], eps=EPS, center=center)
    out = lib.group_norm_bwd(s["dy"], s["x"], groups, s["weight"], s["bias"], s["gate"], mean, rstd)
    return {"y": y, "rstd": rstd, **({"mean": mean} if center else {}), **out}


def check(got, want, rows, C):
    # float32 arithmetic: sums over C columns and over the rows are off by at most (their depth + 16) roundings of terms of about
    # the result's size, of which sqrt would do for independent ones; dx is a difference of terms that are up to 2 / (1 / sqrt(C))
    # of it for the few columns of the narrow groups tested (C >= 3), for which 64 roundings are counted
    f32 = (64 + (C + rows) ** 0.5) * 2.0 ** -24
    assert set(got) <= set(want)
    for k, v in got.items():
        assert rel(v.reshape(want[k].shape), want[k]) <= f32 + (half_step(v.dtype) if v.dtype != torch.float32 else 0), k


FORMS = [(5, 3, 3), (1, 1, 4), (7, 2, 8), (33, 5, 16), (3, 16, 32), (40, 7, 64), (129, 16, 128), (17, 33, 128), (9, 3, 131), (5, 2, 256),
         (6, 4, 257), (4, 3, 512), (5, 1, 1024), (3, 2, 1032), (2, 2, 2048), (3, 1, 2056), (2, 2, 5000), (2000, 1, 20)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,groups,C", FORMS)
def test_forms(rows, groups, C, dtype):
    for k, (center, shared, gate) in enumerate([(True, False, True), (False, True, True), (True, True, False), (False, False, False)]):
        s = make(rows, groups, C, dtype, shared=shared, gate=gate, seed=k)
        check(call(s, groups, center), definition(s, groups, center), rows * (groups if shared else 1), C)


# groups of several warps: their lanes' sums cross them; rows enough for several visits of a block
WIDE = [(700, 1, 512), (3, 5, 520), (9, 3, 1024), (500, 1, 1031), (40, 1, 2048), (500, 2, 1028), (1, 3, 2049), (200, 1, 4096), (7, 2, 4104), (310, 1, 8192),
        (2, 2, 8200), (33, 9, 260)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,groups,C", WIDE)
def test_groups_of_several_warps(rows, groups, C, dtype):
    for k, (center, shared, gate, bias) in enumerate([(True, True, True, True), (False, False, True, False), (True, False, False, False)]):
        s = make(rows, groups, C, dtype, shared=shared, gate=gate, bias=bias, seed=k)
        check(call(s, groups, center), definition(s, groups, center), rows * (groups if shared else 1), C)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_absent_parameters_and_mixed_types(weight, bias):
    for dtype, wdt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        s = make(50, 4, 64, dtype, wdt, weight=weight, bias=bias, shared=True)
        check(call(s, 4, True), definition(s, 4, True), 200, 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides(dtype, shift):
    """Halves of a wider buffer, from an aligned column and from an odd one, in three axes."""
    B, T, G, C = 2, 9, 3, 64
    s = make(B * T, G, C, dtype)
    want = call(s, G, True)
    wide = torch.full((B, T, 4 * G * C + 8), 7.0, device=DEV, dtype=dtype)
    part = lambda k: wide[..., k * G * C + shift:(k + 1) * G * C + shift]  # noqa: E731
    for k, name in enumerate(("x", "gate", "dy")):
        part(k).copy_(s[name].view(B, T, -1))
    y, mean, rstd = lib.group_norm_fwd(part(0), G, s["weight"], s["bias"], part(1), eps=EPS, y=part(3))
    assert rel(y, want["y"].view(B, T, -1).double()) <= 2 * half_step(dtype) and bool((wide[..., 4 * G * C + shift:] == 7).all())
    out = torch.full_like(wide, 5.0)
    grads = dict(dx=out[..., shift:G * C + shift], dgate=out[..., G * C + shift:2 * G * C + shift])
    got = lib.group_norm_bwd(part(2), part(0), G, s["weight"], s["bias"], part(1), mean, rstd, grads=grads)
    for k in ("dx", "dgate", "dweight", "dbias"):
        assert rel(got[k].reshape(want[k].shape), want[k].double()) <= 2 * half_step(dtype) + 1e-5, k
    assert bool((out[..., 2 * G * C + shift:] == 5).all())


@pytest.mark.parametrize("C", [128, 20, 3000])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_infinities_stay_in_their_group(C, bad):
    s = make(11, 3, C, torch.float32)
    clean = call(s, 3, True)
    s["x"][4, C + 1] = bad
    got = call(s, 3, True)
    keep = torch.ones(11, 3, C, dtype=torch.bool, device=DEV)
    keep[4, 1] = False
    for k in ("y", "dx", "dgate"):
        a, b = got[k].view(11, 3, C), clean[k].view(11, 3, C)
        assert torch.equal(a[keep], b[keep]) and not bool(torch.isfinite(a[4, 1]).any() and k == "dx"), k
    out = torch.ones(3, C, dtype=torch.bool, device=DEV)
    out[1] = False
    assert torch.equal(got["dweight"].view(3, C)[out], clean["dweight"].view(3, C)[out])
    assert not bool(torch.isfinite(got["dweight"].view(3, C)[1]).any())


def test_large_offset_cancels_nothing():
    s = make(40, 4, 128, torch.float32)
    s["x"] = (s["x"] * 1e-2 + 100.0).contiguous()
    got, want = call(s, 4, True), definition(s, 4, True)
    # the mean is rounded to half a step of 100 (2^-18 / 2... of 100: 3.8e-6), against deviations of 1.5e-2
    assert rel(got["y"], want["y"]) <= 4 * 3.9e-6 / 1.5e-2


def test_equal_calls_streams_and_graphs():
    s = make(300, 16, 128, torch.bfloat16, shared=True)
    want = call(s, 16, False)
    assert all(torch.equal(v, want[k]) for k, v in call(s, 16, False).items())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _, rstd = lib.group_norm_fwd(s["x"], 16, s["weight"], s["bias"], s["gate"], eps=EPS, center=False, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want["y"]) and torch.equal(rstd, want["rstd"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s, 16, False)
    s["x"].mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    fresh = call(s, 16, False)
    assert all(torch.equal(got[k], fresh[k]) for k in got) and not torch.equal(got["y"], want["y"])


@pytest.mark.parametrize("gate", [False, True])
def test_gradient_of_an_absent_bias(gate):
    """The C call may ask for dbias of a norm without one: the sum of what reaches it."""
    s = make(37, 3, 64, torch.float32, gate=gate, bias=False)
    want = definition({**s, "bias": torch.zeros(192, device=DEV)}, 3, True)
    y, mean, rstd = lib.group_norm_fwd(s["x"], 3, s["weight"], None, s["gate"], eps=EPS)
    out = {k: torch.full_like(s["x"], 7.0) for k in ("dx", "dgate")}
    dw, db = torch.zeros(192, device=DEV), torch.zeros(192, device=DEV)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    a = _lib.GroupNormBwdArgs(37, 3, 64, _lib.KDA_F32, _lib.KDA_F32, _lib.GROUP_NORM_FLAG_CENTER, ptr(s["dy"]), 0, ptr(s["x"]), 0, ptr(s["gate"]), 0,
                              ptr(s["weight"]), None, ptr(mean), ptr(rstd), ptr(out["dx"]), 0, ptr(out["dgate"]) if gate else None, 0,
                              ptr(dw), ptr(db), None, 0)
    n = _lib.load().group_norm_bwd_workspace(ctypes.byref(a))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = ws.data_ptr(), n
    assert _lib.load().group_norm_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    check(dict(dx=out["dx"], dweight=dw, dbias=db), want, 37, 64)


def test_more_groups_than_a_grid_has_rows():
    """Four million groups and more go one by one."""
    groups, C = 4_200_000, 3
    s = make(1, groups, C, torch.float32, shared=True)
    check(call(s, groups, True), definition(s, groups, True), groups, C)


@pytest.mark.parametrize("groups,C", [(4_200_000, 3), (70_000, 1023), (66_000, 2049)])
def test_sums_of_one_sign_over_many_groups(groups, C):
    """One weight for more groups than a grid's second axis has places, every term of dbias the same: a single float32 sum of them would
    stop growing in steps of a term.  The sums here are nested: along any path from a term to the total at most 2^12 additions (a block's
    rows and groups, its slots, then the blocks'), each off by half a step."""
    x = torch.randn(1, groups * C, device=DEV)
    w, b = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    dy = torch.full_like(x, 0.7)
    y, mean, rstd = lib.group_norm_fwd(x, groups, w, b, eps=EPS)
    out = lib.group_norm_bwd(dy, x, groups, w, b, None, mean, rstd)
    want = float(dy[0, 0]) * groups
    assert float((out["dbias"].double() - want).abs().max()) <= 2 ** 12 * 2.0 ** -24 * want
    xh = ((x.view(groups, C).double() - mean.view(groups, 1)) * rstd.view(groups, 1))
    assert rel(y.view(groups, C), xh) <= 8 * 2.0 ** -24
    terms = xh * float(dy[0, 0])
    assert float((out["dweight"].double() - terms.sum(0)).abs().max() / terms.abs().sum(0).max()) <= (2 ** 12 + 8) * 2.0 ** -24


@pytest.mark.parametrize("rows,groups,C", [(2, 4_200_000, 3), (1, 66_000, 520)])
def test_many_groups_with_weights_of_their_own(rows, groups, C):
    s = make(rows, groups, C, torch.bfloat16, torch.float32)
    check(call(s, groups, True), definition(s, groups, True), rows, C)
