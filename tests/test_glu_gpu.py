"""Gated feed-forward product on the GPU against its definition in float64: sizes that end inside every tile, one row to many,
strides, both activations, saved and recomputed products."""
import ctypes
import math

import pytest
import torch

import chunkwise_gated_delta_gb300 as lib
from chunkwise_gated_delta_gb300 import _lib
import layer_ref as ref
from mixer_ref import half_step, rel

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(M, D, F, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + M + 3 * D + 7 * F)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=rn(M, D).to(dtype), wg=(rn(F, D) / math.sqrt(D)).to(dtype), wu=(rn(F, D) / math.sqrt(D)).to(dtype), dh=rn(M, F).to(dtype))


def definition(s, activation):
    f = {k: v.double().requires_grad_(k != "dh") for k, v in s.items()}
    h, g, u = ref.glu(f["x"], f["wg"], f["wu"], activation)
    dx, dg, du = torch.autograd.grad((h * f["dh"]).sum(), [f["x"], f["wg"], f["wu"]])
    return dict(h=h.detach(), g=g.detach(), u=u.detach(), dx=dx, dw_gate=dg, dw_up=du)


def tol(name, dtype, depth):
    """Products in float32: each sum of `depth` terms is off by about sqrt(depth) roundings of its terms, at most the sum's size
    here (16 counted twice over); h, dx and the weights' gradients are rounded to dtype, the last three from dg and du rounded too."""
    f32 = (32 + 4 * math.sqrt(depth)) * 2.0 ** -24
    if dtype == torch.float32 or name in ("g", "u"):
        return f32
    return f32 + half_step(dtype) * (1 if name == "h" else 2)


def check(got, want, dtype, M, D, F):
    for k, v in got.items():
        assert v.dtype == (torch.float32 if k in ("g", "u") else dtype)
        assert rel(v, want[k]) <= tol(k, dtype, max(M, D, F)), (k, rel(v, want[k]))


def call(s, activation="silu", save=True):
    h, g, u = lib.glu_fwd(s["x"], s["wg"], s["wu"], activation=activation, save=True)
    kept = (g, u) if save else (None, None)
    return dict(h=h, g=g, u=u, **lib.glu_bwd(s["x"], s["wg"], s["wu"], s["dh"], *kept, activation=activation))


SIZES = [(1, 1, 1), (1, 64, 128), (2, 8, 8), (3, 40, 72), (8, 128, 64), (9, 256, 136), (16, 512, 264), (17, 72, 520), (33, 136, 128),
         (64, 256, 256), (65, 200, 136), (127, 64, 264), (128, 128, 128), (129, 264, 520), (300, 72, 1000), (257, 513, 129), (70, 517, 1031),
         (1, 517, 1031), (5, 9, 1000), (512, 512, 512), (1000, 24, 40), (20, 264, 2051), (3000, 72, 40)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_sizes(M, D, F, dtype):
    s = make(M, D, F, dtype)
    want = definition(s, "silu")
    got = call(s)
    check(got, want, dtype, M, D, F)
    assert torch.equal(got["h"], lib.glu_fwd(s["x"], s["wg"], s["wu"]))
    check(call(s, save=False), want, dtype, M, D, F)


@pytest.mark.parametrize("M,D,F", [(130, 70, 518), (20, 266, 1030), (301, 1182, 98), (3, 34, 2), (1027, 130, 66)])
def test_even_widths_in_bfloat16(M, D, F):
    """Rows of whole pairs, but not of 16 bytes: operands that move and outputs that leave by pairs."""
    s = make(M, D, F, torch.bfloat16)
    want = definition(s, "silu")
    check(call(s), want, torch.bfloat16, M, D, F)
    check(call(s, save=False), want, torch.bfloat16, M, D, F)


@pytest.mark.parametrize("M,D,F", [(2142, 16, 8320), (1500, 1411, 130), (700, 3000, 2051)])
def test_many_tiles_in_float32(M, D, F):
    s = make(M, D, F, torch.float32)
    want = definition(s, "silu")
    check(call(s), want, torch.float32, M, D, F)
    check(call(s, save=False), want, torch.float32, M, D, F)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_gelu(M, dtype):
    s = make(M, 96, 160, dtype, seed=2)
    want = definition(s, "gelu")
    check(call(s, "gelu"), want, dtype, M, 96, 160)
    check(call(s, "gelu", save=False), want, dtype, M, 96, 160)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,shift,pad", [(6, 0, 8), (6, 1, 9), (150, 0, 8), (150, 1, 9), (150, 0, 1), (6, 2, 10), (150, 2, 10), (50, 4, 14)])
def test_strides(M, shift, pad, dtype):
    """Inputs and outputs inside wider buffers, from aligned columns and from odd ones; three axes."""
    D, F = 136, 264
    s = make(M, D, F, dtype)
    inside = lambda rows, cols, v=7.0: torch.full((rows, cols + pad), v, device=DEV, dtype=dtype)[:, shift:shift + cols]  # noqa: E731
    v = {}
    for k, t in s.items():
        v[k] = inside(*t.shape)
        v[k].copy_(t)
    x3, dh3 = v["x"].unflatten(0, (2, M // 2)), v["dh"].unflatten(0, (2, M // 2))
    want = definition(s, "silu")
    h = inside(M, F)
    got, g, u = lib.glu_fwd(x3, v["wg"], v["wu"], save=True, y=h.unflatten(0, (2, M // 2)))
    assert got.data_ptr() == h.data_ptr() and bool((h._base[:, shift + F:] == 7).all()) and bool((h._base[:, :shift] == 7).all())
    grads = dict(dx=inside(M, D).unflatten(0, (2, M // 2)), dw_gate=inside(F, D), dw_up=inside(F, D))
    out = lib.glu_bwd(x3, v["wg"], v["wu"], dh3, g, u, grads=grads)
    check(dict(h=h, dx=out["dx"].flatten(0, 1), dw_gate=out["dw_gate"], dw_up=out["dw_up"]), want, dtype, M, D, F)
    for t in out.values():
        assert bool((t._base[:, shift + D:] == 7).all()) and bool((t._base[:, :shift] == 7).all())


def test_infinities_stay_in_their_row():
    s = make(140, 64, 130, torch.bfloat16)
    clean = lib.glu_fwd(s["x"], s["wg"], s["wu"])
    s["x"][77, 3] = float("nan")
    got = lib.glu_fwd(s["x"], s["wg"], s["wu"])
    keep = torch.arange(140, device=DEV) != 77
    assert torch.equal(got[keep], clean[keep]) and bool(torch.isnan(got[77]).all())


def test_gradients_against_differences():
    s = make(7, 5, 6, torch.float32)
    got = call(s)

    def loss(k, e):
        t = {n: v.double() for n, v in s.items()}
        t[k] = t[k] + e
        return float((ref.glu(t["x"], t["wg"], t["wu"], "silu")[0] * t["dh"]).sum())
    for k, name in (("x", "dx"), ("wg", "dw_gate"), ("wu", "dw_up")):
        d = torch.randn(s[k].shape, device=DEV, dtype=torch.float64)
        diff = (loss(k, 1e-5 * d) - loss(k, -1e-5 * d)) / 2e-5
        size = float((got[name].double() * d).abs().sum())
        assert abs(float((got[name].double() * d).sum()) - diff) <= tol(name, torch.float32, 7) * size, k


@pytest.mark.parametrize("M", [4, 200])
def test_equal_calls_streams_and_graphs(M):
    s = make(M, 256, 384, torch.bfloat16)
    want = call(s)
    assert all(torch.equal(v, want[k]) for k, v in call(s).items())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = lib.glu_fwd(s["x"], s["wg"], s["wu"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want["h"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s)
    s["x"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    fresh = call(s)
    assert all(torch.equal(got[k], fresh[k]) for k in got) and not torch.equal(got["h"], want["h"])


@pytest.mark.parametrize("M", [100, 700])
def test_a_wait_that_runs_out(M):
    """A budget of one poll is too small for the waits of a real launch: the call ends, says so, and leaves NaN in what it did not
    finish; the next one is unharmed.  One CTA alone, and pairs."""
    s = make(M, 512, 640, torch.bfloat16)
    want = call(s)
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)
    status.view(torch.int32)[7] = 1
    h, g, u = lib.glu_fwd(s["x"], s["wg"], s["wu"], save=True, status=status)
    assert lib.status_read(status) == _lib.KDA_ERR_TIMEOUT
    assert bool(torch.isnan(h).any()) and bool(torch.isnan(g).any()) and lib.status_read(status) == 0
    for kept in ((want["g"], want["u"]), (None, None)):
        out = lib.glu_bwd(s["x"], s["wg"], s["wu"], s["dh"], *kept, status=status)
        assert lib.status_read(status) == _lib.KDA_ERR_TIMEOUT
        assert all(bool(torch.isnan(v).any()) for v in out.values())
    status.zero_()
    h, g, u = lib.glu_fwd(s["x"], s["wg"], s["wu"], save=True, status=status)
    got = dict(h=h, g=g, u=u, **lib.glu_bwd(s["x"], s["wg"], s["wu"], s["dh"], g, u, status=status))
    assert lib.status_read(status) == 0 and all(torch.equal(got[k], want[k]) for k in want)


def test_workspaces_need_no_more_than_16_bytes():
    """Sums of parts of a product (few tiles, a long K) and the products' gradients in a workspace that begins off 32 bytes."""
    M, D, F = 40, 264, 4104
    s = make(M, D, F, torch.bfloat16)
    want = definition(s, "silu")
    out = dict(dx=torch.empty(M, D, device=DEV, dtype=torch.bfloat16), dw_gate=torch.empty(F, D, device=DEV, dtype=torch.bfloat16),
               dw_up=torch.empty(F, D, device=DEV, dtype=torch.bfloat16))
    a = _lib.GluBwdArgs(M, D, F, _lib.KDA_BF16, 0, s["x"].data_ptr(), 0, s["wg"].data_ptr(), 0, s["wu"].data_ptr(), 0, s["dh"].data_ptr(), 0, None, None,
                        out["dx"].data_ptr(), 0, out["dw_gate"].data_ptr(), 0, out["dw_up"].data_ptr(), 0, None, 0, None)
    n = _lib.load().glu_bwd_workspace(ctypes.byref(a))
    assert n > 2 * M * F * 2
    ws = torch.empty(n + 64, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = ws.data_ptr() + 16, n
    assert _lib.load().glu_bwd(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    check(out, want, torch.bfloat16, M, D, F)


@pytest.mark.parametrize("M,D,F", [(4096, 64, 8192), (4096, 4096, 2048), (100, 64, 70000)])
def test_a_wait_that_runs_out_with_many_tiles_to_a_worker(M, D, F):
    """Whatever was not finished is NaN: every element of every output is, or it is what an undisturbed call gives."""
    s = make(M, D, F, torch.bfloat16)
    want = call(s)
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)
    status.view(torch.int32)[7] = 1
    same = lambda a, b: bool((torch.isnan(a) | (a == b)).all())  # noqa: E731
    for _ in range(3):
        h, g, u = lib.glu_fwd(s["x"], s["wg"], s["wu"], save=True, status=status)
        assert lib.status_read(status) == _lib.KDA_ERR_TIMEOUT
        for k, v in dict(h=h, g=g, u=u).items():
            assert same(v, want[k]) and bool(torch.isnan(v).any()), k
        for kept in ((want["g"], want["u"]), (None, None)):
            out = lib.glu_bwd(s["x"], s["wg"], s["wu"], s["dh"], *kept, status=status)
            assert lib.status_read(status) == _lib.KDA_ERR_TIMEOUT
            for k, v in out.items():
                assert same(v, want[k]), k
