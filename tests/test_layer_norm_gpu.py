"""layer_norm_fwd / layer_norm_bwd against the definition in float64.

Tolerances (relative Frobenius), fixed before the first run: one rounding of the
output, half_step(dtype), plus the float32 arithmetic.  Each float32 operation is
off by at most u = 2^-24 relative to its result; a sum of D terms held in pieces
of at most 64 (a thread's share, then two tree levels) adds at most 80 u of the
sum of magnitudes, which for rows of mean m and deviation s is D |m|-like: the
offsets below are at most 4 s, so mean and xh are off by at most 4 * 80 u < 2e-5
of s.  Sums over rows (dweight, dbias) add up to `rows` terms in pieces; their
magnitude exceeds the result by the square root of the count: 1e-4.
"""
import pytest
import torch

from chunkwise_gated_delta_gb300 import layer_norm_bwd, layer_norm_fwd

from mixer_ref import half_step, layer_norm, rel

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(rows, D, dtype, seed, wdtype=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = (rn(rows, D) + 4 * torch.rand(rows, 1, generator=g, device=DEV)).to(dtype)
    w, b = (1 + 0.2 * rn(D)).to(wdtype or dtype), rn(D).to(wdtype or dtype)
    return x, w, b, rn(rows, D).to(dtype)


def _check(x, w, b, dy, eps=1e-5, **outs):
    y, mean, rstd = layer_norm_fwd(x, w, b, eps=eps)
    got = layer_norm_bwd(dy, x, w, mean, rstd, bias=b is not None, **outs)
    torch.cuda.synchronize()
    leaf = [None if t is None else t.double().requires_grad_() for t in (x, w, b)]
    ry, rm, rr = layer_norm(*leaf, eps)
    used = [t for t in leaf if t is not None]
    grads = dict(zip([n for n, t in zip(("dx", "dweight", "dbias"), leaf) if t is not None],
                     torch.autograd.grad((ry * dy.double()).sum(), used)))
    h = half_step(x.dtype)
    assert rel(y, ry) <= h + 2e-5
    rm = rm.detach()
    assert float((mean.double() - rm).abs().max()) <= 2e-5 * max(1.0, float(rm.abs().max()))
    assert rel(rstd, rr) <= 2e-5
    assert set(got) == set(grads)
    for k, r in grads.items():
        hk = h if k == "dx" else half_step(got[k].dtype)
        assert rel(got[k], r) <= hk + (2e-5 if k == "dx" else 1e-4), k
    return y, got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 8), (3, 1), (5, 7), (37, 64), (700, 96), (2, 2051), (129, 1000), (1300, 2048), (9, 4096),
                                    (5, 8200), (3, 16384), (2, 20001), (1, 40000), (2000, 1000), (1301, 3080), (900, 8000), (400, 16390)])
def test_against_the_definition(dtype, rows, D):
    _check(*_inputs(rows, D, dtype, seed=rows + D), eps=1e-5 if D > 1 else 1e-3)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_optional_parameters(weight, bias):
    x, w, b, dy = _inputs(40, 200, torch.float32, 3)
    _check(x, w if weight else None, b if bias else None, dy)


def test_float32_parameters_of_bf16_rows():
    x, w, b, dy = _inputs(300, 512, torch.bfloat16, 4, wdtype=torch.float32)
    _, got = _check(x, w, b, dy)
    assert got["dweight"].dtype == torch.float32


@pytest.mark.parametrize("D,pad,shift", [(64, 8, 0), (64, 3, 1), (65, 7, 2)])
def test_row_strides_and_alignment(D, pad, shift):
    x, w, b, dy = _inputs(33, D + pad, torch.bfloat16, 5)
    sl = slice(shift, shift + D)
    xs, dys = x[:, sl], dy[:, sl]
    y, _ = _check(xs, w[:D].clone(), b[:D].clone(), dys)
    buf = torch.full((33, D + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    layer_norm_fwd(xs, w[:D].clone(), b[:D].clone(), y=buf[:, sl])
    assert torch.equal(buf[:, sl], y)
    assert bool((buf[:, :shift] == 7).all()) and bool((buf[:, shift + D:] == 7).all())


def test_three_axes_and_one_row():
    x, w, b, dy = _inputs(24, 48, torch.float32, 6)
    y, mean, _ = layer_norm_fwd(x.view(2, 12, 48), w, b)
    y2, mean2, _ = layer_norm_fwd(x, w, b)
    assert torch.equal(y.view(24, 48), y2) and torch.equal(mean.view(-1), mean2)
    y3, _, _ = layer_norm_fwd(x[0], w, b)
    assert torch.equal(y3, y2[0])


def test_large_offset_keeps_the_variance():
    """A common offset 2^11 times the deviation.  A thread's 32 terms add up to 2^16 and are off by
    at most 2^-8 at each step, so the mean is off by at most 32 * 2^-8 / 64 < 2^-9 of the deviation at
    the very worst (all roundings to one side) and y with it; the sum of squares in one pass would
    lose 22 of 24 bits."""
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.randn(16, 1024, generator=g, device=DEV) + 2048.0
    y, _, rstd = layer_norm_fwd(x)
    ry, _, rr = layer_norm(x.double(), None, None, 1e-5)
    assert rel(y, ry) <= 2.0 ** -9 and rel(rstd, rr) <= 2.0 ** -9


def test_constant_rows_and_special_values():
    x = torch.full((4, 256), 3.0, device=DEV)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    w, b = torch.ones(256, device=DEV), torch.full((256,), 0.5, device=DEV)
    y, mean, rstd = layer_norm_fwd(x, w, b)
    assert bool((y[0] == 0.5).all()) and bool((y[3] == 0.5).all())     # a row without variance gives the bias
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all())       # the definition's values, in their rows alone
    got = layer_norm_bwd(torch.ones_like(x), x, w, mean, rstd)
    assert bool(torch.isfinite(got["dx"][[0, 3]]).all())


def test_equal_calls_give_equal_bits():
    x, w, b, dy = _inputs(5000, 384, torch.bfloat16, 8)
    _, mean, rstd = layer_norm_fwd(x, w, b)
    one, two = (layer_norm_bwd(dy, x, w, mean, rstd) for _ in range(2))
    assert all(torch.equal(one[k], two[k]) for k in one)


def test_offsets_beyond_32_bits():
    ld = 1_200_000_000                       # row 2 begins past element 2^31
    buf = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 64), (ld, 1))
    src, w, b, dy = _inputs(3, 64, torch.bfloat16, 9)
    x.copy_(src)
    y, mean, rstd = layer_norm_fwd(x, w, b)
    y2, mean2, rstd2 = layer_norm_fwd(src, w, b)
    assert torch.equal(y, y2) and torch.equal(mean, mean2)
    a, c = layer_norm_bwd(dy, x, w, mean, rstd), layer_norm_bwd(dy, src, w, mean2, rstd2)
    assert all(torch.equal(a[k], c[k]) for k in a)
