"""short_conv_fwd / short_conv_bwd / short_conv_step against the definition in float64.

Tolerances (relative Frobenius), fixed before the first run: one rounding of the
output, half_step(dtype), plus float32 arithmetic: five operations and a SiLU
(exponential and reciprocal of 2 units each, u = 2^-24) on terms whose magnitudes
exceed their sum by a factor of about 2 in the norm: below 40 u = 2.4e-6.  Sums
over tokens (dweight, dbias) exceed the result by the square root of the count
and add in pieces of at most 64 and then 8 partial sums: 1e-4.
"""
import pytest
import torch

from chunkwise_gated_delta_gb300 import short_conv_bwd, short_conv_fwd, short_conv_step

from mixer_ref import half_step, rel, short_conv, spans_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(rows, n, D, W, dtype, seed, h0=True, bias=True, wdtype=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    wd = wdtype or dtype
    return dict(x=rn(rows, D).to(dtype), weight=rn(D, W).to(wd), bias=rn(D).to(wd) if bias else None,
                h0=rn(n, W - 1, D).to(dtype) if h0 else None, dy=rn(rows, D).to(dtype), dht=rn(n, W - 1, D).to(dtype))


def _run(d, B, T, cu, silu, **kw):
    x, dy = d["x"].view(B, T, -1) if d["x"].is_contiguous() else d["x"][None], d["dy"].view(B, T, -1)
    act = "silu" if silu else None
    y, ht = short_conv_fwd(x, d["weight"], d["bias"], d["h0"], activation=act, cu_seqlens=cu)
    got = short_conv_bwd(x, d["weight"], d["bias"], d["h0"], dy, d["dht"], activation=act, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    return y, ht, got


def _check(d, lens, silu, y, ht, got):
    leaf = {k: None if v is None else v.double() for k, v in d.items()}
    names = [k for k in ("x", "weight", "bias", "h0") if leaf[k] is not None]
    for k in names:
        leaf[k].requires_grad_()
    ry, rht = short_conv(leaf["x"], leaf["weight"], leaf["bias"], leaf["h0"], spans_of(lens), silu)
    grads = torch.autograd.grad((ry * leaf["dy"]).sum() + (rht * leaf["dht"]).sum(), [leaf[k] for k in names],
                                allow_unused=True)
    h = half_step(d["x"].dtype)
    assert rel(y.reshape(ry.shape), ry) <= h + 2.4e-6
    assert torch.equal(ht.double(), rht)
    assert set(got) == {"d" + k for k in names}
    for k, r in zip(names, grads):
        r = torch.zeros_like(leaf[k]) if r is None else r
        v = got["d" + k]
        tol = half_step(v.dtype) + (1e-4 if k in ("weight", "bias") else 2.4e-6)
        assert rel(v.reshape(r.shape), r) <= tol, k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,D", [(1, 1, 4), (2, 2, 12), (3, 3, 33), (1, 31, 132), (2, 64, 516), (1, 130, 1024), (2, 333, 40)])
def test_dense(dtype, W, B, T, D):
    d = _inputs(B * T, B, D, W, dtype, seed=B + T + D + W, h0=T % 2 == 1, bias=W != 3)
    _check(d, [T] * B, W != 2, *_run(d, B, T, None, W != 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,lens", [(4, [0]), (4, [1, 0, 2, 3, 0, 1]), (4, [64, 17, 0, 200, 33]), (2, [31, 1, 33, 32]),
                                    (3, [0, 0, 5])])
def test_packed(dtype, W, lens):
    T = max(1, sum(lens))
    d = _inputs(T, len(lens), 68, W, dtype, seed=sum(lens) + W)
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV)
    y, ht, got = _run(d, 1, T, cu, True)
    if sum(lens) == 0:                       # no sequence covers the one row: only the states are defined
        assert torch.equal(ht, d["h0"]) and torch.equal(got["dh0"], d["dht"])
        assert not bool(got["dweight"].any()) and not bool(got["dbias"].any())
        return
    _check(d, lens, True, y, ht, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,D,lens", [(4, 1024, [2000, 2000]), (3, 1032, [1999, 3, 0, 1500, 498]), (2, 1025, [3001, 700]),
                                      (4, 1028, [1, 2500, 2, 1100])])
def test_long_segments(dtype, W, D, lens):
    """Enough rows and channels that a thread walks many tokens of one segment."""
    T = sum(lens)
    d = _inputs(T, len(lens), D, W, dtype, seed=T + W)
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV)
    _check(d, lens, True, *_run(d, 1, T, cu, True))


def test_rows_outside_every_sequence_are_left_alone():
    """Rows past the last offset hold NaN on input and a sentinel on output."""
    d = _inputs(20, 2, 16, 4, torch.float32, seed=1)
    d["x"][13:] = float("nan")
    d["dy"][13:] = float("nan")
    cu = torch.tensor([0, 6, 13], dtype=torch.int32, device=DEV)
    y = torch.full((1, 20, 16), 9.0, device=DEV)
    dx = torch.full((1, 20, 16), 9.0, device=DEV)
    short_conv_fwd(d["x"][None], d["weight"], d["bias"], d["h0"], cu_seqlens=cu, y=y)
    got = short_conv_bwd(d["x"][None], d["weight"], d["bias"], d["h0"], d["dy"][None], d["dht"], cu_seqlens=cu,
                         grads=dict(dx=dx))
    assert bool((y[0, 13:] == 9).all()) and bool((dx[0, 13:] == 9).all())
    assert bool(torch.isfinite(y).all()) and all(bool(torch.isfinite(v).all()) for v in got.values())


def test_prefill_in_pieces_equals_one_call():
    d = _inputs(101, 1, 64, 4, torch.bfloat16, seed=2)
    x = d["x"][None]
    whole, ht = short_conv_fwd(x, d["weight"], d["bias"], d["h0"])
    state, parts = d["h0"], []
    for lo, hi in ((0, 40), (40, 42), (42, 43), (43, 101)):
        y, state = short_conv_fwd(x[:, lo:hi].contiguous(), d["weight"], d["bias"], state)
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, ht)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,D", [(4, 64), (3, 33), (2, 520)])
def test_steps_equal_the_prompt_form(dtype, W, D):
    B, T, S = 3, 7, 8
    d = _inputs(B * T, B, D, W, dtype, seed=3, bias=W != 3)
    x = d["x"].view(B, T, D)
    y, ht = short_conv_fwd(x, d["weight"], d["bias"], d["h0"])
    slots = torch.tensor([6, 0, 3], dtype=torch.int32, device=DEV)
    state = torch.full((S, W - 1, D), 5.0, dtype=dtype, device=DEV)
    state[slots.long()] = d["h0"]
    for t in range(T):
        assert torch.equal(short_conv_step(x[:, t], d["weight"], d["bias"], state, slots=slots), y[:, t])
    assert torch.equal(state[slots.long()], ht)
    rest = [i for i in range(S) if i not in (6, 0, 3)]
    assert bool((state[rest] == 5).all())


def test_padding_requests_change_nothing():
    d = _inputs(4, 4, 24, 4, torch.float32, seed=4)
    state = d["h0"].clone()
    slots = torch.tensor([-1, 2, 4, 1 << 30], dtype=torch.int32, device=DEV)
    y = short_conv_step(d["x"], d["weight"], d["bias"], state, slots=slots)
    assert not bool(y[[0, 2, 3]].any()) and bool(y[1].any())
    assert torch.equal(state[[0, 1, 3]], d["h0"][[0, 1, 3]]) and torch.equal(state[2, 2], d["x"][1])


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 8), (4, 3)])
def test_row_strides_and_alignment(shift, pad):
    D, n = 32, 2
    d = _inputs(50, n, D + pad + shift, 4, torch.bfloat16, seed=5)
    sl = slice(shift, shift + D)
    wide = d["x"].view(n, 25, -1)
    args = (d["weight"][sl].clone(), d["bias"][sl].clone(), d["h0"][..., sl].contiguous())
    dy = d["dy"].view(n, 25, -1)
    one = short_conv_fwd(wide[..., sl], *args)
    two = short_conv_fwd(wide[..., sl].contiguous(), *args)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    buf = torch.full_like(wide, 3.0)
    got = short_conv_bwd(wide[..., sl], *args, dy[..., sl], grads=dict(dx=buf[..., sl]))
    ref = short_conv_bwd(wide[..., sl].contiguous(), *args, dy[..., sl].contiguous())
    assert all(torch.equal(got[k], ref[k]) for k in ref)
    assert bool((buf[..., :shift] == 3).all()) and bool((buf[..., shift + D:] == 3).all())


def test_equal_calls_give_equal_bits():
    d = _inputs(4000, 1, 96, 4, torch.bfloat16, seed=6)
    one, two = (_run(d, 1, 4000, None, True)[2] for _ in range(2))
    assert all(torch.equal(one[k], two[k]) for k in one)


def test_float32_taps_of_bf16_rows():
    d = _inputs(90, 1, 64, 4, torch.bfloat16, seed=7, wdtype=torch.float32)
    _check(d, [90], True, *_run(d, 1, 90, None, True))


def test_offsets_beyond_32_bits():
    ld = 1_200_000_000
    buf = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    d = _inputs(3, 1, 64, 4, torch.bfloat16, seed=8)
    x = buf.as_strided((1, 3, 64), (3 * ld, ld, 1))
    x.copy_(d["x"][None])
    args = (d["weight"], d["bias"], d["h0"])
    assert all(torch.equal(a, b) for a, b in zip(short_conv_fwd(x, *args), short_conv_fwd(d["x"][None], *args)))
    a, b = short_conv_bwd(x, *args, d["dy"][None]), short_conv_bwd(d["x"][None], *args, d["dy"][None])
    assert all(torch.equal(a[k], b[k]) for k in b)


def test_large_values_of_the_activation():
    """SiLU far out: 0 on the left (not NaN), the value itself on the right."""
    x = torch.tensor([[[-200.0, -90.0, 90.0, 200.0]]], device=DEV)
    w = torch.zeros(4, 4, device=DEV)
    w[:, 3] = 1.0
    y, _ = short_conv_fwd(x, w)
    assert torch.equal(y[0, 0, 2:], x[0, 0, 2:]) and float(y[0, 0, :2].abs().max()) <= 1e-35
    got = short_conv_bwd(x, w, None, None, torch.ones_like(x))
    assert torch.equal(got["dx"][0, 0, 2:], torch.ones(2, device=DEV)) and float(got["dx"][0, 0, :2].abs().max()) <= 1e-35
