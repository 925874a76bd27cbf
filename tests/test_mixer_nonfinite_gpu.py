"""Infinities and NaN through the operators of include/mixer.h: an output is finite where the definition
(float64, automatic differentiation for the gradients) is finite, and within the operators' tolerances
there; where the definition has an infinity or a NaN, so has the output.  The places are the ones
where a kernel's padding or look-ahead could spread a value: last rows, last tokens, tiles' ends.

Tolerances (relative to the largest finite value of an output, fixed before the first run): those of the
operators' own tests, the output's rounding half_step(dtype) and 1e-4 for the longest sums."""
import pytest
import torch

from chunkwise_gated_delta_gb300 import layer_norm_bwd, layer_norm_fwd, short_conv_bwd, short_conv_fwd, ssm_scan_bwd, ssm_scan_fwd

from mixer_ref import half_step, layer_norm, short_conv, spans_of, ssm_scan

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


def _rand(seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return rn, lambda *s: rn(*s).to(dtype)  # noqa: E731


def _alike(got, ref, what):
    ref = ref.detach().double().reshape(got.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), (what, "not finite at", (torch.isfinite(got) != fin).nonzero()[:4].tolist())
    if bool(fin.any()):
        scale = float(ref[fin].abs().max())
        tol = (half_step(got.dtype) if got.dtype == torch.bfloat16 else 0.0) + 1e-4
        assert float((got.double()[fin] - ref[fin]).abs().max()) <= tol * scale, what


# ------------------------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(77, 64), (1301, 96), (1301, 1000), (701, 4096), (1301, 77), (303, 20001)])
@pytest.mark.parametrize("value", [INF, NAN])
def test_norm_backward_of_a_last_row(dtype, rows, D, value):
    """The infinity of one dy in the last row: an infinity in that column of dweight and dbias, nothing elsewhere."""
    rn, t = _rand(rows + D, dtype)
    x, w, b, dy = t(rows, D), t(D), t(D), t(rows, D)
    dy[-1, 5] = value
    _, mean, rstd = layer_norm_fwd(x, w, b)
    got = layer_norm_bwd(dy, x, w, mean, rstd)
    xh, _, _ = layer_norm(x.double(), None, None, 1e-5)
    _alike(got["dbias"], dy.double().sum(0), "dbias")
    _alike(got["dweight"], (dy.double() * xh).sum(0), "dweight")
    if value == INF:
        assert float(got["dbias"][5]) == INF
        assert float(got["dweight"][5]) == INF * (1 if float(xh[-1, 5]) > 0 else -1)
    assert bool(torch.isfinite(got["dx"][:-1]).all()) and not bool(torch.isfinite(got["dx"][-1]).any())


# ------------------------------------------------------------------------------------ convolution
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 37])
@pytest.mark.parametrize("which,value", [("x", INF), ("x", NAN), ("dy", INF), ("dy", NAN), ("h0", NAN), ("dht", INF)])
@pytest.mark.parametrize("at", ["first", "last", "inside"])
def test_conv(dtype, D, which, value, at):
    W, lens = 4, [5, 0, 70, 1, 41]
    rn, t = _rand(3, dtype)
    T, n = sum(lens), len(lens)
    d = dict(x=t(T, D), weight=t(D, W), bias=t(D), h0=t(n, W - 1, D), dy=t(T, D), dht=t(n, W - 1, D))
    lo, hi = spans_of(lens)[2]
    row = {"first": lo, "last": hi - 1, "inside": lo + 33}[at]
    if which in ("h0", "dht"):
        d[which][2, {"first": 0, "inside": 1, "last": 2}[at], 7] = value
    else:
        d[which][row, 7] = value
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV)
    y, ht = short_conv_fwd(d["x"][None], d["weight"], d["bias"], d["h0"], cu_seqlens=cu)
    got = short_conv_bwd(d["x"][None], d["weight"], d["bias"], d["h0"], d["dy"][None], d["dht"], cu_seqlens=cu)
    leaf = {k: v.double() for k, v in d.items()}
    names = ("x", "weight", "bias", "h0")
    for k in names:
        leaf[k].requires_grad_()
    ry, rht = short_conv(leaf["x"], leaf["weight"], leaf["bias"], leaf["h0"], spans_of(lens), True)
    # a gradient from each output on its own: nothing of autograd's zeros meets an infinity
    grads = torch.autograd.grad((ry, rht), [leaf[k] for k in names], (leaf["dy"], leaf["dht"]))
    _alike(y, ry, "y")
    _alike(ht, rht, "ht")
    for k, r in zip(names, grads):
        _alike(got["d" + k], r, "d" + k)


# ------------------------------------------------------------------------------------ scan
NAMES = ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0")


def _scan_inputs(lens, D, N, dtype, seed):
    rn, t = _rand(seed, dtype)
    T, n = sum(lens), len(lens)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    d = dict(x=t(T, D), delta=t(T, D), A=-(0.5 + torch.arange(N, device=DEV) + torch.rand(D, N, generator=g, device=DEV)), B=t(T, N),
             C=t(T, N), D=rn(D), z=t(T, D), delta_bias=rn(D) - 2.0, h0=rn(n, D, N))
    return d, t(T, D), rn(n, D, N)


def _scan_check(d, dy, dht, lens, grads=True):
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV) if len(lens) > 1 else None
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    y, ht = ssm_scan_fwd(*v, cu_seqlens=cu)
    leaf = {k: d[k].double() for k in NAMES}
    if grads:
        for k in NAMES:
            leaf[k].requires_grad_()
    ry, rht = ssm_scan(*(leaf[k] for k in NAMES), spans_of(lens), True)
    _alike(y, ry, "y")
    _alike(ht, rht, "ht")
    if grads:
        got = ssm_scan_bwd(*v, dy[None], dht, cu_seqlens=cu)
        for k, r in zip(NAMES, torch.autograd.grad((ry, rht), [leaf[k] for k in NAMES], (dy.double(), dht.double()))):
            _alike(got["d" + k], r, "d" + k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,N", [(64, 16), (37, 5), (32, 32)])
@pytest.mark.parametrize("which,value", [("x", INF), ("x", NAN), ("B", INF), ("B", NAN), ("C", INF), ("delta", NAN), ("z", NAN), ("dy", INF),
                                         ("dy", NAN)])
@pytest.mark.parametrize("at", ["last", "inside"])
def test_scan_of_packed_sequences(dtype, D, N, which, value, at):
    lens = [9, 0, 70, 1, 33]
    d, dy, dht = _scan_inputs(lens, D, N, dtype, 5)
    lo, hi = spans_of(lens)[2]
    row = hi - 1 if at == "last" else lo + 40
    (dy if which == "dy" else d[which])[row, 3] = value
    _scan_check(d, dy, dht, lens)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,N,T", [(64, 16, 33), (64, 16, 64), (37, 5, 50), (64, 8, 1100), (1704, 16, 45)])
def test_scan_ends_with_an_infinite_input(dtype, D, N, T):
    """B of the last token: one state of every channel ends infinite, not NaN."""
    d, dy, dht = _scan_inputs([T], D, N, dtype, 6)
    d["B"][-1, 2] = INF
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    _, ht = ssm_scan_fwd(*v)
    assert bool(torch.isinf(ht[0, :, 2]).all())
    assert torch.equal(torch.sign(ht[0, :, 2]), torch.sign(d["x"][-1].float()))
    _scan_check(d, dy, dht, [T], grads=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,N,lens", [(64, 16, [33]), (64, 16, [64]), (37, 5, [9, 0, 50]), (64, 8, [1100]), (64, 16, [1030, 0, 300]), (8, 4, [7])])
def test_states_without_memory(dtype, D, N, lens):
    """A of minus infinity: the state is its last input alone, also where a tile's or a batch of segments'
    end is filled up."""
    d, dy, dht = _scan_inputs(lens, D, N, dtype, 7)
    d["A"][:, 1] = -INF
    _scan_check(d, dy, dht, lens, grads=False)
    # the gradients that do not go through A itself: ddelta and dA have the definition's infinity times 0
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV) if len(lens) > 1 else None
    got = ssm_scan_bwd(*v, dy[None], dht, cu_seqlens=cu)
    leaf = {k: d[k].double() for k in NAMES}
    names = ("x", "B", "C", "D", "z", "h0")
    for k in names:
        leaf[k].requires_grad_()
    ry, rht = ssm_scan(*(leaf[k] for k in NAMES), spans_of(lens), True)
    for k, r in zip(names, torch.autograd.grad((ry, rht), [leaf[k] for k in names], (dy.double(), dht.double()))):
        _alike(got["d" + k], r, "d" + k)
