"""float32 calls large enough that memory traffic binds them, against the definitions in float64: all SMs
busy, several rows, segments or tiles for every block, partial sums over many blocks.

Tolerances (relative Frobenius, u = 2^-24): those of the operators' own tests for outputs by row; a sum over n
rows exceeds its result by sqrt(n) and adds in pieces of at most 80 terms: sqrt(n) 80 u."""
import pytest
import torch

from chunkwise_gated_delta_gb300 import layer_norm_bwd, layer_norm_fwd, short_conv_bwd, short_conv_fwd, ssm_scan_bwd, ssm_scan_fwd

from mixer_ref import layer_norm, rel, short_conv, spans_of, ssm_scan

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _sums(n):
    return n ** 0.5 * 80 * U


@pytest.mark.parametrize("rows,D", [(16384, 1024), (16384, 2048), (8191, 4096), (4099, 8192)])
def test_layer_norm(rows, D):
    g = torch.Generator(device=DEV).manual_seed(D)
    x, dy = (torch.randn(rows, D, generator=g, device=DEV) for _ in range(2))
    w, b = 1 + 0.2 * torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV)
    y, mean, rstd = layer_norm_fwd(x, w, b)
    got = layer_norm_bwd(dy, x, w, mean, rstd)
    leaf = [v.double().requires_grad_() for v in (x, w, b)]
    ry, rm, rr = layer_norm(*leaf, 1e-5)
    grads = torch.autograd.grad((ry * dy.double()).sum(), leaf)
    assert rel(y, ry) <= 2e-5 and rel(rstd, rr) <= 2e-5 and float((mean.double() - rm.detach()).abs().max()) <= 2e-5
    for k, r in zip(("dx", "dweight", "dbias"), grads):
        assert rel(got[k], r) <= (2e-5 if k == "dx" else _sums(rows)), k


@pytest.mark.parametrize("B,T,D,W", [(4, 2048, 2048, 4), (3, 2047, 2044, 3)])
def test_short_conv(B, T, D, W):
    g = torch.Generator(device=DEV).manual_seed(W)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dy, w, b, h0 = rn(B, T, D), rn(B, T, D), rn(D, W), rn(D), rn(B, W - 1, D)
    y, ht = short_conv_fwd(x, w, b, h0)
    got = short_conv_bwd(x, w, b, h0, dy)
    leaf = [v.double().requires_grad_() for v in (x, w, b, h0)]
    ry, rht = short_conv(leaf[0].reshape(B * T, D), *leaf[1:], spans_of([T] * B), True)
    grads = torch.autograd.grad((ry * dy.double().reshape(B * T, D)).sum(), leaf)
    assert rel(y.reshape(B * T, D), ry) <= 2.4e-6 and torch.equal(ht.double(), rht)
    for k, r in zip(("dx", "dweight", "dbias", "dh0"), grads):
        assert rel(got[k], r) <= (_sums(B * T) if k in ("dweight", "dbias") else 2.4e-6), k


def test_ssm_scan():
    B, T, D, N = 4, 600, 2560, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    A = -(0.5 + torch.arange(N, device=DEV) + torch.rand(D, N, generator=g, device=DEV))
    names = ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0")
    v = dict(zip(names, (rn(B, T, D), 0.5 * rn(B, T, D), A, rn(B, T, N), rn(B, T, N), rn(D), rn(B, T, D), rn(D) - 2.0, rn(B, D, N))))
    dy, dht = rn(B, T, D), rn(B, D, N)
    y, ht = ssm_scan_fwd(*v.values())
    got = ssm_scan_bwd(*v.values(), dy, dht)
    sums = {k: torch.zeros_like(v[k], dtype=torch.float64) for k in ("A", "D", "delta_bias")}
    for i in range(B):                       # one sequence's graph at a time
        leaf = {k: (t if k in sums else t[i:i + 1] if k == "h0" else t[i]).double().requires_grad_() for k, t in v.items()}
        ry, rht = ssm_scan(*leaf.values(), [(0, T)], True)
        grads = torch.autograd.grad((ry, rht), list(leaf.values()), (dy[i].double(), dht[i:i + 1].double()))
        assert rel(y[i], ry) <= 2.5e-5 and rel(ht[i:i + 1], rht) <= 2.5e-5
        for k, r in zip(names, grads):
            if k in sums:
                sums[k] += r
            else:
                assert rel(got["d" + k][i], r.reshape(got["d" + k][i].shape)) <= 1e-4, k
        del leaf, ry, rht, grads
    for k, r in sums.items():
        assert rel(got["d" + k], r) <= 1e-4 + _sums(B * T), k
