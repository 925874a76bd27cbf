"""The gated recurrence, the gated norm over groups and the gated feed-forward product in float64, from their
definitions (torch).  Gradients come from automatic differentiation of these functions."""
import torch


def gated_scan(x, decay, gate, rate, h0, spans, scale):
    """x, decay, gate [rows, D]; h0 [n, D] or None; spans: (first row, end row) of each sequence.  (y [rows, D], ht [n, D]):
    rows of no sequence are 0."""
    log_a = -scale * torch.nn.functional.softplus(rate, threshold=700.0) * torch.sigmoid(decay)
    a, v = torch.exp(log_a), (-torch.expm1(2 * log_a)).sqrt() * torch.sigmoid(gate) * x
    rows, hts = [torch.zeros_like(x[0])] * x.shape[0], []
    for i, (lo, hi) in enumerate(spans):
        h = x.new_zeros(x.shape[1]) if h0 is None else h0[i]
        for t in range(lo, hi):
            h = a[t] * h + v[t]
            rows[t] = h
        hts.append(h)
    return torch.stack(rows), torch.stack(hts)


def group_norm(x, groups, weight, bias, gate, eps, center):
    """x, gate [rows, groups C]; weight, bias [groups C] or [C].  (y, mean, rstd)"""
    v = x.unflatten(-1, (groups, -1))
    mean = v.mean(-1) if center else torch.zeros_like(v[..., 0])
    rstd = (((v - mean[..., None]) ** 2).mean(-1) + eps) ** -0.5
    n = (v - mean[..., None]) * rstd[..., None]
    par = lambda p: p if p.numel() == n.shape[-1] else p.unflatten(0, (groups, -1))  # noqa: E731
    if weight is not None:
        n = n * par(weight)
    if bias is not None:
        n = n + par(bias)
    n = n.flatten(-2)
    if gate is not None:
        n = n * gate * torch.sigmoid(gate)
    return n, mean, rstd


def glu(x, w_gate, w_up, activation):
    g, u = x @ w_gate.T, x @ w_up.T
    act = g * torch.sigmoid(g) if activation == "silu" else g * 0.5 * torch.erfc(-g * 0.5 ** 0.5)
    return act * u, g, u
