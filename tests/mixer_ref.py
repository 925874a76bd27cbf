"""The operators of include/mixer.h in float64, from their definitions (torch, token by token).

Gradients come from automatic differentiation of these functions.  Sequences are
given as a list of (first row, end row) of a [rows, ...] tensor.
"""
import torch


def layer_norm(x, weight, bias, eps):
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    rstd = (var + eps) ** -0.5
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def short_conv(x, weight, bias, h0, spans, silu):
    """x [rows, D]; h0 [n, W-1, D] or None.  (y [rows, D], ht [n, W-1, D])"""
    W, D = weight.shape[1], x.shape[1]
    ys, hts = [], []
    for i, (lo, hi) in enumerate(spans):
        front = x.new_zeros(W - 1, D) if h0 is None else h0[i]
        ext = torch.cat([front, x[lo:hi]])
        n = hi - lo
        pre = sum(ext[j:j + n] * weight[:, j] for j in range(W))
        if bias is not None:
            pre = pre + bias
        ys.append(pre * torch.sigmoid(pre) if silu else pre)
        hts.append(ext[n:])
    return torch.cat(ys), torch.stack(hts)


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def ssm_scan(x, delta, A, B, C, D, z, delta_bias, h0, spans, use_softplus):
    """x, delta, z [rows, D]; B, C [rows, N].  (y [rows, D], ht [n, D, N])"""
    dt = delta if delta_bias is None else delta + delta_bias
    if use_softplus:
        dt = softplus(dt)
    ys, hts = [], []
    for i, (lo, hi) in enumerate(spans):
        h = x.new_zeros(A.shape) if h0 is None else h0[i]
        for t in range(lo, hi):
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * B[t]
            ys.append((h * C[t]).sum(-1))
        hts.append(h)
    y = torch.stack(ys) if ys else x.new_zeros(0, x.shape[1])
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, torch.stack(hts)


def spans_of(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rel(got, ref):
    """Relative Frobenius error (absolute where the reference is zero)."""
    ref = ref.detach().double()
    n = float(ref.norm())
    return float((got.double() - ref).norm()) / (n if n else 1.0)
