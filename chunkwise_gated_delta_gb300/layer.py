"""Python binding of include/mixer.h, second part: the gated recurrence, the gated norm over a mixer's heads and
the gated feed-forward product.

Conventions are those of :mod:`.mixer`: sequence tensors with rows that may lie apart, packed batches by
``cu_seqlens``, outputs and workspaces allocated on the stream of the call, no CPU path.
"""
from __future__ import annotations

import torch

from . import _lib
from .mixer import _CODES, _On, _check, _code, _cuda, _dense_out, _known, _out, _rows, _sequences, _tensor

_F32 = torch.float32


# -------------------------------------------------------------------------------- gated recurrence
def _gated_inputs(x, decay, gate, rate, scale, dims):
    """Checks the inputs that the recurrence's calls share; pointers and strides in the C order."""
    dev = _cuda(x, "x")
    if x.dim() != dims:
        raise ValueError("x must be [B, T, D]" if dims == 3 else "x must be [B, D]")
    if not (scale > 0.0 and scale <= 3e38):
        raise ValueError("scale must be positive and finite")
    code = _code(x, "x")
    ptrs = [*_rows(x, "x", x.shape, x.dtype, dev), *_rows(decay, "decay", x.shape, x.dtype, dev),
            *_rows(gate, "gate", x.shape, x.dtype, dev), _tensor(rate, "rate", (x.shape[-1],), _F32, dev)]
    return dev, code, ptrs


def _state_shape(rows, D):
    return (-(-rows // _lib.GATED_SCAN_STATE_ROWS), D)


def gated_scan_fwd(x, decay, gate, rate, h0=None, *, scale=8.0, output_final_state=True, save_states=False, y=None,
                   ht=None, cu_seqlens=None, stream=None):
    """Gated linear recurrence, one state per channel: (y, ht), with ``save_states`` (y, ht, states).

        q = scale softplus(rate) sigmoid(decay);  a = exp(-q)
        h = a h + sqrt(1 - a^2) sigmoid(gate) x;  y = h

    x, decay, gate: [B, T, D] (one dtype, bf16 or fp32); rate: [D] fp32; h0: [B, D] fp32 or None (zeros).
    y has x's dtype, ht is fp32 [B, D] (None when ``output_final_state`` is false).  states: what
    :func:`gated_scan_bwd` would otherwise compute again, fp32 [ceil(B T / 8), D].
    """
    dev, code, ptrs = _gated_inputs(x, decay, gate, rate, scale, 3)
    B, T, D = x.shape
    cu, n = _sequences(cu_seqlens, B, dev)
    hp = None if h0 is None else _tensor(h0, "h0", (n, D), _F32, dev)
    with _On(dev, stream, (x, decay, gate, rate, h0, cu_seqlens)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        htp = sp = None
        if output_final_state or ht is not None:
            ht, htp = _dense_out(on, ht, "ht", (n, D), _F32)
        if save_states:
            states, sp = _dense_out(on, None, "states", _state_shape(B * T, D), _F32)
        args = _lib.GatedScanFwdArgs(n, T, D, code, scale, *ptrs, hp, yp, ldy, htp, sp, None, 0, cu)
        ws = on.workspace("gated_scan_fwd_workspace", args)
        on.launch("gated_scan_fwd", args)
        del ws
    return (y, ht, states) if save_states else (y, ht)


def gated_scan_bwd(x, decay, gate, rate, h0, dy, dht=None, *, states=None, scale=8.0, grads=None, cu_seqlens=None,
                   stream=None):
    """Backward of :func:`gated_scan_fwd`, whose inputs it takes again: a dict with dx, ddecay, dgate (dtype of x) and
    drate (fp32), and dh0 when h0 is given.  dy: [B, T, D]; dht: gradient of ht, fp32 [B, D] or None; states: the
    forward's, or None (the forward runs again for them).  ``grads`` may supply output tensors by the names of those
    that the call returns."""
    dev, code, ptrs = _gated_inputs(x, decay, gate, rate, scale, 3)
    B, T, D = x.shape
    cu, n = _sequences(cu_seqlens, B, dev)
    hp = None if h0 is None else _tensor(h0, "h0", (n, D), _F32, dev)
    dyp = _rows(dy, "dy", x.shape, x.dtype, dev)
    dhp = None if dht is None else _tensor(dht, "dht", (n, D), _F32, dev)
    sp = None if states is None else _tensor(states, "states", _state_shape(B * T, D), _F32, dev)
    out = _known(grads, ("dx", "ddecay", "dgate", "drate", "dh0"), dh0=h0 is not None)
    with _On(dev, stream, (x, decay, gate, rate, h0, dy, dht, states, cu_seqlens)) as on:
        seq = []
        for name in ("dx", "ddecay", "dgate"):
            out[name], p, ld = _out(on, out.get(name), name, x.shape, x.dtype)
            seq += [p, ld]
        out["drate"], drp = _dense_out(on, out.get("drate"), "drate", (D,), _F32)
        dh0p = None
        if h0 is not None:
            out["dh0"], dh0p = _dense_out(on, out.get("dh0"), "dh0", (n, D), _F32)
        args = _lib.GatedScanBwdArgs(n, T, D, code, scale, *ptrs, hp, *dyp, dhp, sp, *seq, drp, dh0p, None, 0, cu)
        ws = on.workspace("gated_scan_bwd_workspace", args)
        on.launch("gated_scan_bwd", args)
        del ws
    return out


def gated_scan_step(x, decay, gate, rate, state, *, scale=8.0, slots=None, y=None, stream=None):
    """One token of each request: y [B, D]; ``state`` [S, D] fp32 is updated in place.

    x, decay, gate: [B, D]; rate as in :func:`gated_scan_fwd`.  slots: int32 CUDA tensor [B], the state of each request
    (no two alike), or None (request b has state b).  A request whose slot lies outside [0, S) is padding: its y is 0,
    no state changes.
    """
    dev, code, ptrs = _gated_inputs(x, decay, gate, rate, scale, 2)
    B, D = x.shape
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a tensor")
    sp = _tensor(state, "state", (state.shape[0], D) if state.dim() == 2 else (None, D), _F32, dev)
    ip = None if slots is None else _tensor(slots, "slots", (B,), torch.int32, dev)
    with _On(dev, stream, (x, decay, gate, rate, state, slots)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        on.launch("gated_scan_step", _lib.GatedScanStepArgs(B, D, state.shape[0], code, scale, *ptrs, sp, ip, yp, ldy))
    return y


# ------------------------------------------------------------------------------------ norm over groups
def _group_inputs(x, groups, weight, bias, gate):
    dev = _cuda(x, "x")
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must have at least one row and one column")
    cols = x.shape[-1]
    if not isinstance(groups, int) or isinstance(groups, bool):
        raise TypeError("groups must be an integer")
    if groups < 1 or cols % groups:
        raise ValueError(f"groups must divide the last axis ({cols})")
    code, C = _code(x, "x"), cols // groups
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
    lead = weight if weight is not None else bias
    wdt = x.dtype if lead is None else lead.dtype
    if wdt not in _CODES:
        raise TypeError(f"weight: unsupported dtype {wdt}")
    shared = lead is not None and lead.dim() == 1 and lead.shape[0] == C and groups > 1
    shape = (C,) if shared else (cols,)
    wp = None if weight is None else _tensor(weight, "weight", shape, wdt, dev)
    bp = None if bias is None else _tensor(bias, "bias", shape, wdt, dev)
    xp = _rows(x, "x", x.shape, x.dtype, dev)
    zp = (None, 0) if gate is None else _rows(gate, "gate", x.shape, x.dtype, dev)
    return dev, code, C, wdt, shape, _lib.GROUP_NORM_FLAG_SHARED if shared else 0, wp, bp, xp, zp


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, *, eps=1e-5, center=True, y=None, stream=None):
    """Norm over each of ``groups`` equal parts of the last axis (a mixer's heads), and a gate: (y, mean, rstd).

        n = (x - mean) rstd weight + bias;  y = n silu(gate)

    x, gate: [..., groups C] bf16 or fp32; weight, bias: [groups C], or [C] for all groups alike (bf16 or fp32, one
    dtype), or None; gate may be None.  ``center=False`` takes the root mean square without subtracting the mean.
    y has x's dtype; mean (None without a centre) and rstd are fp32 [..., groups] for :func:`group_norm_bwd`.
    """
    dev, code, C, wdt, _, flags, wp, bp, xp, zp = _group_inputs(x, groups, weight, bias, gate)
    if not eps >= 0.0:
        raise ValueError("eps must not be negative")
    with _On(dev, stream, (x, weight, bias, gate)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        stat = (*x.shape[:-1], groups)
        mean = torch.empty(stat, dtype=_F32, device=dev) if center else None
        rstd = torch.empty(stat, dtype=_F32, device=dev)
        if center:
            flags |= _lib.GROUP_NORM_FLAG_CENTER
        on.launch("group_norm_fwd", _lib.GroupNormFwdArgs(
            x.numel() // x.shape[-1], groups, C, code, _CODES[wdt], flags, eps, *xp, *zp, wp, bp, yp, ldy,
            mean.data_ptr() if center else None, rstd.data_ptr()))
    return y, mean, rstd


def group_norm_bwd(dy, x, groups, weight, bias, gate, mean, rstd, *, grads=None, stream=None):
    """Backward of :func:`group_norm_fwd`, whose inputs it takes again with its mean (None: without a centre) and rstd:
    a dict with dx (dtype of x), and dweight, dbias and dgate for the inputs that are given.  ``grads`` may supply output
    tensors by the names of those that the call returns."""
    dev, code, C, wdt, shape, flags, wp, bp, xp, zp = _group_inputs(x, groups, weight, bias, gate)
    dyp = _rows(dy, "dy", x.shape, x.dtype, dev)
    stat = (*x.shape[:-1], groups)
    rp = _tensor(rstd, "rstd", stat, _F32, dev)
    mp = None if mean is None else _tensor(mean, "mean", stat, _F32, dev)
    if mean is not None:
        flags |= _lib.GROUP_NORM_FLAG_CENTER
    out = _known(grads, ("dx", "dweight", "dbias", "dgate"), dweight=weight is not None, dbias=bias is not None,
                 dgate=gate is not None)
    with _On(dev, stream, (dy, x, weight, bias, gate, mean, rstd)) as on:
        out["dx"], *dxp = _out(on, out.get("dx"), "dx", x.shape, x.dtype)
        dzp, dwp, dbp = (None, 0), None, None
        if gate is not None:
            out["dgate"], *dzp = _out(on, out.get("dgate"), "dgate", x.shape, x.dtype)
        if weight is not None:
            out["dweight"], dwp = _dense_out(on, out.get("dweight"), "dweight", shape, wdt)
        if bias is not None:
            out["dbias"], dbp = _dense_out(on, out.get("dbias"), "dbias", shape, wdt)
        args = _lib.GroupNormBwdArgs(x.numel() // x.shape[-1], groups, C, code, _CODES[wdt], flags, *dyp, *xp, *zp, wp, bp,
                                     mp, rp, *dxp, *dzp, dwp, dbp, None, 0)
        ws = on.workspace("group_norm_bwd_workspace", args)
        on.launch("group_norm_bwd", args)
        del ws
    return out


# ------------------------------------------------------------------------- gated feed-forward product
def _glu_activation(name):
    if name == "silu":
        return 0
    if name == "gelu":
        return _lib.GLU_FLAG_GELU
    raise ValueError(f"unknown activation {name!r}")


def _glu_inputs(x, w_gate, w_up):
    dev = _cuda(x, "x")
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must have at least one row and one column")
    code, D = _code(x, "x"), x.shape[-1]
    _check(w_gate, "w_gate", (None, D), x.dtype, dev)
    F = w_gate.shape[0]
    if F == 0:
        raise ValueError("w_gate must have at least one row")
    ptrs = [*_rows(x, "x", x.shape, x.dtype, dev), *_rows(w_gate, "w_gate", (F, D), x.dtype, dev),
            *_rows(w_up, "w_up", (F, D), x.dtype, dev)]
    return dev, code, D, F, x.numel() // D, ptrs


def _glu_status(status, dev):
    if status is None:
        return None
    p = _tensor(status, "status", (status.shape[0],) if isinstance(status, torch.Tensor) and status.dim() == 1 else (None,),
                torch.uint8, dev)
    if status.shape[0] < 256:
        raise ValueError("status must have 256 bytes")
    return p


def glu_fwd(x, w_gate, w_up, *, activation="silu", save=False, y=None, status=None, stream=None):
    """First half of a gated feed-forward block in one kernel: h, with ``save`` (h, g, u).

        g = x w_gate^T;  u = x w_up^T;  h = act(g) u

    x: [..., D]; w_gate, w_up: [F, D] (one dtype, bf16 or fp32); activation: "silu" or "gelu" (g Phi(g)).  h is [..., F]
    of x's dtype.  g and u are fp32 [..., F], what :func:`glu_bwd` would otherwise compute again.  status: uint8 [256],
    zero at first, for :func:`.api.status_read`: whether a wait of the bf16 kernels ran out.
    """
    dev, code, D, F, rows, ptrs = _glu_inputs(x, w_gate, w_up)
    flags = _glu_activation(activation)
    shape, stp = (*x.shape[:-1], F), _glu_status(status, dev)
    with _On(dev, stream, (x, w_gate, w_up, status)) as on:
        y, yp, ldy = _out(on, y, "y", shape, x.dtype)
        g = u = gp = up = None
        if save:
            g, gp = _dense_out(on, None, "g", shape, _F32)
            u, up = _dense_out(on, None, "u", shape, _F32)
        args = _lib.GluFwdArgs(rows, D, F, code, flags, *ptrs, yp, ldy, gp, up, None, 0, stp)
        ws = on.workspace("glu_fwd_workspace", args)
        on.launch("glu_fwd", args)
        del ws
    return (y, g, u) if save else y


def glu_bwd(x, w_gate, w_up, dh, g=None, u=None, *, activation="silu", grads=None, status=None, stream=None):
    """Backward of :func:`glu_fwd`, whose inputs it takes again: a dict with dx, dw_gate and dw_up (dtype of x).
    dh: [..., F]; g, u: the forward's, or None (computed again); status as there.  ``grads`` may supply output tensors by name."""
    dev, code, D, F, rows, ptrs = _glu_inputs(x, w_gate, w_up)
    flags = _glu_activation(activation)
    shape = (*x.shape[:-1], F)
    dhp = _rows(dh, "dh", shape, x.dtype, dev)
    if (g is None) != (u is None):
        raise ValueError("g and u come together")
    gp = None if g is None else _tensor(g, "g", shape, _F32, dev)
    up = None if u is None else _tensor(u, "u", shape, _F32, dev)
    out, stp = _known(grads, ("dx", "dw_gate", "dw_up")), _glu_status(status, dev)
    with _On(dev, stream, (x, w_gate, w_up, dh, g, u, status)) as on:
        out["dx"], *dxp = _out(on, out.get("dx"), "dx", x.shape, x.dtype)
        out["dw_gate"], *dgp = _out(on, out.get("dw_gate"), "dw_gate", (F, D), x.dtype)
        out["dw_up"], *dup = _out(on, out.get("dw_up"), "dw_up", (F, D), x.dtype)
        args = _lib.GluBwdArgs(rows, D, F, code, flags, *ptrs, *dhp, gp, up, *dxp, *dgp, *dup, None, 0, stp)
        ws = on.workspace("glu_bwd_workspace", args)
        on.launch("glu_bwd", args)
        del ws
    return out
