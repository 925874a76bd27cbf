"""Python binding of include/mixer.h: layer norm, the short causal convolution and the selective scan.

As in :mod:`.api`, everything is computed in ``libkda.so``; this module checks
shapes, types and strides, allocates the outputs and picks the stream.  There is
no CPU path.

Sequence tensors are [B, T, C] with the last axis contiguous; their rows may lie
apart (parts of a wider projection's output need no copy), as long as one row
stride serves all B T rows.  With ``cu_seqlens`` (int32 CUDA tensor [n + 1]) n
sequences lie back to back in [1, T, C] tensors and states are [n, ...].

Outputs and workspaces are allocated on the stream that the call runs on (the
current one, or ``stream``), so a call captured into a CUDA graph keeps them in
the graph's own pool.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import KdaError

_CODES = {torch.bfloat16: _lib.KDA_BF16, torch.float32: _lib.KDA_F32}
_F32 = torch.float32

# The current stream's handle and the current device without building Python objects for them (a
# decoding step's calls are short); the public functions where a build lacks these.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_functions: dict = {}


def _function(name):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    return fn


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _check(t, name, shape, dtype, device):
    """Shape, dtype and device (a CUDA index; -1 is the CPU).  An axis of None may have any size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on device cuda:{device}, not {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _tensor(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor of this shape and dtype."""
    if type(t) is not torch.Tensor or t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _check(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, dtype, device):
    """Pointer and row stride of a tensor whose rows (last axis) may lie apart."""
    if type(t) is not torch.Tensor or t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _check(t, name, shape, dtype, device)
    width = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), width
    st = t.stride()
    if width > 1 and st[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last axis")
    rows = [k for k in range(len(shape) - 1) if shape[k] > 1]
    ld = step = st[rows[-1]] if rows else width
    for k in reversed(rows):             # every axis of rows follows from the one stride
        if st[k] != step:
            raise ValueError(f"{name}: one row stride must serve all rows")
        step *= shape[k]
    if ld < width:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld


def _cuda(t, name):
    """The index of the tensor's CUDA device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _sequences(cu_seqlens, B, device):
    """Pointer to the offsets and the number of sequences."""
    if cu_seqlens is None:
        return None, B
    if not isinstance(cu_seqlens, torch.Tensor):
        raise TypeError("cu_seqlens must be a tensor")
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if B != 1 or cu_seqlens.numel() < 2:
        raise ValueError("with cu_seqlens (at least two offsets) the tensors are [1, T, C]")
    return _tensor(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, device), cu_seqlens.numel() - 1


class _On:
    """The stream of a call: allocations inside go to it, launches too."""

    __slots__ = ("device", "handle", "ctx", "side")

    def __init__(self, device, stream, inputs):
        self.device = device
        self.handle = _raw_stream(device)
        self.ctx = None
        self.side = None                 # a stream other than the current one
        if stream is not None and stream.device.index != device:
            raise ValueError(f"stream must be on device cuda:{device}, not {stream.device}")
        if stream is not None and stream.cuda_stream != self.handle:
            self.ctx = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
            self.side = stream
            for t in inputs:
                if t is not None:
                    self.uses(t)
        elif _device_index() != device:
            self.ctx = torch.cuda.device(device)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)

    def uses(self, t):
        """The allocator must not hand out a caller's tensor while another stream reads or writes it."""
        if self.side is not None:
            t.record_stream(self.side)

    def launch(self, name, args):
        rc = _function(name)(ctypes.byref(args), self.handle)
        if rc:
            raise KdaError(rc, name)

    def workspace(self, name, args):
        """Points args at a workspace of the size that the library asks for."""
        need = _function(name)(ctypes.byref(args))
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            args.workspace, args.workspace_bytes = ws.data_ptr(), need
            return ws
        return None


def _out(on, given, name, shape, dtype):
    """An output tensor of a call (rows may lie apart): the caller's, or a new one."""
    if given is None:
        given = torch.empty(shape, dtype=dtype, device=on.device)
        return given, given.data_ptr(), shape[-1]
    rows = _rows(given, name, shape, dtype, on.device)
    on.uses(given)
    return (given, *rows)


def _dense_out(on, given, name, shape, dtype):
    if given is None:
        given = torch.empty(shape, dtype=dtype, device=on.device)
        return given, given.data_ptr()
    ptr = _tensor(given, name, shape, dtype, on.device)
    on.uses(given)
    return given, ptr


def _known(grads, names, **inputs):
    """The caller's gradient tensors by name.  ``inputs``: for names that depend on it, whether the call has the
    input (or asks for the gradient): a tensor for another would come back unwritten."""
    grads = {k: v for k, v in (grads or {}).items() if v is not None or k not in names}
    extra = set(grads) - set(names)
    if extra:
        raise ValueError(f"unknown gradients: {sorted(extra)}")
    idle = sorted(k for k in grads if not inputs.get(k, True))
    if idle:
        raise ValueError(f"gradients that this call does not compute: {idle}")
    return grads


def _weights(weight, bias, wname, shape, D, device, default):
    """Pointers of weight and bias, and their dtype's code.  A weight of two axes (the convolution's) is needed."""
    if not isinstance(weight, torch.Tensor) and (weight is not None or len(shape) == 2):
        raise TypeError(f"{wname} must be a tensor")
    if bias is not None and not isinstance(bias, torch.Tensor):
        raise TypeError("bias must be a tensor")
    dt = weight.dtype if weight is not None else bias.dtype if bias is not None else default
    if weight is not None and len(shape) == 2 and weight.dim() == 2:
        shape = (D, weight.shape[1])     # [D, W], any W
    w = None if weight is None else _tensor(weight, wname, shape, dt, device)
    b = None if bias is None else _tensor(bias, "bias", (D,), dt, device)
    if dt not in _CODES:
        raise TypeError(f"{wname}: unsupported dtype {dt}")
    return w, b, dt


# ------------------------------------------------------------------------------------ layer norm
def layer_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, y=None, stream=None):
    """Layer norm over the last axis: (y, mean, rstd).

    x: [..., D] bf16 or fp32; weight, bias: [D] (bf16 or fp32, one dtype) or None.
    y has x's dtype; mean and rstd are fp32 [...] for :func:`layer_norm_bwd`.
    """
    dev = _cuda(x, "x")
    D = x.shape[-1] if x.dim() else 0
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must have at least one row and one column")
    code = _code(x, "x")
    xp, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    wp, bp, wdt = _weights(weight, bias, "weight", (D,), D, dev, x.dtype)
    with _On(dev, stream, (x, weight, bias)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
        on.launch("layer_norm_fwd", _lib.LayerNormFwdArgs(
            x.numel() // D, D, code, _CODES[wdt], eps, xp, ldx, wp, bp, yp, ldy, mean.data_ptr(), rstd.data_ptr()))
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, *, bias=True, grads=None, stream=None):
    """Backward of :func:`layer_norm_fwd`: a dict with dx (dtype of x), dweight when weight is
    given, and dbias when ``bias`` is set (both in weight's dtype; x's without a weight).
    ``grads`` may supply output tensors by the names of those that the call returns."""
    dev = _cuda(x, "x")
    D = x.shape[-1] if x.dim() else 0
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must have at least one row and one column")
    code = _code(x, "x")
    xp, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    dyp, lddy = _rows(dy, "dy", x.shape, x.dtype, dev)
    wp, _, wdt = _weights(weight, None, "weight", (D,), D, dev, x.dtype)
    mp = _tensor(mean, "mean", tuple(x.shape[:-1]), torch.float32, dev)
    rp = _tensor(rstd, "rstd", tuple(x.shape[:-1]), torch.float32, dev)
    out = _known(grads, ("dx", "dweight", "dbias"), dweight=weight is not None, dbias=bias)
    with _On(dev, stream, (x, dy, weight, mean, rstd)) as on:
        out["dx"], dxp, lddx = _out(on, out.get("dx"), "dx", x.shape, x.dtype)
        dwp = dbp = None
        if weight is not None:
            out["dweight"], dwp = _dense_out(on, out.get("dweight"), "dweight", (D,), wdt)
        if bias:
            out["dbias"], dbp = _dense_out(on, out.get("dbias"), "dbias", (D,), wdt)
        args = _lib.LayerNormBwdArgs(x.numel() // D, D, code, _CODES[wdt], dyp, lddy, xp, ldx, wp, mp, rp, dxp, lddx,
                                     dwp, dbp, None, 0)
        ws = on.workspace("layer_norm_bwd_workspace", args)
        on.launch("layer_norm_bwd", args)
        del ws
    return out


# --------------------------------------------------------------------------- short causal convolution
def _activation(name):
    if name in (None, "none"):
        return 0
    if name == "silu":
        return _lib.SHORT_CONV_FLAG_SILU
    raise ValueError(f"unknown activation {name!r}")


def short_conv_fwd(x, weight, bias=None, h0=None, *, activation="silu", output_final_state=True, y=None, ht=None,
                   cu_seqlens=None, stream=None):
    """Causal convolution of W taps per channel: (y, ht).

    x: [B, T, D]; weight: [D, W], W = 2, 3 or 4, the last tap on the current token; bias: [D] or None;
    h0: [B, W-1, D], the inputs before the first token (oldest first), or None (zeros).
    activation: "silu" or None.  ht: the last W-1 inputs, the h0 of a continuation (None when
    ``output_final_state`` is false).
    """
    dev = _cuda(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    code, flags = _code(x, "x"), _activation(activation)
    cu, n = _sequences(cu_seqlens, B, dev)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    wp, bp, wdt = _weights(weight, bias, "weight", (D, None), D, dev, x.dtype)
    W = weight.shape[1]
    hp = None if h0 is None else _tensor(h0, "h0", (n, W - 1, D), x.dtype, dev)
    with _On(dev, stream, (x, weight, bias, h0, cu_seqlens)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        htp = None
        if output_final_state or ht is not None:
            ht, htp = _dense_out(on, ht, "ht", (n, W - 1, D), x.dtype)
        on.launch("short_conv_fwd", _lib.ShortConvFwdArgs(n, T, D, W, code, _CODES[wdt], flags, xp, ldx, wp, bp, hp, yp,
                                                          ldy, htp, cu))
    return y, ht


def short_conv_bwd(x, weight, bias, h0, dy, dht=None, *, activation="silu", grads=None, cu_seqlens=None, stream=None):
    """Backward of :func:`short_conv_fwd`: a dict with dx, dweight (weight's dtype), dbias when bias is
    given and dh0 when h0 is given.  dht: gradient of ht, or None.  ``grads`` may supply output
    tensors by the names of those that the call returns."""
    dev = _cuda(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    code, flags = _code(x, "x"), _activation(activation)
    cu, n = _sequences(cu_seqlens, B, dev)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    dyp, lddy = _rows(dy, "dy", x.shape, x.dtype, dev)
    wp, bp, wdt = _weights(weight, bias, "weight", (D, None), D, dev, x.dtype)
    W = weight.shape[1]
    hp = None if h0 is None else _tensor(h0, "h0", (n, W - 1, D), x.dtype, dev)
    dhp = None if dht is None else _tensor(dht, "dht", (n, W - 1, D), x.dtype, dev)
    out = _known(grads, ("dx", "dweight", "dbias", "dh0"), dbias=bias is not None, dh0=h0 is not None)
    with _On(dev, stream, (x, weight, bias, h0, dy, dht, cu_seqlens)) as on:
        out["dx"], dxp, lddx = _out(on, out.get("dx"), "dx", x.shape, x.dtype)
        out["dweight"], dwp = _dense_out(on, out.get("dweight"), "dweight", (D, W), wdt)
        dbp = dh0p = None
        if bias is not None:
            out["dbias"], dbp = _dense_out(on, out.get("dbias"), "dbias", (D,), wdt)
        if h0 is not None:
            out["dh0"], dh0p = _dense_out(on, out.get("dh0"), "dh0", (n, W - 1, D), x.dtype)
        args = _lib.ShortConvBwdArgs(n, T, D, W, code, _CODES[wdt], flags, xp, ldx, wp, bp, hp, dyp, lddy, dhp, dxp, lddx,
                                     dh0p, dwp, dbp, None, 0, cu)
        ws = on.workspace("short_conv_bwd_workspace", args)
        on.launch("short_conv_bwd", args)
        del ws
    return out


def short_conv_step(x, weight, bias, state, *, activation="silu", slots=None, y=None, stream=None):
    """One token of each request: y [B, D]; ``state`` [S, W-1, D] is updated in place.

    slots: int32 CUDA tensor [B], the state of each request (no two alike), or None (request b has
    state b).  A request whose slot lies outside [0, S) is padding: its y is 0, no state changes.
    """
    dev = _cuda(x, "x")
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a tensor")
    if x.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [B, D] and state [S, W-1, D]")
    B, D = x.shape
    code, flags = _code(x, "x"), _activation(activation)
    xp, ldx = _rows(x, "x", x.shape, x.dtype, dev)
    wp, bp, wdt = _weights(weight, bias, "weight", (D, None), D, dev, x.dtype)
    W = weight.shape[1]
    sp = _tensor(state, "state", (state.shape[0], W - 1, D), x.dtype, dev)
    ip = None if slots is None else _tensor(slots, "slots", (B,), torch.int32, dev)
    with _On(dev, stream, (x, weight, bias, state, slots)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        on.launch("short_conv_step", _lib.ShortConvStepArgs(B, D, W, state.shape[0], code, _CODES[wdt], flags, xp, ldx,
                                                            wp, bp, sp, ip, yp, ldy))
    return y


# ------------------------------------------------------------------------- selective state-space scan
def _scan_inputs(x, delta, A, B, C, D, z, delta_bias, dims):
    """Checks the inputs that the scan's calls share; pointers and strides in the C order."""
    dev = _cuda(x, "x")
    if x.dim() != dims:
        raise ValueError("x must be [B, T, D]" if dims == 3 else "x must be [B, D]")
    if not isinstance(A, torch.Tensor):
        raise TypeError("A must be a tensor")
    if A.dim() != 2:
        raise ValueError("A must be [D, N]")
    ch, n = x.shape[-1], A.shape[1]
    code, lead = _code(x, "x"), x.shape[:-1]
    ptrs = [*_rows(x, "x", x.shape, x.dtype, dev), *_rows(delta, "delta", x.shape, x.dtype, dev),
            *_rows(B, "B", (*lead, n), x.dtype, dev), *_rows(C, "C", (*lead, n), x.dtype, dev)]
    ptrs += [None, 0] if z is None else _rows(z, "z", x.shape, x.dtype, dev)
    f32 = torch.float32
    ptrs += [_tensor(A, "A", (ch, n), f32, dev), None if D is None else _tensor(D, "D", (ch,), f32, dev),
             None if delta_bias is None else _tensor(delta_bias, "delta_bias", (ch,), f32, dev)]
    return dev, code, ch, n, ptrs


def ssm_scan_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, h0=None, *, delta_softplus=True,
                 output_final_state=True, y=None, ht=None, cu_seqlens=None, stream=None):
    """Selective scan: (y, ht).

        dt = softplus(delta + delta_bias);  h = exp(dt A) h + dt x B;  y = (C . h + D x) silu(z)

    x, delta, z: [B, T, D]; B, C: [B, T, N] (one dtype, bf16 or fp32); A: [D, N], D, delta_bias: [D],
    h0: [B, D, N], all fp32; N up to 32.  z, D, delta_bias and h0 may be None; ``delta_softplus=False``
    takes dt = delta + delta_bias.  y has x's dtype, ht is fp32 [B, D, N] (None when
    ``output_final_state`` is false).
    """
    dev, code, ch, n, ptrs = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, 3)
    bt, T = x.shape[:2]
    cu, seqs = _sequences(cu_seqlens, bt, dev)
    hp = None if h0 is None else _tensor(h0, "h0", (seqs, ch, n), torch.float32, dev)
    with _On(dev, stream, (x, delta, A, B, C, D, z, delta_bias, h0, cu_seqlens)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        htp = None
        if output_final_state or ht is not None:
            ht, htp = _dense_out(on, ht, "ht", (seqs, ch, n), torch.float32)
        args = _lib.SsmScanFwdArgs(seqs, T, ch, n, code, int(delta_softplus), *ptrs, hp, yp, ldy, htp, None, 0, cu)
        ws = on.workspace("ssm_scan_fwd_workspace", args)
        on.launch("ssm_scan_fwd", args)
        del ws
    return y, ht


def ssm_scan_bwd(x, delta, A, B, C, D, z, delta_bias, h0, dy, dht=None, *, delta_softplus=True, grads=None,
                 cu_seqlens=None, stream=None):
    """Backward of :func:`ssm_scan_fwd`, whose inputs it takes again: a dict with dx, ddelta, dB, dC
    (dtype of x) and dA (fp32), and dz, dD, ddelta_bias, dh0 for the inputs that are given.
    dy: [B, T, D]; dht: gradient of ht, fp32 [B, D, N] or None.  ``grads`` may supply output tensors by
    the names of those that the call returns."""
    dev, code, ch, n, ptrs = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, 3)
    bt, T = x.shape[:2]
    cu, seqs = _sequences(cu_seqlens, bt, dev)
    f32 = torch.float32
    hp = None if h0 is None else _tensor(h0, "h0", (seqs, ch, n), f32, dev)
    dyp = _rows(dy, "dy", x.shape, x.dtype, dev)
    dhp = None if dht is None else _tensor(dht, "dht", (seqs, ch, n), f32, dev)
    out = _known(grads, ("dx", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0"), dD=D is not None, dz=z is not None,
                 ddelta_bias=delta_bias is not None, dh0=h0 is not None)
    with _On(dev, stream, (x, delta, A, B, C, D, z, delta_bias, h0, dy, dht, cu_seqlens)) as on:
        seq = []
        for name, shape in (("dx", x.shape), ("ddelta", x.shape), ("dB", B.shape), ("dC", C.shape)):
            out[name], p, ld = _out(on, out.get(name), name, shape, x.dtype)
            seq += [p, ld]
        if z is not None:
            out["dz"], p, ld = _out(on, out.get("dz"), "dz", x.shape, x.dtype)
            seq += [p, ld]
        else:
            seq += [None, 0]
        par = []
        for name, src, shape in (("dA", A, (ch, n)), ("dD", D, (ch,)), ("ddelta_bias", delta_bias, (ch,)),
                                 ("dh0", h0, (seqs, ch, n))):
            p = None
            if src is not None:
                out[name], p = _dense_out(on, out.get(name), name, shape, f32)
            par.append(p)
        args = _lib.SsmScanBwdArgs(seqs, T, ch, n, code, int(delta_softplus), *ptrs, hp, *dyp, dhp, *seq, *par, None, 0,
                                   cu)
        ws = on.workspace("ssm_scan_bwd_workspace", args)
        on.launch("ssm_scan_bwd", args)
        del ws
    return out


def ssm_scan_step(x, delta, A, B, C, state, D=None, z=None, delta_bias=None, *, delta_softplus=True, slots=None, y=None,
                  stream=None):
    """One token of each request: y [B, D]; ``state`` [S, D, N] fp32 is updated in place.

    x, delta, z: [B, D]; B, C: [B, N]; A, D, delta_bias as in :func:`ssm_scan_fwd`; slots as in
    :func:`short_conv_step`.
    """
    dev, code, ch, n, ptrs = _scan_inputs(x, delta, A, B, C, D, z, delta_bias, 2)
    bt = x.shape[0]
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a tensor")
    sp = _tensor(state, "state", (state.shape[0], ch, n) if state.dim() == 3 else (None, ch, n), _F32, dev)
    ip = None if slots is None else _tensor(slots, "slots", (bt,), torch.int32, dev)
    with _On(dev, stream, (x, delta, A, B, C, state, D, z, delta_bias, slots)) as on:
        y, yp, ldy = _out(on, y, "y", x.shape, x.dtype)
        on.launch("ssm_scan_step", _lib.SsmScanStepArgs(bt, ch, n, state.shape[0], code, int(delta_softplus), *ptrs, sp, ip,
                                                        yp, ldy))
    return y
