"""Host-side checks of the gated recurrence, the norm over groups and the gated feed-forward product that need no GPU: refusals
before any launch, workspace sizes, and the Python binding's checks."""
import ctypes
import re

import pytest
import torch

from chunkwise_gated_delta_gb300 import _lib, layer, mixer
from chunkwise_gated_delta_gb300 import build as kbuild

BAD, SPACE = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_WORKSPACE
BASE = 1 << 40                               # made-up, well separated addresses; never dereferenced

_SIZES = {"gated_scan_fwd": dict(B=2, T=500, D=64, scale=8.0), "gated_scan_bwd": dict(B=2, T=500, D=64, scale=8.0),
          "gated_scan_step": dict(B=4, D=64, slots=9, scale=8.0),
          "group_norm_fwd": dict(rows=8, groups=4, C=16, eps=1e-5, flags=1), "group_norm_bwd": dict(rows=8, groups=4, C=16, flags=1),
          "glu_fwd": dict(rows=8, D=64, F=128), "glu_bwd": dict(rows=8, D=64, F=128)}


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


def _args(name, **over):
    a = _lib.MIXER_EXPORTS[name][0]()
    for i, (f, t) in enumerate(a._fields_):
        if t is ctypes.c_void_p and f != "cu_seqlens":
            setattr(a, f, BASE + i * (1 << 32))
    for k, v in {**_SIZES[name], "workspace_bytes": 1 << 30, **over}.items():
        if any(f == k for f, _ in a._fields_):
            setattr(a, k, v)
    return a


def _at(name, field, plus=0):
    return getattr(_args(name), field) + plus


_CASES = []
for _n in _SIZES:
    _CASES += [(_n, dict(dtype=5), BAD), (_n, dict(x=None), BAD), (_n, dict(x=BASE + 1), BAD), (_n, dict(ld_x=63), BAD),
               (_n, dict(ld_x=-64), BAD), (_n, dict(ld_x=1 << 41), BAD)]
    if "scan" in _n:
        _CASES += [(_n, dict(D=0), BAD), (_n, dict(B=0), BAD), (_n, dict(decay=None), BAD), (_n, dict(gate=None), BAD), (_n, dict(rate=None), BAD),
                   (_n, dict(scale=0.0), BAD), (_n, dict(scale=-1.0), BAD), (_n, dict(scale=float("nan")), BAD),
                   (_n, dict(scale=float("inf")), BAD), (_n, dict(rate=BASE + 2), BAD)]
    if "group" in _n:
        _CASES += [(_n, dict(rows=0), BAD), (_n, dict(groups=0), BAD), (_n, dict(C=0), BAD), (_n, dict(rows=1 << 29, groups=4), BAD),
                   (_n, dict(groups=1 << 16, C=1 << 15), BAD), (_n, dict(flags=4), BAD), (_n, dict(w_dtype=3), BAD)]
    if "glu" in _n:
        _CASES += [(_n, dict(rows=0), BAD), (_n, dict(D=0), BAD), (_n, dict(F=0), BAD), (_n, dict(w_gate=None), BAD), (_n, dict(w_up=None), BAD),
                   (_n, dict(flags=2), BAD), (_n, dict(g=None), BAD), (_n, dict(u=None), BAD), (_n, dict(ld_w_up=63), BAD),
                   (_n, dict(status=BASE + (1 << 45) + 8), BAD)]
_CASES += [("gated_scan_fwd", dict(T=0), BAD), ("gated_scan_fwd", dict(B=1 << 16, T=1 << 16), BAD), ("gated_scan_fwd", dict(y=None), BAD),
           ("gated_scan_fwd", dict(cu_seqlens=BASE + 2), BAD), ("gated_scan_fwd", dict(workspace=None), SPACE),
           ("gated_scan_fwd", dict(workspace_bytes=64), SPACE), ("gated_scan_fwd", dict(workspace=BASE + (1 << 45) + 4), BAD),
           ("gated_scan_fwd", dict(y=_at("gated_scan_fwd", "gate", 64)), BAD), ("gated_scan_fwd", dict(ht=_at("gated_scan_fwd", "h0")), BAD),
           ("gated_scan_fwd", dict(states=_at("gated_scan_fwd", "x", 256)), BAD),
           ("gated_scan_bwd", dict(dy=None), BAD), ("gated_scan_bwd", dict(dx=None), BAD), ("gated_scan_bwd", dict(drate=None), BAD),
           ("gated_scan_bwd", dict(workspace=None), SPACE), ("gated_scan_bwd", dict(workspace_bytes=1024), SPACE),
           ("gated_scan_bwd", dict(dgate=_at("gated_scan_bwd", "dx", 64)), BAD), ("gated_scan_bwd", dict(dh0=_at("gated_scan_bwd", "dht")), BAD),
           ("gated_scan_bwd", dict(workspace=_at("gated_scan_bwd", "states")), BAD),
           ("gated_scan_step", dict(slots=0), BAD), ("gated_scan_step", dict(slot=None, slots=3), BAD), ("gated_scan_step", dict(state=None), BAD),
           ("gated_scan_step", dict(y=_at("gated_scan_step", "state", 128)), BAD),
           ("group_norm_fwd", dict(eps=-1.0), BAD), ("group_norm_fwd", dict(eps=float("nan")), BAD), ("group_norm_fwd", dict(y=None), BAD),
           ("group_norm_fwd", dict(flags=0), BAD),                       # a mean without a centre
           ("group_norm_fwd", dict(y=_at("group_norm_fwd", "gate")), BAD),
           ("group_norm_bwd", dict(flags=0), BAD), ("group_norm_bwd", dict(mean=None), BAD), ("group_norm_bwd", dict(rstd=None), BAD),
           ("group_norm_bwd", dict(gate=None), BAD), ("group_norm_bwd", dict(dgate=None), BAD), ("group_norm_bwd", dict(workspace=None), SPACE),
           ("group_norm_bwd", dict(workspace_bytes=16), SPACE), ("group_norm_bwd", dict(dx=_at("group_norm_bwd", "dy", 32)), BAD),
           ("glu_fwd", dict(h=None), BAD), ("glu_fwd", dict(h=_at("glu_fwd", "x", 128)), BAD), ("glu_fwd", dict(u=_at("glu_fwd", "g", 64)), BAD),
           ("glu_fwd", dict(x=BASE + 2, workspace=None), SPACE),         # an operand that has to move
           ("glu_bwd", dict(dh=None), BAD), ("glu_bwd", dict(dx=None), BAD), ("glu_bwd", dict(dw_up=None), BAD), ("glu_bwd", dict(workspace=None), SPACE),
           ("glu_bwd", dict(workspace_bytes=4095), SPACE), ("glu_bwd", dict(dw_up=_at("glu_bwd", "dw_gate", 64)), BAD),
           ("glu_bwd", dict(workspace=_at("glu_bwd", "g")), BAD)]


@pytest.mark.parametrize("name,over,code", _CASES)
def test_refusals_before_any_launch(lib, name, over, code):
    assert getattr(lib, name)(ctypes.byref(_args(name, **over)), None) == code
    query = name + "_workspace"
    if query in _lib.MIXER_EXPORTS and code != SPACE and "workspace" not in over:
        assert getattr(lib, query)(ctypes.byref(_args(name, **over))) == 0


def test_workspace_sizes(lib):
    size = lambda n, **o: getattr(lib, n + "_workspace")(ctypes.byref(_args(n, **o)))  # noqa: E731
    assert size("gated_scan_fwd", B=1, T=128) == 0 and size("gated_scan_fwd") > 0           # one segment takes none
    assert size("gated_scan_bwd", B=1, T=128) == 0 and size("gated_scan_bwd", B=1, T=128, states=None) >= 16 * 64 * 4
    kept, again = size("gated_scan_bwd"), size("gated_scan_bwd", states=None)
    assert again >= kept + 125 * 64 * 4                                                     # a state before every eighth of 1000 rows
    # a packed batch has as many rows as tokens
    assert size("gated_scan_bwd", B=2048, T=1 << 20, cu_seqlens=1 << 30, D=8) > 0
    assert size("gated_scan_bwd", B=2048, T=1 << 20, D=8) == 0
    assert size("group_norm_bwd", dweight=None, dbias=None) == 0 and size("group_norm_bwd") >= 8 * 64
    assert size("glu_fwd") == 0 and size("glu_fwd", x=BASE + 2) >= 8 * 64 * 2 and size("glu_fwd", dtype=_lib.KDA_F32, x=BASE + 4) == 0
    assert size("glu_fwd", ld_w_gate=65) >= 128 * 64 * 2
    assert size("glu_bwd") >= 2 * 8 * 128 * 2


@pytest.mark.parametrize("T", [129, 144, 160, 192])
def test_a_backward_without_states_has_the_forwards_space(lib, T):
    """Its rows may be one segment where the forward's, which it runs for the states, are several."""
    size = lambda n, **o: getattr(lib, n + "_workspace")(ctypes.byref(_args(n, B=1, T=T, **o)))  # noqa: E731
    for D in (64, 77888, 77890, 104000, 166400, 230016):
        states = (-(-T // 8) * D * 4 + 15) // 16 * 16
        assert size("gated_scan_bwd", D=D, ld_x=D, states=None) >= states + size("gated_scan_fwd", D=D, ld_x=D), D


def test_state_rows_are_the_headers():
    src = open(kbuild.INCLUDE + "/mixer.h").read()
    for name in ("GATED_SCAN_STATE_ROWS", "GROUP_NORM_FLAG_CENTER", "GROUP_NORM_FLAG_SHARED", "GLU_FLAG_GELU"):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == getattr(_lib, name)


# ------------------------------------------------------------------------------ Python binding
def test_no_cpu_path():
    x, w = torch.zeros(2, 3, 8), torch.zeros(16, 8)
    r = torch.zeros(8)
    for call in (lambda: layer.gated_scan_fwd(x, x, x, r), lambda: layer.gated_scan_bwd(x, x, x, r, None, x),
                 lambda: layer.gated_scan_step(x[0], x[0], x[0], r, torch.zeros(3, 8)), lambda: layer.group_norm_fwd(x, 2),
                 lambda: layer.group_norm_bwd(x, x, 2, None, None, None, None, torch.zeros(2, 3, 2)), lambda: layer.glu_fwd(x, w, w),
                 lambda: layer.glu_bwd(x, w, w, torch.zeros(2, 3, 16))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


class _Cuda:
    """Checks with tensors that lie on the CPU: they count as device -1."""

    def __enter__(self):
        self.mp = pytest.MonkeyPatch()
        for mod in (layer, mixer):
            self.mp.setattr(mod, "_cuda", lambda t, name: t.get_device())

    def __exit__(self, *exc):
        self.mp.undo()


@pytest.mark.parametrize("call,err,match", [
    (lambda x, r: layer._gated_inputs(x[0], x[0], x[0], r, 8.0, 3), ValueError, r"\[B, T, D\]"),
    (lambda x, r: layer._gated_inputs(x, x, x, r, 0.0, 3), ValueError, "scale"),
    (lambda x, r: layer._gated_inputs(x, x, x, r, float("nan"), 3), ValueError, "scale"),
    (lambda x, r: layer._gated_inputs(x, x[:, :2], x, r, 8.0, 3), ValueError, "decay must have shape"),
    (lambda x, r: layer._gated_inputs(x, x, x.bfloat16(), r, 8.0, 3), TypeError, "gate must be"),
    (lambda x, r: layer._gated_inputs(x, x, x, r.double(), 8.0, 3), TypeError, "rate must be"),
    (lambda x, r: layer._gated_inputs(x, x, x, None, 8.0, 3), TypeError, "rate must be a tensor"),
    (lambda x, r: layer._gated_inputs(x.half(), x.half(), x.half(), r, 8.0, 3), TypeError, "unsupported dtype"),
    (lambda x, r: layer._group_inputs(x, 3, None, None, None), ValueError, "groups must divide"),
    (lambda x, r: layer._group_inputs(x, 0, None, None, None), ValueError, "groups must divide"),
    (lambda x, r: layer._group_inputs(x, 2.0, None, None, None), TypeError, "groups must be an integer"),
    (lambda x, r: layer._group_inputs(x, True, None, None, None), TypeError, "groups must be an integer"),
    (lambda x, r: layer._group_inputs(x, 2, r[:4], r, None), ValueError, "bias must have shape"),
    (lambda x, r: layer._group_inputs(x, 2, r[:3], None, None), ValueError, "weight must have shape"),
    (lambda x, r: layer._group_inputs(x, 2, [1.0], None, None), TypeError, "weight must be a tensor"),
    (lambda x, r: layer._group_inputs(x, 2, None, None, x[:, :2]), ValueError, "gate must have shape"),
    (lambda x, r: layer._glu_inputs(x, torch.zeros(16, 7), torch.zeros(16, 7)), ValueError, "w_gate must have shape"),
    (lambda x, r: layer._glu_inputs(x, torch.zeros(16, 8), torch.zeros(15, 8)), ValueError, "w_up must have shape"),
    (lambda x, r: layer._glu_inputs(x, torch.zeros(0, 8), torch.zeros(0, 8)), ValueError, "at least one row"),
    (lambda x, r: layer._glu_inputs(x, None, torch.zeros(16, 8)), TypeError, "w_gate must be a tensor"),
    (lambda x, r: layer._glu_inputs(x, torch.zeros(8, 16).t(), torch.zeros(16, 8)), ValueError, "contiguous in its last axis"),
    (lambda x, r: layer._glu_activation("relu"), ValueError, "unknown activation"),
    (lambda x, r: layer._glu_status(torch.zeros(8, dtype=torch.uint8), -1), ValueError, "256"),
    (lambda x, r: layer._glu_status(r, -1), TypeError, "status must be"),
    (lambda x, r: layer.glu_bwd(x, torch.zeros(16, 8), torch.zeros(16, 8), torch.zeros(2, 3, 16), torch.zeros(2, 3, 16)), ValueError, "come together"),
    (lambda x, r: layer.group_norm_bwd(x, x, 2, None, None, None, None, torch.zeros(2, 3, 2), grads=dict(dweight=r)), ValueError, "does not compute"),
    (lambda x, r: layer.gated_scan_bwd(x, x, x, r, None, x, grads=dict(dh0=r)), ValueError, "does not compute"),
    (lambda x, r: layer.gated_scan_bwd(x, x, x, r, None, x, states=torch.zeros(2, 8)), ValueError, "states must have shape"),
])
def test_refusals_by_name(call, err, match):
    with _Cuda():
        with pytest.raises(err, match=match):
            call(torch.zeros(2, 3, 8), torch.zeros(8))
