"""Host-side checks of include/mixer.h that need no GPU: exports, argument refusals before any
launch, the layout of the argument blocks, the segment arithmetic of packed batches, and the
Python binding's checks of shapes and strides."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from chunkwise_gated_delta_gb300 import _lib, mixer
from chunkwise_gated_delta_gb300 import build as kbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP, SPACE = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE
BASE = 1 << 40                               # made-up, well separated addresses; never dereferenced


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


def _header():
    src = open(os.path.join(ROOT, "include", "mixer.h")).read()
    return re.sub(r"/\*.*?\*/", "", src, flags=re.S)


def test_exports_every_declared_symbol(lib):
    declared = set(re.findall(r"^(?:kda_status|size_t) (\w+)\(", _header(), flags=re.M))
    assert declared == set(_lib.MIXER_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def test_argument_blocks_have_the_headers_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    blocks = {n: a for n, (a, _) in _lib.MIXER_EXPORTS.items() if not n.endswith("_workspace")}
    lines = [f'printf("{n} %zu\\n", sizeof({n}_args));' for n in blocks]
    lines += [f'printf("{n}.{f} %zu\\n", offsetof({n}_args, {f}));' for n, a in blocks.items() for f, _ in a._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "mixer.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True, timeout=120)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True,
                                                       timeout=60).stdout.splitlines())
    for n, a in blocks.items():
        assert int(got[n]) == ctypes.sizeof(a)
        for f, _ in a._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(a, f).offset, (n, f)


_SIZES = {"layer_norm_fwd": dict(rows=8, D=64, eps=1e-5), "layer_norm_bwd": dict(rows=8, D=64),
          "short_conv_fwd": dict(B=2, T=50, D=64, W=4), "short_conv_bwd": dict(B=2, T=50, D=64, W=4),
          "short_conv_step": dict(B=4, D=64, W=4, slots=9),
          "ssm_scan_fwd": dict(B=2, T=50, D=64, N=16), "ssm_scan_bwd": dict(B=2, T=50, D=64, N=16),
          "ssm_scan_step": dict(B=4, D=64, N=16, slots=9)}


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
    _s = _SIZES[_n]
    _CASES += [(_n, dict(dtype=5), BAD), (_n, dict(D=0), BAD), (_n, dict(x=None), BAD)]
    _CASES += [(_n, dict(x=BASE + 1), BAD), (_n, dict(ld_x=63), BAD), (_n, dict(ld_x=-64), BAD)]
    if "flags" in dict(_lib.MIXER_EXPORTS[_n][0]._fields_):
        _CASES.append((_n, dict(flags=2), BAD))
    if "B" in _s:
        _CASES.append((_n, dict(B=0), BAD))
    if "T" in _s:
        _CASES += [(_n, dict(T=0), BAD), (_n, dict(B=1 << 16, T=1 << 16), BAD), (_n, dict(cu_seqlens=BASE + 2), BAD)]
    if "W" in _s:
        _CASES += [(_n, dict(W=0), BAD), (_n, dict(W=1), UNSUP), (_n, dict(W=5), UNSUP), (_n, dict(weight=None), BAD),
                   (_n, dict(w_dtype=9), BAD)]
    if "N" in _s:
        _CASES += [(_n, dict(N=0), BAD), (_n, dict(N=33), UNSUP), (_n, dict(A=None), BAD), (_n, dict(delta=None), BAD),
                   (_n, dict(ld_B=15), BAD), (_n, dict(A=BASE + 2), BAD)]
    if "slots" in _s:
        _CASES += [(_n, dict(slots=0), BAD), (_n, dict(slot=None, slots=3), BAD), (_n, dict(state=None), BAD)]
_CASES += [("layer_norm_fwd", dict(rows=0), BAD), ("layer_norm_fwd", dict(eps=-1.0), BAD),
           ("layer_norm_fwd", dict(eps=float("nan")), BAD), ("layer_norm_fwd", dict(y=None), BAD),
           ("layer_norm_bwd", dict(mean=None), BAD), ("layer_norm_bwd", dict(rows=5000, workspace=None), SPACE),
           ("layer_norm_bwd", dict(rows=5000, workspace_bytes=64), SPACE),
           ("layer_norm_bwd", dict(rows=5000, workspace=BASE + (1 << 45) + 4), BAD),
           ("short_conv_bwd", dict(workspace=None), SPACE), ("short_conv_bwd", dict(dx=None), BAD),
           ("ssm_scan_bwd", dict(workspace_bytes=1024), SPACE), ("ssm_scan_bwd", dict(dz=None), BAD),
           ("ssm_scan_bwd", dict(z=None), BAD), ("ssm_scan_bwd", dict(dA=None), BAD),
           # outputs over inputs, or over each other
           ("layer_norm_fwd", dict(y=_at("layer_norm_fwd", "x", 128)), BAD),
           ("layer_norm_bwd", dict(dbias=_at("layer_norm_bwd", "dweight", 64)), BAD),
           ("short_conv_fwd", dict(y=_at("short_conv_fwd", "x")), BAD),
           ("short_conv_step", dict(y=_at("short_conv_step", "state", 1024)), BAD),
           ("ssm_scan_fwd", dict(ht=_at("ssm_scan_fwd", "h0")), BAD),
           ("ssm_scan_bwd", dict(dx=_at("ssm_scan_bwd", "dy", 6272)), BAD),
           ("ssm_scan_bwd", dict(workspace=_at("ssm_scan_bwd", "dBm")), BAD),
           # columns of one buffer that meet
           ("ssm_scan_fwd", dict(ld_z=128, ld_y=128, y=_at("ssm_scan_fwd", "z", 126)), BAD)]


@pytest.mark.parametrize("name,over,code", _CASES)
def test_refusals_before_any_launch(lib, name, over, code):
    assert getattr(lib, name)(ctypes.byref(_args(name, **over)), None) == code
    query = name + "_workspace"
    if query in _lib.MIXER_EXPORTS and code != SPACE and "workspace" not in over:
        assert getattr(lib, query)(ctypes.byref(_args(name, **over))) == 0


@pytest.mark.parametrize("name", sorted(_lib.MIXER_EXPORTS))
def test_null_argument_block(lib, name):
    fn = getattr(lib, name)
    assert (fn(None, None) == BAD) if _lib.MIXER_EXPORTS[name][1] else (fn(None) == 0)


def test_workspace_sizes(lib):
    size = lambda n, **o: getattr(lib, n + "_workspace")(ctypes.byref(_args(n, **o)))  # noqa: E731
    assert size("layer_norm_bwd", rows=5000) >= 8 * 2 * 64 * 4 and size("layer_norm_bwd", dweight=None, dbias=None) == 0
    assert size("short_conv_bwd") >= 64 * 5 * 4 and size("short_conv_bwd", dweight=None, dbias=None) == 0
    dense, packed = size("ssm_scan_bwd", T=640), size("ssm_scan_bwd", B=2, T=1280, cu_seqlens=BASE)
    assert 0 < dense < packed                # a packed batch has a slot more per sequence
    # halves of one buffer side by side are no overlap
    ok = dict(ld_z=128, ld_x=128, x=_at("ssm_scan_bwd", "z", 128), ld_dx=128, ld_dz=128, dx=_at("ssm_scan_bwd", "dz", 128))
    assert size("ssm_scan_bwd", **ok) > 0


def test_segment_arithmetic(tmp_path):
    nvcc = kbuild._nvcc()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("nvcc not found")
    exe = tmp_path / "mixer_seq_check"
    r = subprocess.run([nvcc, "-O1", "-std=c++17", "-I", kbuild.CSRC, os.path.join(ROOT, "tests", "host", "mixer_seq_check.cu"),
                        "-o", str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# ------------------------------------------------------------------------------ Python binding
CPU = -1                                     # the index of tensors that are on no GPU


def test_rows_takes_what_one_stride_serves():
    buf = torch.zeros(2, 5, 24)
    for t, ld in ((buf, 24), (buf[..., 3:11], 24), (buf[:1, :, 4:6], 24), (buf[:, :1, 0:8], 120), (buf[0, 2:3], 24),
                  (buf[:1, :1, :7], 7), (buf[..., :1], 24)):
        assert mixer._rows(t, "t", t.shape, torch.float32, CPU) == (t.data_ptr(), ld if t.numel() != 24 else 24)


@pytest.mark.parametrize("t,err", [
    (torch.zeros(2, 5, 24).transpose(1, 2), ValueError),        # last axis not contiguous
    (torch.zeros(4, 5, 24)[::2], ValueError),                   # two strides
    (torch.zeros(2, 6, 24)[:, :5], ValueError),
    (torch.zeros(1, 1, 24).expand(2, 5, 24), ValueError),       # rows on top of each other
    (torch.zeros(2, 5, 24, dtype=torch.float64), TypeError),
])
def test_rows_refuses_others(t, err):
    with pytest.raises(err):
        mixer._rows(t, "t", t.shape, torch.float32, CPU)


def test_no_cpu_path():
    x, w = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    for call in (lambda: mixer.layer_norm_fwd(x), lambda: mixer.short_conv_fwd(x, w),
                 lambda: mixer.short_conv_step(x[0], w, None, torch.zeros(3, 3, 8)),
                 lambda: mixer.ssm_scan_fwd(x, x, torch.zeros(8, 4), x[..., :4], x[..., :4])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="activation"):
        mixer._activation("gelu")
    with pytest.raises(TypeError, match="int32"):
        mixer._sequences(torch.zeros(3, dtype=torch.int64), 1, CPU)
    with pytest.raises(ValueError, match="unknown"):
        mixer._known({"dq": None}, ("dx",))
