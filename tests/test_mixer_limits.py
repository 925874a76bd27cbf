"""Limits of the operators of include/mixer.h that need no GPU: what the types of the kernels' accesses
assume, counters near 2^31, sizes that are taken or refused, and the Python binding's refusals."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from chunkwise_gated_delta_gb300 import build as kbuild
from chunkwise_gated_delta_gb300 import _lib, mixer


def _nvcc():
    nvcc = kbuild._nvcc()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("nvcc not found")
    return nvcc


def _compile(tmp_path, src, *flags):
    f = tmp_path / "check.cu"
    f.write_text(src)
    return subprocess.run([_nvcc(), "-O1", "-std=c++17", *flags, "-I", kbuild.CSRC, str(f), "-o", str(tmp_path / "check")],
                          capture_output=True, text=True, timeout=600)


@pytest.mark.parametrize("kind,count,ok", [("float", 4, True), ("mixer::bf16", 8, True), ("float", 8, False), ("mixer::bf16", 16, False)])
def test_no_access_is_wider_than_the_workspaces_alignment(tmp_path, kind, count, ok):
    """Workspaces are promised 16-byte alignment, so a type whose alignment is more must not exist."""
    r = _compile(tmp_path, f'#include "mixer_common.cuh"\nsize_t n = alignof(mixer::Vec<{kind}, {count}>);\n', *kbuild.ARCH, "-c")
    assert (r.returncode == 0) is ok, r.stderr[-2000:]
    assert ok or "at most 16 bytes" in r.stderr


def test_positions_past_the_longest_length(tmp_path):
    """The scan's forward walks whole sequences of up to 2^31 - 1 tokens and looks some tiles ahead."""
    exe = tmp_path / "mixer_limits_check"
    r = subprocess.run([_nvcc(), "-O1", "-std=c++17", "-I", kbuild.CSRC, os.path.join(kbuild.ROOT, "tests", "host", "mixer_limits_check.cu"),
                        "-o", str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_rows_that_the_gated_recurrence_reads(tmp_path):
    """None but covered rows, also where all packed sequences are empty and lie at the end."""
    exe = tmp_path / "extent_check"
    r = subprocess.run([_nvcc(), "-O1", "-std=c++17", "-I", kbuild.CSRC, os.path.join(kbuild.ROOT, "tests", "host", "extent_check.cu"),
                        "-o", str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# ------------------------------------------------------------------------------------ Python binding
class _Stream:
    """Stands in for a CUDA stream."""

    def __init__(self, index, handle):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


@pytest.mark.parametrize("handle", [0, 7])
def test_streams_of_other_devices_are_refused(monkeypatch, handle):
    """Their kernels would run where the tensors are not; the handle may even be the current stream's (both 0)."""
    monkeypatch.setattr(mixer, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(mixer, "_device_index", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert mixer._On(0, _Stream(0, handle), ()).handle == handle
    with pytest.raises(ValueError, match="stream must be on device cuda:0, not cuda:1"):
        mixer._On(0, _Stream(1, handle), ())


def test_gradients_that_a_call_does_not_compute_are_refused():
    t = torch.zeros(3)
    names = ("dx", "dweight", "dbias")
    assert mixer._known(dict(dx=t, dbias=None), names, dweight=False, dbias=False) == dict(dx=t)
    assert mixer._known(dict(dx=t, dweight=t), names, dweight=True, dbias=False) == dict(dx=t, dweight=t)
    with pytest.raises(ValueError, match="does not compute.*dbias"):
        mixer._known(dict(dx=t, dbias=t), names, dweight=True, dbias=False)


def test_arguments_that_are_no_tensors_are_refused_by_name():
    w = torch.zeros(8, 4)
    assert mixer._weights(w, None, "weight", (8, None), 8, -1, w.dtype) == (w.data_ptr(), None, w.dtype)
    assert mixer._weights(None, None, "weight", (8,), 8, -1, w.dtype) == (None, None, w.dtype)
    for call, name in ((lambda: mixer._weights(None, None, "weight", (8, None), 8, -1, w.dtype), "weight"),
                       (lambda: mixer._weights([1.0], None, "weight", (1,), 1, -1, w.dtype), "weight"),
                       (lambda: mixer._weights(w, [1.0], "weight", (8, None), 8, -1, w.dtype), "bias"),
                       (lambda: mixer._sequences([0, 3], 1, -1), "cu_seqlens"), (lambda: mixer._cuda(None, "x"), "x")):
        with pytest.raises(TypeError, match=f"{name} must be a tensor"):
            call()


# ------------------------------------------------------------------------------------ sizes
def _workspace(name, **sizes):
    """The workspace that the library asks for: checks of the arguments and no launch (the addresses are made up)."""
    kbuild.build()
    a = _lib.MIXER_EXPORTS[name][0]()
    for i, (f, t) in enumerate(a._fields_):
        if t is ctypes.c_void_p and f != "cu_seqlens":
            setattr(a, f, (i + 1) << 40)
    for k, v in {**dict(workspace_bytes=1 << 33), **sizes}.items():
        if any(f == k for f, _ in a._fields_):
            setattr(a, k, v)
    return getattr(_lib.load(), name + "_workspace")(ctypes.byref(a))


@pytest.mark.parametrize("name", ["short_conv_bwd", "ssm_scan_bwd"])
def test_a_packed_batch_has_as_many_rows_as_tokens(name):
    """2048 sequences in 2^20 packed tokens are 2^20 rows; dense they would be 2^31, one too many.  (Workspace
    queries, which check the arguments and launch nothing; the addresses are made up.)"""
    size = lambda **over: _workspace(name, **{**dict(B=2048, T=1 << 20, D=8, W=4, N=16), **over})  # noqa: E731
    assert size(cu_seqlens=1 << 30) > 0
    assert size() == 0 and size(T=(1 << 20) - 1) > 0


_WHOLE_SPLIT = [  # dtype, N, B, D, T and the two forms' times in us on one GB300 (152 SMs)
    ("bf16", 4, 2, 2048, 4096, 176, 119), ("bf16", 4, 4, 2048, 4096, 179, 219), ("bf16", 8, 1, 2048, 2048, 90, 43), ("bf16", 8, 4, 2048, 16384, 698, 896),
    ("bf16", 16, 1, 1024, 16384, 527, 161), ("bf16", 16, 1, 2048, 4096, 135, 88), ("bf16", 16, 2, 2048, 2048, 70, 88),
    ("bf16", 16, 2, 2048, 4096, 136, 162), ("bf16", 16, 2, 2048, 16384, 527, 590), ("bf16", 12, 4, 1216, 8192, 267, 324),
    ("bf16", 16, 1, 256, 512, 21, 27), ("bf16", 32, 1, 2048, 4096, 221, 181), ("bf16", 32, 2, 1216, 8192, 478, 373),
    ("f32", 4, 2, 2048, 2048, 144, 90), ("f32", 8, 2, 2048, 4096, 185, 158), ("f32", 8, 4, 2048, 8192, 370, 560), ("f32", 16, 1, 1024, 2048, 82, 43),
    ("f32", 16, 2, 2048, 16384, 616, 754), ("f32", 16, 4, 1216, 16384, 620, 796), ("f32", 32, 1, 2048, 16384, 851, 756),
    ("f32", 32, 1, 1024, 1024, 54, 41)]


@pytest.mark.parametrize("dtype,N,B,D,T,whole,split", _WHOLE_SPLIT)
def test_the_scan_is_split_where_that_was_measured_faster(dtype, N, B, D, T, whole, split):
    code = _lib.KDA_BF16 if dtype == "bf16" else _lib.KDA_F32
    assert (_workspace("ssm_scan_fwd", B=B, T=T, D=D, N=N, dtype=code) > 0) == (split < whole)
