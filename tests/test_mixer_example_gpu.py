"""examples/mixer_block.py: the block's training step against automatic differentiation of the same block
in float64, and prompt-then-decode against one pass.

Tolerances, fixed before the first run: float32 parameters and inputs; the block chains about ten
operators, each off by at most 1e-4 (the scan's gradients) in the relative Frobenius norm, and the matrix
products (float32, sums of up to 64 terms) by 1e-5: 1e-3 in all.  In bfloat16 every intermediate is rounded
(half a step, 2^-8) in both orders of work, about ten times on the way: 2^-8 * 10 = 4e-2.
"""
import importlib.util
import os

import pytest
import torch

from mixer_ref import layer_norm, rel, short_conv, spans_of, ssm_scan

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")


def _module():
    spec = importlib.util.spec_from_file_location("mixer_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(block, u, p):
    B, T, _ = u.shape
    n, _, _ = layer_norm(u, p["norm_w"], p["norm_b"], 1e-5)
    xz = (n @ p["w_in"].t()).reshape(B * T, -1)
    spans, d = spans_of([T] * B), block.inner
    x, _ = short_conv(xz[:, :d], p["conv_w"], p["conv_b"], None, spans, True)
    low, bm, cm = block._parts(x @ p["w_x"].t())
    y, _ = ssm_scan(x, low @ p["w_dt"].t(), p["A"], bm, cm, p["D"], xz[:, d:], p["dt_bias"], None, spans, True)
    return (y @ p["w_out"].t()).reshape(B, T, -1)


def test_training_step_against_automatic_differentiation(monkeypatch):
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_tf32", False)
    block = _module().SsmBlock(model=24, inner=48, states=8, rank=8, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    u, dout = (torch.randn(2, 40, 24, generator=g, device="cuda") for _ in range(2))
    out, grads = block.train(u, dout)
    leaf = {k: v.double().requires_grad_() for k, v in {**block.p, "u": u}.items()}
    ref = _reference(block, leaf["u"], leaf)
    assert rel(out, ref) <= 1e-3
    names = sorted(grads)
    for k, r in zip(names, torch.autograd.grad((ref * dout.double()).sum(), [leaf[k] for k in names])):
        assert rel(grads[k], r) <= 1e-3, (k, rel(grads[k], r))


def test_prompt_and_single_tokens_equal_one_pass():
    assert _module().main() <= 4e-2
