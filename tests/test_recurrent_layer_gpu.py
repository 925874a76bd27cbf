"""examples/mixer_block.py's RecurrentLayer, whose every product but the plain matrix products is the library's: its training step
against automatic differentiation of the same layer in float64, and a prompt in parts, then single tokens through slots.

Tolerances, fixed before the first run: in float32 about ten operators in a row, each off by at most 1e-4 in the relative
Frobenius norm, and matrix products of up to 256 terms by 1e-5: 1e-3 in all.  In bfloat16 every intermediate is
rounded (half a step, 2^-8) in both orders of work, about ten times on the way: 2^-8 * 10 = 4e-2."""
import importlib.util
import os

import pytest
import torch

import layer_ref as ref
from mixer_ref import layer_norm, rel, short_conv, spans_of

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")


def _layer(**kw):
    spec = importlib.util.spec_from_file_location("mixer_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.RecurrentLayer(**kw)


def _reference(layer, u, p):
    B, T, M = u.shape
    spans, d = spans_of([T] * B), layer.d
    n, _, _ = layer_norm(u.reshape(B * T, M), p["norm1"], None, 1e-5)
    proj = n @ p["w_in"].t()
    x, _ = short_conv(proj[:, :d], p["conv_w"], None, None, spans, True)
    y, _ = ref.gated_scan(x, proj[:, d:2 * d], proj[:, 2 * d:3 * d], p["rate"], None, spans, 8.0)
    o, _, _ = ref.group_norm(y, layer.heads, p["head_norm"], None, proj[:, 3 * d:], 1e-5, False)
    v = u.reshape(B * T, M) + o @ p["w_out"].t()
    n, _, _ = layer_norm(v, p["norm2"], None, 1e-5)
    h, _, _ = ref.glu(n, p["w_gate"], p["w_up"], "silu")
    return (v + h @ p["w_down"].t()).reshape(B, T, M)


@pytest.mark.parametrize("dtype,bound", [(torch.float32, 1e-3), (torch.bfloat16, 4e-2)], ids=["f32", "bf16"])
def test_training_step_against_automatic_differentiation(monkeypatch, dtype, bound):
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_tf32", False)
    layer = _layer(model=40, heads=3, width=16, inner=72, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    u, dout = (torch.randn(2, 45, 40, generator=g, device="cuda").to(dtype) for _ in range(2))
    out, grads = layer.train(u, dout)
    leaf = {k: v.double().requires_grad_() for k, v in {**layer.p, "u": u}.items()}
    want = _reference(layer, leaf["u"], leaf)
    assert rel(out, want) <= bound
    names = sorted(grads)
    assert set(names) == set(leaf)
    for k, r in zip(names, torch.autograd.grad((want * dout.double()).sum(), [leaf[k] for k in names])):
        assert rel(grads[k], r) <= bound, (k, rel(grads[k], r))


@pytest.mark.parametrize("dtype,bound", [(torch.float32, 1e-3), (torch.bfloat16, 4e-2)], ids=["f32", "bf16"])
def test_prompt_in_parts_then_single_tokens_in_slots(monkeypatch, dtype, bound):
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_tf32", False)
    layer = _layer(model=64, heads=2, width=32, dtype=dtype)
    u = torch.randn(3, 90, 64, device="cuda").to(dtype)
    whole, _ = layer.prompt(u)
    a, state = layer.prompt(u[:, :50].contiguous())
    b, state = layer.prompt(u[:, 50:80].contiguous(), state)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cache = [torch.zeros(6, *s.shape[1:], device="cuda", dtype=s.dtype) for s in state]
    for c, s in zip(cache, state):
        c[slots.long()] = s
    tail = torch.stack([layer.step(u[:, t].contiguous(), cache, slots) for t in range(80, 90)], 1)
    assert rel(torch.cat([a, b, tail], 1), whole.double()) <= bound
    assert all(not bool(c[[1, 3, 5]].any()) for c in cache)


def test_a_captured_decoding_step():
    layer = _layer(model=64, heads=2, width=32)
    u = torch.randn(3, 64, device="cuda").bfloat16()
    state = [torch.randn(3, 3, 64, device="cuda").bfloat16(), torch.randn(3, 64, device="cuda")]
    first = [s.clone() for s in state]
    want = layer.step(u, state)
    after = [s.clone() for s in state]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(u, state)
    for s, f in zip(state, first):
        s.copy_(f)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(s, a) for s, a in zip(state, after))
