"""The gated delta-rule block of examples/mixer_block.py (norm, projection, short convolution, kda_chunk_fwd)
against the same block in float64, whole, in parts with its states carried, and token by token.

Tolerances (relative Frobenius), fixed before the first run: as for the example's other block, 1e-3 in float32
(norm and convolution 2e-5, the delta rule 1e-5, three matrix products and the normalisations 1e-5 each,
with room for a factor of ten through the rule's products of them) and 10 * 2^-8 = 4e-2 in bfloat16 (about ten
roundings of half a step on the way)."""
import importlib.util
import os

import pytest
import torch

import oracle
from mixer_ref import layer_norm, rel, short_conv, spans_of

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 1e-3, torch.bfloat16: 4e-2}

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")


def _block(dtype):
    spec = importlib.util.spec_from_file_location("mixer_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    block = m.KdaBlock(model=96, heads=2, dtype=dtype, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    block.p["norm_w"] += 0.1 * torch.randn(96, generator=g, device="cuda").to(dtype)
    block.p["norm_b"] += 0.1 * torch.randn(96, generator=g, device="cuda").to(dtype)
    return block, torch.randn(2, 150, 96, generator=g, device="cuda").to(dtype)


def _reference(block, u):
    p, h = {k: v.double() for k, v in block.p.items()}, block.heads
    B, T, _ = u.shape
    n, _, _ = layer_norm(u.double(), p["norm_w"], p["norm_b"], 1e-5)
    qkv, conv = short_conv((n @ p["w_qkv"].t()).reshape(B * T, -1), p["conv_w"], None, None, spans_of([T] * B), True)
    q, k, v = (t.reshape(B, T, h, 128) for t in qkv.chunk(3, -1))
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    gate = (-0.1 * torch.nn.functional.softplus(n @ p["w_gate"].t())).reshape(B, T, h, 128)
    beta = torch.sigmoid(n @ p["w_beta"].t())
    o, ht = oracle.kda_fwd(*(t.cpu().numpy() for t in (q, k, v, gate, beta)))
    return torch.from_numpy(o).to(u.device).reshape(B, T, -1) @ p["w_out"].t(), conv, torch.from_numpy(ht).to(u.device)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cuts", [(), (100,), (64, 65, 128), tuple(range(1, 7)) + (90, 91)])
def test_prompt_whole_in_parts_and_by_tokens(dtype, cuts, monkeypatch):
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_tf32", False)
    block, u = _block(dtype)
    ref, conv, ht = _reference(block, u)
    outs, state = [], (None, None)
    for lo, hi in zip((0,) + cuts, cuts + (u.shape[1],)):
        y, state = block.prompt(u[:, lo:hi].contiguous(), state)
        outs.append(y)
    for got, r in ((torch.cat(outs, 1), ref), (state[0], conv), (state[1], ht)):
        assert got.shape == r.shape and rel(got, r) <= TOL[dtype], rel(got, r)
