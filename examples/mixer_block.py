"""Two token-mixer blocks on the library's operators: train a step, read a prompt, then decode.

    python examples/mixer_block.py            # needs the GPU and the built library

SsmBlock   norm -> projection to x and a gate z -> short causal convolution -> projection of x to the
           step, B and C -> selective scan with the gate -> projection back.
           ``train`` runs forward and backward and returns every gradient, ``prompt`` returns the
           outputs and the two states (convolution and scan), ``step`` takes one token of each
           request and updates the states in place.
KdaBlock   norm -> one projection to q, k and v -> short causal convolution over all of their
           channels -> the gated delta rule (kda_chunk_fwd): the same first operators in front of
           the other mixer.

The gradient buffers of x and z are halves of one tensor, those of the step, B and C parts of another,
so the projections' gradients are one matrix product each and nothing is copied together.
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import chunkwise_gated_delta_gb300 as lib  # noqa: E402


class SsmBlock:
    def __init__(self, model: int, inner: int, states: int = 16, width: int = 4, rank: int | None = None,
                 dtype=torch.bfloat16, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        ru = lambda *s: torch.rand(*s, generator=g, device=device)  # noqa: E731
        self.inner, self.states, self.width, self.rank = inner, states, width, rank or max(16, inner // 16)
        step0 = torch.exp(ru(inner) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        self.p = dict(
            norm_w=torch.ones(model, dtype=dtype, device=device), norm_b=torch.zeros(model, dtype=dtype, device=device),
            w_in=(rn(2 * inner, model) / math.sqrt(model)).to(dtype),
            conv_w=((2 * ru(inner, width) - 1) / math.sqrt(width)).to(dtype), conv_b=torch.zeros(inner, dtype=dtype, device=device),
            w_x=(rn(self.rank + 2 * states, inner) / math.sqrt(inner)).to(dtype),
            w_dt=(rn(inner, self.rank) / math.sqrt(self.rank)).to(dtype),
            dt_bias=step0 + torch.log(-torch.expm1(-step0)),
            A=-torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1), D=torch.ones(inner, device=device),
            w_out=(rn(model, inner) / math.sqrt(inner)).to(dtype))

    def _parts(self, proj):
        r, n = self.rank, self.states
        return proj[..., :r], proj[..., r:r + n], proj[..., r + n:]

    def _forward(self, u, conv_state=None, scan_state=None):
        p, d = self.p, self.inner
        n, mean, rstd = lib.layer_norm_fwd(u, p["norm_w"], p["norm_b"])
        xz = n @ p["w_in"].t()
        x, conv_state = lib.short_conv_fwd(xz[..., :d], p["conv_w"], p["conv_b"], conv_state)
        proj = x @ p["w_x"].t()
        low, B, C = self._parts(proj)
        delta = low @ p["w_dt"].t()
        args = (x, delta, p["A"], B, C, p["D"], xz[..., d:], p["dt_bias"])
        y, scan_state = lib.ssm_scan_fwd(*args, scan_state)
        return y @ p["w_out"].t(), (conv_state, scan_state), dict(u=u, n=n, mean=mean, rstd=rstd, xz=xz, x=x, proj=proj, delta=delta,
                                                                  args=args, y=y)

    def prompt(self, u, state=(None, None)):
        """u [B, T, model]: (outputs, states); ``state`` continues an earlier part of the prompt."""
        out, state, _ = self._forward(u, *state)
        return out, state

    def step(self, u, state, slots=None):
        """u [B, model], one token of each request; the states are updated in place."""
        p, d = self.p, self.inner
        n, _, _ = lib.layer_norm_fwd(u, p["norm_w"], p["norm_b"])
        xz = n @ p["w_in"].t()
        x = lib.short_conv_step(xz[..., :d], p["conv_w"], p["conv_b"], state[0], slots=slots)
        proj = x @ p["w_x"].t()
        low, B, C = self._parts(proj)
        y = lib.ssm_scan_step(x, low @ p["w_dt"].t(), p["A"], B, C, state[1], p["D"], xz[..., d:], p["dt_bias"], slots=slots)
        return y @ p["w_out"].t()

    def train(self, u, dout):
        """Forward and backward: (outputs, gradients of u and of every parameter by its name)."""
        p, d, flat = self.p, self.inner, lambda t: t.reshape(-1, t.shape[-1])
        out, _, k = self._forward(u)
        g = {}
        dy = dout @ p["w_out"]
        g["w_out"] = flat(dout).t() @ flat(k["y"])
        dxz, dproj = torch.empty_like(k["xz"]), torch.empty_like(k["proj"])
        dlow, dB, dC = self._parts(dproj)
        s = lib.ssm_scan_bwd(*k["args"], None, dy, grads=dict(dz=dxz[..., d:], dB=dB, dC=dC))
        g["A"], g["D"], g["dt_bias"] = s["dA"], s["dD"], s["ddelta_bias"]
        dlow.copy_(s["ddelta"] @ p["w_dt"])
        g["w_dt"] = flat(s["ddelta"]).t() @ flat(self._parts(k["proj"])[0])
        g["w_x"] = flat(dproj).t() @ flat(k["x"])
        dx = s["dx"] + dproj @ p["w_x"]
        c = lib.short_conv_bwd(k["xz"][..., :d], p["conv_w"], p["conv_b"], None, dx, grads=dict(dx=dxz[..., :d]))
        g["conv_w"], g["conv_b"] = c["dweight"], c["dbias"]
        g["w_in"] = flat(dxz).t() @ flat(k["n"])
        m = lib.layer_norm_bwd(dxz @ p["w_in"], u, p["norm_w"], k["mean"], k["rstd"])
        g["norm_w"], g["norm_b"], g["u"] = m["dweight"], m["dbias"], m["dx"]
        return out, g


class KdaBlock:
    def __init__(self, model: int, heads: int, dtype=torch.bfloat16, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.heads, c = heads, heads * 128
        self.p = dict(norm_w=torch.ones(model, dtype=dtype, device=device), norm_b=torch.zeros(model, dtype=dtype, device=device),
                      w_qkv=(rn(3 * c, model) / math.sqrt(model)).to(dtype), w_gate=(rn(c, model) / math.sqrt(model)).to(dtype),
                      w_beta=(rn(heads, model) / math.sqrt(model)).to(dtype),
                      conv_w=((2 * torch.rand(3 * c, 4, generator=g, device=device) - 1) / 2).to(dtype),
                      w_out=(rn(model, c) / math.sqrt(c)).to(dtype))

    def prompt(self, u, state=(None, None)):
        p, h = self.p, self.heads
        n, _, _ = lib.layer_norm_fwd(u, p["norm_w"], p["norm_b"])
        qkv, conv_state = lib.short_conv_fwd(n @ p["w_qkv"].t(), p["conv_w"], None, state[0])
        q, k, v = (t.unflatten(-1, (h, 128)) for t in qkv.chunk(3, -1))
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(u.dtype) for t in (q, k))
        gate = (-0.1 * torch.nn.functional.softplus((n @ p["w_gate"].t()).float())).to(u.dtype).unflatten(-1, (h, 128))
        beta = torch.sigmoid((n @ p["w_beta"].t()).float()).to(u.dtype)
        o, ht = lib.kda_chunk_fwd(q.contiguous(), k.contiguous(), v.contiguous(), gate.contiguous(), beta.contiguous(), state[1])
        return o.flatten(-2) @ p["w_out"].t(), (conv_state, ht)


def main():
    torch.manual_seed(0)
    block = SsmBlock(model=512, inner=1024)
    u = torch.randn(2, 200, 512, device="cuda").to(torch.bfloat16)
    out, grads = block.train(u, torch.randn_like(u))
    print("training step:", {k: tuple(v.shape) for k, v in grads.items()})
    # a prompt of 192 tokens in two parts, then eight tokens one at a time
    a, state = block.prompt(u[:, :100].contiguous())
    b, state = block.prompt(u[:, 100:192].contiguous(), state)
    tail = torch.stack([block.step(u[:, t], state) for t in range(192, 200)], 1)
    diff = float((torch.cat([a, b, tail], 1).float() - out.float()).norm() / out.float().norm())
    print(f"prompt in parts, then single tokens, against one pass: relative difference {diff:.2e}")
    kda = KdaBlock(model=512, heads=4)
    whole, _ = kda.prompt(u)
    print("gated delta-rule block:", tuple(whole.shape))
    return diff


if __name__ == "__main__":
    main()
