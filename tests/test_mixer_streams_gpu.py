"""The operators of include/mixer.h on other streams and under CUDA graph capture.

- A call given ``stream`` runs there, its outputs and workspace allocated in that
  stream's order; calls on two unordered streams give the results of calls in a row.
- A captured training pass (norm, convolution, scan, forward and backward) replays to
  the eager results bit for bit, also after its inputs changed and while other calls
  with larger workspaces ran in between.
- A captured decoding step advances the states in place at every replay.
"""
import pytest
import torch

import chunkwise_gated_delta_gb300 as lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _block(seed, B=2, T=150, D=64, N=16, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    t = lambda *s: rn(*s).to(dtype)  # noqa: E731
    return dict(u=t(B, T, D), nw=t(D), nb=t(D), cw=t(D, 4), cb=t(D), delta=t(B, T, D), A=-torch.rand(D, N, device=DEV) - 0.2,
                Bm=t(B, T, N), Cm=t(B, T, N), D=rn(D), z=t(B, T, D), dbias=rn(D) - 2, dy=t(B, T, D))


def _train(v, stream=None):
    kw = dict(stream=stream)
    n, mean, rstd = lib.layer_norm_fwd(v["u"], v["nw"], v["nb"], **kw)
    x, _ = lib.short_conv_fwd(n, v["cw"], v["cb"], **kw)
    args = (x, v["delta"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["dbias"], None)
    y, ht = lib.ssm_scan_fwd(*args, **kw)
    gs = lib.ssm_scan_bwd(*args, v["dy"], **kw)
    gc = lib.short_conv_bwd(n, v["cw"], v["cb"], None, gs["dx"], **kw)
    gn = lib.layer_norm_bwd(gc["dx"], v["u"], v["nw"], mean, rstd, **kw)
    out = {"y": y, "ht": ht}
    for name, grads in (("scan", gs), ("conv", gc), ("norm", gn)):
        out.update({f"{name}.{k}": t for k, t in grads.items()})
    return out


def _same(a, b):
    assert set(a) == set(b)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_unordered_streams_match_calls_in_a_row():
    vs = [_block(1), _block(2, T=333)]
    refs = [_train(v) for v in vs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        outs = [_train(v, stream=s) for v, s in zip(vs, streams)]
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        _same(o, r)


def test_captured_training_pass_replays_to_the_eager_bits():
    static, other = _block(3), _block(4)
    refs = {k: _train(v) for k, v in (("static", static), ("other", other))}
    saved = {k: t.clone() for k, t in static.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _train(static)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _train(static)
    for which, src in (("static", saved), ("other", other), ("static", saved)):
        for k in static:
            static[k].copy_(src[k])
        _train(_block(5, B=3, T=700))            # an eager call with larger workspaces
        graph.replay()
        torch.cuda.synchronize()
        _same(out, refs[which])


def test_captured_step_advances_the_states():
    v = _block(6, B=4, T=6)
    conv = torch.zeros(4, 3, 64, dtype=torch.bfloat16, device=DEV)
    scan = torch.zeros(4, 64, 16, device=DEV)
    cur = {k: v[k][:, 0].contiguous() for k in ("u", "delta", "Bm", "Cm", "z")}

    def step(conv, scan):
        x = lib.short_conv_step(cur["u"], v["cw"], v["cb"], conv)
        return lib.ssm_scan_step(x, cur["delta"], v["A"], cur["Bm"], cur["Cm"], scan, v["D"], cur["z"], v["dbias"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(conv.clone(), scan.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(conv, scan)
    c2, s2 = torch.zeros_like(conv), torch.zeros_like(scan)
    for t in range(6):
        for k in cur:
            cur[k].copy_(v[k][:, t])
        graph.replay()
        ref = step(c2, s2)
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(conv, c2) and torch.equal(scan, s2)
