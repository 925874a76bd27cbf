"""The operators of include/mixer.h at the limits of what they take: workspaces at the promised alignment
and no more, non-finite values, supplied outputs on other streams, gradients that nothing asks for."""
import ctypes

import pytest
import torch

from chunkwise_gated_delta_gb300 import (_lib, layer_norm_bwd, layer_norm_fwd, mixer, short_conv_bwd, short_conv_step, ssm_scan_bwd,
                                         ssm_scan_fwd)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rand(seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return rn, lambda *s: rn(*s).to(dtype)  # noqa: E731


# ------------------------------------------------------------------------------------ workspaces
class _Shifted(mixer._On):
    """Workspaces at 16 bytes past a multiple of 512, and no longer than asked for."""

    seen = 0

    def workspace(self, name, args):
        need = getattr(_lib.load(), name)(ctypes.byref(args))
        if not need:
            return None
        buf = torch.full((need + 32,), 0x5A, dtype=torch.uint8, device=DEV)
        assert buf.data_ptr() % 512 == 0
        args.workspace, args.workspace_bytes = buf.data_ptr() + 16, need
        type(self).seen += 1
        self.buf = buf
        return buf

    def launch(self, name, args):
        super().launch(name, args)
        if getattr(self, "buf", None) is not None:
            assert bool((self.buf[:16] == 0x5A).all()) and bool((self.buf[-16:] == 0x5A).all()), "written outside"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_workspaces_of_sixteen_byte_alignment(dtype, monkeypatch):
    rn, t = _rand(1, dtype)
    x, w, dy = t(700, 96), t(96), t(700, 96)
    _, mean, rstd = layer_norm_fwd(x, w)
    cx, cw, cdy = t(1, 300, 64), t(64, 4), t(1, 300, 64)
    sx = [t(1, 1500, 64), t(1, 1500, 64), -torch.rand(64, 16, device=DEV) - 0.5, t(1, 1500, 16), t(1, 1500, 16), rn(64), t(1, 1500, 64), rn(64), None]
    sdy = t(1, 1500, 64)

    def run():
        y, ht = ssm_scan_fwd(*sx)
        out = {"y": y, "ht": ht}
        for name, grads in (("norm", layer_norm_bwd(dy, x, w, mean, rstd)), ("conv", short_conv_bwd(cx, cw, None, None, cdy)),
                            ("scan", ssm_scan_bwd(*sx, sdy))):
            out.update({f"{name}.{k}": v for k, v in grads.items()})
        return out

    ref = run()
    monkeypatch.setattr(mixer, "_On", _Shifted)
    got = run()
    torch.cuda.synchronize()
    assert _Shifted.seen >= 4
    _Shifted.seen = 0
    for k in ref:
        assert torch.equal(got[k], ref[k]), k


# ------------------------------------------------------------------------------------ sizes near 2^31
def test_rows_of_more_columns_than_a_signed_step_reaches():
    """One row of 2^31 - 1 values, half of them 1, half -1 and a last 0: every sum is a whole number that
    float32 holds, so the mean is 0 and a normalised value is 1 / sqrt(1 + eps) up to a few units of
    float32, which bfloat16 rounds to 1.  The same row as dy: mean(g xh) = rstd (D - 1) / D, so dx =
    x rstd (1 - xh rstd) < 2 eps, and 0 at the end."""
    D = (1 << 31) - 1
    x = torch.ones(1, D, dtype=torch.bfloat16, device=DEV)
    x[0, 1::2] = -1
    x[0, -1] = 0
    y, mean, rstd = layer_norm_fwd(x, eps=1e-5)
    assert float(mean[0]) == 0.0 and abs(float(rstd[0]) - (1 + 1e-5) ** -0.5) <= 1e-6
    assert torch.equal(y, x)
    got = layer_norm_bwd(x, x, None, mean, rstd, bias=False, grads=dict(dx=y))
    assert set(got) == {"dx"} and float(y[0, -1]) == 0.0
    assert float(y.max()) <= 2e-5 and float(y.min()) >= -2e-5


def test_parameter_sums_of_more_column_blocks_than_a_grid_has_in_y():
    """65536 blocks of 256 columns and five more.  x of ones and minus ones (mean 0, whole sums), dy of small
    whole numbers: dbias is exact, dweight = rstd sum(dy x) off by two roundings of each of three
    products and of their sums, 5 u of at most 6."""
    D, rows = 65536 * 256 + 5, 3
    x = torch.ones(rows, D, device=DEV)
    x[:, 1::2] = -1
    x[:, -1] = 0
    g = torch.Generator(device=DEV).manual_seed(2)
    dy = torch.randint(-2, 3, (rows, D), generator=g, device=DEV).float()
    w = torch.ones(D, device=DEV)
    _, mean, rstd = layer_norm_fwd(x, w)
    got = layer_norm_bwd(dy, x, w, mean, rstd)
    assert torch.equal(got["dbias"], dy.sum(0))
    ref = (dy.double() * x.double() * rstd.double()[:, None]).sum(0)
    assert float((got["dweight"].double() - ref).abs().max()) <= 5 * 2.0 ** -24 * 6


def test_single_tokens_of_more_requests_than_blocks_end_at():
    """2^31 - 1 requests of one channel: the last block has a thread past them."""
    B = (1 << 31) - 1
    x = torch.full((B, 1), 2.0, dtype=torch.bfloat16, device=DEV)
    x[-1] = 3
    state = torch.full((B, 1, 1), 5.0, dtype=torch.bfloat16, device=DEV)
    state[-1] = 7
    w = torch.tensor([[1.0, 10.0]], dtype=torch.bfloat16, device=DEV)
    y = short_conv_step(x, w, None, state, activation=None)
    assert float(y[0]) == 25.0 and float(y[-2]) == 25.0 and float(y[-1]) == 37.0 and bool((y[:-1] == 25).all())
    assert torch.equal(state[:, 0], x)


def test_many_sequences_of_many_packed_tokens():
    """4096 sequences of 256 tokens each, packed: more than 2^31 as a product, 2^20 rows in memory.  Against
    the same sequences as a dense batch: bit for bit where a sequence is walked alone, in another order of sums
    over the sequences (relative 1e-4 as in the operators' own tests) for the parameters' gradients."""
    n, T, D, N = 4096, 256, 8, 4
    rn, t = _rand(7, torch.float32)
    x, w, b, dy = t(n, T, D), t(D, 4), t(D), t(n, T, D)
    delta, A, bc, z = t(n, T, D), -torch.rand(D, N, device=DEV) - 0.5, t(n, T, N), t(n, T, D)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV) * T
    flat = lambda v: v.reshape(1, n * T, -1)  # noqa: E731

    def run(f, cu):
        y, ht = mixer.short_conv_fwd(f(x), w, b, cu_seqlens=cu)
        out = dict(y=y, ht=ht, **short_conv_bwd(f(x), w, b, None, f(dy), cu_seqlens=cu))
        args = (f(x), f(delta), A, f(bc), f(bc), b, f(z), b, None)
        out["scan"], out["state"] = ssm_scan_fwd(*args, cu_seqlens=cu)
        out.update({"scan." + k: v for k, v in ssm_scan_bwd(*args, f(dy), cu_seqlens=cu).items()})
        return out

    one, two = run(lambda v: v, None), run(flat, cu)
    for k, v in one.items():
        if k in ("y", "ht", "dx", "scan", "state", "scan.dx", "scan.ddelta", "scan.dB", "scan.dC", "scan.dz"):
            assert torch.equal(v.reshape(-1), two[k].reshape(-1)), k
        else:
            assert float((v.double() - two[k].double()).norm()) <= 1e-4 * float(v.double().norm()), k


# ------------------------------------------------------------------------------------ outputs on other streams
def _calls(T=2000, D=1024, N=16):
    """Every operator with all of its outputs supplied: (name, names and shapes of the outputs, call)."""
    rn, t = _rand(4, torch.float32)
    x, w, b, cw, h, bc = t(1, T, D), t(D), t(D), t(D, 4), t(1, 3, D), t(1, T, N)
    A, sh = -torch.rand(D, N, device=DEV) - 0.5, rn(1, D, N)
    _, mean, rstd = layer_norm_fwd(x, w, b)
    seq, vec = (1, T, D), (D,)
    yield "layer_norm_fwd", dict(y=seq), lambda o, s: layer_norm_fwd(x, w, b, y=o["y"], stream=s)
    yield ("layer_norm_bwd", dict(dx=seq, dweight=vec, dbias=vec),
           lambda o, s: layer_norm_bwd(x, x, w, mean, rstd, grads=o, stream=s))
    yield "short_conv_fwd", dict(y=seq, ht=(1, 3, D)), lambda o, s: mixer.short_conv_fwd(x, cw, b, h, y=o["y"], ht=o["ht"], stream=s)
    yield ("short_conv_bwd", dict(dx=seq, dweight=(D, 4), dbias=vec, dh0=(1, 3, D)),
           lambda o, s: short_conv_bwd(x, cw, b, h, x, grads=o, stream=s))
    state = t(T, 3, D)
    yield "short_conv_step", dict(y=(T, D)), lambda o, s: short_conv_step(x[0], cw, b, state, y=o["y"], stream=s)
    args = (x, x, A, bc, bc, w, x, b, sh)
    yield "ssm_scan_fwd", dict(y=seq, ht=(1, D, N)), lambda o, s: ssm_scan_fwd(*args, y=o["y"], ht=o["ht"], stream=s)
    yield ("ssm_scan_bwd", dict(dx=seq, ddelta=seq, dz=seq, dB=(1, T, N), dC=(1, T, N), dA=(D, N), dD=vec, ddelta_bias=vec, dh0=(1, D, N)),
           lambda o, s: ssm_scan_bwd(*args, x, grads=o, stream=s))
    st = t(T, D, N)
    yield ("ssm_scan_step", dict(y=(T, D)),
           lambda o, s: mixer.ssm_scan_step(x[0], x[0], A, bc[0], bc[0], st, w, x[0], b, y=o["y"], stream=s))


def test_supplied_outputs_are_not_handed_out_while_the_call_runs():
    """The call waits on its stream behind a quarter of a second of other work; the outputs' memory, given up by the caller
    meanwhile, must not come back from the allocator."""
    side = torch.cuda.Stream()
    for name, shapes, call in _calls():
        call({k: torch.empty(v, device=DEV) for k, v in shapes.items()}, None)        # (compiled modules loaded, pools warm)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out = {k: torch.empty(v, device=DEV) for k, v in shapes.items()}
        at = {t.data_ptr() for t in out.values()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(500_000_000)
        res = call(dict(out), side)
        busy = not side.query()
        del out, res
        new = [torch.empty(v, device=DEV) for v in shapes.values()]
        assert busy and not at & {t.data_ptr() for t in new}, name
        torch.cuda.synchronize()


# ------------------------------------------------------------------------------------ refusals
def test_gradient_buffers_without_their_inputs_are_refused():
    """They would come back in the result as they were."""
    rn, t = _rand(5, torch.float32)
    x, w, h, A, bc = t(1, 20, 8), t(8), t(1, 3, 8), -torch.rand(8, 4, device=DEV), t(1, 20, 4)
    _, mean, rstd = layer_norm_fwd(x, w)
    norm = lambda **g: layer_norm_bwd(x, x, g.pop("weight", None), mean, rstd, bias=g.pop("bias", False), grads=g)  # noqa: E731
    conv = lambda **g: short_conv_bwd(x, t(8, 4), None, None, x, grads=g)  # noqa: E731
    scan = lambda **g: ssm_scan_bwd(x, x, A, bc, bc, None, None, None, None, x, grads=g)  # noqa: E731
    for call, buffers in ((norm, dict(dweight=w, dbias=w)), (conv, dict(dbias=w, dh0=h)),
                          (scan, dict(dD=w, ddelta_bias=w, dz=torch.empty_like(x), dh0=t(1, 8, 4)))):
        given = set(call())
        for k, v in buffers.items():
            assert k not in given
            with pytest.raises(ValueError, match=f"does not compute.*{k}"):
                call(**{k: v})
            assert set(call(**{k: None})) == given
    assert set(norm(weight=w, bias=True, dweight=torch.empty_like(w), dbias=torch.empty_like(w))) == {"dx", "dweight", "dbias"}


def test_arguments_that_are_no_tensors_are_refused_by_name():
    rn, t = _rand(6, torch.float32)
    x, w, A, bc = t(1, 20, 8), t(8, 4), -torch.rand(8, 4, device=DEV), t(1, 20, 4)
    state, scan_state = t(20, 3, 8), t(20, 8, 4)
    for call, name in ((lambda: mixer.short_conv_fwd(x, None), "weight"), (lambda: short_conv_bwd(x, None, None, None, x), "weight"),
                       (lambda: short_conv_step(x[0], None, None, state), "weight"), (lambda: short_conv_step(x[0], w, None, None), "state"),
                       (lambda: mixer.short_conv_fwd(x, w, cu_seqlens=[0, 20]), "cu_seqlens"),
                       (lambda: ssm_scan_fwd(x, x, None, bc, bc), "A"), (lambda: ssm_scan_fwd(x, x, A, None, bc), "B"),
                       (lambda: ssm_scan_fwd(x, None, A, bc, bc), "delta"), (lambda: ssm_scan_bwd(x, x, A, bc, bc, None, None, None, None, None), "dy"),
                       (lambda: mixer.ssm_scan_step(x[0], x[0], A, bc[0], bc[0], None), "state"),
                       (lambda: layer_norm_fwd(x, [1.0]), "weight"), (lambda: layer_norm_bwd(x, x, None, None, None), "mean")):
        with pytest.raises(TypeError, match=f"{name} must be a tensor"):
            call()
    assert mixer.ssm_scan_step(x[0], x[0], A, bc[0], bc[0], scan_state).shape == (20, 8)
