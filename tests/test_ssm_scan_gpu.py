"""ssm_scan_fwd / ssm_scan_bwd / ssm_scan_step against the definition in float64.

Tolerances (relative Frobenius), fixed before the first run.  One rounding of the
output, half_step(dtype).  In float32 (u = 2^-24): a decay exp(dt A) is off by the
exponential's 4 u and by the rounding of its argument, at most 3 u |dt A|, and a
state that remembers m tokens gathers m such errors; with the inputs below
dt |A| >= 0.01 for all but a few states and T <= 300, so a state is off by at most
m (4 u) + 8 u with m <= 100: 2.5e-5, and each gradient, a product of two such
recurrences, by twice that plus its sums' rounding: 1e-4.
"""
import ctypes

import pytest
import torch

from chunkwise_gated_delta_gb300 import _lib, ssm_scan_bwd, ssm_scan_fwd, ssm_scan_step

from mixer_ref import half_step, rel, spans_of, ssm_scan

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F_TOL, B_TOL = 2.5e-5, 1e-4
NAMES = ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0")


def _inputs(rows, n, D, N, dtype, seed, gate=True, skip=True, bias=True, h0=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    d = dict(x=rn(rows, D).to(dtype), delta=(0.5 * rn(rows, D) - (0.0 if bias else 2.0)).to(dtype),
             A=-(0.5 + torch.arange(N, device=DEV) + torch.rand(D, N, generator=g, device=DEV)),
             B=rn(rows, N).to(dtype), C=rn(rows, N).to(dtype), D=rn(D) if skip else None,
             z=rn(rows, D).to(dtype) if gate else None, delta_bias=rn(D) - 2.0 if bias else None,
             h0=rn(n, D, N) if h0 else None)
    return d, rn(rows, D).to(dtype), rn(n, D, N)


def _call(d, dy, dht, B, T, cu=None, softplus=True, **kw):
    v = [d[k] if d[k] is None or k in ("A", "D", "delta_bias", "h0") else d[k].reshape(B, T, -1) for k in NAMES]
    y, ht = ssm_scan_fwd(*v, delta_softplus=softplus, cu_seqlens=cu)
    got = ssm_scan_bwd(*v, dy.reshape(B, T, -1), dht, delta_softplus=softplus, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    return y, ht, got


def _reference(d, dy, dht, lens, softplus=True):
    leaf = {k: None if v is None else v.double() for k, v in d.items()}
    names = [k for k in NAMES if leaf[k] is not None]
    for k in names:
        leaf[k].requires_grad_()
    ry, rht = ssm_scan(*(leaf[k] for k in NAMES), spans_of(lens), softplus)
    loss = (ry * dy[:ry.shape[0]].double()).sum() + (rht * dht.double()).sum()
    grads = torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True)
    return ry, rht, {"d" + k: torch.zeros_like(leaf[k]) if r is None else r for k, r in zip(names, grads)}


def _check(d, dy, dht, lens, out, softplus=True):
    y, ht, got = out
    ry, rht, grads = _reference(d, dy, dht, lens, softplus)
    h = half_step(d["x"].dtype)
    assert rel(y.reshape(ry.shape), ry) <= h + F_TOL
    assert rel(ht, rht) <= F_TOL
    assert set(got) == set(grads)
    for k, r in grads.items():
        tol = B_TOL + (h if got[k].dtype == torch.bfloat16 else 0.0)
        assert rel(got[k].reshape(r.shape), r) <= tol, (k, rel(got[k].reshape(r.shape), r))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 4, 5, 8, 16, 24, 32])
def test_state_counts(dtype, N):
    d, dy, dht = _inputs(2 * 75, 2, 37, N, dtype, seed=N)
    _check(d, dy, dht, [75] * 2, _call(d, dy, dht, 2, 75))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D", [(1, 1, 16), (3, 2, 1), (1, 7, 130), (2, 8, 32), (1, 31, 33), (2, 32, 64), (1, 33, 200),
                                   (1, 64, 128), (1, 65, 96), (2, 129, 48), (1, 300, 257)])
def test_lengths_and_channels(dtype, B, T, D):
    d, dy, dht = _inputs(B * T, B, D, 16, dtype, seed=T + D, h0=T % 2 == 1)
    _check(d, dy, dht, [T] * B, _call(d, dy, dht, B, T))


@pytest.mark.parametrize("gate,skip,bias,softplus", [(False, False, False, True), (True, False, True, True),
                                                     (False, True, False, True), (True, True, True, False)])
def test_optional_inputs(gate, skip, bias, softplus):
    d, dy, dht = _inputs(90, 1, 40, 16, torch.float32, seed=11, gate=gate, skip=skip, bias=bias)
    if not softplus:                         # dt itself: positive steps
        d["delta"], d["delta_bias"] = d["delta"].abs() * 0.2 + 0.01, d["delta_bias"].abs() * 0.01
    _check(d, dy, dht, [90], _call(d, dy, dht, 1, 90, softplus=softplus), softplus)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[1, 0, 63, 64, 65, 0, 3], [0, 0, 150], [200, 0], [5]])
def test_packed(dtype, lens):
    T = sum(lens)
    d, dy, dht = _inputs(T, len(lens), 50, 16, dtype, seed=T)
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV)
    _check(d, dy, dht, lens, _call(d, dy, dht, 1, T, cu))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D,lens", [(16, 70, [1500]), (5, 24, [1030, 0, 300, 257, 1]), (32, 100, [900]), (3, 36, [2050]),
                                      (16, 64, [0, 1100]), (16, 48, [1153])])
def test_long_sequences_on_few_channels(dtype, N, D, lens):
    """Few blocks, long sequences: the forward cuts them into segments (256 tokens and more) that
    run side by side; against the definition and against the unsplit form of the same call.
    The tolerance of the module holds for T <= 300; the states' memory, not T, bounds the error, and
    dt |A| >= 0.01 keeps it at 100 tokens here too."""
    T = sum(lens)
    d, dy, dht = _inputs(T, len(lens), D, N, dtype, seed=T + N)
    cu = torch.tensor([0] + [b for _, b in spans_of(lens)], dtype=torch.int32, device=DEV) if len(lens) > 1 else None
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    y, ht = ssm_scan_fwd(*v, cu_seqlens=cu)
    ry, rht = ssm_scan(*(d[k].double() for k in NAMES), spans_of(lens), True)
    assert rel(y[0], ry) <= half_step(dtype) + F_TOL and rel(ht, rht) <= F_TOL
    # the unsplit form: no workspace
    code = _lib.KDA_BF16 if dtype == torch.bfloat16 else _lib.KDA_F32
    y1, ht1 = torch.empty_like(y), torch.empty_like(ht)
    p = lambda t: t.data_ptr()  # noqa: E731
    args = _lib.SsmScanFwdArgs(len(lens), T, D, N, code, 1, p(v[0]), 0, p(v[1]), 0, p(v[3]), 0, p(v[4]), 0, p(v[6]), 0, p(v[2]),
                               p(v[5]), p(v[7]), p(v[8]), p(y1), 0, p(ht1), None, 0, None if cu is None else p(cu))
    lib = _lib.load()
    assert lib.ssm_scan_fwd_workspace(ctypes.byref(args)) > 0
    assert lib.ssm_scan_fwd(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == _lib.KDA_OK
    torch.cuda.synchronize()
    assert rel(y1[0], ry) <= half_step(dtype) + F_TOL and rel(ht1, rht) <= F_TOL


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,D,N", [(3, 1704, 16), (3, 1699, 16), (6, 1704, 8), (2, 1312, 32), (8, 1304, 4), (3, 1704, 12)])
def test_many_channels(dtype, B, D, N):
    """Enough blocks to fill the SMs: full blocks, whole sequences, several tiles and a ragged last one."""
    d, dy, dht = _inputs(B * 75, B, D, N, dtype, seed=B + D + N)
    _check(d, dy, dht, [75] * B, _call(d, dy, dht, B, 75))


def test_empty_batch_of_sequences_passes_the_states():
    d, dy, dht = _inputs(1, 2, 20, 16, torch.float32, seed=12)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    _, ht, got = _call(d, dy, dht, 1, 1, cu)
    assert torch.equal(ht, d["h0"]) and torch.equal(got["dh0"], dht)
    assert not any(bool(got[k].any()) for k in ("dA", "dD", "ddelta_bias"))


def test_rows_outside_every_sequence_are_left_alone():
    d, dy, dht = _inputs(100, 2, 24, 16, torch.float32, seed=13)
    for k in ("x", "delta", "B", "C", "z"):
        d[k][70:] = float("nan")
    dy[70:] = float("nan")
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device=DEV)
    outs = {k: torch.full((1, 100, w), 9.0, device=DEV) for k, w in (("dx", 24), ("ddelta", 24), ("dz", 24), ("dB", 16),
                                                                     ("dC", 16))}
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    y = torch.full((1, 100, 24), 9.0, device=DEV)
    ssm_scan_fwd(*v, y=y, cu_seqlens=cu)
    got = ssm_scan_bwd(*v, dy[None], dht, grads=outs, cu_seqlens=cu)
    assert bool((y[0, 70:] == 9).all()) and all(bool((outs[k][0, 70:] == 9).all()) for k in outs)
    assert bool(torch.isfinite(y).all()) and all(bool(torch.isfinite(t).all()) for t in got.values())


def test_offsets_out_of_range_are_clamped():
    """Offsets below 0 and above T act as 0 and T."""
    d, dy, dht = _inputs(80, 2, 24, 16, torch.float32, seed=14)
    good = torch.tensor([0, 33, 80], dtype=torch.int32, device=DEV)
    bad = torch.tensor([-7, 33, 1 << 30], dtype=torch.int32, device=DEV)
    (y, ht, g1), (y2, ht2, g2) = _call(d, dy, dht, 1, 80, good), _call(d, dy, dht, 1, 80, bad)
    assert torch.equal(y, y2) and torch.equal(ht, ht2) and all(torch.equal(g1[k], g2[k]) for k in g1)


def test_no_final_state_gradient_is_zero():
    d, dy, _ = _inputs(70, 1, 24, 16, torch.float32, seed=15)
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    one = ssm_scan_bwd(*v, dy[None])
    two = ssm_scan_bwd(*v, dy[None], torch.zeros(1, 24, 16, device=DEV))
    assert all(torch.equal(one[k], two[k]) for k in one)
    y, ht = ssm_scan_fwd(*v, output_final_state=False)
    assert ht is None and torch.equal(y, ssm_scan_fwd(*v)[0])


def test_extreme_steps():
    """delta far to the left: no step, the state stays; far to the right: dt = delta, the past is gone."""
    d, dy, dht = _inputs(40, 1, 8, 4, torch.float32, seed=16, bias=False)
    d["delta"][:20] = -100.0
    _, ht, got = _call({k: (v[:20].contiguous() if k in ("x", "delta", "B", "C", "z") else v) for k, v in d.items()},
                       dy[:20], dht, 1, 20)
    assert torch.equal(ht, d["h0"]) and rel(got["dh0"] - dht, _reference(
        {k: (v[:20] if k in ("x", "delta", "B", "C", "z") else v) for k, v in d.items()}, dy[:20], dht, [20])[2]["dh0"] - dht) <= B_TOL
    d["delta"][20:] = 100.0
    out = _call(d, dy, dht, 1, 40)
    _check(d, dy, dht, [40], out)
    # the step's derivative for tiny steps: exp(delta), not zero, to relative precision
    d["delta"][:] = -20.0
    _check(d, dy, dht, [40], _call(d, dy, dht, 1, 40))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decays_of_a_long_memory_have_no_drift(dtype):
    """x = 0, h0 = 1: ht is the product of T decays.  A decay's error may be 1.2e-8 in the mean; the
    products' and arguments' roundings have mean zero, but for log2 e's own, at most 2^-25 of an exponent
    of about 8 in all."""
    T, D, N = 512, 64, 16
    g = torch.Generator(device=DEV).manual_seed(24)
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    delta, A = (0.01 * (0.5 + rand(1, T, D))).to(dtype), -(1 + rand(D, N))
    x, bc, h0 = delta.new_zeros(1, T, D), delta.new_ones(1, T, N), torch.ones(1, D, N, device=DEV)
    exact = (delta[0].double().sum(0)[:, None] * A.double()).exp()
    tol = T * 1.2e-8 + 8 * 2.0 ** -25
    _, ht = ssm_scan_fwd(x, delta, A, bc, bc, h0=h0, delta_softplus=False)
    assert abs(float((ht[0].double() / exact - 1).mean())) <= tol
    state = h0.clone()
    for t in range(T):
        ssm_scan_step(x[:, t], delta[:, t], A, bc[:, t], bc[:, t], state, delta_softplus=False)
    assert abs(float((state[0].double() / exact - 1).mean())) <= tol


def test_non_finite_values_stay_in_their_channel():
    d, dy, dht = _inputs(50, 1, 40, 16, torch.float32, seed=17)
    y0, ht0, _ = _call(d, dy, dht, 1, 50)
    d["x"][10, 3], d["delta"][5, 9], d["z"][7, 20] = float("nan"), float("inf"), float("inf")
    y, ht, _ = _call(d, dy, dht, 1, 50)
    keep = [c for c in range(40) if c not in (3, 9, 20)]
    assert torch.equal(y[0, :, keep], y0[0, :, keep]) and torch.equal(ht[0, keep], ht0[0, keep])
    assert torch.equal(y[0, :10, 3], y0[0, :10, 3]) and bool(y[0, 10:, 3].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_in_pieces_equals_one_call(dtype):
    d, dy, dht = _inputs(140, 1, 48, 16, dtype, seed=18)
    v = {k: t if k in ("A", "D", "delta_bias", "h0") else t[None] for k, t in d.items()}
    whole, ht = ssm_scan_fwd(*(v[k] for k in NAMES))
    state, parts = v["h0"], []
    for lo, hi in ((0, 50), (50, 51), (51, 140)):
        w = {k: t if k in ("A", "D", "delta_bias") else t[:, lo:hi].contiguous() for k, t in v.items() if k != "h0"}
        y, state = ssm_scan_fwd(*(w[k] for k in NAMES[:-1]), state)
        parts.append(y)
    assert rel(torch.cat(parts, 1), whole) <= 2 * half_step(dtype) + F_TOL and rel(state, ht) <= F_TOL


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D", [(16, 64), (5, 33), (32, 130), (1, 7), (8, 40)])
def test_steps_against_the_definition(dtype, N, D):
    B, T, S = 3, 5, 7
    d, _, _ = _inputs(B * T, B, D, N, dtype, seed=19 + N)
    ry, rht, _ = _reference(d, torch.zeros(B * T, D, device=DEV), torch.zeros(B, D, N, device=DEV), [T] * B)
    v = {k: t if k in ("A", "D", "delta_bias", "h0") else t.view(B, T, -1) for k, t in d.items()}
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device=DEV)
    state = torch.full((S, D, N), 5.0, device=DEV)
    state[slots.long()] = v["h0"]
    for t in range(T):
        y = ssm_scan_step(v["x"][:, t], v["delta"][:, t], v["A"], v["B"][:, t], v["C"][:, t], state, v["D"], v["z"][:, t],
                          v["delta_bias"], slots=slots)
        assert rel(y, ry.view(B, T, D)[:, t]) <= half_step(dtype) + F_TOL
    assert rel(state[slots.long()], rht) <= F_TOL
    assert bool((state[[1, 2, 3, 5]] == 5).all())


def test_padding_requests_change_nothing():
    d, _, _ = _inputs(4, 4, 24, 16, torch.float32, seed=20)
    state = d["h0"].clone()
    slots = torch.tensor([-1, 2, 4, -(1 << 31)], dtype=torch.int32, device=DEV)
    y = ssm_scan_step(d["x"], d["delta"], d["A"], d["B"], d["C"], state, d["D"], d["z"], d["delta_bias"], slots=slots)
    assert not bool(y[[0, 2, 3]].any()) and bool(y[1].any())
    assert torch.equal(state[[0, 1, 3]], d["h0"][[0, 1, 3]]) and not torch.equal(state[2], d["h0"][2])


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 4), (3, 2)])
def test_row_strides_and_alignment(shift, pad):
    """x and z as halves of one buffer, B and C as parts of another, the gradients likewise."""
    D, N, B, T = 40, 16, 2, 70
    d, dy, dht = _inputs(B * T, B, D, N, torch.bfloat16, seed=21)
    xz = torch.zeros(B, T, 2 * D + pad + shift, dtype=torch.bfloat16, device=DEV)
    bc = torch.zeros(B, T, 2 * N + pad + shift, dtype=torch.bfloat16, device=DEV)
    view = dict(x=xz[..., shift:shift + D], z=xz[..., shift + D:shift + 2 * D], B=bc[..., shift:shift + N],
                C=bc[..., shift + N:shift + 2 * N])
    for k in view:
        view[k].copy_(d[k].view(B, T, -1))
    ref = _call(d, dy, dht, B, T)
    dxz, dbc = torch.full_like(xz, 3.0), torch.full_like(bc, 3.0)
    grads = dict(dx=dxz[..., shift:shift + D], dz=dxz[..., shift + D:shift + 2 * D], dB=dbc[..., shift:shift + N],
                 dC=dbc[..., shift + N:shift + 2 * N])
    v = [view.get(k, d[k] if k in ("A", "D", "delta_bias", "h0") else d[k].view(B, T, -1)) for k in NAMES]
    y, ht = ssm_scan_fwd(*v)
    got = ssm_scan_bwd(*v, dy.view(B, T, D), dht, grads=grads)
    assert torch.equal(y, ref[0]) and torch.equal(ht, ref[1]) and all(torch.equal(got[k], ref[2][k]) for k in got)
    for buf, n in ((dxz, 2 * D), (dbc, 2 * N)):
        assert bool((buf[..., :shift] == 3).all()) and bool((buf[..., shift + n:] == 3).all())


def test_equal_calls_give_equal_bits():
    d, dy, dht = _inputs(1500, 3, 160, 16, torch.bfloat16, seed=22)
    one, two = (_call(d, dy, dht, 3, 500) for _ in range(2))
    assert torch.equal(one[0], two[0]) and all(torch.equal(one[2][k], two[2][k]) for k in one[2])


def test_gradients_against_differences():
    """Central differences of the definition in float64 (step 1e-5: off by about 1e-9 relative)
    on entries of every input."""
    d, dy, dht = _inputs(9, 1, 5, 3, torch.float32, seed=23)
    _, _, got = _call(d, dy, dht, 1, 9)
    base = {k: v.double().cpu() for k, v in d.items()}
    wy, wh = dy.double().cpu(), dht.double().cpu()

    def loss(v):
        y, ht = ssm_scan(*(v[k] for k in NAMES), [(0, 9)], True)
        return float((y * wy).sum() + (ht * wh).sum())

    g = torch.Generator().manual_seed(24)
    for k in NAMES:
        scale = float(got["d" + k].abs().max())
        for at in torch.randperm(base[k].numel(), generator=g)[:4].tolist():
            hi, lo = ({**base, k: base[k].clone()} for _ in range(2))
            hi[k].view(-1)[at] += 1e-5
            lo[k].view(-1)[at] -= 1e-5
            diff = (loss(hi) - loss(lo)) / 2e-5
            assert abs(float(got["d" + k].reshape(-1)[at]) - diff) <= B_TOL * scale + 1e-7, (k, at)


def test_offsets_beyond_32_bits():
    ld = 1_200_000_000
    buf = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    d, dy, dht = _inputs(3, 1, 64, 16, torch.bfloat16, seed=25)
    ref = _call(d, dy, dht, 1, 3)
    v = [d[k] if k in ("A", "D", "delta_bias", "h0") else d[k][None] for k in NAMES]
    for k in ("x", "z", "B"):
        far = buf.as_strided((1, 3, d[k].shape[1]), (3 * ld, ld, 1))
        far.copy_(d[k][None])
        w = [far if n == k else t for n, t in zip(NAMES, v)]
        y, ht = ssm_scan_fwd(*w)
        got = ssm_scan_bwd(*w, dy[None], dht)
        assert torch.equal(y, ref[0]) and all(torch.equal(got[n], ref[2][n]) for n in got), k
