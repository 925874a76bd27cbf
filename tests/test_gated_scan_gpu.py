"""Gated recurrence on the GPU against its definition in float64: forward, gradients, single tokens, packed batches,
sequences cut anywhere in a tile, strides, infinities, streams and graphs."""
import pytest
import torch

import chunkwise_gated_delta_gb300 as lib
import layer_ref as ref
from mixer_ref import half_step, rel, spans_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 8.0

# A state carries a product of up to n = 1 / (1 - a) decays, here a <= 0.9995 where its gate is half open or more, so n of at
# most 2000; each decay is off by its rounding (2^-24) and by the exponent's relative error (sigmoid's exponential,
# sum, reciprocal, two products: 6 roundings) times -log a, which over n decays adds up to 6 roundings in all.  The
# roundings of a add up as sqrt(n) of independent ones, 45, and at most 2^-24 * 2000 = 1.2e-4 should all of them point one way; the
# bound here takes 8 times the independent sum.
STATE = (8 * 45 + 6) * 2.0 ** -24


def tol(dtype):
    return STATE if dtype == torch.float32 else half_step(dtype) + STATE


def make(rows, n, D, dtype, seed=0, slow=False, h0=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = dict(x=rn(rows, D).to(dtype), decay=rn(rows, D).to(dtype), gate=rn(rows, D).to(dtype), rate=rn(D) - (6 if slow else 1),
             h0=rn(n, D) if h0 else None, dy=rn(rows, D).to(dtype), dht=rn(n, D))
    return s


def definition(s, spans, grads=False):
    f = {k: v.double().requires_grad_(grads and k not in ("dy", "dht")) for k, v in s.items() if v is not None}
    y, ht = ref.gated_scan(f["x"], f["decay"], f["gate"], f["rate"], f.get("h0"), spans, SCALE)
    out = {"y": y, "ht": ht}
    if grads:
        names = [k for k in ("x", "decay", "gate", "rate", "h0") if k in f]
        loss = sum((y[lo:hi] * f["dy"][lo:hi]).sum() for lo, hi in spans) + (ht * f["dht"]).sum()
        got = torch.autograd.grad(loss, [f[k] for k in names], allow_unused=True)
        out.update({"d" + k: torch.zeros_like(f[k]) if v is None else v for k, v in zip(names, got)})
    return {k: v.detach() for k, v in out.items()}


def call(s, shape, cu=None, states=True):
    """Forward and backward; sequence tensors viewed as `shape` [B, T, D]."""
    v = {k: t.view(shape) if k in ("x", "decay", "gate", "dy") else t for k, t in s.items() if t is not None}
    args = (v["x"], v["decay"], v["gate"], v["rate"], v.get("h0"))
    y, ht, st = lib.gated_scan_fwd(*args, scale=SCALE, save_states=True, cu_seqlens=cu)
    g = lib.gated_scan_bwd(*args, v["dy"], v["dht"], states=st if states else None, scale=SCALE, cu_seqlens=cu)
    return {"y": y, "ht": ht, **g}


def compare(got, want, dtype, rows=None):
    for k, w in want.items():
        v = got[k].reshape(w.shape)
        if rows is not None and k not in ("ht", "dh0", "drate"):
            v, w = v[:rows], w[:rows]
        assert rel(v, w) <= tol(v.dtype if k in ("ht", "drate", "dh0") else dtype), k


# (up to 128 rows are one segment)
DENSE = [(1, 1, 1), (2, 64, 70), (1, 128, 34), (1, 129, 34), (4, 100, 20), (1, 1, 64), (3, 1, 130), (2, 2, 2), (1, 31, 63), (2, 32, 64), (1, 33, 65), (2, 63, 66), (1, 64, 128), (3, 65, 8),
         (2, 200, 514), (9, 17, 37)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", DENSE)
def test_dense(B, T, D, dtype):
    s = make(B * T, B, D, dtype, seed=T)
    got = call(s, (B, T, D))
    compare(got, definition(s, spans_of([T] * B), True), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,D,h0", [([5, 1, 0, 64, 3, 31, 1, 1, 40], 70, True), ([0, 0, 7], 64, True), ([129, 1, 300, 0, 62], 33, True),
                                       ([1] * 77, 12, True), ([1] * 200, 12, True), ([100, 0, 28], 34, True), ([64, 64, 32, 32], 128, False), ([333], 2, False), ([0], 3, True)])
def test_packed(lens, D, h0, dtype):
    n, rows = len(lens), max(1, sum(lens))
    s = make(rows, n, D, dtype, seed=D, h0=h0)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    got = call(s, (1, rows, D), cu)
    compare(got, definition(s, spans_of(lens), True), dtype, sum(lens))


@pytest.mark.parametrize("B,T,D", [(1, 5000, 64), (1, 3000, 130), (2, 2100, 40)])
def test_long_memories_and_clusters(B, T, D):
    """Few channels: a chain's tiles go round a cluster of blocks.  Rates of a long memory."""
    s = make(B * T, B, D, torch.float32, seed=3, slow=True)
    compare(call(s, (B, T, D)), definition(s, spans_of([T] * B), True), torch.float32)


def test_one_long_sequence_among_short_ones():
    lens = [3, 0, 2500, 1, 40]
    s = make(sum(lens), len(lens), 66, torch.float32, seed=8, slow=True)
    cu = torch.tensor([0, 3, 3, 2503, 2504, 2544], dtype=torch.int32, device=DEV)
    compare(call(s, (1, sum(lens), 66), cu), definition(s, spans_of(lens), True), torch.float32)


def test_without_saved_states_the_same_bits():
    s = make(2 * 150, 2, 96, torch.bfloat16)
    a, b = call(s, (2, 150, 96)), call(s, (2, 150, 96), states=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("T", [129, 160])
def test_states_again_where_only_the_forward_has_segments(T):
    """So many channels that the backward's rows are one segment and the forward's, which it runs for the states, several."""
    s = make(T, 1, 77890, torch.bfloat16)
    a, b = call(s, (1, T, 77890)), call(s, (1, T, 77890), states=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    compare(b, definition(s, spans_of([T]), True), torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strided_rows_and_supplied_outputs(dtype):
    B, T, D = 2, 70, 64
    s = make(B * T, B, D, dtype)
    want = call(s, (B, T, D))
    wide = torch.zeros(B, T, 4 * D + 1, device=DEV, dtype=dtype)       # odd stride: single elements
    parts = [wide[..., 1 + k * D:1 + (k + 1) * D] for k in range(3)]
    for p, k in zip(parts, ("x", "decay", "gate")):
        p.copy_(s[k].view(B, T, D))
    out = torch.full((B, T, 2 * D), 7.0, device=DEV, dtype=dtype)
    y, ht = lib.gated_scan_fwd(*parts, s["rate"], s["h0"], scale=SCALE, y=out[..., D:])
    assert rel(y, want["y"].double()) <= half_step(dtype) * 2 and bool((out[..., :D] == 7).all())
    grads = torch.full((B, T, 3 * D), 7.0, device=DEV, dtype=dtype)
    g = lib.gated_scan_bwd(*parts, s["rate"], s["h0"], s["dy"].view(B, T, D), s["dht"], scale=SCALE,
                           grads=dict(dx=grads[..., :D], ddecay=grads[..., D:2 * D], dgate=grads[..., 2 * D:]))
    for k in ("dx", "ddecay", "dgate", "drate", "dh0"):
        assert rel(g[k], want[k].double()) <= half_step(dtype) * 2, k


def test_rows_behind_the_last_sequence_stay():
    D, cu = 40, torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    s = make(80, 2, D, torch.float32)
    for k in ("x", "decay", "gate", "dy"):
        s[k][50:] = float("nan")
    v = {k: t.view(1, 80, D) if k in ("x", "decay", "gate", "dy") else t for k, t in s.items()}
    buf = {k: torch.full((1, 80, D), 7.0, device=DEV) for k in ("y", "dx", "ddecay", "dgate")}
    args = (v["x"], v["decay"], v["gate"], v["rate"], v["h0"])
    _, ht = lib.gated_scan_fwd(*args, scale=SCALE, y=buf["y"], cu_seqlens=cu)
    g = lib.gated_scan_bwd(*args, v["dy"], v["dht"], scale=SCALE, cu_seqlens=cu, grads={k: buf[k] for k in ("dx", "ddecay", "dgate")})
    for t in buf.values():
        assert bool((t[0, 50:] == 7).all()) and bool(torch.isfinite(t).all())
    want = definition({k: t[:50] if k in ("x", "decay", "gate", "dy") else t for k, t in s.items()}, [(0, 20), (20, 50)], True)
    compare({"y": buf["y"][0, :50], "ht": ht, **{k: t[0, :50] if t.dim() == 3 else t for k, t in g.items()}}, want, torch.float32)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_infinities_stay_in_their_sequence(bad):
    lens, D = [10, 90, 3, 70], 48
    s = make(sum(lens), 4, D, torch.float32)
    cu = torch.tensor([0, 10, 100, 103, 173], dtype=torch.int32, device=DEV)
    clean = call(s, (1, 173, D), cu)
    s["x"][60, 5] = bad
    s["dy"][120, 7] = bad
    got = call(s, (1, 173, D), cu)
    y = got["y"][0]
    assert not bool(torch.isfinite(y[60:100, 5]).any()) and not bool(torch.isfinite(got["ht"][1, 5]))
    keep = torch.ones(173, D, dtype=torch.bool, device=DEV)
    keep[60:100, 5] = False
    assert torch.equal(y[keep], clean["y"][0][keep])
    for k in ("dx", "ddecay", "dgate"):
        keep = torch.ones(173, D, dtype=torch.bool, device=DEV)
        keep[10:100, 5] = False
        keep[103:121, 7] = False
        assert torch.equal(got[k][0][keep], clean[k][0][keep]), k
        assert not bool(torch.isfinite(got["dx"][0, 103:121, 7]).any())
    assert torch.equal(got["drate"][torch.arange(D, device=DEV) > 7], clean["drate"][torch.arange(D, device=DEV) > 7])


def test_gates_that_are_shut():
    """A gate of minus infinity lets nothing in, a decay of minus infinity keeps the state as it is: exactly, and with finite
    gradients."""
    T, D = 80, 34
    s = make(T, 1, D, torch.float32)
    s["decay"][:] = -float("inf")
    got = call(s, (1, T, D))
    assert torch.equal(got["y"][0], s["h0"].expand(T, D)) and torch.equal(got["ht"], s["h0"])
    assert all(bool(torch.isfinite(t).all()) for t in got.values()) and not bool(got["ddecay"].any())
    s = make(T, 1, D, torch.float32)
    s["gate"][:] = -float("inf")
    s["h0"] = None
    got = call(s, (1, T, D))
    assert not bool(got["y"].any()) and not bool(got["dx"].any()) and all(bool(torch.isfinite(t).all()) for t in got.values())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 63, 64, 200])
def test_step(D, dtype):
    B, S = 5, 9
    s = make(B, B, D, dtype)
    slots = torch.tensor([7, 0, -1, 3, 9], dtype=torch.int32, device=DEV)
    state = torch.randn(S, D, device=DEV)
    before = state.clone()
    y = lib.gated_scan_step(s["x"], s["decay"], s["gate"], s["rate"], state, scale=SCALE, slots=slots)
    live, at = [0, 1, 3], [7, 0, 3]
    h0 = torch.zeros(B, D, device=DEV)
    h0[live] = before[at]
    want = definition({**s, "h0": h0}, [(b, b + 1) for b in range(B)])
    assert rel(y[live], want["y"][live]) <= tol(dtype) and rel(state[at], want["ht"][live]) <= STATE
    assert not bool(y[[2, 4]].any())
    rest = [k for k in range(S) if k not in at]
    assert torch.equal(state[rest], before[rest])
    whole = before[:B].clone()
    y2 = lib.gated_scan_step(s["x"], s["decay"], s["gate"], s["rate"], whole, scale=SCALE)
    want = definition({**s, "h0": before[:B]}, [(b, b + 1) for b in range(B)])
    assert rel(y2, want["y"]) <= tol(dtype)


def test_prompt_in_parts_then_single_tokens():
    B, T, D = 2, 100, 66
    s = make(B * T, B, D, torch.float32)
    v = {k: s[k].view(B, T, D) for k in ("x", "decay", "gate")}
    whole, ht = lib.gated_scan_fwd(*v.values(), s["rate"], s["h0"], scale=SCALE)
    part = lambda lo, hi: [t[:, lo:hi].contiguous() for t in v.values()]  # noqa: E731
    a, h = lib.gated_scan_fwd(*part(0, 37), s["rate"], s["h0"], scale=SCALE)
    b, h = lib.gated_scan_fwd(*part(37, 95), s["rate"], h, scale=SCALE)
    tail = torch.stack([lib.gated_scan_step(*(t[:, k].contiguous() for t in v.values()), s["rate"], h, scale=SCALE) for k in range(95, T)], 1)
    assert rel(torch.cat([a, b, tail], 1), whole.double()) <= STATE and rel(h, ht.double()) <= STATE


def test_gradients_against_differences():
    lens, D = [6, 0, 4], 3
    s = make(10, 3, D, torch.float32, seed=5)
    cu = torch.tensor([0, 6, 6, 10], dtype=torch.int32, device=DEV)
    got = call(s, (1, 10, D), cu)

    def loss(k, e):
        t = {n: v.double() if v is not None else None for n, v in s.items()}
        t[k] = t[k] + e
        y, ht = ref.gated_scan(t["x"], t["decay"], t["gate"], t["rate"], t["h0"], spans_of(lens), SCALE)
        return float((y * t["dy"]).sum() + (ht * t["dht"]).sum())
    for k in ("x", "decay", "gate", "rate", "h0"):
        d = torch.randn(s[k].shape, device=DEV, dtype=torch.float64)
        diff = (loss(k, 1e-5 * d) - loss(k, -1e-5 * d)) / 2e-5
        size = float((got["d" + k].double().reshape(d.shape) * d).abs().sum())
        assert abs(float((got["d" + k].double().reshape(d.shape) * d).sum()) - diff) <= STATE * size + 1e-7 * size, k


def test_equal_calls_other_streams_and_graphs():
    s = make(2 * 300, 2, 192, torch.bfloat16)
    want = call(s, (2, 300, 192))
    again = call(s, (2, 300, 192))
    assert all(torch.equal(want[k], again[k]) for k in want)
    side = torch.cuda.Stream()
    v = {k: s[k].view(2, 300, 192) for k in ("x", "decay", "gate")}
    side.wait_stream(torch.cuda.current_stream())
    y, ht = lib.gated_scan_fwd(*v.values(), s["rate"], s["h0"], scale=SCALE, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want["y"]) and torch.equal(ht, want["ht"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s, (2, 300, 192))
    s["x"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    fresh = call(s, (2, 300, 192))
    assert all(torch.equal(got[k], fresh[k]) for k in got) and not torch.equal(got["y"], want["y"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,D,cu", [(5, 40, [5, 5]), (150, 33, [150, 150, 150]), (150, 64, [151, 400]), (300, 70, [300, 300]), (300, 70, [77, 77, 77])])
def test_none_but_empty_sequences_anywhere(T, D, cu, dtype):
    """States and their gradients pass through, no row is written, the sum of drate is 0; what the uncovered rows hold does not matter."""
    n = len(cu) - 1
    s = make(T, n, D, dtype)
    for k in ("x", "decay", "gate", "dy"):
        s[k][:] = float("nan")
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    v = {k: t.view(1, T, D) if k in ("x", "decay", "gate", "dy") else t for k, t in s.items()}
    args = (v["x"], v["decay"], v["gate"], v["rate"], v["h0"])
    buf = {k: torch.full((1, T, D), 7.0, device=DEV, dtype=dtype) for k in ("y", "dx", "ddecay", "dgate")}
    _, ht, states = lib.gated_scan_fwd(*args, scale=SCALE, y=buf["y"], save_states=True, cu_seqlens=off)
    for kept in (states, None):
        g = lib.gated_scan_bwd(*args, v["dy"], v["dht"], states=kept, scale=SCALE, cu_seqlens=off, grads={k: buf[k] for k in ("dx", "ddecay", "dgate")})
        assert torch.equal(ht, s["h0"]) and torch.equal(g["dh0"], s["dht"]) and not bool(g["drate"].any())
        assert all(bool((t == 7).all()) for t in buf.values())


# Fast decays.  The exponent q = coefficient times sigmoid is off by at most 10 roundings of its size (sigmoid's exponential, sum and
# reciprocal, softplus' two functions, the products with scale, coefficient and log2 e), so a = exp(-q) by 10 q roundings of its own
# size and 4 of the exponential.  Rates reach 3 here: q <= 8 softplus(3) = 24.4.  The factor 1 - sigmoid(decay) of ddecay is
# at least 1 - sigmoid(3) = 0.047, from a sigmoid off by 3 roundings: 64 more.  The rest of a gradient's factors: 12.
FAST = (10 * 24.4 + 4 + 64 + 12) * 2.0 ** -24


def make_fast(rows, n, D, dtype, seed=0):
    """Rates from a memory of hundreds of tokens to one of less than a token, decays' gates open."""
    s = make(rows, n, D, dtype, seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    s["rate"] = torch.linspace(-5, 3, D, device=DEV)[torch.randperm(D, generator=g, device=DEV)]
    s["decay"] = (2 + 0.5 * torch.randn(rows, D, generator=g, device=DEV)).clamp(max=3).to(dtype)
    return s


def by_channel(got, want):
    """The largest relative error of a channel."""
    d = (got.double().reshape(want.shape) - want).flatten(0, -2).norm(dim=0)
    return float((d / want.flatten(0, -2).norm(dim=0)).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,D,packed", [([256], 64, False), ([150, 150], 130, False), ([70, 0, 1, 200, 33], 67, True), ([40], 128, False)])
def test_gradients_of_fast_decays_by_channel(lens, D, packed, dtype):
    rows, n = sum(lens), len(lens)
    s = make_fast(rows, n, D, dtype, seed=D)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV) if packed else None
    got = call(s, (1, rows, D) if packed else (n, rows // n, D), cu)
    want = definition(s, spans_of(lens), True)
    bound = FAST + STATE
    for k in ("y", "dx", "ddecay", "dgate"):
        assert by_channel(got[k], want[k]) <= bound + (half_step(dtype) if dtype != torch.float32 else 0), k
    # ht = sum of v_t a_{t+1} .. a_T (and of h0 a_1 .. a_T), dh0 = sum of a_1 .. a_t dy_t (and dht): terms of both signs, where a channel may
    # have one such sum that cancels, so each is relative to the sum of its terms' sizes, which the same recurrence gives for the
    # sizes of x, h0, dy and dht (no decay or gate is negative).  A term of k decays is off by k (10 q + 4) roundings and e^(-q k) of the
    # whole, at most 10 q + 4 for fast decays; STATE has the slow ones.
    size = definition({**s, **{k: s[k].abs() for k in ("x", "h0", "dy", "dht")}}, spans_of(lens), True)
    for k in ("ht", "dh0"):
        assert float(((got[k].double() - want[k]).abs() / size[k]).max()) <= bound, k
    # drate sums terms of both signs: relative to their sizes, scale sigmoid(rate) |ddecay| s / (q (1 - s))
    sg, rate = torch.sigmoid(s["decay"].double()), s["rate"].double()
    size = (want["ddecay"].abs() / (torch.nn.functional.softplus(rate) * (1 - sg)) * torch.sigmoid(rate)).sum(0)
    assert float(((got["drate"].double() - want["drate"]).abs() / size).max()) <= bound


def test_states_of_fast_decays_by_element():
    """With nothing let in, a state is the product of its decays: each as exact as its exponent."""
    T, D = 5, 66
    s = make_fast(T, 1, D, torch.float32)
    s["gate"][:] = -float("inf")
    s["h0"] = torch.full((1, D), 1e7, device=DEV)
    y, ht = lib.gated_scan_fwd(*(s[k].view(1, T, D) for k in ("x", "decay", "gate")), s["rate"], s["h0"], scale=SCALE)
    want = definition(s, [(0, T)])["y"]
    some = want > 1e-30                      # (below, float32 has no digits to lose)
    t = torch.arange(1, T + 1, device=DEV, dtype=torch.float64)[:, None].expand(T, D)
    off = ((y[0].double() - want).abs() / want)[some]
    assert bool((off <= t[some] * (10 * 24.4 + 5) * 2.0 ** -24).all()) and torch.equal(ht[0], y[0, -1])
    state = s["h0"].clone()
    y1 = lib.gated_scan_step(s["x"][:1], s["decay"][:1], s["gate"][:1], s["rate"], state, scale=SCALE)
    assert float(((y1.double() - want[:1]).abs() / want[:1]).max()) <= (10 * 24.4 + 5) * 2.0 ** -24 and torch.equal(state, y1)


@pytest.mark.parametrize("lens", [[300], [200, 0, 250]])
def test_an_infinite_state_stays_infinite(lens):
    """Products of a segment's decays underflow where each of them is positive: an infinity that enters is one that leaves, with its sign,
    and so are the gradients that an infinite one of the final state has."""
    D, n, rows = 40, len(lens), sum(lens)
    s = make(rows, n, D, torch.float32, seed=4)
    s["rate"][:] = 0.0
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    clean = call(s, (1, rows, D), cu)
    inf = float("inf")
    s["h0"][0, 5], s["h0"][0, 9], s["dht"][0, 7], s["dht"][0, 11] = inf, -inf, inf, -inf
    got = call(s, (1, rows, D), cu)
    first = lens[0]
    for c, sign in ((5, 1), (9, -1)):
        assert bool((got["y"][0, :first, c] == sign * inf).all()) and float(got["ht"][0, c]) == sign * inf
    for c, sign in ((7, 1), (11, -1)):
        assert bool((got["dx"][0, :first, c] == sign * inf).all()) and float(got["dh0"][0, c]) == sign * inf
    keep = torch.ones(rows, D, dtype=torch.bool, device=DEV)
    keep[:first, [5, 7, 9, 11]] = False
    for k in ("y", "dx", "ddecay", "dgate"):
        assert torch.equal(got[k][0][keep], clean[k][0][keep]), k


def test_a_huge_state_decays_to_nothing():
    """A product of decays that underflows, times a state near the largest float32: what is left of it is below the rounding of what comes in."""
    T, D = 400, 34
    s = make(T, 1, D, torch.float32)
    s["rate"][:] = 0.0
    s["h0"][:] = 1e38
    want = definition(s, [(0, T)])
    y, ht = lib.gated_scan_fwd(*(s[k].view(1, T, D) for k in ("x", "decay", "gate")), s["rate"], s["h0"], scale=SCALE)
    assert rel(ht, want["ht"]) <= STATE and rel(y[0, 200:], want["y"][200:]) <= STATE
