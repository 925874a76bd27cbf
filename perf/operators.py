"""What is measured of the operators around a state-space mixer: the short causal convolution, the selective
state-space scan and layer norm, each in its forward pass, its backward pass and, where it has one, its form for
single tokens.

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges.  ``prepare()`` makes a case's inputs,
``run()`` makes one pass: with ``own`` false in elementary torch operations in 32 bits, with ``own`` true through the
package's entry points.  ``exact()`` is the operators' definition in 64 bits, written apart from the plain form
(its gradients come from automatic differentiation of the definition).

The operators, per channel d and state n (x, delta, z [B, T, D]; B, C [B, T, N]; A [D, N] < 0):

    conv   y_t = silu(bias + sum_j weight[:, j] x_{t-W+1+j}),  x before the start taken from a state [B, W-1, D]
    scan   dt_t = softplus(delta_t + delta_bias),  h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,
           y_t = (sum_n C_t[n] h_t[:, n] + D x_t) silu(z_t)
    norm   y = (x - mean) / sqrt(var + eps) * weight + bias, over the last axis
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a batch of prompts through one mixer of the width of 16 heads of 128
        dict(name="scan_fwd_b4t4096d2048", op="scan", way="fwd", batch=4, lens="", tokens=4096, channels=2048, states=16,
             dtype="bf16", gate=True, h0=False),
        # one long prompt, continued from an earlier part's state: few rows, a long axis
        dict(name="scan_fwd_b1t16384d1024", op="scan", way="fwd", batch=1, lens="", tokens=16384, channels=1024, states=16,
             dtype="bf16", gate=True, h0=True),
        # prompts of very different lengths packed back to back, an empty one among them; odd channel and state counts
        dict(name="scan_fwd_packed_f32", op="scan", way="fwd", batch=7, lens="1,0,333,1500,64,17,82", tokens=1997,
             channels=517, states=10, dtype="f32", gate=False, h0=True),
        # a training step of the mixer's scan: outputs, then every gradient
        dict(name="scan_train_b2t2048d2048", op="scan", way="train", batch=2, lens="", tokens=2048, channels=2048, states=16,
             dtype="bf16", gate=True, h0=False),
        # packed documents in training, 32 bits, few channels
        dict(name="scan_train_packed_f32", op="scan", way="train", batch=5, lens="129,1,400,0,62", tokens=592,
             channels=390, states=12, dtype="f32", gate=True, h0=True),
        # one token for each of 64 requests, states in slots of a larger cache
        dict(name="scan_step_b64d4096", op="scan", way="step", batch=64, lens="", tokens=1, channels=4096, states=16,
             dtype="bf16", gate=True, h0=True),
        # the convolution over a large batch of prompts: all of q, k and v of 32 heads of 128, or a mixer of that width
        dict(name="conv_fwd_b8t2048d4096", op="conv", way="fwd", batch=8, lens="", tokens=2048, channels=4096, width=4,
             dtype="bf16", h0=False),
        # a training step of the convolution over packed documents
        dict(name="conv_train_packed_d2048", op="conv", way="train", batch=6, lens="4096,2,1021,0,2500,572", tokens=8191,
             channels=2048, width=4, dtype="bf16", h0=True),
        # one token of one request: the latency of a call
        dict(name="conv_step_b1d2048", op="conv", way="step", batch=1, lens="", tokens=1, channels=2048, width=4,
             dtype="bf16", h0=True),
        # the norm before a mixer, over a batch of prompts
        dict(name="norm_fwd_16384x2048", op="norm", way="fwd", rows=16384, channels=2048, dtype="bf16"),
        # a training step of the norm
        dict(name="norm_train_16384x2048", op="norm", way="train", rows=16384, channels=2048, dtype="bf16"),
        # few rows of an odd width, 32 bits
        dict(name="norm_train_77x2051_f32", op="norm", way="train", rows=77, channels=2051, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        channels = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            channels = max(16, channels // 8 * 8)
        rows = min(_log(rng, 1, 16384), max(1, 16384 * 2048 // channels))
        return dict(op=op, way=rng.choice(["fwd", "train"]), rows=rows, channels=channels, dtype=dtype)
    way = rng.choice(["fwd", "train", "step"])
    channels = _log(rng, 16, 4096)
    if rng.random() < 0.6:
        channels = max(16, channels // 16 * 16)
    case = dict(op=op, way=way, channels=channels, dtype=dtype, h0=way == "step" or rng.random() < 0.5)
    if op == "scan":
        case.update(states=rng.choice([16, 16, 16, 8, 4, 1, 5, 24, 32]), gate=rng.random() < 0.7)
    else:
        case.update(width=rng.choice([4, 4, 3, 2]))
    if way == "step":
        case.update(batch=_log(rng, 1, 128), tokens=1, lens="")
        return case
    most = (1 << 23) if way == "train" else (1 << 25)      # tokens x channels (x states / 16)
    most //= max(1, case.get("states", 16) // 16 + (case.get("states", 16) % 16 > 0))
    tokens = max(1, min(_log(rng, 1, 4096), most // channels))
    if rng.random() < 0.5:                                  # packed: sequences of any length, empty ones too
        n = rng.randint(2, 9)
        cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
        case.update(batch=n, tokens=tokens, lens=",".join(map(str, lens)))
    else:
        case.update(batch=max(1, min(_log(rng, 1, 8), most // (tokens * channels))), tokens=tokens, lens="")
    return case


def _lens(case):
    """Lengths of the sequences, and the shape [rows, tokens] in which they lie."""
    if case["lens"]:
        return [int(v) for v in case["lens"].split(",")], (1, case["tokens"])
    return [case["tokens"]] * case["batch"], (case["batch"], case["tokens"])


# ------------------------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    """The tensors that a program has in hand before the call.  As in a mixer block, x and z are halves of one
    projection's output, and delta, B and C parts of another's (strided views, not copies)."""
    dev, dt = torch.device("cuda"), _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    ru = lambda *shape: torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    d = case["channels"]
    s = {"case": case}
    if case["op"] == "norm":
        # residual-stream rows: an offset and a scale of their own
        rows = case["rows"]
        s["x"] = (rn(rows, d) * (0.5 + 2.0 * ru(rows, 1)) + 0.3 * rn(rows, 1)).to(dt)
        s["weight"] = (1.0 + 0.1 * rn(d)).to(dt)
        s["bias"] = (0.1 * rn(d)).to(dt)
        if case["way"] == "train":
            s["dy"] = rn(rows, d).to(dt)
        return s
    n_seq, step = case["batch"], case["way"] == "step"
    lens, (rows, tokens) = _lens(case)
    lead = (n_seq,) if step else (rows, tokens)
    slots = 2 * n_seq + 3
    if case["lens"]:
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    else:
        s["cu"] = None
    if step:
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:n_seq].to(torch.int32)
    xz = rn(*lead, 2 * d).to(dt)
    if case["op"] == "conv":
        w = case["width"]
        s["x"] = xz[..., :d]
        s["weight"] = ((2.0 * ru(d, w) - 1.0) / math.sqrt(w)).to(dt)
        s["bias"] = ((2.0 * ru(d) - 1.0) / math.sqrt(w)).to(dt)
        if step:
            s["state"] = rn(slots, w - 1, d).to(dt)
            return s
        s["h0"] = rn(n_seq, w - 1, d).to(dt) if case["h0"] else None
        if case["way"] == "train":
            s["dy"] = rn(*lead, d).to(dt)
            s["dht"] = rn(n_seq, w - 1, d).to(dt)
        return s
    n = case["states"]
    # the usual initialisation: A = -(1 ... N), steps log-uniform in [1e-3, 1e-1] through softplus's inverse
    step0 = torch.exp(ru(d) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    s["delta_bias"] = step0 + torch.log(-torch.expm1(-step0))
    s["A"] = -torch.arange(1, n + 1, device=dev, dtype=torch.float32).repeat(d, 1) * (0.8 + 0.4 * ru(d, n))
    s["D"] = 1.0 + 0.1 * rn(d)
    s["x"] = torch.nn.functional.silu(rn(*lead, d)).to(dt)
    s["delta"] = (0.5 * rn(*lead, d)).to(dt)
    s["z"] = xz[..., d:] if case["gate"] else None
    rank = max(1, d // 16)
    proj = rn(*lead, rank + 2 * n).to(dt)
    s["B"], s["C"] = proj[..., rank:rank + n], proj[..., rank + n:]
    if step:
        s["state"] = 0.1 * rn(slots, d, n)
        return s
    s["h0"] = 0.1 * rn(n_seq, d, n) if case["h0"] else None
    if case["way"] == "train":
        s["dy"] = rn(*lead, d).to(dt)
        s["dht"] = 0.1 * rn(n_seq, d, n)
    return s


def work(case):
    """Bytes: each input read once, each output written once.  Operations: the definition's (an exponential counts 1)."""
    es, d = (2 if case["dtype"] == "bf16" else 4), case["channels"]
    if case["op"] == "norm":
        m = case["rows"] * d
        if case["way"] == "fwd":
            return {"bytes": 2 * m * es + 2 * d * es + 8 * case["rows"], "flops": 8 * m}
        return {"bytes": 4 * m * es + 4 * d * es + 8 * case["rows"], "flops": 21 * m}
    seqs, step = case["batch"], case["way"] == "step"
    tokens = seqs if step else sum(_lens(case)[0])
    if case["op"] == "conv":
        w, m = case["width"], tokens * d
        par, st = (w + 1) * d * es, seqs * (w - 1) * d * es
        if case["way"] == "train":
            return {"bytes": 4 * m * es + 2 * par + (4 if case["h0"] else 2) * st, "flops": (6 * w + 16) * m}
        return {"bytes": 2 * m * es + par + (2 if case["h0"] else 1) * st, "flops": (2 * w + 5) * m}
    n, m = case["states"], tokens * d
    z = 1 if case["gate"] else 0
    par, st, bc = (d * n + 2 * d) * 4, seqs * d * n * 4, 2 * tokens * n * es
    if case["way"] == "train":
        # x, delta, z, dy in; y and the three gradients out; B, C in, dB, dC out
        return {"bytes": (6 + 2 * z) * m * es + 2 * bc + 2 * par + (4 if case["h0"] else 2) * st,
                "flops": m * (22 * n + 40)}
    return {"bytes": (3 + z) * m * es + bc + par + (2 if case["h0"] else 1) * st, "flops": m * (7 * n + 16)}


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"scan": _plain_scan, "conv": _plain_conv, "norm": _plain_norm}[case["op"]](state, case)


def _run_own(s, case):
    import chunkwise_gated_delta_gb300 as lib
    op, way = case["op"], case["way"]
    if op == "norm":
        y, mean, rstd = lib.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        if way == "fwd":
            return {"y": y, "mean": mean, "rstd": rstd}
        return {"y": y, **lib.layer_norm_bwd(s["dy"], s["x"], s["weight"], mean, rstd)}
    if op == "conv":
        if way == "step":
            return {"y": lib.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], slots=s["slots"]),
                    "state": s["state"]}
        y, ht = lib.short_conv_fwd(s["x"], s["weight"], s["bias"], s["h0"], cu_seqlens=s["cu"])
        out = {"y": y, "ht": ht}
        if way == "train":
            out.update(lib.short_conv_bwd(s["x"], s["weight"], s["bias"], s["h0"], s["dy"], s["dht"],
                                          cu_seqlens=s["cu"]))
        return {k: v for k, v in out.items() if v is not None}
    if way == "step":
        return {"y": lib.ssm_scan_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["state"], s["D"], s["z"],
                                       s["delta_bias"], slots=s["slots"]), "state": s["state"]}
    args = (s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"], s["h0"])
    y, ht = lib.ssm_scan_fwd(*args, cu_seqlens=s["cu"])
    out = {"y": y, "ht": ht}
    if way == "train":
        out.update(lib.ssm_scan_bwd(*args, s["dy"], s["dht"], cu_seqlens=s["cu"]))
    return {k: v for k, v in out.items() if v is not None}


# --- plain forms: elementary operations, 32 bits, rounded once at the end
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_norm(s, case):
    x, dt = s["x"].float(), s["x"].dtype
    w, b = s["weight"].float(), s["bias"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    xhat = c * rstd
    out = {"y": (xhat * w + b).to(dt)}
    if case["way"] == "fwd":
        return {**out, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy = s["dy"].float()
    gw = dy * w
    dx = rstd * (gw - gw.mean(-1, keepdim=True) - xhat * (gw * xhat).mean(-1, keepdim=True))
    return {**out, "dx": dx.to(dt), "dweight": (dy * xhat).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}


def _pad(v, lens):
    """Packed [1, T, ...] to [sequences, longest, ...] with zeros behind each end; dense batches as they are."""
    if lens is None:
        return v
    out = v.new_zeros(len(lens), max(lens), *v.shape[2:])
    at = 0
    for i, n in enumerate(lens):
        out[i, :n] = v[0, at:at + n]
        at += n
    return out


def _unpad(v, lens):
    return v if lens is None else torch.cat([v[i, :n] for i, n in enumerate(lens)]).unsqueeze(0)


def _plain_conv(s, case):
    w, dt = case["width"], s["x"].dtype
    weight, bias = s["weight"].float(), s["bias"].float()
    if case["way"] == "step":
        at = s["slots"].long()
        full = torch.cat([s["state"][at], s["x"].unsqueeze(1)], 1)
        pre = bias + (full.float() * weight.t()).sum(1)
        s["state"][at] = full[:, 1:]
        return {"y": (pre * _sigmoid(pre)).to(dt), "state": s["state"]}
    lens = _lens(case)[0] if case["lens"] else None
    x = _pad(s["x"].float(), lens)
    n_seq, t, d = x.shape
    h0 = s["h0"].float() if s["h0"] is not None else x.new_zeros(n_seq, w - 1, d)
    full = torch.cat([h0, x], 1)
    pre = bias + sum(full[:, j:j + t] * weight[:, j] for j in range(w))
    sg = _sigmoid(pre)
    out = {"y": _unpad(pre * sg, lens).to(dt)}
    ends = lens if lens is not None else [t] * n_seq
    out["ht"] = torch.stack([full[i, n:n + w - 1] for i, n in enumerate(ends)]).to(dt)
    if case["way"] == "fwd":
        return out
    dpre = _pad(s["dy"].float(), lens) * sg * (1.0 + pre * (1.0 - sg))
    dfull = torch.zeros_like(full)
    for j in range(w):
        dfull[:, j:j + t] += dpre * weight[:, j]
    for i, n in enumerate(ends):
        dfull[i, n:n + w - 1] += s["dht"][i].float()
    out["dx"] = _unpad(dfull[:, w - 1:], lens).to(dt)
    if s["h0"] is not None:
        out["dh0"] = dfull[:, :w - 1].to(dt)
    out["dweight"] = torch.stack([(dpre * full[:, j:j + t]).sum((0, 1)) for j in range(w)], 1).to(dt)
    out["dbias"] = dpre.sum((0, 1)).to(dt)
    return out


def _plain_scan(s, case):
    dt_, a_mat = s["x"].dtype, s["A"]
    if case["way"] == "step":
        at = s["slots"].long()
        x, step = s["x"].float(), _softplus(s["delta"].float() + s["delta_bias"])
        h = torch.exp(step.unsqueeze(-1) * a_mat) * s["state"][at] + (step * x).unsqueeze(-1) * s["B"].float().unsqueeze(1)
        s["state"][at] = h
        y = (h * s["C"].float().unsqueeze(1)).sum(-1) + s["D"] * x
        if s["z"] is not None:
            z = s["z"].float()
            y = y * z * _sigmoid(z)
        return {"y": y.to(dt_), "state": s["state"]}
    lens = _lens(case)[0] if case["lens"] else None
    train = case["way"] == "train"
    pre = s["delta"].float() + s["delta_bias"]
    step = _pad(_softplus(pre), lens)                       # zero behind an end: the state stays as it is there
    x = _pad(s["x"].float(), lens)
    bm, cm = _pad(s["B"].float(), lens), _pad(s["C"].float(), lens)
    n_seq, t, d = x.shape
    n = a_mat.shape[1]
    u = step * x
    h = s["h0"].clone() if s["h0"] is not None else x.new_zeros(n_seq, d, n)
    y = x.new_empty(n_seq, t, d)
    part = 128
    entry = []
    for t0 in range(0, t, part):
        k = slice(t0, min(t, t0 + part))
        if train:
            entry.append(h)
        hs = _states(h, step[:, k], u[:, k], a_mat, bm[:, k])
        h = hs[-1]
        y[:, k] = torch.stack([(v * cm[:, t0 + i].unsqueeze(1)).sum(-1) for i, v in enumerate(hs)], 1)
    y = y + s["D"] * x
    z = _pad(s["z"].float(), lens) if s["z"] is not None else None
    out = {"ht": h}
    if z is not None:
        sg = _sigmoid(z)
        out["y"] = _unpad(y * z * sg, lens).to(dt_)
    else:
        out["y"] = _unpad(y, lens).to(dt_)
    if not train:
        return out
    dy = _pad(s["dy"].float(), lens)
    if z is not None:
        out["dz"] = _unpad(dy * y * sg * (1.0 + z * (1.0 - sg)), lens).to(dt_)
        dy = dy * z * sg
    carry = s["dht"].clone()                                # gradient of the state after a token, from what follows
    dx, dstep = s["D"] * dy, torch.empty_like(step)
    d_b, d_c, d_a = torch.empty_like(bm), torch.empty_like(cm), torch.zeros_like(a_mat)
    for t0 in reversed(range(0, t, part)):
        k = slice(t0, min(t, t0 + part))
        h_in = entry[t0 // part]
        hs = torch.stack([h_in] + _states(h_in, step[:, k], u[:, k], a_mat, bm[:, k]), 1)
        a = torch.exp(step[:, k].unsqueeze(-1) * a_mat)
        gs = []
        for i in reversed(range(k.stop - k.start)):
            gt = torch.addcmul(carry, dy[:, t0 + i].unsqueeze(-1), cm[:, t0 + i].unsqueeze(1))
            gs.append(gt)
            carry = gt * a[:, i]
        gs = torch.stack(gs[::-1], 1)
        d_c[:, k] = (dy[:, k].unsqueeze(-1) * hs[:, 1:]).sum(2)
        d_b[:, k] = (gs * u[:, k].unsqueeze(-1)).sum(2)
        du = (gs * bm[:, k].unsqueeze(2)).sum(-1)
        q = gs * a * hs[:, :-1]                             # gradient of dt A
        d_a += (q * step[:, k].unsqueeze(-1)).sum((0, 1))
        dx[:, k] += du * step[:, k]
        dstep[:, k] = (q * a_mat).sum(-1) + du * x[:, k]
    dpre = _unpad(dstep, lens) * _sigmoid(pre)
    out.update(dx=_unpad(dx, lens).to(dt_), ddelta=dpre.to(dt_), dA=d_a, dB=_unpad(d_b, lens).to(dt_),
               dC=_unpad(d_c, lens).to(dt_), dD=(dy * x).sum((0, 1)), ddelta_bias=dpre.sum((0, 1)))
    if s["h0"] is not None:
        out["dh0"] = carry
    return out


def _states(h, step, u, a_mat, bm):
    """The states after each token, as a list."""
    a = torch.exp(step.transpose(0, 1).unsqueeze(-1) * a_mat)
    v = u.transpose(0, 1).unsqueeze(-1) * bm.transpose(0, 1).unsqueeze(2)
    out = []
    for i in range(a.shape[0]):
        h = torch.addcmul(v[i], a[i], h)
        out.append(h)
    return out


# ------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    train = case["way"] == "train"
    leaf = {}
    for k, v in s.items():
        if isinstance(v, torch.Tensor) and v.is_floating_point():
            v = v.detach().to(torch.float64, memory_format=torch.contiguous_format)
            leaf[k] = v.requires_grad_(True) if train and k not in ("dy", "dht") else v
    with torch.enable_grad() if train else torch.no_grad():
        out = {"scan": _exact_scan, "conv": _exact_conv, "norm": _exact_norm}[case["op"]](s, leaf, case)
    if not train:
        return out
    names = {"scan": ["x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0"], "conv": ["x", "weight", "bias", "h0"],
             "norm": ["x", "weight", "bias"]}[case["op"]]
    names = [k for k in names if k in leaf]
    loss = (out["y"] * leaf["dy"]).sum()
    if "dht" in leaf:
        loss = loss + (out["ht"] * leaf["dht"]).sum()
    grads = torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True)
    out.update({"d" + k: torch.zeros_like(leaf[k]) if v is None else v for k, v in zip(names, grads)})
    return {k: v.detach() for k, v in out.items()}


def _spans(s, case):
    """For each sequence: its row, its first token and the token after its last."""
    if s["cu"] is None:
        return [(i, 0, case["tokens"]) for i in range(case["batch"])]
    cu = s["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def _exact_norm(s, f, case):
    mean = f["x"].sum(1) / f["x"].shape[1]
    var = ((f["x"] - mean[:, None]) ** 2).sum(1) / f["x"].shape[1]
    rstd = (var + EPS) ** -0.5
    y = torch.addcmul(f["bias"], (f["x"] - mean[:, None]) * rstd[:, None], f["weight"])
    return {"y": y, "mean": mean, "rstd": rstd} if case["way"] == "fwd" else {"y": y}


def _exact_conv(s, f, case):
    w = case["width"]
    if case["way"] == "step":
        at, ext = s["slots"].long(), None
        ext = torch.cat([f["state"][at], f["x"][:, None]], 1)
        pre = torch.einsum("bjd,dj->bd", ext, f["weight"]) + f["bias"]
        state = f["state"].clone()
        state[at] = ext[:, 1:]
        return {"y": pre * torch.sigmoid(pre), "state": state}
    ys, hts = [], []
    for i, (row, a, b) in enumerate(_spans(s, case)):
        seq = f["x"][row, a:b]
        front = f["h0"][i] if s["h0"] is not None else seq.new_zeros(w - 1, seq.shape[1])
        ext = torch.cat([front, seq], 0)
        pre = torch.einsum("tdj,dj->td", ext.unfold(0, w, 1), f["weight"]) + f["bias"] if b > a else seq
        ys.append(pre * torch.sigmoid(pre))
        hts.append(ext[b - a:])
    y = torch.stack(ys) if s["cu"] is None else torch.cat(ys)[None]
    return {"y": y, "ht": torch.stack(hts)}


def _exact_scan(s, f, case):
    dt = torch.nn.functional.softplus(f["delta"] + f["delta_bias"], threshold=60.0)
    if case["way"] == "step":
        at = s["slots"].long()
        h = torch.exp(dt[..., None] * f["A"]) * f["state"][at] + torch.einsum("bd,bd,bn->bdn", dt, f["x"], f["B"])
        y = torch.einsum("bdn,bn->bd", h, f["C"]) + f["x"] * f["D"]
        state = f["state"].clone()
        state[at] = h
        return {"y": y * torch.nn.functional.silu(f["z"]) if s["z"] is not None else y, "state": state}
    dense = s["cu"] is None
    d, n = f["A"].shape
    ys, hts = [], []
    for i, (row, a, b) in enumerate([(slice(None), 0, case["tokens"])] if dense else _spans(s, case)):
        x, step, bm, cm = (v[row, a:b] for v in (f["x"], dt, f["B"], f["C"]))
        if s["h0"] is not None:
            h = f["h0"] if dense else f["h0"][i]
        else:
            h = x.new_zeros(*((case["batch"],) if dense else ()), d, n)
        rows = []
        for xt, st, bt, ct in zip(*(v.unbind(-2) for v in (x, step, bm, cm))):
            h = h * torch.exp(st[..., None] * f["A"]) + (st * xt)[..., None] * bt[..., None, :]
            rows.append((h @ ct[..., None])[..., 0])
        ys.append(torch.stack(rows, -2) if rows else x)
        hts.append(h)
    y = (ys[0] if dense else torch.cat(ys)[None]) + f["x"] * f["D"]
    if s["z"] is not None:
        y = y * torch.nn.functional.silu(f["z"])
    return {"y": y, "ht": hts[0] if dense else torch.stack(hts)}
