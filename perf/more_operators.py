"""What is measured of the operators of a gated recurrent layer: the gated linear recurrence, the gated group norm over
its heads, and the gated feed-forward product that follows it; forward, backward and single tokens.

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges.  ``prepare()`` makes a case's inputs,
``run()`` makes one pass: with ``own`` false in elementary torch operations in 32 bits, with ``own`` true through the
package's entry points.  ``exact()`` is the operators' definition in 64 bits, written apart from the plain form
(its gradients come from automatic differentiation of the definition).

The operators (sequence tensors [B, T, D]; rate [D]; W [F, D]; G groups of neighbouring channels):

    scan   q_t = scale softplus(rate) sigmoid(decay_t),  a_t = exp(-q_t),
           h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t,  y_t = h_t
    norm   n = (x - mean) / sqrt(var + eps) * weight + bias over each group of a row (or, without a centre,
           x / sqrt(mean of squares + eps) * weight),  y = n silu(gate)
    glu    g = x W_gate^T,  u = x W_up^T,  h = silu(g) u
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
SCALE = 8.0


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a batch of prompts through one mixer of the width of 16 heads of 128
        dict(name="scan_fwd_b4t4096d2048", op="scan", way="fwd", batch=4, lens="", tokens=4096, channels=2048,
             dtype="bf16", h0=False),
        # one long prompt, continued from an earlier part's state: few rows, a long axis
        dict(name="scan_fwd_b1t16384d1024", op="scan", way="fwd", batch=1, lens="", tokens=16384, channels=1024,
             dtype="bf16", h0=True),
        # a training step of the recurrence: outputs, then every gradient
        dict(name="scan_train_b2t2048d2048", op="scan", way="train", batch=2, lens="", tokens=2048, channels=2048,
             dtype="bf16", h0=False),
        # packed documents in training, 32 bits, an empty one and one of a single token among them, odd channel count
        dict(name="scan_train_packed_f32", op="scan", way="train", batch=6, lens="129,1,700,0,462,33", tokens=1325,
             channels=517, dtype="f32", h0=True),
        # one token for each of 64 requests, states in slots of a larger cache
        dict(name="scan_step_b64d4096", op="scan", way="step", batch=64, lens="", tokens=1, channels=4096,
             dtype="bf16", h0=True),
        # the norm and gate behind a mixer of 16 heads of 128, over a batch of prompts
        dict(name="norm_fwd_16384x16x128", op="norm", way="fwd", rows=16384, groups=16, width=128, dtype="bf16",
             gate=True, center=False, shared=True, affine=True),
        # a training step of the norm and gate behind 32 heads of 128
        dict(name="norm_train_8192x32x128", op="norm", way="train", rows=8192, groups=32, width=128, dtype="bf16",
             gate=True, center=False, shared=True, affine=True),
        # few rows, centred groups of an odd width with weights of their own, no gate, 32 bits
        dict(name="norm_train_77x8x131_f32", op="norm", way="train", rows=77, groups=8, width=131, dtype="f32",
             gate=False, center=True, shared=False, affine=True),
        # the feed-forward block's first half over a batch of prompts, four times as wide as the model
        dict(name="glu_fwd_8192x2048x8192", op="glu", way="fwd", rows=8192, model=2048, inner=8192, dtype="bf16"),
        # a training step of it: the product, then every gradient
        dict(name="glu_train_4096x2048x5632", op="glu", way="train", rows=4096, model=2048, inner=5632, dtype="bf16"),
        # one token: the weights pass by once
        dict(name="glu_fwd_1x4096x11008", op="glu", way="fwd", rows=1, model=4096, inner=11008, dtype="bf16"),
        # a small training step in 32 bits, odd sizes throughout
        dict(name="glu_train_77x517x1031_f32", op="glu", way="train", rows=77, model=517, inner=1031, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "norm", "glu", "glu"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "glu":
        way = rng.choice(["fwd", "train"])
        most = (1 << 32) if dtype == "f32" else 4096 * 2048 * 5632      # rows x model x inner
        rows, model, inner = _log(rng, 1, 8192), _log(rng, 16, 4096), _log(rng, 16, 11008)
        if rng.random() < 0.7:
            model, inner = max(16, model // 16 * 16), max(16, inner // 16 * 16)
        rows = max(1, min(rows, most // (model * inner)))
        return dict(op=op, way=way, rows=rows, model=model, inner=inner, dtype=dtype)
    if op == "norm":
        width, groups = rng.choice([64, 128, 128, 256, 32, 96, 131, 512, 16, 20]), _log(rng, 1, 64)
        rows = max(1, min(_log(rng, 1, 16384), 8192 * 4096 // (width * groups)))
        return dict(op=op, way=rng.choice(["fwd", "train"]), rows=rows, groups=groups, width=width, dtype=dtype,
                    gate=rng.random() < 0.7, center=rng.random() < 0.4, shared=rng.random() < 0.5, affine=rng.random() < 0.8)
    way = rng.choice(["fwd", "train", "step"])
    channels = _log(rng, 16, 4096)
    if rng.random() < 0.6:
        channels = max(16, channels // 16 * 16)
    case = dict(op=op, way=way, channels=channels, dtype=dtype, h0=way == "step" or rng.random() < 0.5)
    if way == "step":
        case.update(batch=_log(rng, 1, 128), tokens=1, lens="")
        return case
    most = (1 << 23) if way == "train" else (1 << 25)                    # tokens x channels
    tokens = max(1, min(_log(rng, 1, 16384), most // channels))
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
    """The tensors that a program has in hand before the call.  As in a layer, both gates of the recurrence are halves
    of one projection's output, and the norm's gate is a part of another's (strided views, not copies)."""
    dev, dt = torch.device("cuda"), _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    ru = lambda *shape: torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    train = case["way"] == "train"
    s = {"case": case}
    if case["op"] == "glu":
        m, d, f = case["rows"], case["model"], case["inner"]
        s["x"] = rn(m, d).to(dt)                                         # normalised rows
        s["w_gate"], s["w_up"] = ((rn(f, d) / math.sqrt(d)).to(dt) for _ in range(2))
        if train:
            s["dh"] = rn(m, f).to(dt)
        return s
    if case["op"] == "norm":
        m, n, w = case["rows"], case["groups"], case["width"]
        # a mixer's outputs: each head with an offset and a scale of its own
        s["x"] = (rn(m, n, w) * (0.2 + 2.0 * ru(m, n, 1)) + 0.3 * rn(m, n, 1)).reshape(m, n * w).to(dt)
        c = w if case["shared"] else n * w
        s["weight"] = (1.0 + 0.1 * rn(c)).to(dt) if case["affine"] else None
        s["bias"] = (0.1 * rn(c)).to(dt) if case["affine"] and case["center"] else None
        s["gate"] = rn(m, 2 * n * w).to(dt)[:, n * w:] if case["gate"] else None
        if train:
            s["dy"] = rn(m, n * w).to(dt)
        return s
    d, n_seq = case["channels"], case["batch"]
    lens, (rows, tokens) = _lens(case)
    step = case["way"] == "step"
    lead = (n_seq,) if step else (rows, tokens)
    s["cu"] = None
    if case["lens"]:
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["x"] = rn(*lead, d).to(dt)
    gates = rn(*lead, 2 * d).to(dt)
    s["decay"], s["gate"] = gates[..., :d], gates[..., d:]
    # the usual initialisation: a channel keeps 0.9 to 0.999 of its state where its gate is wide open
    s["rate"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * ru(d)) / SCALE))
    if step:
        slots = 2 * n_seq + 3
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:n_seq].to(torch.int32)
        s["state"] = rn(slots, d)
        return s
    s["h0"] = rn(n_seq, d) if case["h0"] else None
    if train:
        s["dy"] = rn(*lead, d).to(dt)
        s["dht"] = rn(n_seq, d)
    return s


def work(case):
    """Bytes: each input read once, each output written once.  Operations: the definition's (an exponential counts 1)."""
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "glu":
        m, d, f = case["rows"], case["model"], case["inner"]
        if case["way"] == "train":
            return {"bytes": (2 * m * d + 4 * f * d + 2 * m * f) * es, "flops": 12 * m * d * f + 20 * m * f}
        return {"bytes": (m * d + 2 * f * d + m * f) * es, "flops": 4 * m * d * f + 6 * m * f}
    if case["op"] == "norm":
        rows, n, w = case["rows"], case["groups"], case["width"]
        m, z = rows * n * w, 1 if case["gate"] else 0
        par = (w if case["shared"] else n * w) * (int(case["affine"]) + int(case["affine"] and case["center"])) * es
        stat = rows * n * 4 * (1 + int(case["center"]))
        if case["way"] == "train":
            return {"bytes": (4 + 2 * z) * m * es + 2 * par + stat, "flops": (20 + 14 * z) * m}
        return {"bytes": (2 + z) * m * es + par + stat, "flops": (6 + 5 * z) * m}
    d, seqs, step = case["channels"], case["batch"], case["way"] == "step"
    m = (seqs if step else sum(_lens(case)[0])) * d
    st = seqs * d * 4
    if case["way"] == "train":
        # x, decay, gate, dy in; y and three gradients out
        return {"bytes": 8 * m * es + 2 * d * 4 + (4 if case["h0"] else 2) * st, "flops": 55 * m}
    return {"bytes": 4 * m * es + d * 4 + (2 if case["h0"] else 1) * st, "flops": 20 * m}


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"scan": _plain_scan, "norm": _plain_norm, "glu": _plain_glu}[case["op"]](state, case)


def _run_own(s, case):
    import chunkwise_gated_delta_gb300 as lib
    op, train = case["op"], case["way"] == "train"
    if op == "glu":
        if not train:
            return {"h": lib.glu_fwd(s["x"], s["w_gate"], s["w_up"])}
        h, g, u = lib.glu_fwd(s["x"], s["w_gate"], s["w_up"], save=True)
        return {"h": h, **lib.glu_bwd(s["x"], s["w_gate"], s["w_up"], s["dh"], g, u)}
    if op == "norm":
        y, mean, rstd = lib.group_norm_fwd(s["x"], case["groups"], s["weight"], s["bias"], s["gate"], eps=EPS,
                                           center=case["center"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if train:
            out = {"y": y, **lib.group_norm_bwd(s["dy"], s["x"], case["groups"], s["weight"], s["bias"], s["gate"], mean, rstd)}
        return {k: v for k, v in out.items() if v is not None}
    args = (s["x"], s["decay"], s["gate"], s["rate"])
    if case["way"] == "step":
        return {"y": lib.gated_scan_step(*args, s["state"], scale=SCALE, slots=s["slots"]), "state": s["state"]}
    if not train:
        y, ht = lib.gated_scan_fwd(*args, s["h0"], scale=SCALE, cu_seqlens=s["cu"])
        return {"y": y, "ht": ht}
    y, ht, states = lib.gated_scan_fwd(*args, s["h0"], scale=SCALE, save_states=True, cu_seqlens=s["cu"])
    return {"y": y, "ht": ht, **lib.gated_scan_bwd(*args, s["h0"], s["dy"], s["dht"], states=states, scale=SCALE,
                                                   cu_seqlens=s["cu"])}


# --- plain forms: elementary operations, 32 bits, rounded once at the end
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_glu(s, case):
    x, wg, wu, dt = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["x"].dtype
    g, u = x @ wg.t(), x @ wu.t()
    sg = _sigmoid(g)
    out = {"h": (g * sg * u).to(dt)}
    if case["way"] == "fwd":
        return out
    dh = s["dh"].float()
    dg, du = dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg
    return {**out, "dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}


def _plain_norm(s, case):
    rows, n, w, dt = case["rows"], case["groups"], case["width"], s["x"].dtype
    heads = lambda v: v.float().reshape(rows, n, w)  # noqa: E731
    par = lambda v: v.float() if case["shared"] else v.float().reshape(n, w)  # noqa: E731
    x, c = heads(s["x"]), heads(s["x"])
    out = {}
    if case["center"]:
        mean = x.mean(-1, keepdim=True)
        c = x - mean
        out["mean"] = mean[..., 0]
    rstd = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)
    out["rstd"] = rstd[..., 0]
    xhat = c * rstd
    y = xhat
    if s["weight"] is not None:
        y = y * par(s["weight"])
    if s["bias"] is not None:
        y = y + par(s["bias"])
    if s["gate"] is not None:
        z = heads(s["gate"])
        sg = _sigmoid(z)
    out["y"] = (y if s["gate"] is None else y * z * sg).reshape(rows, n * w).to(dt)
    if case["way"] == "fwd":
        return out
    out, dy = {"y": out["y"]}, heads(s["dy"])
    if s["gate"] is not None:
        out["dgate"] = (dy * y * sg * (1.0 + z * (1.0 - sg))).reshape(rows, n * w).to(dt)
        dy = dy * z * sg
    lead = (0, 1) if case["shared"] else 0
    if s["weight"] is not None:
        out["dweight"] = (dy * xhat).sum(lead).reshape(-1).to(dt)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(lead).reshape(-1).to(dt)
    gw = dy if s["weight"] is None else dy * par(s["weight"])
    dx = gw - xhat * (gw * xhat).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - gw.mean(-1, keepdim=True)
    out["dx"] = (rstd * dx).reshape(rows, n * w).to(dt)
    return out


def _doubling(a, v):
    """States h_t = a_t h_{t-1} + v_t along axis 1 (from 0), in log2(T) passes over both tensors."""
    a, v, k = a.clone(), v.clone(), 1
    while k < v.shape[1]:
        v[:, k:] = torch.addcmul(v[:, k:], a[:, k:], v[:, :-k])
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return v


def _plain_scan(s, case):
    dt, train = s["x"].dtype, case["way"] == "train"
    x, sd, sx = s["x"].float(), _sigmoid(s["decay"].float()), _sigmoid(s["gate"].float())
    coef = SCALE * _softplus(s["rate"])
    q = coef * sd
    a, m = torch.exp(-q), torch.sqrt(-torch.expm1(-2.0 * q))
    v = m * sx * x
    if case["way"] == "step":
        at = s["slots"].long()
        h = torch.addcmul(v, a, s["state"][at])
        s["state"][at] = h
        return {"y": h.to(dt), "state": s["state"]}
    lens = _lens(case)[0]
    ends, live = [], []                                     # rows' ends, and the sequences that are not empty
    for i, n in enumerate(lens):
        ends.append((ends[-1] if ends else 0) + n)
        live += [i] if n else []
    d, dev = x.shape[-1], x.device
    first = torch.tensor([ends[i] - lens[i] for i in live], device=dev)
    last = torch.tensor([ends[i] - 1 for i in live], device=dev)
    live = torch.tensor(live, device=dev)
    flat = lambda t: t.reshape(-1, d)  # noqa: E731
    keep = a.clone()                                        # a without the link into each first token
    flat(keep)[first] = 0.0
    if s["h0"] is not None:
        flat(v)[first] += flat(a)[first] * s["h0"][live]
    h = _doubling(keep, v)
    ht = s["h0"].clone() if s["h0"] is not None else x.new_zeros(len(lens), d)
    ht[live] = flat(h)[last]
    out = {"y": h.to(dt), "ht": ht}
    if not train:
        return out
    # gradients of the states: the same recurrence from the end, its coefficient the next token's
    grad = s["dy"].float().clone()
    flat(grad)[last] += s["dht"][live]
    follow = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
    grad = _doubling(follow.flip(1), grad.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    flat(before)[first] = s["h0"][live] if s["h0"] is not None else 0.0
    dq = grad * (sx * x * a * a / m - a * before)
    dv = grad * m
    dpre = dq * sd
    out.update(dx=(dv * sx).to(dt), ddecay=(dpre * coef * (1.0 - sd)).to(dt), dgate=(dv * x * sx * (1.0 - sx)).to(dt),
               drate=flat(dpre).sum(0) * SCALE * _sigmoid(s["rate"]))
    if s["h0"] is not None:
        dh0 = s["dht"].clone()                              # an empty sequence hands its state through
        dh0[live] = flat(a * grad)[first]
        out["dh0"] = dh0
    return out


# ------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    train = case["way"] == "train"
    leaf = {}
    for k, v in s.items():
        if isinstance(v, torch.Tensor) and v.is_floating_point():
            v = v.detach().to(torch.float64, memory_format=torch.contiguous_format)
            leaf[k] = v.requires_grad_(True) if train and k not in ("dy", "dht", "dh") else v
    with torch.enable_grad() if train else torch.no_grad():
        out = {"scan": _exact_scan, "norm": _exact_norm, "glu": _exact_glu}[case["op"]](s, leaf, case)
    if not train:
        return out
    names = {"scan": ["x", "decay", "gate", "rate", "h0"], "norm": ["x", "weight", "bias", "gate"],
             "glu": ["x", "w_gate", "w_up"]}[case["op"]]
    names = [k for k in names if k in leaf]
    loss = (out["h"] * leaf["dh"]).sum() if case["op"] == "glu" else (out["y"] * leaf["dy"]).sum()
    if "dht" in leaf:
        loss = loss + (out["ht"] * leaf["dht"]).sum()
    grads = torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True)
    out.update({"d" + k: torch.zeros_like(leaf[k]) if v is None else v for k, v in zip(names, grads)})
    return {k: v.detach() for k, v in out.items()}


def _exact_glu(s, f, case):
    g = torch.einsum("md,fd->mf", f["x"], f["w_gate"])
    return {"h": torch.nn.functional.silu(g) * torch.einsum("md,fd->mf", f["x"], f["w_up"])}


def _exact_norm(s, f, case):
    x = f["x"].unflatten(1, (case["groups"], case["width"]))
    mean = x.sum(2) / case["width"] if case["center"] else torch.zeros_like(x[..., 0])
    power = ((x - mean[..., None]) ** 2).sum(2) / case["width"]
    rstd = (power + EPS) ** -0.5
    y = (x - mean[..., None]) * rstd[..., None]
    reps = case["groups"] if case["shared"] else 1
    if "weight" in f:
        y = y * f["weight"].repeat(reps).unflatten(0, (case["groups"], case["width"]))
    if "bias" in f:
        y = y + f["bias"].repeat(reps).unflatten(0, (case["groups"], case["width"]))
    y = y.flatten(1)
    if "gate" in f:
        y = y * torch.nn.functional.silu(f["gate"])
    if case["way"] == "train":
        return {"y": y}
    return {"y": y, "rstd": rstd, **({"mean": mean} if case["center"] else {})}


def _exact_scan(s, f, case):
    log_a = -SCALE * torch.nn.functional.softplus(f["rate"], threshold=60.0) * torch.sigmoid(f["decay"])
    a = torch.exp(log_a)
    v = (-torch.expm1(2.0 * log_a)) ** 0.5 * torch.sigmoid(f["gate"]) * f["x"]
    if case["way"] == "step":
        at = s["slots"].long()
        h = a * f["state"][at] + v
        state = f["state"].clone()
        state[at] = h
        return {"y": h, "state": state}
    if s["cu"] is None:
        spans = [(slice(None), 0, case["tokens"])]
    else:
        cu = s["cu"].tolist()
        spans = [(0, lo, hi) for lo, hi in zip(cu[:-1], cu[1:])]
    ys, hts = [], []
    for i, (row, lo, hi) in enumerate(spans):
        if s["h0"] is not None:
            h = f["h0"] if s["cu"] is None else f["h0"][i]
        else:
            h = f["x"].new_zeros(*((case["batch"],) if s["cu"] is None else ()), case["channels"])
        rows = []
        for at, vt in zip(a[row, lo:hi].unbind(-2), v[row, lo:hi].unbind(-2)):
            h = at * h + vt
            rows.append(h)
        ys.append(torch.stack(rows, -2) if rows else f["x"][row, lo:hi])
        hts.append(h)
    if s["cu"] is None:
        return {"y": ys[0], "ht": hts[0]}
    return {"y": torch.cat(ys)[None], "ht": torch.stack(hts)}
