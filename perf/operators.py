"""The operators of a gated recurrent mixer, as a user's program calls them, for measurement.

Two operators, each with the directions it is used in:

  gated linear recurrence    h_t = a_t h_{t-1} + u_t per channel, channels last (b, L, D)
      scan        the whole sequence from an initial state; the states h as y, and the last one
      scan_bwd    the gradients of x, the gate and the initial state
      step        one token (or a short run) on a resident state
  group norm with an activation, channels last (n, S, C)
      norm        statistics over (S, C / G) of each sample and group, affine map, activation or gate
      norm_bwd    the gradients of x, the gate, the weight and the bias

The decay a_t comes from the gate tensor: "decay" a = g, "log" a = exp(g), "logit" a = sigmoid(g); the input
is u = x, or u = (1 - a) x where `complement` is true.  A token with a = 0 starts a new sequence of a packed
batch (g = 0, -inf, -inf).  The norm's `act`: "none" y = n, "silu" y = silu(n), "gate" y = n silu(z),
"gate_first" y = norm(x silu(z)), with n = w xhat + b; `rms` leaves out the mean.
"""
import math

import torch

own = False

BLOCK = 64  # tokens between two of the states that the scan's backward pass starts from

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def scan_case(name, op, b, L, D, dtype, kind, complement, init):
    return {"name": name, "op": op, "b": b, "L": L, "D": D, "dtype": dtype, "kind": kind, "complement": complement,
            "init": init}


def norm_case(name, op, n, S, C, G, dtype, act, rms):
    return {"name": name, "op": op, "n": n, "S": S, "C": C, "G": G, "dtype": dtype, "act": act, "rms": rms}


def listed():
    return [
        # serving one request with the 130M layer's width: nothing but latency
        scan_case("step b1 d1536", "step", 1, 1, 1536, "bf16", "logit", True, True),
        # serving 64 requests at once with the 2.7B layer's width
        scan_case("step b64 d5120", "step", 64, 1, 5120, "bf16", "log", False, True),
        # the forward pass of the 130M layer: few steps for each chain, a launch counts
        scan_case("scan 130m layer", "scan", 4, 2048, 1536, "bf16", "logit", True, False),
        # one long document of 256K tokens: few channels, the work has to be split over the sequence
        scan_case("scan 256k", "scan", 1, 262144, 2048, "bf16", "log", False, True),
        # training the 2.7B layer
        scan_case("scan_bwd 2.7b layer", "scan_bwd", 2, 8192, 5120, "bf16", "logit", True, True),
        # training in 32 bits at odd sizes: rows that no wide load fits
        scan_case("scan_bwd odd f32", "scan_bwd", 3, 4099, 1001, "f32", "decay", False, True),
        # the norm behind the serving step: one row a request, the gate applied first
        norm_case("norm step b64 c5120", "norm", 64, 1, 5120, 1, "bf16", "gate_first", True),
        # the gated norm of the 2.7B layer, 16384 tokens, 8 groups
        norm_case("norm tokens 2.7b layer", "norm", 16384, 1, 5120, 8, "bf16", "gate_first", True),
        # training the 130M layer with one group a head of 64 channels, mean taken out, gate behind the norm
        norm_case("norm_bwd tokens 130m", "norm_bwd", 8192, 1, 1536, 24, "bf16", "gate", False),
        # feature maps of 64 x 64 positions, 16 channels a group
        norm_case("norm map 4096x512", "norm", 8, 4096, 512, 32, "bf16", "silu", False),
        # odd positions, channels and groups in 32 bits
        norm_case("norm_bwd odd f32", "norm_bwd", 3, 1001, 330, 11, "f32", "silu", False),
        # training on long sequences: a group's values fill more than the on-chip memory of a cluster
        norm_case("norm_bwd long 65536x256", "norm_bwd", 4, 65536, 256, 8, "bf16", "silu", False),
    ]


def spread(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; every third one is rounded to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // 64 * 64)) if v >= 128 and rng.random() < 0.34 else max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_bwd", "scan_bwd", "norm", "norm", "norm_bwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        c = scan_case("", op, spread(rng, 1, 128), rng.choice([1, 1, 1, 2, 5]), spread(rng, 64, 8192), dtype,
                      rng.choice(["decay", "log", "logit"]), rng.random() < 0.5, True)
    elif op in ("scan", "scan_bwd"):
        most = 160_000_000 if op == "scan" else 40_000_000
        while True:
            b, L, D = spread(rng, 1, 16), spread(rng, 16, 262144), spread(rng, 64, 8192)
            if 20_000 <= b * L * D <= most:
                break
        c = scan_case("", op, b, L, D, dtype, rng.choice(["decay", "log", "logit"]), rng.random() < 0.5,
                      rng.random() < 0.5)
    else:
        most = 64_000_000 if op == "norm" else 32_000_000
        act, rms = rng.choice(["none", "silu", "gate", "gate_first"]), rng.random() < 0.5
        while True:
            tokens = rng.random() < 0.5
            n, S = (spread(rng, 1, 16384), 1) if tokens else (spread(rng, 1, 32), spread(rng, 2, 65536))
            G = rng.choice([1, 1, 4, 8, 11, 24, 32])
            C = G * max(1, spread(rng, 64, 6144) // G)
            if 20_000 <= n * S * C <= most:
                break
        c = norm_case("", op, n, S, C, G, dtype, act, rms)
    del c["name"]
    return c


# ------------------------------------------------------------------ the plain forms

def decay_of(g, kind):
    """The decay a and 1 - a."""
    if kind == "decay":
        return g, 1 - g
    if kind == "log":
        return torch.exp(g), -torch.expm1(g)
    return 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))


def linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 from h_{-1} = 0: after the pass with step d each entry spans 2 d tokens."""
    d = 1
    while d < u.shape[1]:
        u = torch.cat([u[:, :d], u[:, d:] + a[:, d:] * u[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return u


def states_of(x, g, init, kind, complement):
    """The states h (b, L, D), the decay and 1 - a, in 32 bits."""
    a, s = decay_of(g.float(), kind)
    u = s * x.float() if complement else x.float()
    if init is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * init[:, None], u[:, 1:]], 1)
    return linear_scan(a, u), a, s


def before(h, init):
    """The state that each token starts from."""
    first = torch.zeros_like(h[:, 0]) if init is None else init
    return torch.cat([first[:, None], h[:, :-1]], 1)


def plain_scan(t, c):
    h, _, _ = states_of(t["x"], t["gate"], t["init"], c["kind"], c["complement"])
    return {"y": h.to(t["x"].dtype), "final": h[:, -1].clone()}


def plain_scan_bwd(t, c):
    x, dtype = t["x"].float(), t["x"].dtype
    h, a, s = states_of(t["x"], t["gate"], t["init"], c["kind"], c["complement"])
    was = before(h, t["init"])
    dy = t["dy"].float()
    dy = torch.cat([dy[:, :-1], dy[:, -1:] + t["dfinal"][:, None]], 1)
    follow = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    dh = linear_scan(follow.flip(1), dy.flip(1)).flip(1)
    da = dh * (was - x) if c["complement"] else dh * was
    if c["kind"] == "log":
        da = da * a
    elif c["kind"] == "logit":
        da = da * a * s
    dx = dh * s if c["complement"] else dh
    return {"dx": dx.to(dtype), "dgate": da.to(dtype), "dinit": a[:, 0] * dh[:, 0]}


def grouped(v, G):
    n, S, C = v.shape
    return v.reshape(n, S, G, C // G)


def sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def stats_of(v, G, eps, rms):
    v = grouped(v, G)
    mean = torch.zeros_like(v[:, 0, :, 0]) if rms else v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def normed(v, mean, rstd, G):
    return ((grouped(v, G) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(v.shape)


def plain_norm(t, c):
    x = t["x"].float()
    if c["act"] == "gate_first":
        z = t["z"].float()
        x = x * z * sigmoid(z)
    mean, rstd = stats_of(x, c["G"], t["eps"], c["rms"])
    y = normed(x, mean, rstd, c["G"]) * t["weight"] + t["bias"]
    if c["act"] == "silu":
        y = y * sigmoid(y)
    elif c["act"] == "gate":
        z = t["z"].float()
        y = y * (z * sigmoid(z))
    return {"y": y.to(t["x"].dtype), "mean": mean, "rstd": rstd}


def plain_norm_bwd(t, c):
    x, dp, act, G, dtype = t["x"].float(), t["dy"].float(), c["act"], c["G"], t["x"].dtype
    out = {}
    v = x
    if "z" in t:
        z = t["z"].float()
        sz = sigmoid(z)
        dsilu = sz * (1 + z * (1 - sz))
    if act == "gate_first":
        v = x * z * sz
    xhat = normed(v, t["mean"], t["rstd"], G)
    if act in ("silu", "gate"):
        p = xhat * t["weight"] + t["bias"]
    if act == "silu":
        sp = sigmoid(p)
        dp = dp * (sp * (1 + p * (1 - sp)))
    elif act == "gate":
        out["dz"] = (dp * p * dsilu).to(dtype)
        dp = dp * (z * sz)
    out["dweight"], out["dbias"] = (dp * xhat).sum((0, 1)), dp.sum((0, 1))
    q = dp * t["weight"]
    m1 = grouped(q, G).mean((1, 3), keepdim=True)
    m2 = grouped(q * xhat, G).mean((1, 3), keepdim=True)
    dv = grouped(q, G) - grouped(xhat, G) * m2
    if not c["rms"]:
        dv = dv - m1
    dv = (dv * t["rstd"][:, None, :, None]).reshape(x.shape)
    if act == "gate_first":
        out["dz"] = (dv * x * dsilu).to(dtype)
        dv = dv * (z * sz)
    out["dx"] = dv.to(dtype)
    return out


# ------------------------------------------------------------------ what a user's program has and does

def scan_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, L, D, dtype = c["b"], c["L"], c["D"], DTYPE[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    # half lives from about one token to a few hundred, each channel around its own
    rate = torch.exp(uniform(D) * 5 - 5.5)
    if c["kind"] == "logit":
        gate = -torch.log(rate) + normal(b, L, D)
        start = -math.inf
    else:
        gate = -rate * torch.exp(0.5 * normal(b, L, D))
        start = -math.inf
        if c["kind"] == "decay":
            gate, start = torch.exp(gate), 0.0
    if L >= 256:  # a few sequences in one row: a token that forgets all before it
        at = torch.randint(1, L, (b, 1 + L // 4096), generator=g, device="cuda")
        gate[torch.arange(b, device="cuda")[:, None], at] = start
    t = {"x": normal(b, L, D).to(dtype), "gate": gate.to(dtype), "init": normal(b, D) if c["init"] else None}
    if c["op"] == "scan_bwd":
        t["dy"] = normal(b, L, D).to(dtype)
        t["dfinal"] = normal(b, D)
        h, _, _ = states_of(t["x"], t["gate"], t["init"], c["kind"], c["complement"])
        t["states"] = before(h, t["init"])[:, ::BLOCK].contiguous()  # the forward pass leaves them behind
    if c["op"] == "step":
        t["next"] = torch.empty_like(t["init"])
    return t


def norm_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, S, C, dtype = c["n"], c["S"], c["C"], DTYPE[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = normal(n, S, C) * (0.5 + torch.rand(C, generator=g, device="cuda")) + 0.3 * normal(C)
    t = {"x": x.to(dtype), "weight": 1 + 0.2 * normal(C), "bias": 0.2 * normal(C), "eps": 1e-5}
    if c["act"] in ("gate", "gate_first"):
        t["z"] = normal(n, S, C).to(dtype)
    if c["op"] == "norm_bwd":
        t["dy"] = normal(n, S, C).to(dtype)
        v = t["x"].float()
        if c["act"] == "gate_first":
            z = t["z"].float()
            v = v * z * sigmoid(z)
        t["mean"], t["rstd"] = stats_of(v, c["G"], t["eps"], c["rms"])  # the forward pass leaves them behind
    return t


def prepare(case, seed):
    t = norm_inputs(case, seed) if case["op"].startswith("norm") else scan_inputs(case, seed)
    return {"case": case, "t": t}


def own_run(t, c):
    from state_space_model_02_gb300 import ssd

    if c["op"].startswith("norm"):
        kw = {"groups": c["G"], "z": t.get("z"), "act": c["act"], "rms": c["rms"]}
        if c["op"] == "norm":
            y, mean, rstd = ssd.group_norm(t["x"], t["weight"], t["bias"], eps=t["eps"], want_stats=True, **kw)
            return {"y": y, "mean": mean, "rstd": rstd}
        d = ssd.group_norm_bwd(t["x"], t["dy"], t["mean"], t["rstd"], t["weight"], t["bias"], **kw)
        return {k: v for k, v in d.items() if v is not None}
    kw = {"kind": c["kind"], "complement": c["complement"]}
    if c["op"] == "step":
        return {"y": ssd.gated_decode(t["x"], t["gate"], t["init"], new_state=t["next"], **kw), "final": t["next"]}
    if c["op"] == "scan":
        y, final = ssd.gated_scan(t["x"], t["gate"], t["init"], **kw)
        return {"y": y, "final": final}
    return ssd.gated_scan_bwd(t["x"], t["gate"], t["dy"], t["states"], t["dfinal"], **kw)


PLAIN = {"step": plain_scan, "scan": plain_scan, "scan_bwd": plain_scan_bwd, "norm": plain_norm,
         "norm_bwd": plain_norm_bwd}


def run(state):
    c = state["case"]
    return own_run(state["t"], c) if own else PLAIN[c["op"]](state["t"], c)


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"].startswith("norm"):
        n, S, C, G = (case[k] for k in ("n", "S", "C", "G"))
        gated = case["act"] in ("gate", "gate_first")
        if case["op"] == "norm":  # x (and z) in, y out, the statistics out, weight and bias in
            return {"bytes": n * S * C * e * (2 + gated) + 8 * n * G + 8 * C, "flops": n * S * C * (12 if gated else 8)}
        # x, dy (and z) in, dx (and dz) out, the statistics in, weight and bias in, their gradients out
        return {"bytes": n * S * C * e * (3 + 2 * gated) + 8 * n * G + 16 * C, "flops": n * S * C * (30 if gated else 20)}
    b, L, D = case["b"], case["L"], case["D"]
    if case["op"] == "scan_bwd":  # x, gate, dy in, dx and dgate out; a state of each block, dfinal in and dinit out
        return {"bytes": b * L * D * e * 5 + 4 * b * D * (-(-L // BLOCK) + 2), "flops": b * L * D * 16}
    # x, gate in, y out; the first state (if any) in, the last one out
    return {"bytes": b * L * D * e * 3 + 4 * b * D * (2 if case["init"] else 1), "flops": b * L * D * 8}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact_scan(t, c):
    """Token after token."""
    x, g = t["x"].double(), t["gate"].double()
    a = g if c["kind"] == "decay" else g.exp() if c["kind"] == "log" else g.sigmoid()
    u = (1 - a) * x if c["complement"] else x
    h = torch.empty_like(x)
    last = torch.zeros_like(x[:, 0]) if t["init"] is None else t["init"].double()
    for i in range(c["L"]):
        last = torch.addcmul(u[:, i], a[:, i], last, out=h[:, i])
    if c["op"] != "scan_bwd":
        return {"y": h, "final": h[:, -1]}
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    dh = t["dfinal"].double()
    for i in reversed(range(c["L"])):
        dh = dh + t["dy"][:, i].double()
        was = h[:, i - 1] if i else torch.zeros_like(dh) if t["init"] is None else t["init"].double()
        dx[:, i] = dh * (1 - a[:, i]) if c["complement"] else dh
        dg[:, i] = dh * (was - x[:, i]) if c["complement"] else dh * was
        dh = dh * a[:, i]
    if c["kind"] == "log":
        dg *= a
    elif c["kind"] == "logit":
        dg *= a * (1 - a)
    return {"dx": dx, "dgate": dg, "dinit": dh}


def exact_norm(t, c):
    """The definition; the gradients by differentiating it."""
    n, S, C, G = c["n"], c["S"], c["C"], c["G"]
    leaf = {k: t[k].double().requires_grad_(c["op"] == "norm_bwd") for k in ("x", "z", "weight", "bias") if k in t}
    v = leaf["x"]
    gate = leaf["z"] * torch.sigmoid(leaf["z"]) if "z" in leaf else None
    if c["act"] == "gate_first":
        v = v * gate
    by = v.reshape(n, S, G, C // G).transpose(1, 2).reshape(n, G, -1)
    mean = by.mean(2) * (0.0 if c["rms"] else 1.0)
    rstd = (by.square().mean(2) - mean.square() + t["eps"]).rsqrt()
    hat = ((by - mean[..., None]) * rstd[..., None]).reshape(n, G, S, C // G).transpose(1, 2).reshape(n, S, C)
    y = hat * leaf["weight"] + leaf["bias"]
    y = y * torch.sigmoid(y) if c["act"] == "silu" else y * gate if c["act"] == "gate" else y
    if c["op"] == "norm":
        return {"y": y, "mean": mean, "rstd": rstd}
    names = {"x": "dx", "z": "dz", "weight": "dweight", "bias": "dbias"}
    grads = torch.autograd.grad(y, [leaf[k] for k in leaf], t["dy"].double())
    return {names[k]: v for k, v in zip(leaf, grads)}


def exact(case, seed):
    t = prepare(case, seed)["t"]
    return exact_norm(t, case) if case["op"].startswith("norm") else exact_scan(t, case)
