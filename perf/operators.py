"""The operators around the sequence scan, as measured workloads.

Three families that sit next to the state-space scan in a layer:

  gated   a gated linear recurrence over long sequences, one decay per channel:
            r = sigmoid(r_raw), g = sigmoid(g_raw), a = exp(-c softplus(lam) r)
            h_t = a_t h_{t-1} + sqrt(1 - a_t^2) g_t x_t,   y = h
          forward ("gated_scan"), forward and backward ("gated_train"), one
          token with the state updated in place ("gated_step")
  norm    the RMS norm of B and C (the scan's keys and queries) per group and
          the rotation of their pairs by the token's position, in one pass:
          forward ("norm"), forward and backward ("norm_train")
  linear  the projections into and out of a layer,
          out = act(x W^T + bias) + residual: forward ("linear"), backward
          from the saved pre-activation ("linear_bwd")

`run` computes them in elementary torch operations, or with `own` set through
the package's entry points.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_C = 8.0                      # decay scale of the gated recurrence
_EPS = 1e-5

# Largest work a drawn case may ask for, by what bounds each family: those of
# the largest listed ones.
_MAX_GATED = 65536 * 5120     # tokens x channels, forward
_MAX_TRAIN = 8 * 4096 * 5120  # tokens x channels, forward and backward
_MAX_NORM = 65536 * 8 * 128   # elements of B (and of C)
_MAX_LINEAR = 32768 * 10576 * 2560
_MAX_LINEAR_BWD = 8192 * 5120 * 2560


def listed():
    return [
        # one user's decode step in a wide layer: latency
        {"name": "gated step, 1 row", "op": "gated_step", "b": 1, "D": 2560, "dtype": "bf16"},
        # a full serving batch's decode step
        {"name": "gated step, 256 rows", "op": "gated_step", "b": 256, "D": 5120, "dtype": "f32"},
        # one long prompt
        {"name": "gated scan, 64k tokens", "op": "gated_scan", "b": 1, "L": 65536, "D": 5120, "dtype": "bf16",
         "packed": False, "init": True},
        # documents packed into ragged rows, odd channel count
        {"name": "gated scan, packed odd", "op": "gated_scan", "b": 3, "L": 1777, "D": 1003, "dtype": "f32",
         "packed": True, "init": True},
        # a training step's share of a wide layer
        {"name": "gated train, 8 x 4096", "op": "gated_train", "b": 8, "L": 4096, "D": 5120, "dtype": "bf16",
         "packed": False, "init": False},
        # a small layer trained in full precision on packed rows
        {"name": "gated train, packed f32", "op": "gated_train", "b": 2, "L": 777, "D": 1536, "dtype": "f32",
         "packed": True, "init": True},
        # the keys and queries of one long prompt, eight groups
        {"name": "norm, 64k tokens", "op": "norm", "b": 1, "L": 65536, "G": 8, "N": 128, "R": 128, "dtype": "bf16",
         "interleaved": False, "far": 0},
        # a training step on ragged rows far into a document, partly rotated
        {"name": "norm train, 8 x 4095", "op": "norm_train", "b": 8, "L": 4095, "G": 2, "N": 128, "R": 64,
         "dtype": "bf16", "interleaved": True, "far": 900000},
        # a decode step's projection back into the residual stream
        {"name": "linear, 4 rows", "op": "linear", "M": 4, "N": 2560, "K": 5120, "dtype": "bf16", "act": "none",
         "bias": False, "residual": True},
        # a prompt's projection into a wide layer
        {"name": "linear, 32768 rows", "op": "linear", "M": 32768, "N": 10576, "K": 2560, "dtype": "bf16",
         "act": "none", "bias": False, "residual": False},
        # ragged sizes in full precision with the whole epilogue
        {"name": "linear, odd f32", "op": "linear", "M": 333, "N": 1001, "K": 771, "dtype": "f32", "act": "gelu",
         "bias": True, "residual": True},
        # the backward of a training step's gated projection
        {"name": "linear backward, 8192 rows", "op": "linear_bwd", "M": 8192, "N": 5120, "K": 2560, "dtype": "bf16",
         "act": "silu", "bias": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_step", "gated_scan", "gated_train", "norm", "norm_train", "linear", "linear_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = {"op": op, "dtype": dtype}
    if op == "gated_step":
        c["b"] = _log(rng, 1, 512)
        c["D"] = rng.choice([_log(rng, 200, 5120), 64 * rng.randint(4, 80)])
    elif op in ("gated_scan", "gated_train"):
        most = _MAX_GATED if op == "gated_scan" else _MAX_TRAIN
        most //= 2 if dtype == "f32" else 1
        c["D"] = rng.choice([_log(rng, 200, 5120), 64 * rng.randint(4, 80)])
        c["L"] = _log(rng, 1, 65536 if op == "gated_scan" else 16384)
        c["L"] = max(1, min(c["L"], most // c["D"]))
        c["b"] = _log(rng, 1, max(1, min(16, most // (c["D"] * c["L"]))))
        c["packed"] = rng.random() < 0.4
        c["init"] = rng.random() < 0.5
    elif op in ("norm", "norm_train"):
        c["G"] = rng.choice([1, 2, 3, 4, 8])
        c["N"] = rng.choice([64, 128, 128, 256, 96, 80, 112])
        c["R"] = rng.choice([c["N"], c["N"] // 2])
        most = _MAX_NORM // (2 if dtype == "f32" else 1) // (2 if op == "norm_train" else 1)
        c["L"] = max(1, min(_log(rng, 1, 65536), most // (c["G"] * c["N"])))
        c["b"] = _log(rng, 1, max(1, min(256, most // (c["G"] * c["N"] * c["L"]))))
        c["interleaved"] = rng.random() < 0.5
        c["far"] = rng.choice([0, rng.randint(1, 1 << 20)])
    else:
        most = _MAX_LINEAR if op == "linear" else _MAX_LINEAR_BWD
        most //= 16 if dtype == "f32" else 1
        side = lambda: rng.choice([_log(rng, 128, 8192), 8 * _log(rng, 16, 1024)])  # noqa: E731
        c["N"], c["K"] = side(), side()
        c["M"] = max(1, min(_log(rng, 1, 32768), most // (c["N"] * c["K"])))
        c["act"] = rng.choice(["none", "silu", "gelu"])
        c["bias"] = rng.random() < 0.5
        if op == "linear":
            c["residual"] = rng.random() < 0.5
    return c


# --------------------------------------------------------------------------
# inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _gated_inputs(c, g):
    t = _T[c["dtype"]]
    rows = (c["b"],) if c["op"] == "gated_step" else (c["b"], c["L"])
    D = c["D"]
    # the two gates leave one projection side by side: r_raw and g_raw are its halves
    gates = _randn(g, *rows, 2 * D).to(t)
    # decay at an open gate between 0.9 and 0.999: c softplus(lam) = -log(a)
    a = 0.9 + 0.099 * torch.rand(D, generator=g, device="cuda", dtype=torch.float64)
    s = {"x": _randn(g, *rows, D).to(t), "r": gates[..., :D], "g": gates[..., D:],
         "lam": torch.log(torch.expm1(-torch.log(a) / _C)).float()}
    if c["op"] == "gated_step":
        s["state"] = _randn(g, c["b"], D)
        return s
    s["init"] = _randn(g, c["b"], D) if c["init"] else None
    s["seq_idx"] = None
    if c["packed"]:
        # documents of about 100 tokens on average, some of a single one
        start = torch.rand(c["b"], c["L"], generator=g, device="cuda") < 0.01
        start[:, 1::97] |= start[:, ::97][:, :start[:, 1::97].shape[1]]
        s["seq_idx"] = torch.cumsum(start, 1).to(torch.int32)
    if c["op"] == "gated_train":
        s["dy"] = _randn(g, *rows, D).to(t)
        s["dfinal"] = _randn(g, c["b"], D)
    return s


def _norm_inputs(c, g):
    t = _T[c["dtype"]]
    shape = (c["b"], c["L"], c["G"], c["N"])
    s = {"B": _randn(g, *shape).to(t), "C": _randn(g, *shape).to(t),
         "wB": 1.0 + 0.1 * _randn(g, c["N"]), "wC": 1.0 + 0.1 * _randn(g, c["N"])}
    j = torch.arange(c["R"] // 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = (10000.0 ** (-2.0 * j / c["R"])).float()
    s["positions"] = None
    if c["far"]:
        first = torch.randint(0, c["far"], (c["b"], 1), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = first + torch.arange(c["L"], device="cuda", dtype=torch.int32)
    s["interleaved"] = c["interleaved"]
    if c["op"] == "norm_train":
        s["dB"], s["dC"] = _randn(g, *shape).to(t), _randn(g, *shape).to(t)
    return s


def _linear_inputs(c, g):
    t = _T[c["dtype"]]
    s = {"x": _randn(g, c["M"], c["K"]).to(t), "W": (_randn(g, c["N"], c["K"]) / math.sqrt(c["K"])).to(t),
         "act": c["act"]}
    s["bias"] = 0.1 * _randn(g, c["N"]) if c["bias"] else None
    if c["op"] == "linear":
        s["residual"] = _randn(g, c["M"], c["N"]).to(t) if c["residual"] else None
    else:
        s["dy"] = _randn(g, c["M"], c["N"]).to(t)
        # what the forward saved: the pre-activation (unit variance plus the bias), in the layer's type
        z = _randn(g, c["M"], c["N"])
        s["z"] = None if c["act"] == "none" else (z if s["bias"] is None else z + s["bias"]).to(t)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = (_gated_inputs if op.startswith("gated") else _norm_inputs if op.startswith("norm") else _linear_inputs)(case, g)
    s["op"] = op
    return s


# --------------------------------------------------------------------------
# the package's entry points


def _run_own(s):
    from state_space_sequence_scan_b200 import ssd

    op = s["op"]
    if op == "gated_step":
        y = ssd.gated_step(s["x"], s["r"], s["g"], s["lam"], s["state"], decay_scale=_C)
        return {"y": y, "state": s["state"]}
    if op == "gated_scan":
        y, final = ssd.gated_scan_fwd(s["x"], s["r"], s["g"], s["lam"], init_state=s["init"], seq_idx=s["seq_idx"],
                                      decay_scale=_C)
        return {"y": y, "final": final}
    if op == "gated_train":
        y, final, states = ssd.gated_scan_fwd_states(s["x"], s["r"], s["g"], s["lam"], init_state=s["init"],
                                                     seq_idx=s["seq_idx"], decay_scale=_C)
        d = ssd.gated_scan_bwd(s["x"], s["r"], s["g"], s["lam"], states, s["dy"], dfinal_state=s["dfinal"],
                               init_state=s["init"], seq_idx=s["seq_idx"], decay_scale=_C)
        return {"y": y, "final": final, "dx": d["x"], "dr": d["r_raw"], "dg": d["g_raw"], "dlam": d["lam"],
                "dinit": d["init_state"]}
    if op in ("norm", "norm_train"):
        B, C = ssd.bc_norm_rotate_fwd(s["B"], s["C"], s["wB"], s["wC"], s["inv_freq"], positions=s["positions"],
                                      eps=_EPS, interleaved=s["interleaved"])
        if op == "norm":
            return {"B": B, "C": C}
        d = ssd.bc_norm_rotate_bwd(s["B"], s["C"], s["wB"], s["wC"], s["inv_freq"], s["dB"], s["dC"],
                                   positions=s["positions"], eps=_EPS, interleaved=s["interleaved"])
        return {"B": B, "C": C, "dB": d["B"], "dC": d["C"], "dwB": d["weight_B"], "dwC": d["weight_C"]}
    if op == "linear":
        return ssd.linear_fwd(s["x"], s["W"], bias=s["bias"], residual=s["residual"], activation=s["act"])
    d = ssd.linear_bwd(s["x"], s["W"], s["dy"], preact=s["z"], activation=s["act"], want_dbias=s["bias"] is not None)
    return {"dx": d["x"], "dW": d["weight"], "db": d["bias"]}


# --------------------------------------------------------------------------
# the plain forms


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling spans."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _gates(s):
    x, r, g = s["x"].float(), torch.sigmoid(s["r"].float()), torch.sigmoid(s["g"].float())
    la = -_C * torch.log1p(torch.exp(s["lam"])) * r
    return x, r, g, torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))


def _kept(s):
    """1 where a token continues its predecessor's document, 0 at a start; [b, L, 1]."""
    i = s["seq_idx"]
    kept = torch.ones(s["x"].shape[0], s["x"].shape[1], 1, device=s["x"].device)
    if i is not None:
        kept[:, 1:, 0] = (i[:, 1:] == i[:, :-1]).float()
    return kept


def _gated_fwd(s):
    x, r, g, a, beta = _gates(s)
    b = beta * g * x
    if s["init"] is not None:
        b[:, 0] += a[:, 0] * s["init"]
    return _scan(a * _kept(s), b)


def _gated_train(s):
    x, r, g, a, beta = _gates(s)
    kept = _kept(s)
    h = _gated_fwd(s)
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["init"] is None else s["init"][:, None], h[:, :-1]], 1) * kept
    dy = s["dy"].to(torch.float32, copy=True)
    dy[:, -1] += s["dfinal"]
    later = torch.cat([(a * kept)[:, 1:], torch.zeros_like(a[:, :1])], 1)
    dh = _scan(later.flip(1), dy.flip(1)).flip(1)
    dla = dh * (a * before - a * a / beta * g * x)
    k = _C * torch.log1p(torch.exp(s["lam"]))
    t = s["x"].dtype
    return {"y": h.to(t), "final": h[:, -1].clone(), "dx": (dh * beta * g).to(t),
            "dr": (-dla * k * r * (1 - r)).to(t), "dg": (dh * beta * x * g * (1 - g)).to(t),
            "dlam": ((-_C * torch.sigmoid(s["lam"])).double() * (dla * r).double().sum((0, 1))).float(),
            "dinit": dh[:, 0] * a[:, 0]}


def _turn(s, L):
    """cos and sin of each token's angles, [b or 1, L, 1, R / 2]; the angles in
    64 bits, where far positions need them."""
    p = s["positions"]
    p = torch.arange(L, device="cuda")[None] if p is None else p
    angle = p.double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(v, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    p, q = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
    p, q = p * cos - q * sin, q * cos + p * sin
    both = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([both, v[..., R:]], -1)


def _norm_one(v, w, cos, sin, interleaved):
    v = v.float()
    rs = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)
    return _rotate(v * rs * w, cos, sin, interleaved)


def _norm_one_bwd(v, w, d, cos, sin, interleaved):
    v, d = v.float(), _rotate(d.float(), cos, -sin, interleaved)
    rs = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)
    n = v * rs
    dn = d * w
    return rs * (dn - n * (dn * n).mean(-1, keepdim=True)), (d * n).double().sum((0, 1, 2)).float()


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5))) if act == "gelu" else z


def _act_slope(z, act):
    if act == "silu":
        q = torch.sigmoid(z)
        return q * (1.0 + z * (1.0 - q))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _run_plain(s):
    op = s["op"]
    if op == "gated_step":
        x, r, g, a, beta = _gates(s)
        s["state"].copy_(a * s["state"] + beta * g * x)
        return {"y": s["state"].to(s["x"].dtype), "state": s["state"]}
    if op == "gated_scan":
        h = _gated_fwd(s)
        return {"y": h.to(s["x"].dtype), "final": h[:, -1].clone()}
    if op == "gated_train":
        return _gated_train(s)
    if op in ("norm", "norm_train"):
        t, il = s["B"].dtype, s["interleaved"]
        cos, sin = _turn(s, s["B"].shape[1])
        out = {"B": _norm_one(s["B"], s["wB"], cos, sin, il).to(t), "C": _norm_one(s["C"], s["wC"], cos, sin, il).to(t)}
        if op == "norm_train":
            dB, out["dwB"] = _norm_one_bwd(s["B"], s["wB"], s["dB"], cos, sin, il)
            dC, out["dwC"] = _norm_one_bwd(s["C"], s["wC"], s["dC"], cos, sin, il)
            out["dB"], out["dC"] = dB.to(t), dC.to(t)
        return out
    x, W = s["x"].float(), s["W"].float()
    if op == "linear":
        z = x @ W.T
        z = _act(z if s["bias"] is None else z + s["bias"], s["act"])
        return (z if s["residual"] is None else z + s["residual"].float()).to(s["x"].dtype)
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    t = s["x"].dtype
    return {"dx": (dz @ W).to(t), "dW": (dz.T @ x).to(t),
            "db": None if s["bias"] is None else dz.double().sum(0).float()}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op.startswith("gated"):
        rows = case["b"] * case.get("L", 1)
        n, state = rows * case["D"], case["b"] * case["D"] * 4
        ids = rows * 4 if case.get("packed") else 0
        init = state if case.get("init") else 0
        if op == "gated_step":
            return {"bytes": 4 * n * e + 2 * state + 4 * case["D"], "flops": 12 * n}
        if op == "gated_scan":
            return {"bytes": 4 * n * e + ids + init + state + 4 * case["D"], "flops": 12 * n}
        # x and the gates once for both directions, dy; y, dx, dr, dg; states and the decay's gradient
        return {"bytes": 8 * n * e + ids + init + 3 * state + 8 * case["D"], "flops": 40 * n}
    if op.startswith("norm"):
        n = 2 * case["b"] * case["L"] * case["G"] * case["N"]
        small = 8 * case["N"] + 2 * case["R"] + (4 * case["b"] * case["L"] if case["far"] else 0)
        if op == "norm":
            return {"bytes": 2 * n * e + small, "flops": 8 * n}
        return {"bytes": 4 * n * e + small + 8 * case["N"], "flops": 24 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear":
        return {"bytes": e * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + (4 * N if case["bias"] else 0),
                "flops": 2.0 * M * N * K}
    return {"bytes": e * (2 * M * K + 2 * N * K + M * N * (1 if case["act"] == "none" else 2)) + (4 * N if case["bias"] else 0),
            "flops": 4.0 * M * N * K}


# --------------------------------------------------------------------------
# the definitions in 64 bits, token by token


def _exact_gated(s):
    f = torch.float64
    x, rr, gg, lam = (s[k].to(f) for k in ("x", "r", "g", "lam"))
    r, g = 1 / (1 + torch.exp(-rr)), 1 / (1 + torch.exp(-gg))
    k = _C * torch.logaddexp(lam, torch.zeros_like(lam))
    a = torch.exp(-k * r)
    beta = torch.sqrt(-torch.expm1(-2 * k * r))
    if s["op"] == "gated_step":
        h = a * s["state"].to(f) + beta * g * x
        return {"y": h, "state": h}
    b, L, D = x.shape
    first = torch.zeros(b, L, dtype=torch.bool, device=x.device)
    if s["seq_idx"] is not None:
        first[:, 1:] = s["seq_idx"][:, 1:] != s["seq_idx"][:, :-1]
    a_in = a.masked_fill(first[..., None], 0.0)
    b_in = beta * g * x
    h = torch.zeros(b, D, dtype=f, device=x.device) if s["init"] is None else s["init"].to(f)
    hs = torch.empty_like(x)
    for t in range(L):
        h = torch.addcmul(b_in[:, t], a_in[:, t], h, out=hs[:, t])
    if s["op"] == "gated_scan":
        return {"y": hs, "final": hs[:, -1]}
    dhs = s["dy"].to(f)
    dhs[:, -1] += s["dfinal"].to(f)
    for t in range(L - 2, -1, -1):
        dhs[:, t] += a_in[:, t + 1] * dhs[:, t + 1]
    prev = torch.zeros_like(hs)
    prev[:, 1:] = hs[:, :-1]
    if s["init"] is not None:
        prev[:, 0] = s["init"].to(f)
    prev.masked_fill_(first[..., None], 0.0)
    # d h / d (k r) = -a h_prev + g x a^2 / beta
    dkr = dhs * (g * x * a * a / beta - a * prev)
    return {"y": hs, "final": hs[:, -1], "dx": dhs * beta * g, "dr": dkr * k * r * (1 - r),
            "dg": dhs * beta * x * g * (1 - g),
            "dlam": (dkr * r).sum((0, 1)) * _C / (1 + torch.exp(-lam)), "dinit": a_in[:, 0] * dhs[:, 0]}


def _exact_norm(s):
    f = torch.float64
    b, L, G, N = s["B"].shape
    R, dev = 2 * s["inv_freq"].numel(), s["B"].device
    pos = torch.arange(L, device=dev).expand(b, L) if s["positions"] is None else s["positions"]
    # the rotation as multiplication by e^(i angle) of the pairs, the rest by 1
    turn = torch.polar(torch.ones(b, L, R // 2, dtype=f, device=dev), pos.to(f)[..., None] * s["inv_freq"].to(f))[:, :, None]
    j = torch.arange(R // 2, device=dev)
    re, im = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + R // 2)

    def rotated(v, by):
        z = torch.complex(v[..., re], v[..., im]) * by
        out = v.clone()
        out[..., re], out[..., im] = z.real, z.imag
        return out

    out = {}
    for k in "BC":
        v, w = s[k].to(f), s["w" + k].to(f)
        size = torch.sqrt(v.square().sum(-1, keepdim=True) / N + _EPS)
        out[k] = rotated(v / size * w, turn)
        if s["op"] == "norm_train":
            d = rotated(s["d" + k].to(f), turn.conj())
            out["dw" + k] = (d * v / size).sum((0, 1, 2))
            out["d" + k] = d * w / size - v * (d * w * v).sum(-1, keepdim=True) / (N * size ** 3)
    return out


def _exact_linear(s):
    f = torch.float64
    x, W = s["x"].to(f), s["W"].to(f)
    if s["op"] == "linear":
        z = torch.einsum("mk,nk->mn", x, W)
        if s["bias"] is not None:
            z += s["bias"].to(f)
        if s["act"] == "silu":
            z = z / (1 + torch.exp(-z))
        elif s["act"] == "gelu":
            z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z if s["residual"] is None else z + s["residual"].to(f)
    dz = s["dy"].to(f)
    if s["act"] == "silu":
        z = s["z"].to(f)
        e = torch.exp(-z)
        dz = dz * (1 + e + z * e) / (1 + e) ** 2
    elif s["act"] == "gelu":
        z = s["z"].to(f)
        dz = dz * (0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi))
    return {"dx": torch.einsum("mn,nk->mk", dz, W), "dW": torch.einsum("mn,mk->nk", dz, x),
            "db": None if s["bias"] is None else dz.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    return (_exact_gated if op.startswith("gated") else _exact_norm if op.startswith("norm") else _exact_linear)(s)
