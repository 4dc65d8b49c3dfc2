"""Cases, inputs and plain forms of the selective scan, of the short causal convolution before it
and of layer norm.

Three operators, each with its passes:

  conv   y_t = act(bias + sum_j w_j x_{t-K+1+j})  a channel, over whole prompts (fwd), its gradients
         (bwd) and one token a sequence on the cache of the last K-1 inputs (step)
  scan   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,  y_t = (C_t . h_t + D x_t) silu(z_t)  a channel with
         S states, d_t = softplus(dt_t + bias) or given: fwd, bwd and step
  norm   h = residual + x,  n = (h - mean h) / sqrt(var h + eps) * w + b  a row: fwd and bwd

Where `own` is false `run` computes them from elementary torch operations in 32 bits (long sums
in 64); where it is true it calls the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------- cases
def _conv(name, pas, B, T, D, K, dtype, act, state, view, lens=""):
    c = {"op": "conv", "pass": pas, "B": B, "T": T, "D": D, "K": K, "dtype": dtype, "act": act,
         "state": state, "view": view, "lens": lens}
    return dict(c, name=name) if name else c


def _scan(name, pas, B, T, D, S, G, dtype, steps, z, state, view, lens=""):
    c = {"op": "scan", "pass": pas, "B": B, "T": T, "D": D, "S": S, "G": G, "dtype": dtype,
         "steps": steps, "z": z, "state": state, "view": view, "lens": lens}
    return dict(c, name=name) if name else c


def _norm(name, pas, rows, d, dtype, residual, bias):
    c = {"op": "norm", "pass": pas, "rows": rows, "d": d, "dtype": dtype, "residual": residual,
         "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    packed = "20000,1,8191,0,63,5021,1333,129,2048,65,3149"
    return [
        # a layer's training or prefill batch, its input one half of a projection's output
        _conv("conv fwd layer", "fwd", 8, 4096, 2048, 4, "bf16", "silu", False, True),
        # prompts of all lengths (one empty) continued from caches, an odd width in float32
        _conv("conv fwd packed", "fwd", 1, 40000, 1001, 3, "f32", "none", True, False, packed),
        # the training step's backward of the layer
        _conv("conv bwd layer", "bwd", 8, 4096, 2048, 4, "bf16", "silu", False, True),
        # a few sequences being decoded: latency
        _conv("conv step few", "step", 4, 1, 1024, 4, "bf16", "silu", True, False),
        # a layer's training or prefill batch, gated, its inputs parts of projections' outputs
        _scan("scan fwd layer", "fwd", 8, 4096, 2048, 16, 1, "bf16", "logits", True, False, True),
        # a serving batch of prompts of all lengths (one empty), one of them long, continued from states
        _scan("scan fwd packed", "fwd", 1, 40000, 2048, 16, 1, "bf16", "logits", True, True, True, packed),
        # the training step's backward of the layer
        _scan("scan bwd layer", "bwd", 8, 4096, 2048, 16, 1, "bf16", "logits", True, False, True),
        # a small float32 layer of odd sizes with groups and states, steps given: gradient checks
        _scan("scan bwd odd", "bwd", 2, 333, 234, 10, 2, "f32", "values", False, True, False),
        # a full decode batch
        _scan("scan step batch", "step", 256, 1, 4096, 16, 1, "bf16", "logits", True, True, False),
        # the output norm of a layer's heads (every token and head a row)
        _norm("norm heads", "fwd", 524288, 128, "bf16", False, True),
        # the norm between two blocks while decoding: latency
        _norm("norm decode", "fwd", 64, 2048, "bf16", True, True),
        # the norm between two blocks in a training step's backward
        _norm("norm bwd layer", "bwd", 32768, 2048, "bf16", True, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        d = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            d = -(-d // 16) * 16
        rows = _log(rng, 1, max(1, min(65536, (1 << 25) // d)))
        return _norm("", rng.choice(["fwd", "bwd"]), rows, d, dtype, rng.random() < 0.6, rng.random() < 0.6)
    pas = rng.choice(["fwd", "fwd", "bwd", "step"] if op == "conv" else ["fwd", "fwd", "bwd", "bwd", "step"])
    G = rng.choice([1, 1, 2, 4]) if op == "scan" else 1
    D = G * _log(rng, 4, 4096 // G)
    if rng.random() < 0.6:
        D = -(-D // (8 * G)) * 8 * G
    S = rng.choice([16, 16, rng.randint(1, 32)])
    per = D * S if op == "scan" else D
    most = (1 << (30 if op == "scan" else 26)) // per // (2 if pas == "bwd" else 1)
    lens = ""
    if pas == "step":
        B, T = _log(rng, 1, 256), 1
    else:
        B, T = rng.choice([1, 2, 3, 8]), 1
        tokens = _log(rng, 1, min(most, 65536 if pas == "fwd" else 16384))
        if rng.random() < 0.4:
            n = rng.randint(1, 12)
            cut = sorted(rng.randint(0, tokens) for _ in range(n - 1))
            lens = ",".join(str(b - a) for a, b in zip([0] + cut, cut + [tokens]))
            B, T = 1, tokens
        else:
            T = max(1, tokens // B)
    state = pas == "step" or rng.random() < 0.5
    view = pas != "step" and rng.random() < 0.5
    if op == "conv":
        return _conv("", pas, B, T, D, rng.randint(2, 4), dtype, rng.choice(["silu", "silu", "none"]), state, view, lens)
    return _scan("", pas, B, T, D, S, G, dtype, rng.choice(["logits", "logits", "values"]), rng.random() < 0.6, state,
                 view, lens)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["dtype"]]

    def randn(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return torch.randn(shape, device=DEV, generator=g).mul_(std).add_(mean).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = randn(rows, d, mean=0.3, std=1.5, dtype=t)
        s["r"] = randn(rows, d, dtype=t) if case["residual"] else None
        s["w"] = randn(d, mean=1.0, std=0.2)
        s["b"] = randn(d, std=0.2) if case["bias"] else None
        if case["pass"] == "bwd":
            s["dn"] = randn(rows, d, dtype=t)
            s["dh"] = randn(rows, d, dtype=t) if case["residual"] else None
        return s
    B, T, D = case["B"], case["T"], case["D"]
    lead, n = (B,) if case["pass"] == "step" else (B, T), B
    s["cu"], s["longest"] = None, T
    if case["lens"]:
        lens = [int(x) for x in case["lens"].split(",")]
        n, s["longest"] = len(lens), max(lens)
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    s["n"] = n
    wide = randn(*lead, 2 * D if case["view"] else D, dtype=t)  # x, and z beside it in a view
    s["x"] = wide[..., :D]
    if case["op"] == "conv":
        K = case["K"]
        s["w"] = randn(D, K, std=K ** -0.5)
        s["bias"] = randn(D, std=0.2)
        s["h0"] = randn(n, K - 1, D, dtype=t) if case["state"] else None
        if case["pass"] == "bwd":
            s["dout"] = randn(*lead, D, dtype=t)
            s["dht"] = randn(n, K - 1, D, dtype=t) if case["state"] else None
        return s
    S, G = case["S"], case["G"]
    s["z"] = None if not case["z"] else wide[..., D:] if case["view"] else randn(*lead, D, dtype=t)
    if case["view"]:  # B and C as parts of one projection, the steps from another
        both = randn(*lead, 2 * G * S, dtype=t)
        s["Bm"], s["Cm"] = (x.unflatten(-1, (G, S)) for x in both.split(G * S, -1))
    else:
        s["Bm"], s["Cm"] = (randn(*lead, G, S, dtype=t) for _ in range(2))
    # decays 1, 2, .. S a unit of time (a little apart from channel to channel), steps of 0.001 to 0.1
    s["A"] = -(torch.arange(1, S + 1, device=DEV).float() * torch.exp(randn(D, S, std=0.1)))
    at = torch.exp(torch.rand(D, device=DEV, generator=g) * math.log(100.0) + math.log(0.001))
    if case["steps"] == "logits":
        s["dt"] = randn(*lead, D, std=0.7, dtype=t)
        s["dt_bias"] = at + torch.log(-torch.expm1(-at))
    else:
        s["dt"] = (at * torch.exp(randn(*lead, D, std=0.7))).to(t)
        s["dt_bias"] = None
    s["Dv"] = randn(D, mean=1.0, std=0.2)
    if case["pass"] == "step":
        s["state"] = randn(n, D, S, std=0.5)
        return s
    s["h0"] = randn(n, D, S, std=0.5) if case["state"] else None
    if case["pass"] == "bwd":
        s["dout"] = randn(*lead, D, dtype=t)
        s["dht"] = randn(n, D, S, std=0.5) if case["state"] else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _kernels(state)
    return _PLAIN[state["op"], state["pass"]](state)


def _kernels(s):
    import gated_delta_rule_ckda_amd as ck
    at = s["op"], s["pass"]
    if at == ("norm", "fwd"):
        n, h = ck.layer_norm(s["x"], s["w"], s["b"], residual=s["r"], eps=EPS)
        return {"n": n, "h": h}
    if at == ("norm", "bwd"):
        return dict(zip(("dx", "dw", "db"), ck.layer_norm_bwd(
            s["x"], s["w"], s["dn"], dh=s["dh"], eps=EPS, output_dbias=s["b"] is not None)))
    if at == ("conv", "fwd"):
        y, ht = ck.conv_fwd(s["x"], s["w"], bias=s["bias"], act=s["act"], h0=s["h0"], cu_seqlens=s["cu"])
        return {"y": y, "ht": ht}
    if at == ("conv", "bwd"):
        return dict(zip(("dx", "dw", "dbias", "dh0"), ck.conv_bwd(
            s["x"], s["w"], s["dout"], bias=s["bias"], act=s["act"], h0=s["h0"], dht=s["dht"],
            cu_seqlens=s["cu"])))
    if at == ("conv", "step"):
        y = ck.conv_step(s["x"], s["w"], s["h0"], bias=s["bias"], act=s["act"])
        return {"y": y, "state": s["h0"]}
    with_ = dict(D=s["Dv"], z=s["z"], dt_bias=s["dt_bias"], steps=s["steps"])
    if at == ("scan", "step"):
        y = ck.scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], **with_)
        return {"y": y, "state": s["state"]}
    if at == ("scan", "fwd"):
        y, ht = ck.scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], h0=s["h0"], cu_seqlens=s["cu"], **with_)
        return {"y": y, "ht": ht}
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0"), ck.scan_bwd(
        s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dout"], h0=s["h0"], dht=s["dht"], cu_seqlens=s["cu"], **with_)))


# ---------------------------------------------------------------- plain forms
def _spread(s, x):
    """[B,T,...] or packed [1,T,...] -> [n, longest,...] in 32 bits: sequences side by side, zeros
    behind the shorter ones."""
    if s["cu"] is None:
        return x.float()
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(s["longest"], device=x.device)
    inside = (at < cu[1:, None]).reshape(at.shape + (1,) * (x.dim() - 2))
    return torch.where(inside, x[0][at.clamp(max=max(s["T"] - 1, 0))].float(), 0.0)


def _gather(s, y):
    """The inverse of _spread, for tokens of [n, longest,...]."""
    if s["cu"] is None:
        return y
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=y.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return y[seq, t - cu[seq]][None]


def _lengths(s):
    if s["cu"] is None:
        return torch.full((s["n"],), s["T"], device=DEV)
    return (s["cu"][1:] - s["cu"][:-1]).long()


def _silu(x):
    """silu and its derivative."""
    p = torch.sigmoid(x)
    return x * p, p * (1 + x * (1 - p))


def _conv_pre(s):
    """The inputs behind the cached ones, the sums before the activation, and the places of the
    last K-1 inputs."""
    K, L = s["K"], s["longest"]
    x = _spread(s, s["x"])
    h0 = x.new_zeros(s["n"], K - 1, s["D"]) if s["h0"] is None else s["h0"].float()
    x = torch.cat([h0, x], 1)
    pre = sum(s["w"][:, j] * x[:, j:j + L] for j in range(K)) + s["bias"]
    last = _lengths(s)[:, None] + torch.arange(K - 1, device=DEV)
    return x, pre, last[..., None].expand(-1, -1, s["D"])


def _plain_conv(s):
    x, pre, last = _conv_pre(s)
    y = _silu(pre)[0] if s["act"] == "silu" else pre
    io = s["x"].dtype
    return {"y": _gather(s, y).to(io), "ht": x.gather(1, last).to(io)}


def _plain_conv_bwd(s):
    x, pre, last = _conv_pre(s)
    K, L, io = s["K"], s["longest"], s["x"].dtype
    d = _spread(s, s["dout"])
    if s["act"] == "silu":
        d = d * _silu(pre)[1]
    dx = torch.zeros_like(x)
    for j in range(K):
        dx[:, j:j + L] += d * s["w"][:, j]
    if s["dht"] is not None:
        dx.scatter_add_(1, last, s["dht"].float())
    dw = torch.stack([(d * x[:, j:j + L]).sum((0, 1), dtype=torch.float64) for j in range(K)], -1)
    return {"dx": _gather(s, dx[:, K - 1:]).to(io), "dw": dw.float(),
            "dbias": d.sum((0, 1), dtype=torch.float64).float(), "dh0": dx[:, :K - 1].to(io)}


def _plain_conv_step(s):
    x = torch.cat([s["h0"], s["x"][:, None]], 1)
    y = (x.float() * s["w"].t()).sum(1) + s["bias"]
    s["h0"].copy_(x[:, 1:])
    return {"y": (_silu(y)[0] if s["act"] == "silu" else y).to(s["x"].dtype), "state": s["h0"]}


CHUNK = 64


def _steps(s, dt):
    """The steps d and their derivative by what `dt` holds."""
    v = dt if s["dt_bias"] is None else dt + s["dt_bias"]
    if s["steps"] == "values":
        return v, torch.ones_like(v)
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())), torch.sigmoid(v)


def _chunks(s, x, D=False):
    """[n, longest, ...] -> [n, chunks, CHUNK, ...], the channels of a D split into groups."""
    more = -x.shape[1] % CHUNK
    if more:
        x = torch.cat([x, x.new_zeros((x.shape[0], more) + x.shape[2:])], 1)
    x = x.unflatten(1, (-1, CHUNK))
    return x.unflatten(-1, (s["G"], -1)) if D else x


def _tokens(s, rows, D=False):
    """The inverse of _chunks, from a list of CHUNK rows, and packed again."""
    x = torch.stack(rows, 2).flatten(1, 2)[:, :s["longest"]]
    return _gather(s, x.flatten(2) if D else x)


def _laid(s):
    """x, d and d x, B and C in chunks; the channels' A in groups."""
    r = {"x": _chunks(s, _spread(s, s["x"]), True)}
    d, slope = _steps(s, s["dt"].float())
    r["d"] = _chunks(s, _spread(s, d), True)
    r["slope"] = slope
    r["u"] = r["x"] * r["d"]
    r["B"], r["C"] = (_chunks(s, _spread(s, s[m])) for m in ("Bm", "Cm"))
    r["A"] = s["A"].unflatten(0, (s["G"], -1))
    return r


def _decay(r, i):
    return torch.exp(r["d"][:, :, i, ..., None] * r["A"])


def _passed(decay, first, add):
    """H_{m+1} = decay_m H_m + add_m over the chunks: what enters each, and what leaves the last."""
    into, h = [], first
    for m in range(add.shape[1]):
        into.append(h)
        h = decay[:, m] * h + add[:, m]
    return torch.stack(into, 1), h


def _entered(s, r):
    """The states entering the chunks and leaving the last one; a chunk's decay."""
    h = torch.zeros(r["d"].shape[:2] + r["A"].shape, device=DEV)
    for i in range(CHUNK):
        h = _decay(r, i) * h + r["u"][:, :, i, ..., None] * r["B"][:, :, i, :, None]
    first = h.new_zeros(h[:, 0].shape) if s["h0"] is None else s["h0"].unflatten(1, (s["G"], -1))
    r["decay"] = torch.exp(r["d"].sum(2, dtype=torch.float64).float()[..., None] * r["A"])
    return _passed(r["decay"], first, h)


def _plain_scan(s):
    r = _laid(s)
    h, ht = _entered(s, r)
    ys = []
    for i in range(CHUNK):
        h = _decay(r, i) * h + r["u"][:, :, i, ..., None] * r["B"][:, :, i, :, None]
        ys.append((h * r["C"][:, :, i, :, None]).sum(-1))
    y = _tokens(s, ys, True) + s["Dv"] * s["x"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())[0]
    return {"y": y.to(s["x"].dtype), "ht": ht.flatten(1, 2)}


def _plain_scan_bwd(s):
    r = _laid(s)
    h0, _ = _entered(s, r)
    x, dout, io = s["x"].float(), s["dout"].float(), s["x"].dtype
    dy = dout
    if s["z"] is not None:
        act, slope = _silu(s["z"].float())
        dy = dout * act
    dyc = _chunks(s, _spread(s, dy), True)
    hs, ys = [h0], []
    for i in range(CHUNK):
        hs.append(_decay(r, i) * hs[-1] + r["u"][:, :, i, ..., None] * r["B"][:, :, i, :, None])
        ys.append((hs[-1] * r["C"][:, :, i, :, None]).sum(-1))
    g = torch.zeros_like(h0)
    for i in reversed(range(CHUNK)):
        g = _decay(r, i) * (g + dyc[:, :, i, ..., None] * r["C"][:, :, i, :, None])
    last = torch.zeros_like(g[:, 0]) if s["dht"] is None else s["dht"].unflatten(1, (s["G"], -1))
    g, dh0 = _passed(r["decay"].flip(1), last, g.flip(1))
    g = g.flip(1)
    dA = torch.zeros(r["A"].shape, device=DEV, dtype=torch.float64)
    through, given, dB, dC = [], [], [], []
    for i in reversed(range(CHUNK)):
        di, ui, gi = r["d"][:, :, i, ..., None], r["u"][:, :, i, ..., None], dyc[:, :, i, ..., None]
        G = g + gi * r["C"][:, :, i, :, None]
        through.append((G * r["B"][:, :, i, :, None]).sum(-1))
        g = _decay(r, i) * G
        w = g * hs[i]
        given.append((w * r["A"]).sum(-1))
        dA += (w * di).sum((0, 1), dtype=torch.float64)
        dB.append((G * ui).sum(3))
        dC.append((gi * hs[i + 1]).sum(3))
    through, given, dB, dC = (m[::-1] for m in (through, given, dB, dC))
    through = _tokens(s, through, True)
    ddt = (x * through + _tokens(s, given, True)) * r["slope"]
    lead = tuple(range(x.dim() - 1))
    out = {"dx": (_steps(s, s["dt"].float())[0] * through + s["Dv"] * dy).to(io), "ddt": ddt.to(io),
           "dA": dA.float().flatten(0, 1), "dB": _tokens(s, dB).to(io), "dC": _tokens(s, dC).to(io),
           "dD": (dy * x).sum(lead, dtype=torch.float64).float(), "dz": None, "dbias": None,
           "dh0": dh0.flatten(1, 2)}
    if s["z"] is not None:
        out["dz"] = (dout * slope * (_tokens(s, ys, True) + s["Dv"] * x)).to(io)
    if s["dt_bias"] is not None:
        out["dbias"] = ddt.sum(lead, dtype=torch.float64).float()
    return out


def _plain_scan_step(s):
    x, st = s["x"].float(), s["state"]
    rep = s["D"] // s["G"]
    d = _steps(s, s["dt"].float())[0][..., None]
    B, C = (s[m].float().repeat_interleave(rep, 1) for m in ("Bm", "Cm"))
    st.mul_(torch.exp(d * s["A"])).add_(d * x[..., None] * B)
    y = (st * C).sum(-1) + s["Dv"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())[0]
    return {"y": y.to(s["x"].dtype), "state": st}


def _centred(h):
    c = h - h.mean(-1, keepdim=True)
    return c, torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    h, io = s["x"].float(), s["x"].dtype
    if s["r"] is not None:
        h = h + s["r"].float()
    c, r = _centred(h)
    n = c * r * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    return {"n": n.to(io), "h": None if s["r"] is None else h.to(io)}


def _plain_norm_bwd(s):
    c, r = _centred(s["x"].float())
    c, dn = c * r, s["dn"].float()
    m = dn * s["w"]
    dx = r * (m - m.mean(-1, keepdim=True) - c * (m * c).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dn * c).sum(0, dtype=torch.float64).float(),
            "db": None if s["b"] is None else dn.sum(0, dtype=torch.float64).float()}


_PLAIN = {("conv", "fwd"): _plain_conv, ("conv", "bwd"): _plain_conv_bwd, ("conv", "step"): _plain_conv_step,
          ("scan", "fwd"): _plain_scan, ("scan", "bwd"): _plain_scan_bwd, ("scan", "step"): _plain_scan_step,
          ("norm", "fwd"): _plain_norm, ("norm", "bwd"): _plain_norm_bwd}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        if case["pass"] == "fwd":  # x, n; the residual and h
            return {"bytes": rows * d * es * (2 + 2 * case["residual"]) + 4 * d * (1 + case["bias"]), "flops": 0}
        return {"bytes": rows * d * es * (3 + case["residual"]) + 4 * d * (2 + case["bias"]), "flops": 0}
    D, tokens = case["D"], case["B"] * case["T"]
    n = len(case["lens"].split(",")) if case["lens"] else case["B"]
    row = tokens * D * es
    if case["op"] == "conv":
        K = case["K"]
        state, vecs = n * (K - 1) * D * es, 4 * D * (K + 1)
        if case["pass"] == "bwd":  # x, dout in, dx out; the caches and their gradients
            return {"bytes": 3 * row + 2 * vecs + state * (1 + 2 * case["state"]), "flops": 6 * tokens * D * K}
        return {"bytes": 2 * row + vecs + state * (1 + case["state"]), "flops": 2 * tokens * D * K}
    S, G = case["S"], case["G"]
    state, bc = 4 * n * D * S, 2 * tokens * G * S * es
    vecs = 4 * D * (S + 1 + (case["steps"] == "logits"))
    if case["pass"] == "bwd":  # x, dt, dout in, dx, ddt out; z in, dz out
        return {"bytes": row * (5 + 2 * case["z"]) + 2 * bc + 2 * vecs + state * (1 + 2 * case["state"]),
                "flops": 20 * tokens * D * S}
    return {"bytes": row * (3 + case["z"]) + bc + vecs + state * (1 + case["state"]),
            "flops": 7 * tokens * D * S}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "conv":
        return _exact_conv(s)
    return _exact_scan(s)


def _bounds(s):
    """(first, last) token of every sequence in the tokens laid end to end."""
    if s["cu"] is not None:
        cu = s["cu"].tolist()
        return list(zip(cu[:-1], cu[1:]))
    T = 1 if s["pass"] == "step" else s["T"]
    return [(i * T, (i + 1) * T) for i in range(s["n"])]


def _exact_conv(s):
    """A sequence at a time; gradients by torch's differentiation of the definition."""
    K, D, grads = s["K"], s["D"], s["pass"] == "bwd"
    w, bias = (s[m].double().requires_grad_(grads) for m in ("w", "bias"))
    flat = s["x"].reshape(-1, D).double()
    ys, hts, dxs, dh0s = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for i, (a, b) in enumerate(_bounds(s)):
        x = flat[a:b].clone().requires_grad_(grads)
        h0 = torch.zeros(K - 1, D, dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"][i].double()
        h0 = h0.clone().requires_grad_(grads)
        seen = torch.cat([h0, x])
        y = bias.expand(b - a, D)
        for j in range(K):
            y = y + seen[j:j + b - a] * w[:, j]
        if s["act"] == "silu":
            y = y / (1 + torch.exp(-y))
        ht = seen[b - a:]
        if not grads:
            ys.append(y)
            hts.append(ht)
            continue
        to = (y * s["dout"].reshape(-1, D)[a:b].double()).sum()
        if s["dht"] is not None:
            to = to + (ht * s["dht"][i].double()).sum()
        got = torch.autograd.grad(to, [x, h0, w, bias], allow_unused=True)
        dxs.append(got[0] if got[0] is not None else torch.zeros_like(x))
        dh0s.append(got[1] if got[1] is not None else torch.zeros_like(h0))
        dw = dw + (got[2] if got[2] is not None else 0)
        db = db + (got[3] if got[3] is not None else 0)
    if grads:
        return {"dx": torch.cat(dxs).reshape(s["x"].shape), "dw": dw.detach(), "dbias": db.detach(), "dh0": torch.stack(dh0s)}
    return {"y": torch.cat(ys).reshape(s["x"].shape), ("state" if s["pass"] == "step" else "ht"): torch.stack(hts)}


def _exact_scan(s):
    """Token by token, all sequences side by side (a sequence that has ended has steps of zero)."""
    D, S, G, n, grads = s["D"], s["S"], s["G"], s["n"], s["pass"] == "bwd"
    spans = _bounds(s)
    T = max(b - a for a, b in spans)

    def rows(x, *shape):  # [T, n, *shape]
        x = x.reshape((-1,) + shape)
        out = x.new_zeros((T, n) + shape)
        for i, (a, b) in enumerate(spans):
            out[:b - a, i] = x[a:b]
        return out

    def back(y, like):
        return torch.cat([y[:b - a, i] for i, (a, b) in enumerate(spans)]).reshape(like.shape)

    A, rep = s["A"].double(), D // G
    v = s["dt"].double()
    if s["dt_bias"] is not None:
        v = v + s["dt_bias"].double()
    d64 = torch.logaddexp(v, torch.zeros_like(v)) if s["steps"] == "logits" else v
    d, x, Bm, Cm = rows(d64, D), rows(s["x"].double(), D), rows(s["Bm"], G, S), rows(s["Cm"], G, S)
    h = s["state"] if s["pass"] == "step" else s["h0"]
    h = torch.zeros(n, D, S, dtype=torch.float64, device=DEV) if h is None else h.double()

    def on_channels(m, t):
        return m[t].double()[:, :, None].expand(n, G, rep, S).reshape(n, D, S)

    def step(h, t):
        return torch.exp(d[t][..., None] * A) * h + (d[t] * x[t])[..., None] * on_channels(Bm, t)

    block, kept = 64, []
    y = torch.empty(T, n, D, dtype=torch.float64, device=DEV)
    for t in range(T):
        if grads and t % block == 0:
            kept.append(h)
        h = step(h, t)
        y[t] = (h * on_channels(Cm, t)).sum(-1)
    y = back(y, s["x"]) + s["Dv"].double() * s["x"].double()
    gate = None if s["z"] is None else torch.sigmoid(s["z"].double())
    act = 1.0 if gate is None else s["z"].double() * gate
    if not grads:
        return {"y": y * act, ("state" if s["pass"] == "step" else "ht"): h}
    dout = s["dout"].double()
    dy64 = dout * act
    dy = rows(dy64, D)
    g = torch.zeros_like(h) if s["dht"] is None else s["dht"].double()
    dA = torch.zeros_like(A)
    dx, dd = torch.zeros_like(x), torch.zeros_like(d)
    dB, dC = (torch.zeros(T, n, G, S, dtype=torch.float64, device=DEV) for _ in range(2))
    for b in reversed(range(len(kept))):
        lo, hi = b * block, min(T, (b + 1) * block)
        hs = [kept[b]]
        for t in range(lo, hi):
            hs.append(step(hs[-1], t))
        for t in reversed(range(lo, hi)):
            dC[t] = (dy[t][..., None] * hs[t - lo + 1]).reshape(n, G, rep, S).sum(2)
            g = g + dy[t][..., None] * on_channels(Cm, t)
            dB[t] = (g * (d[t] * x[t])[..., None]).reshape(n, G, rep, S).sum(2)
            gb = (g * on_channels(Bm, t)).sum(-1)
            dx[t] = d[t] * gb
            a = torch.exp(d[t][..., None] * A)
            w = g * a * hs[t - lo]
            dd[t] = x[t] * gb + (w * A).sum(-1)
            dA = dA + (w * d[t][..., None]).sum(0)
            g = g * a
    dd = back(dd, s["dt"])
    if s["steps"] == "logits":
        dd = dd / (1 + torch.exp(-v))
    dims = tuple(range(dout.dim() - 1))
    dz = None
    if gate is not None:
        dz = dout * y * (gate + s["z"].double() * gate * (1 - gate))
    return {"dx": back(dx, s["x"]) + s["Dv"].double() * dy64, "ddt": dd, "dA": dA, "dB": back(dB, s["Bm"]),
            "dC": back(dC, s["Cm"]), "dD": (dy64 * s["x"].double()).sum(dims), "dz": dz,
            "dbias": None if s["dt_bias"] is None else dd.sum(dims), "dh0": g}


def _exact_norm(s):
    """Forward from the definition; gradients by torch's differentiation of it."""
    grads = s["pass"] == "bwd"
    h = s["x"].double()
    if not grads and s["r"] is not None:
        h = h + s["r"].double()
    h, w = h.requires_grad_(grads), s["w"].double().requires_grad_(grads)
    b = None if s["b"] is None else s["b"].double().requires_grad_(grads)
    var = (h * h).mean(-1, keepdim=True) - h.mean(-1, keepdim=True) ** 2
    n = (h - h.mean(-1, keepdim=True)) / torch.sqrt(var + EPS) * w
    n = n if b is None else n + b
    if not grads:
        return {"n": n, "h": None if s["r"] is None else h}
    to = (n * s["dn"].double()).sum()
    if s["dh"] is not None:
        to = to + (h * s["dh"].double()).sum()
    got = torch.autograd.grad(to, [h, w] + ([] if b is None else [b]))
    return {"dx": got[0], "dw": got[1], "db": got[2] if b is not None else None}
