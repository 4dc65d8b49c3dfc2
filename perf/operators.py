"""Cases, inputs and plain forms of the decay linear attention and of the block norms.

Five operators:

  decay_fwd    S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t  over whole prompts (one decay a
               a head and token, or one a head), dense or packed, with initial and final states
  decay_bwd    its gradients
  decay_step   one token a sequence, the state updated in place
  norm_fwd     h = x + s * act(g) * rmsnorm(y; w),  n = rmsnorm(h; w')  a row
  norm_bwd     its gradients

Where `own` is false `run` computes them from elementary torch operations in 32 bits (sums of
logarithms of gates in 64); where it is true it calls the package's entry points.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _attn(name, op, B, T, H, Hk, dk, dv, dtype, gates, gate, h0, lens=""):
    c = {"op": op, "B": B, "T": T, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype,
         "gates": gates, "gate": gate, "h0": h0, "lens": lens}
    return dict(c, name=name) if name else c


def _step(name, N, H, Hk, dk, dv, dtype, gates, gate):
    c = {"op": "decay_step", "N": N, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype,
         "gates": gates, "gate": gate}
    return dict(c, name=name) if name else c


def _norm(name, op, rows, d, dtype, act, residual, nxt):
    c = {"op": op, "rows": rows, "d": d, "dtype": dtype, "act": act, "residual": residual,
         "next": nxt}
    return dict(c, name=name) if name else c


def listed():
    packed = ("8191,1024,5021,1,3500,64,0,2777,4096,63,1333,7000,129,2048,65,4688")
    return [
        # a training or prefill batch of a layer: the repository's language-model layer
        _attn("fwd layer", "decay_fwd", 8, 4096, 16, 16, 128, 128, "bf16", "logits", "ckda", False),
        # one long document with few heads in flight: the token axis has to be split
        _attn("fwd long", "decay_fwd", 1, 65536, 16, 16, 128, 128, "bf16", "values", "kda", False),
        # a serving batch of prompts of all lengths (one empty), continued from states, grouped heads
        _attn("fwd packed", "decay_fwd", 1, 40000, 16, 4, 128, 128, "bf16", "logits", "kda", True, packed),
        # a short prompt in float32 with one fixed decay a head: latency
        _attn("fwd short", "decay_fwd", 2, 100, 4, 4, 64, 64, "f32", "head", "kda", False),
        # the training step's backward of the language-model layer
        _attn("bwd layer", "decay_bwd", 8, 4096, 16, 16, 128, 128, "bf16", "logits", "kda", False),
        # a small float32 layer of odd sizes with signed gates and states: gradient checks
        _attn("bwd odd", "decay_bwd", 2, 333, 4, 2, 48, 64, "f32", "values", "ckda", True),
        # a full decode batch: the repository's decode step
        _step("step batch", 256, 32, 32, 128, 128, "bf16", "logits", "kda"),
        # a few sequences being decoded: latency
        _step("step few", 4, 8, 2, 64, 64, "bf16", "values", "ckda"),
        # the gated output norm of a layer's heads (every token and head a row)
        _norm("norm heads", "norm_fwd", 524288, 128, "bf16", "sigmoid", False, False),
        # the norms between two blocks while decoding: latency
        _norm("norm decode", "norm_fwd", 64, 2048, "bf16", "silu", True, True),
        # the norms between two blocks in a training step's backward
        _norm("norm bwd layer", "norm_bwd", 32768, 2048, "bf16", "sigmoid", True, True),
        # a small float32 model of an odd width
        _norm("norm bwd odd", "norm_bwd", 77, 1001, "f32", "silu", True, True),
    ]


def _log(rng, lo, hi):
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_bwd", "decay_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            d = -(-d // 16) * 16
        rows = _log(rng, 1, max(1, min(32768, (1 << 25) // d)))
        full = rng.random() < 0.6
        return _norm("", op, rows, d, dtype, rng.choice(["none", "sigmoid", "silu"]), full,
                     full and rng.random() < 0.7)
    Hk = rng.choice([1, 2, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 4])
    dk, dv = (8 * rng.randint(2, 16) for _ in range(2))
    if rng.random() < 0.5:
        dk = dv = rng.choice([32, 64, 128])
    gates = rng.choice(["values", "logits", "head"])
    gate = rng.choice(["kda", "ckda"])
    if op == "decay_step":
        return _step("", _log(rng, 1, 256), H, Hk, dk, dv, dtype, gates, gate)
    most = (1 << 25) // (H * max(dk, dv))
    tokens = _log(rng, 1, min(most, 65536) if op == "decay_fwd" else min(most // 4, 16384))
    if rng.random() < 0.4:
        n = rng.randint(1, 12)
        cut = sorted(rng.randint(0, tokens) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cut, cut + [tokens])]
        return _attn("", op, 1, tokens, H, Hk, dk, dv, dtype, gates, gate, rng.random() < 0.5,
                     ",".join(map(str, lens)))
    B = rng.choice([1, 2, 3, 8])
    return _attn("", op, B, max(1, tokens // B), H, Hk, dk, dv, dtype, gates, gate,
                 rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["dtype"]]

    def randn(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return torch.randn(shape, device=DEV, generator=g).mul_(std).add_(mean).to(dtype)

    s = dict(case)
    if case["op"].startswith("norm"):
        rows, d = case["rows"], case["d"]
        s["y"] = randn(rows, d, std=1.5, dtype=t)
        s["w"] = randn(d, mean=1.0, std=0.2)
        s["g"] = randn(rows, d, dtype=t) if case["act"] != "none" else None
        s["x"] = randn(rows, d, dtype=t) if case["residual"] else None
        s["s"] = randn(d, mean=0.5, std=0.1) if case["residual"] else None
        s["w2"] = randn(d, mean=1.0, std=0.2) if case["next"] else None
        if case["op"] == "norm_bwd":
            s["dh"] = randn(rows, d, dtype=t)
            s["dn"] = randn(rows, d, dtype=t) if case["next"] else None
        return s
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    if case["op"] == "decay_step":
        lead, n = (case["N"],), case["N"]
    else:
        lead, n = (case["B"], case["T"]), case["B"]
        s["cu"], s["longest"] = None, case["T"]
        if case["lens"]:
            lens = [int(x) for x in case["lens"].split(",")]
            n, s["longest"] = len(lens), max(lens)
            s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    s["scale"] = float(dk) ** -0.5
    s["q"], s["k"] = (randn(*lead, Hk, dk, dtype=t) for _ in range(2))
    s["v"] = randn(*lead, H, dv, dtype=t)
    # memories of some tens to some thousands of tokens; signed gates flip now and then
    if case["gates"] == "head":
        s["alpha"] = 1.0 - torch.exp2(-torch.linspace(4.0, 9.0, H, device=DEV) - torch.rand(H, device=DEV, generator=g))
    else:
        a = randn(*lead, H, mean=4.0, std=1.5)
        if case["gates"] == "logits":
            s["alpha"] = a.to(t)
        else:
            s["alpha"] = torch.sigmoid(a) if case["gate"] == "kda" else torch.tanh(0.5 * a)
    if case["op"] == "decay_step":
        s["state"] = randn(n, H, dk, dv, std=0.5)
        return s
    s["h0"] = randn(n, H, dk, dv, std=0.5) if case["h0"] else None
    if case["op"] == "decay_bwd":
        s["dout"] = randn(*lead, H, dv, dtype=t)
        s["dht"] = randn(n, H, dk, dv, std=0.5) if case["h0"] else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _kernels(state)
    return _PLAIN[state["op"]](state)


def _kernels(s):
    import gated_delta_rule_ckda_amd as ck
    if s["op"] == "norm_fwd":
        h, n = ck.block_norm(s["y"], s["w"], gate=s["g"], act=s["act"], residual=s["x"],
                             scale=s["s"], next_weight=s["w2"], eps=EPS)
        return {"h": h, "n": n}
    if s["op"] == "norm_bwd":
        return dict(zip(("dy", "dw", "dg", "dx", "ds", "dw2"), ck.block_norm_bwd(
            s["y"], s["w"], s["dh"], dnext=s["dn"], gate=s["g"], act=s["act"], residual=s["x"],
            scale=s["s"], next_weight=s["w2"], eps=EPS)))
    gates = "logits" if s["gates"] == "logits" else "values"
    if s["op"] == "decay_step":
        o = ck.decay_step(s["q"], s["k"], s["v"], s["alpha"], s["state"], gate=s["gate"],
                          gates=gates, scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if s["op"] == "decay_fwd":
        o, ht = ck.decay_fwd(s["q"], s["k"], s["v"], s["alpha"], h0=s["h0"], cu_seqlens=s["cu"],
                             gate=s["gate"], gates=gates, scale=s["scale"])
        return {"o": o, "ht": ht}
    return dict(zip(("dq", "dk", "dv", "dalpha", "dh0"), ck.decay_bwd(
        s["q"], s["k"], s["v"], s["alpha"], s["dout"], h0=s["h0"], dht=s["dht"],
        cu_seqlens=s["cu"], gate=s["gate"], gates=gates, scale=s["scale"])))


# ---------------------------------------------------------------- plain forms
CHUNK = 64


def _gate64(s):
    """The gates in 64 bits, and their derivative by what `alpha` holds."""
    a = s["alpha"].double()
    if s["gates"] != "logits":
        return a, torch.ones_like(a)
    p = torch.sigmoid(a)
    if s["gate"] == "kda":
        return p, p * (1 - p)
    return 2 * p - 1, 2 * p * (1 - p)


def _spread(x, n, T, cu, longest, fill=0.0):
    """[B,T,...] or packed [1,T,...] -> [n, longest,...]: sequences side by side."""
    if cu is None:
        return x
    at = cu[:-1, None].long() + torch.arange(longest, device=x.device)
    inside = at < cu[1:, None]
    y = x[0][at.clamp(max=max(T - 1, 0))]
    return torch.where(inside.reshape(inside.shape + (1,) * (y.dim() - 2)), y, torch.full((), fill, device=x.device, dtype=x.dtype))


def _gather(y, T, cu):
    """The inverse of _spread, for tokens of [n, longest,...]."""
    if cu is None:
        return y
    t = torch.arange(T, device=y.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return y[seq, t - cu[seq].long()][None]


def _chunks(x):
    """[n,T,H,...] -> [n,H,chunks,CHUNK,...] (T a multiple of CHUNK)."""
    n, T, H = x.shape[:3]
    x = x.reshape((n, T // CHUNK, CHUNK, H) + x.shape[3:])
    return x.permute((0, 3, 1, 2) + tuple(range(4, x.dim()))).contiguous()


def _tokens(x, T):
    """The inverse of _chunks."""
    x = x.permute((0, 2, 3, 1) + tuple(range(4, x.dim())))
    return x.reshape((x.shape[0], -1, x.shape[3]) + x.shape[4:])[:, :T]


def _pad(x, fill=0.0):
    more = -x.shape[1] % CHUNK
    return torch.cat([x, x.new_full((x.shape[0], more) + x.shape[2:], fill)], 1) if more else x


def _between(L, S, Z, L2, S2, Z2):
    """The products of the gates after place 2 up to place 1, from sums of logarithms, counts of
    signs and counts of zeros."""
    return torch.where(Z == Z2, torch.exp(L - L2) * (1 - 2 * ((S - S2) % 2)), torch.zeros((), dtype=L.dtype, device=L.device)).float()


def _laid(s):
    """What both directions need: the tokens in chunks, the products of gates inside a chunk (D),
    from its start (E) and to its end (F), and over chunks (W)."""
    n = s["B"] if s["cu"] is None else s["cu"].numel() - 1
    H, rep = s["H"], s["H"] // s["Hk"]

    def lay(x, fill=0.0):
        x = _spread(x, n, s["T"], s["cu"], s["longest"], fill)
        return _chunks(_pad(x, fill))

    r = {"n": n, "lay": lay}
    r["q"], r["k"] = (lay(s[x].float()).repeat_interleave(rep, 1) for x in ("q", "k"))
    r["v"] = lay(s["v"].float())
    a, _ = _gate64(s)
    if s["gates"] == "head":
        a = a.expand(s["B"], s["T"], H)
    a = lay(a, 1.0)
    zero, L = a == 0, torch.log(torch.where(a == 0, torch.ones_like(a), a.abs()))
    L, S, Z = L.cumsum(-1), (a < 0).long().cumsum(-1), zero.long().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=a.device).tril()
    r["D"] = low * torch.nan_to_num(_between(L[..., None], S[..., None], Z[..., None], L[..., None, :], S[..., None, :], Z[..., None, :]) * low, nan=0.0, posinf=0.0)
    o = torch.zeros((), device=a.device, dtype=L.dtype)
    r["E"] = _between(L, S, Z, o, o.long(), o.long())
    r["F"] = r["D"][..., -1, :]

    def over(x):
        y = x[..., -1].cumsum(-1)
        return torch.cat([torch.zeros_like(y[..., :1]), y], -1)

    L, S, Z = over(L), over(S), over(Z)
    m = L.shape[-1]
    low = torch.ones(m, m, device=a.device).tril()
    r["W"] = low * torch.nan_to_num(_between(L[..., None], S[..., None], Z[..., None], L[..., None, :], S[..., None, :], Z[..., None, :]) * low, nan=0.0, posinf=0.0)
    return r


def _states(r, s, first, w, a, b):
    """The states before every chunk and after the last, of additions sum w a b^T a chunk."""
    u = (a * w[..., None]).transpose(-1, -2).contiguous() @ b
    u = torch.cat([u.new_zeros(u[:, :, :1].shape) if first is None else first[:, :, None], u], 2)
    return (r["W"] @ u.flatten(-2)).reshape(u.shape)


def _plain_fwd(s):
    r = _laid(s)
    st = _states(r, s, s["h0"], r["F"], r["k"], r["v"])
    p = (r["q"] @ r["k"].transpose(-1, -2).contiguous()) * r["D"]
    o = p @ r["v"] + r["E"][..., None] * (r["q"] @ st[:, :, :-1])
    o = _gather(_tokens(o, s["longest"]), s["T"], s["cu"]) * s["scale"]
    return {"o": o.to(s["v"].dtype), "ht": st[:, :, -1].contiguous()}


def _plain_bwd(s):
    r = _laid(s)
    q, k, v, D, E, F = (r[x] for x in ("q", "k", "v", "D", "E", "F"))
    do = r["lay"](s["dout"].float()) * s["scale"]
    st = _states(r, s, s["h0"], F, k, v)[:, :, :-1]
    u = (q * E[..., None]).transpose(-1, -2).contiguous() @ do
    u = torch.cat([u, u.new_zeros(u[:, :, :1].shape) if s["dht"] is None else s["dht"][:, :, None]], 2)
    ad = (r["W"].transpose(-1, -2).contiguous() @ u.flatten(-2)).reshape(u.shape)
    dh0, ad = ad[:, :, 0].contiguous(), ad[:, :, 1:]
    p, n = q @ k.transpose(-1, -2).contiguous(), do @ v.transpose(-1, -2).contiguous()
    zq = do @ st.transpose(-1, -2).contiguous()            # S do
    yk = v @ ad.transpose(-1, -2).contiguous()             # dS v
    dq = E[..., None] * zq + (n * D) @ k
    dk = F[..., None] * yk + (n * D).transpose(-1, -2).contiguous() @ q
    dv = F[..., None] * (k @ ad) + (p * D).transpose(-1, -2).contiguous() @ do
    # da_t: every pair of a write before t and a read from t on, without the gate a_t itself
    before = torch.cat([torch.zeros_like(D[..., :1, :]), D[..., :-1, :]], -2)
    e = torch.cat([torch.ones_like(E[..., :1]), E[..., :-1]], -1)
    z, y, x = (q * zq).sum(-1), (k * yk).sum(-1), (st * ad).sum((-1, -2))
    rect = (p * n) @ before.transpose(-1, -2).contiguous() + z[..., None] * e[..., None, :]
    da = (D * rect).sum(-2) + F * ((before @ y[..., None])[..., 0] + e * x[..., None])

    def back(t, rep=1):
        t = _gather(_tokens(t, s["longest"]), s["T"], s["cu"])
        return t if rep == 1 else t.reshape(t.shape[:2] + (-1, rep) + t.shape[3:]).sum(3)

    rep, io = s["H"] // s["Hk"], s["v"].dtype
    da = back(da) * _gate64(s)[1].float()
    if s["gates"] == "head":
        da = da.sum((0, 1))
    return {"dq": back(dq, rep).to(io), "dk": back(dk, rep).to(io), "dv": back(dv).to(io),
            "dalpha": da.to(io), "dh0": dh0}


def _plain_step(s):
    rep, st = s["H"] // s["Hk"], s["state"]
    q, k = (s[x].float().repeat_interleave(rep, 1) for x in ("q", "k"))
    a = _gate64(s)[0].float().expand(s["N"], s["H"])
    st.mul_(a[..., None, None]).add_(k[..., None] * s["v"].float()[..., None, :])
    o = (st * q[..., None]).sum(-2) * s["scale"]
    return {"o": o.to(s["v"].dtype), "state": st}


def _act(s):
    """act(g) and its derivative."""
    if s["g"] is None:
        return 1.0, None
    g = s["g"].float()
    p = torch.sigmoid(g)
    return (p, p * (1 - p)) if s["act"] == "sigmoid" else (g * p, p * (1 + g * (1 - p)))


def _plain_norm(s):
    y, io = s["y"].float(), s["y"].dtype
    u = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w"] * _act(s)[0]
    h = u if s["x"] is None else s["x"].float() + s["s"] * u
    if s["w2"] is None:
        return {"h": h.to(io), "n": None}
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w2"]
    return {"h": h.to(io), "n": n.to(io)}


def _plain_norm_bwd(s):
    y, io, dh = s["y"].float(), s["y"].dtype, s["dh"].float()
    act, dact = _act(s)
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    yh = y * r
    u = yh * s["w"]
    ua = u * act
    out = {"dg": None, "dx": None, "ds": None, "dw2": None}
    if s["w2"] is not None:
        h = ua if s["x"] is None else s["x"].float() + s["s"] * ua
        r2 = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        hh, dn = h * r2, s["dn"].float()
        out["dw2"] = (dn * hh).sum(0)
        dn = dn * s["w2"]
        dh = dh + r2 * (dn - hh * (dn * hh).mean(-1, keepdim=True))
    if s["x"] is not None:
        out["dx"] = dh.to(io)
        out["ds"] = (dh * ua).sum(0)
        dh = dh * s["s"]
    if s["g"] is not None:
        out["dg"] = (dh * u * dact).to(io)
    du = dh * act
    out["dw"] = (du * yh).sum(0)
    du = du * s["w"]
    out["dy"] = (r * (du - yh * (du * yh).mean(-1, keepdim=True))).to(io)
    return out


_PLAIN = {"decay_fwd": _plain_fwd, "decay_bwd": _plain_bwd, "decay_step": _plain_step,
          "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        rows, d = case["rows"], case["d"]
        acts = 2 + (case["act"] != "none") + case["residual"] + case["next"]  # y, h, g, x, n
        vecs = 1 + case["residual"] + case["next"]
        if case["op"] == "norm_bwd":  # y, g, x, dh, dn in; dy, dg, dx out
            acts = 3 + 2 * (case["act"] != "none") + (2 if case["residual"] else 0) + case["next"]
            acts -= 1 if case["residual"] and not case["next"] else 0  # x is not needed then
            vecs *= 2
        return {"bytes": rows * d * es * acts + 4 * d * vecs, "flops": 0}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    if case["op"] == "decay_step":
        n = tokens = case["N"]
        states = 2
    else:
        n = len(case["lens"].split(",")) if case["lens"] else case["B"]
        tokens = case["B"] * case["T"]
        states = 1 + case["h0"]
    gate = H * tokens * (es if case["gates"] == "logits" else 4) if case["gates"] != "head" else 4 * H
    state = 4 * n * H * dk * dv
    qk, vo = tokens * Hk * dk * es, tokens * H * dv * es
    if case["op"] == "decay_bwd":  # q, k, v, dout, h0, dht in; dq, dk, dv, dalpha, dh0 out
        return {"bytes": 4 * qk + 3 * vo + 2 * gate + state * (1 + 2 * case["h0"]),
                "flops": 12 * tokens * H * dk * dv}
    return {"bytes": 2 * qk + 2 * vo + gate + states * state, "flops": 4 * tokens * H * dk * dv}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case["op"] == "norm_bwd")
    if case["op"] == "decay_step":
        rep = s["H"] // s["Hk"]
        a = _exact_gate(s, s["alpha"].double()).expand(s["N"], s["H"])
        q, k = (s[x].double().repeat_interleave(rep, 1) for x in ("q", "k"))
        st = a[:, :, None, None] * s["state"].double() + torch.einsum("nhk,nhv->nhkv", k, s["v"].double())
        return {"o": torch.einsum("nhkv,nhk->nhv", st, q) * s["scale"], "state": st}
    return _exact_recurrence(s, case["op"] == "decay_bwd")


def _exact_gate(s, a):
    if s["gates"] != "logits":
        return a
    return 1 / (1 + torch.exp(-a)) if s["gate"] == "kda" else torch.tanh(a / 2)


def _exact_recurrence(s, grads):
    """Token by token, all sequences side by side (a sequence that has ended keeps its state)."""
    H, dk, dv, rep, T = s["H"], s["dk"], s["dv"], s["H"] // s["Hk"], s["longest"]
    cu = None if s["cu"] is None else s["cu"].tolist()
    n = s["B"] if cu is None else len(cu) - 1

    def rows(x, fill=0.0):  # [T, n, ...]
        if cu is None:
            return x.transpose(0, 1).contiguous()
        y = x.new_full((T, n) + x.shape[2:], fill)
        for i in range(n):
            y[: cu[i + 1] - cu[i], i] = x[0, cu[i]: cu[i + 1]]
        return y

    def packed(y):
        if cu is None:
            return y.transpose(0, 1).contiguous()
        return torch.cat([y[: cu[i + 1] - cu[i], i] for i in range(n)])[None]

    q, k = (rows(s[x]) for x in ("q", "k"))
    v = rows(s["v"])
    raw = s["alpha"] if s["gates"] != "head" else s["alpha"].expand(s["B"], s["T"], H)
    a64 = _exact_gate(s, raw.double())
    alpha = rows(a64, 1.0)

    def at(x, t):  # one token's q or k, on the value heads
        return x[t].double().repeat_interleave(rep, 1)

    st = torch.zeros(n, H, dk, dv, dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
    block, kept = 64, []
    if not grads:
        o = torch.empty(T, n, H, dv, dtype=torch.float64, device=DEV)
        for t in range(T):
            st = torch.baddbmm((st * alpha[t][:, :, None, None]).view(n * H, dk, dv), at(k, t).reshape(n * H, dk, 1), v[t].double().reshape(n * H, 1, dv)).view(n, H, dk, dv)
            o[t] = (at(q, t)[:, :, None, :] @ st)[:, :, 0]
        return {"o": packed(o) * s["scale"], "ht": st}

    def step(st, t):
        return st * alpha[t][:, :, None, None] + at(k, t)[..., None] * v[t].double()[:, :, None, :]

    for t in range(T):
        if t % block == 0:
            kept.append(st)
        st = step(st, t)
    do = rows(s["dout"])
    ad = torch.zeros_like(st) if s["dht"] is None else s["dht"].double()
    dq, dk_ = (torch.zeros(T, n, s["Hk"], dk, dtype=torch.float64, device=DEV) for _ in range(2))
    dv_ = torch.empty(T, n, H, dv, dtype=torch.float64, device=DEV)
    da = torch.empty(T, n, H, dtype=torch.float64, device=DEV)
    for b in reversed(range(len(kept))):
        lo, hi = b * block, min(T, (b + 1) * block)
        before = [kept[b]]
        for t in range(lo, hi):
            before.append(step(before[-1], t))
        for t in reversed(range(lo, hi)):
            d = do[t].double() * s["scale"]
            kt, vt = at(k, t), v[t].double()
            dq[t] = (before[t - lo + 1] @ d[..., None])[..., 0].view(n, s["Hk"], rep, dk).sum(2)
            ad = ad + at(q, t)[..., None] * d[:, :, None, :]
            dk_[t] = (ad @ vt[..., None])[..., 0].view(n, s["Hk"], rep, dk).sum(2)
            dv_[t] = (kt[:, :, None, :] @ ad)[:, :, 0]
            da[t] = (ad * before[t - lo]).sum((-1, -2))
            ad = ad * alpha[t][:, :, None, None]
    da = packed(da)
    if s["gates"] == "logits":
        da = da * (a64 * (1 - a64) if s["gate"] == "kda" else (1 - a64 * a64) / 2)
    if s["gates"] == "head":
        da = da.sum((0, 1))
    return {"dq": packed(dq), "dk": packed(dk_), "dv": packed(dv_), "dalpha": da, "dh0": ad}


def _exact_norm(s, grads):
    """Forward from the definition; gradients by torch's differentiation of it."""
    names = ("y", "w", "g", "x", "s", "w2")
    t = {m: None if s[m] is None else s[m].double().requires_grad_(grads) for m in names}

    def rms(z, w):
        return z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS) * w

    def value(y, g, x):
        u = rms(y, t["w"])
        if g is not None:
            u = u * (torch.sigmoid(g) if s["act"] == "sigmoid" else torch.nn.functional.silu(g))
        h = u if x is None else x + t["s"] * u
        return h, None if t["w2"] is None else rms(h, t["w2"])

    if not grads:
        return dict(zip(("h", "n"), value(t["y"], t["g"], t["x"])))
    h, n = value(t["y"], t["g"], t["x"])
    have = [m for m in names if t[m] is not None]
    to = (h * s["dh"].double()).sum() + (0 if n is None else (n * s["dn"].double()).sum())
    got = dict(zip(have, torch.autograd.grad(to, [t[m] for m in have])))
    return {"d" + m: got.get(m) for m in names}
