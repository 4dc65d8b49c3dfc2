"""Inputs, calls and checks shared by the tests of the selective scan, the short
convolution and layer norm."""
import numpy as np
import torch

from gated_delta_rule_ckda_amd.inputs import round_bf16
from tests import scan_fp64 as ref
from tests.gpu_util import dev, host

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rounded(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return round_bf16(x) if dtype == "bf16" else x


def within(name, got, value, bound, half):
    got = host(got)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert np.isfinite(got).all(), name
    if not got.size:
        return 0.0
    off = np.abs(got - value) / (half * (np.abs(value) + bound) + bound + 1e-30)
    assert off.max() <= 1, "%s: %.3g of its bound" % (name, off.max())
    return float(off.max())


def view(x, dtype, pad=3):
    """x [..., w] on the device as a part of wider rows."""
    wide = np.zeros(x.shape[:-1] + (x.shape[-1] + 2 * pad,), np.float32)
    wide[..., :pad] = wide[..., -pad:] = np.nan  # never to be read
    wide[..., pad:-pad] = x
    return dev(wide, dtype)[..., pad:-pad]


def spans_of(lens, B, T):
    if lens is None:
        return [(i, 0, T) for i in range(B)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def make_scan(seed, B, T, D, S, G, dtype, lens=None, steps="logits", z=True, states=True, skip=True, tail=0):
    """float32 arrays (bf16-representable where the io type is bf16); with lens a packed batch."""
    rng = np.random.default_rng(seed)
    if lens is not None:
        B, T = 1, int(sum(lens)) + tail
    n = B if lens is None else len(lens)
    r = lambda *s: rounded(rng.standard_normal(s), dtype)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    c = dict(x=r(B, T, D), B=r(B, T, G, S), C=r(B, T, G, S), dy=r(B, T, D), z=r(B, T, D) if z else None)
    c["A"] = (-np.arange(1, S + 1) * np.exp(0.1 * f(D, S))).astype(np.float32)
    c["D"] = (1 + 0.2 * f(D)) if skip else None
    if steps == "logits":
        c["dt"], c["bias"] = r(B, T, D), (-3.5 + f(D)) if skip else None
        if not skip:
            c["dt"] = rounded(c["dt"] - 3, dtype)
    else:
        c["dt"], c["bias"] = rounded(np.exp(rng.uniform(-7, -1.5, (B, T, D))), dtype), None
    c["h0"], c["dht"] = (f(n, D, S), f(n, D, S)) if states else (None, None)
    return dict(c, dtype=dtype, steps=steps, lens=lens, n=n, spans=spans_of(lens, B, T), T=T, tail=tail)


def scan_tensors(c, strided=False):
    put = (lambda a: view(a, c["dtype"])) if strided else (lambda a: dev(a, c["dtype"]))
    g = {m: None if c[m] is None else put(c[m]) for m in ("x", "dt", "z")}
    for m in ("B", "C"):
        flat = c[m].reshape(c[m].shape[:2] + (-1,))
        g[m] = put(flat).unflatten(-1, c[m].shape[2:])
    for m in ("A", "D", "bias", "h0", "dht"):
        g[m] = None if c[m] is None else dev(c[m])
    g["dy"] = dev(c["dy"], c["dtype"])
    g["cu"] = None
    if c["lens"] is not None:
        g["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(c["lens"])]), dtype=torch.int32, device="cuda")
    return g


def scan_kw(c, g):
    return dict(D=g["D"], z=g["z"], dt_bias=g["bias"], steps=c["steps"], h0=g["h0"], cu_seqlens=g["cu"])


def scan_reference(c, grads=True, cut=0):
    """{name: (value, bound)} over the batch; rows past the last sequence are NaN."""
    out = {}
    for m in ("y", "dx", "ddt", "dz"):
        out[m] = (np.full(c["x"].shape, np.nan), np.zeros(c["x"].shape))
    for m in ("dB", "dC"):
        out[m] = (np.full(c["B"].shape, np.nan), np.zeros(c["B"].shape))
    sums, states = {}, {"ht": [], "dh0": []}
    for i, (b, lo, hi) in enumerate(c["spans"]):
        at = lambda t: None if t is None else t[b, lo:hi]
        one = lambda t: None if t is None else t[i]
        r = ref.scan(at(c["x"]), at(c["dt"]), c["A"], at(c["B"]), at(c["C"]), c["D"], at(c["z"]), c["bias"],
                     c["steps"] == "logits", one(c["h0"]), at(c["dy"]) if grads else None, one(c["dht"]), cut)
        for m, (v, e) in r.items():
            if m in out:
                out[m][0][b, lo:hi], out[m][1][b, lo:hi] = v, e
            elif m in states:
                states[m].append((v, e))
            else:
                have = sums.get(m, (0.0, 0.0, 0.0))
                sums[m] = (have[0] + v, have[1] + e + 40 * ref.EPS * np.abs(v), 0.0)
    for m, v in states.items():
        if v:
            out[m] = (np.stack([t[0] for t in v]), np.stack([t[1] for t in v]))
    for m, v in sums.items():
        out[m] = v[:2]
    return out
