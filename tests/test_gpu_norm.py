"""The norms around a block on the GPU against the float64 formulas of
norm_fp64.py.  Everything is computed in float32 and rounded once, so an output
is off by half a step of its type plus `depth` float32 half steps of its
magnitude: a thread's own elements (32 at most), the trees over threads and
waves (6 + 16), and the elementwise operations and powers of one value (the
bfloat16 form's sigmoid is good to 16 half steps; 64 covers all)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from gated_delta_rule_ckda_amd.inputs import round_bf16
from tests import norm_fp64 as ref
from tests.gpu_util import announce, dev, host

pytestmark = pytest.mark.gpu

DEPTH = 32 + 6 + 16 + 64
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-5

# (post-norm weight, gate, residual, scale, next norm)
PARTS = {"all": "wgxsn", "heads": "wg", "plain": "w", "stream": "xn", "scaled": "wxsn", "gate": "gxs",
         "next": "wgn", "nothing": ""}


def make(seed, rows, d, dtype, parts):
    rng = np.random.default_rng(seed)
    rnd = round_bf16 if dtype == "bf16" else (lambda x: x)
    row = lambda std=1.0: rnd((std * rng.standard_normal((rows, d))).astype(np.float32))
    vec = lambda m: (m + 0.3 * rng.standard_normal(d)).astype(np.float32)
    c = dict(y=row(1.7), dh=row(), dn=row() if "n" in parts else None)
    c["w"] = vec(1) if "w" in parts else None
    c["g"] = row(2.0) if "g" in parts else None
    c["x"] = row() if "x" in parts else None
    c["s"] = vec(0.5) if "s" in parts else None
    c["w2"] = vec(1) if "n" in parts else None
    return c


def on_gpu(c, dtype):
    return {m: None if a is None else dev(a, dtype if a.ndim == 2 else "f32") for m, a in c.items()}


def within(name, x, want, mag, half, depth):
    x = host(x)
    assert np.isfinite(x).all(), name
    off = np.abs(x - want) / (half * np.abs(want) + depth * 2.0 ** -24 * mag + 1e-30)
    assert off.max() <= 1, "%s: %.3g of the bound" % (name, off.max())
    return float(off.max())


def check(c, dtype, act):
    g = on_gpu(c, dtype)
    kw = dict(gate=g["g"], act=act, residual=g["x"], scale=g["s"], next_weight=g["w2"], eps=EPS)
    h, n = ck.block_norm(g["y"], g["w"], **kw)
    grads = ck.block_norm_bwd(g["y"], g["w"], g["dh"], dnext=g["dn"], **kw)
    torch.cuda.synchronize()
    (rh, rn), (hm, nm) = ref.fwd(c["y"], c["w"], c["g"], act, c["x"], c["s"], c["w2"], EPS)
    at = [within("h", h, rh, hm, HALF[dtype], DEPTH)]
    if n is not None:
        at.append(within("n", n, rn, nm, HALF[dtype], DEPTH))
    want, mag = ref.bwd(c["y"], c["w"], c["dh"], c["dn"], c["g"], act, c["x"], c["s"], c["w2"], EPS)
    rows = c["y"].shape[0]
    for name, got, given in zip(("dy", "dw", "dg", "dx", "ds", "dw2"), grads,
                                (1, c["w"], c["g"], c["x"], c["s"], c["w2"])):
        assert (got is None) == (given is None), name
        if got is not None:
            vec = name in ("dw", "ds", "dw2")
            at.append(within(name, got, want[name], mag[name], HALF["f32" if vec else dtype],
                             2 * DEPTH + (rows if vec else 0)))
    announce("at %s of the bounds" % " ".join("%.2g" % a for a in at))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 24, 33, 64, 100, 128, 256, 1000, 1001, 1002, 1024, 2048, 2050,
                               4096, 5000, 8192, 8200, 16383, 16384])
def test_widths(dtype, d):
    check(make(d, 5, d, dtype, "wgxsn"), dtype, "silu")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", sorted(PARTS))
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_parts(dtype, parts, act):
    check(make(3, 37, 64, dtype, PARTS[parts]), dtype, act)
    check(make(4, 3, 1536, dtype, PARTS[parts]), dtype, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 128), (63, 128), (65, 16), (2049, 24), (4097, 128), (3000, 512)])
def test_rows(dtype, rows, d):
    check(make(rows, rows, d, dtype, "wgxsn"), dtype, "sigmoid")


def test_residual_in_place_and_gate_of_minus_infinity():
    c = make(9, 12, 96, "bf16", "wgxsn")
    c["g"][3, 5] = -np.inf
    g = on_gpu(c, "bf16")
    for act in ("sigmoid", "silu"):
        kw = dict(gate=g["g"], act=act, scale=g["s"], next_weight=g["w2"], eps=EPS)
        h, n = ck.block_norm(g["y"], g["w"], residual=g["x"], **kw)
        x = g["x"].clone()
        h2, n2 = ck.block_norm(g["y"], g["w"], residual=x, out=x, **kw)
        torch.cuda.synchronize()
        assert h2 is x and torch.equal(h, h2) and torch.equal(n, n2)
        assert h[3, 5] == g["x"][3, 5]
        r = ck.block_norm_bwd(g["y"], g["w"], g["dh"], dnext=g["dn"], residual=g["x"], **kw)
        assert all(torch.isfinite(t).all() for t in r)


def test_rows_of_zeros_and_no_rows():
    y = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, n = ck.block_norm(y, w, next_weight=w)
    assert (h == 0).all() and (n == 0).all()
    r = ck.block_norm_bwd(y, w, y + 1, dnext=y + 1, next_weight=w)
    assert all(torch.isfinite(t).all() for t in r if t is not None)
    e = y[:0]
    assert ck.block_norm(e, w, next_weight=w)[1].shape == (0, 64)
    r = ck.block_norm_bwd(e, w, e, dnext=e, next_weight=w)
    assert r[0].shape == (0, 64) and (r[1] == 0).all() and (r[5] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(5, 64), (37, 128), (3, 24), (70, 1001)])
@pytest.mark.parametrize("parts", ["wgxsn", "w", "xn", "wn"])
def test_no_eps_and_rows_that_leave_threads_idle(dtype, rows, d, parts):
    """eps = 0 with rows that do not fill a workgroup: the sums over rows hold
    the rows there are, and nothing of the idle threads."""
    c = make(rows, rows, d, dtype, parts)
    g = on_gpu(c, dtype)
    kw = dict(gate=g["g"], act="silu", residual=g["x"], scale=g["s"], next_weight=g["w2"], eps=0.0)
    h, n = ck.block_norm(g["y"], g["w"], **kw)
    grads = ck.block_norm_bwd(g["y"], g["w"], g["dh"], dnext=g["dn"], **kw)
    torch.cuda.synchronize()
    (rh, rn), (hm, nm) = ref.fwd(c["y"], c["w"], c["g"], "silu", c["x"], c["s"], c["w2"], 0.0)
    within("h", h, rh, hm, HALF[dtype], DEPTH)
    if n is not None:
        within("n", n, rn, nm, HALF[dtype], DEPTH)
    want, mag = ref.bwd(c["y"], c["w"], c["dh"], c["dn"], c["g"], "silu", c["x"], c["s"], c["w2"], 0.0)
    for name, got in zip(("dy", "dw", "dg", "dx", "ds", "dw2"), grads):
        if got is not None:
            vec = name in ("dw", "ds", "dw2")
            within(name, got, want[name], mag[name], HALF["f32" if vec else dtype], 2 * DEPTH + (rows if vec else 0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gradients_of_saturated_gates(dtype, act):
    """Gates far from zero keep the digits of their gradients: dg = dh u act'(g)
    is a product, so it is off by half a step of its type and DEPTH float32 half
    steps of the value: u's (as in `h`), a power e = exp(-|g|) (|g| half steps of
    it, 20 here, where it runs on powers of two), and a few operations on
    e / (1 + e)^2, which subtracts nothing.  silu' = p + g e / (1 + e)^2 is off by
    that of the sum of its terms' magnitudes."""
    c = make(17, 40, 128, dtype, "wg")
    rng = np.random.default_rng(18)
    far = rng.uniform(8, 20, c["g"].shape) * rng.choice([-1, 1], c["g"].shape)
    c["g"] = round_bf16(far.astype(np.float32)) if dtype == "bf16" else far.astype(np.float32)
    g = on_gpu(c, dtype)
    got = ck.block_norm_bwd(g["y"], g["w"], g["dh"], gate=g["g"], act=act, eps=EPS)[2]
    torch.cuda.synchronize()
    u = ref.parts(c["y"], c["w"], c["g"], act, None, None, EPS)[2]
    e = np.exp(-np.abs(ref.f64(c["g"])))
    p, q = np.where(c["g"] >= 0, 1, e) / (1 + e), e / (1 + e) ** 2
    to = ref.f64(c["dh"]) * u
    want = to * (q if act == "sigmoid" else p + ref.f64(c["g"]) * q)
    mag = np.abs(to) * (q if act == "sigmoid" else p + np.abs(ref.f64(c["g"])) * q)
    announce("dg at %.2g of its bound" % within("dg", got, want, mag, HALF[dtype], 2 * DEPTH))
