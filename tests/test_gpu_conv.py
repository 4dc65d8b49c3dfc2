"""The short convolution on the GPU against the formulas in float64 with their
bounds (scan_fp64.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests import scan_fp64 as ref
from tests.gpu_util import announce, dev
from tests.ssm_util import HALF, rounded, spans_of, view, within

pytestmark = pytest.mark.gpu


def make(seed, B, T, D, K, dtype, lens=None, bias=True, states=True, tail=0):
    rng = np.random.default_rng(seed)
    if lens is not None:
        B, T = 1, int(sum(lens)) + tail
    n = B if lens is None else len(lens)
    r = lambda *s: rounded(rng.standard_normal(s), dtype)
    c = dict(x=r(B, T, D), dy=r(B, T, D), w=(rng.standard_normal((D, K)) / K ** 0.5).astype(np.float32),
             bias=(0.3 * rng.standard_normal(D)).astype(np.float32) if bias else None,
             h0=r(n, K - 1, D) if states else None, dht=r(n, K - 1, D) if states else None)
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return dict(c, dtype=dtype, spans=spans_of(lens, B, T), cu=cu, T=T, tail=tail)


def check(c, act="silu", strided=False):
    dtype, half = c["dtype"], HALF[c["dtype"]]
    x = view(c["x"], dtype) if strided else dev(c["x"], dtype)
    put = lambda m, t=dtype: None if c[m] is None else dev(c[m], t)
    w, bias, h0, dht, dy = put("w", "f32"), put("bias", "f32"), put("h0"), put("dht"), put("dy")
    cu = None if c["cu"] is None else torch.from_numpy(c["cu"]).cuda()
    kw = dict(bias=bias, act=act, h0=h0, cu_seqlens=cu)
    out = torch.full_like(dy, 7.0)
    y, ht = ck.conv_fwd(x, w, out=out, **kw)
    dx, dw, db, dh0 = ck.conv_bwd(x, w, dy, dht=dht, **kw)
    torch.cuda.synchronize()
    end = c["T"] - c["tail"]
    assert (out[:, end:] == 7).all(), "rows past the last sequence"
    at, sums = [], {"dw": [0, 0], "dbias": [0, 0]}
    for i, (b, lo, hi) in enumerate(c["spans"]):
        one = lambda m: None if c[m] is None else c[m][i]
        r = ref.conv(c["x"][b, lo:hi], c["w"], c["bias"], act, one("h0"), c["dy"][b, lo:hi], one("dht"))
        at.append(within("y", y[b, lo:hi], *r["y"], half))
        at.append(within("dx", dx[b, lo:hi], *r["dx"], half))
        assert np.array_equal(ht[i].float().cpu().numpy(), r["ht"][0].astype(np.float32))
        at.append(within("dh0", dh0[i], *r["dh0"], half))
        for m in sums:
            sums[m][0] = sums[m][0] + r[m][0]
            sums[m][1] = sums[m][1] + r[m][1] + 40 * ref.EPS * np.abs(r[m][0])
    at.append(within("dw", dw, *sums["dw"], HALF["f32"]))
    assert (db is None) == (c["bias"] is None)
    if db is not None:
        at.append(within("dbias", db, *sums["dbias"], HALF["f32"]))
    announce("at %.2g of the bounds" % max(at))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 64, 65, 130])
def test_lengths(dtype, K, T):
    check(make(T + K, 2, T, 24, K, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 7, 8, 63, 64, 65, 130, 256, 257, 1000])
def test_widths(dtype, D):
    check(make(100 + D, 2, 37, D, 4, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("bias,states", [(True, False), (False, True), (False, False)])
def test_parts(dtype, act, bias, states):
    check(make(200, 3, 50, 40, 4, dtype, bias=bias, states=states), act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("lens,tail", [([0, 1, 40, 0, 2, 3, 100], 0), ([5], 9), ([0, 0], 2), ([64, 64], 0)])
def test_packed(dtype, K, lens, tail):
    check(make(300, 1, 0, 20, K, dtype, lens=lens, tail=tail))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 40, 41])
def test_parts_of_wider_rows(dtype, D):
    check(make(400 + D, 2, 40, D, 4, dtype), strided=True)


def test_long_tiles():
    """Channels enough for the longest tiles of tokens."""
    check(make(500, 8, 600, 1028, 4, "bf16", states=False))


def test_no_tokens():
    x, h0 = torch.ones(2, 0, 8, device="cuda"), torch.randn(2, 3, 8, device="cuda")
    w = torch.ones(8, 4, device="cuda")
    y, ht = ck.conv_fwd(x, w, h0=h0)
    dx, dw, db, dh0 = ck.conv_bwd(x, w, x, bias=w[:, 0].contiguous(), h0=h0, dht=2 * h0)
    assert y.shape == (2, 0, 8) and torch.equal(ht, h0) and torch.equal(dh0, 2 * h0) and (dw == 0).all() and (db == 0).all()


def test_no_sequences():
    x = torch.full((1, 6, 8), 3.0, device="cuda")
    w, b = torch.ones(8, 4, device="cuda"), torch.ones(8, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    y, ht = ck.conv_fwd(x, w, bias=b, cu_seqlens=cu, out=out)
    dx, dw, db, dh0 = ck.conv_bwd(x, w, x, bias=b, cu_seqlens=cu)
    assert (y == 7).all() and ht.shape == (0, 3, 8) and (dw == 0).all() and (db == 0).all() and dh0.shape == (0, 3, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,K", [(1, 1, 2), (3, 40, 4), (2, 33, 3), (300, 8, 4)])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_steps_are_the_convolution(dtype, N, D, K, act):
    c = make(600 + N, N, 1, D, K, dtype)
    x, w, b, h0 = dev(c["x"], dtype)[:, 0], dev(c["w"]), dev(c["bias"]), dev(c["h0"], dtype)
    state, new = h0.clone(), torch.empty_like(h0)
    y2 = ck.conv_step(x, w, state, bias=b, act=act, new_state=new)
    assert torch.equal(state, h0)
    y = ck.conv_step(x, w, state, bias=b, act=act)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(state, new)
    for i in range(N):
        r = ref.conv(c["x"][i], c["w"], c["bias"], act, c["h0"][i])
        within("y", y[i][None], *r["y"], HALF[dtype])
        assert np.array_equal(state[i].float().cpu().numpy(), r["ht"][0].astype(np.float32))


def test_cache_in_place_with_many_tiles():
    """h0 and ht in one buffer: a sequence of many tiles reads the old cache in its
    first and writes the new one; sequences shorter than the cache shift it."""
    for T in (1, 2, 500):
        c = make(700 + T, 3, T, 24, 4, "bf16")
        x, w, h0 = dev(c["x"], "bf16"), dev(c["w"]), dev(c["h0"], "bf16")
        y, ht = ck.conv_fwd(x, w, h0=h0)
        state = h0.clone()
        y2, ht2 = ck.conv_fwd(x, w, h0=state, final_state=state)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(ht, ht2)


def test_non_finite_inputs_stay_near():
    c = make(800, 1, 0, 16, 4, "f32", lens=[20, 20])
    x, w, dy = dev(c["x"]), dev(c["w"]), dev(c["dy"])
    cu = torch.from_numpy(c["cu"]).cuda()
    y, _ = ck.conv_fwd(x, w, cu_seqlens=cu)
    dx, dw, _, _ = ck.conv_bwd(x, w, dy, cu_seqlens=cu)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = x.clone()
        bad[0, 18, 3] = value
        y2, _ = ck.conv_fwd(bad, w, cu_seqlens=cu)
        dx2, dw2, _, _ = ck.conv_bwd(bad, w, dy, cu_seqlens=cu)
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[0, 18:20, 3] = True
        assert torch.equal(y[~hit], y2[~hit])
        hit[0, 15:20, 3] = True  # gradients of the inputs under those outputs
        assert torch.equal(dx[~hit], dx2[~hit])
        other = [i for i in range(16) if i != 3]
        assert torch.equal(dw[other], dw2[other])
