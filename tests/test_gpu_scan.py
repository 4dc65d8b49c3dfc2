"""The selective scan on the GPU against the recurrence in float64, within bounds
carried along with it (scan_fp64.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.gpu_util import announce, dev, host
from tests.ssm_util import HALF, make_scan, scan_kw, scan_reference, scan_tensors, within

pytestmark = pytest.mark.gpu

GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


def check(c, strided=False, grads=True, cut=0):
    g, half = scan_tensors(c, strided), HALF[c["dtype"]]
    want = scan_reference(c, grads, cut)
    end = c["T"] - c["tail"]
    kw = scan_kw(c, g)
    out = torch.full_like(g["dy"], 7.0)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], out=out, **kw)
    torch.cuda.synchronize()
    assert y is out and (y[:, end:] == 7).all(), "rows past the last sequence"
    at = [within("y", y[:, :end], want["y"][0][:, :end], want["y"][1][:, :end], half),
          within("ht", ht, *want["ht"], HALF["f32"])]
    if grads:
        got = dict(zip(GRADS, ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)))
        torch.cuda.synchronize()
        for m in GRADS:
            given = {"dz": c["z"], "dD": c["D"], "dbias": c["bias"]}.get(m, 1)
            assert (got[m] is None) == (given is None), m
            if got[m] is None:
                continue
            v, e = want[m]
            rows = m in ("dx", "ddt", "dz", "dB", "dC")
            if rows:
                got[m], v, e = got[m][:, :end], v[:, :end], e[:, :end]
            at.append(within(m, got[m], v, e, half if rows else HALF["f32"]))
    announce("at %s of the bounds" % " ".join("%.2g" % a for a in at))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 100])
def test_lengths(dtype, T):
    check(make_scan(T, 2, T, 72, 16, 1, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 2, 5, 8, 9, 15, 16, 17, 24, 32, 33, 50, 64])
def test_states_a_channel(dtype, S):
    check(make_scan(100 + S, 1, 37, 40, S, 2, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (7, 1), (8, 1), (31, 1), (32, 1), (33, 1), (64, 2), (65, 1), (96, 3),
                                 (128, 8), (130, 2), (264, 1)])
def test_channels_and_groups(dtype, D, G):
    check(make_scan(200 + D + G, 1, 21, D, 16, G, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("steps", ["logits", "values"])
@pytest.mark.parametrize("z,states,skip", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
def test_parts(dtype, steps, z, states, skip):
    check(make_scan(300, 2, 35, 48, 12, 1, dtype, steps=steps, z=z, states=states, skip=skip))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,tail", [([0, 1, 40, 0, 17, 2], 0), ([33], 5), ([0, 0], 3), ([16, 16, 16], 0), ([], 4)])
def test_packed(dtype, lens, tail):
    """Empty sequences keep their states; rows past the last sequence stay as they are."""
    if not lens:
        c = make_scan(400, 1, 4, 24, 16, 1, dtype, lens=[4])
        g = scan_tensors(c)
        kw = dict(scan_kw(c, g), h0=None, cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
        out = torch.full_like(g["dy"], 7.0)
        y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], out=out, **kw)
        got = dict(zip(GRADS, ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], **kw)))
        assert (y == 7).all() and ht.shape == (0, 24, 16)
        assert all((got[m] == 0).all() for m in ("dA", "dD", "dbias"))
        return
    check(make_scan(401, 1, 0, 40, 16, 2, dtype, lens=lens, tail=tail))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [24, 64, 25])
def test_parts_of_wider_rows(dtype, D):
    """Inputs that start at odd addresses inside wider rows, NaN around them."""
    check(make_scan(500 + D, 2, 20, D, 16, 1, dtype), strided=True)


# pieces of 128 tokens at these sizes: their joins are powers of sums of 128 steps
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(300, None), (257, None), (1000, None), (0, [700, 3, 0, 129, 128, 300])])
def test_cut_sequences(dtype, T, lens):
    check(make_scan(600 + T, 1, T, 24, 16, 1, dtype, lens=lens), cut=128)


def test_many_channels_walk_whole_sequences():
    """Enough workgroups that no sequence is cut, for every shape of a workgroup."""
    check(make_scan(702, 8, 20, 4096, 9, 1, "bf16"))
    check(make_scan(700, 6, 290, 4096, 3, 1, "bf16"), grads=False)
    check(make_scan(701, 2, 300, 6200, 10, 2, "f32", z=False), grads=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,S,G", [(1, 8, 16, 1), (3, 33, 16, 1), (5, 40, 5, 2), (2, 12, 64, 3), (4, 7, 1, 7), (9, 65, 20, 5)])
def test_steps_are_the_scan(dtype, N, D, S, G):
    c = make_scan(800 + N, N, 1, D, S, G, dtype)
    g, want = scan_tensors(c), scan_reference(c, False)
    one = {m: g[m][:, 0] for m in ("x", "dt", "z", "B", "C")}
    kw = dict(D=g["D"], z=one["z"], dt_bias=g["bias"], steps=c["steps"])
    state, new = g["h0"].clone(), torch.empty_like(g["h0"])
    y2 = ck.scan_step(one["x"], one["dt"], g["A"], one["B"], one["C"], state, new_state=new, **kw)
    assert torch.equal(state, g["h0"])
    y = ck.scan_step(one["x"], one["dt"], g["A"], one["B"], one["C"], state, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(state, new)
    within("y", y[:, None], *want["y"], HALF[dtype])
    within("state", state, *want["ht"], HALF["f32"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_tokens_leave_the_states(dtype):
    """A step of exactly 0, by a logit of -inf or the type's lowest value, is no step:
    the decay is 1 and nothing is written, forwards and backwards."""
    c = make_scan(900, 1, 40, 16, 16, 1, dtype, z=False)
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    for value in (-np.inf, low, -200.0):
        masked = dict(c, dt=c["dt"].copy())
        masked["dt"][0, 10:30] = value
        g = scan_tensors(masked)
        y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **scan_kw(masked, g))
        keep = np.r_[0:10, 30:40]
        short = dict(c, **{m: c[m][:, keep] for m in ("x", "dt", "B", "C", "dy")}, spans=[(0, 0, 20)], T=20)
        s = scan_tensors(short)
        ys, hts = ck.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], **scan_kw(short, s))
        assert torch.equal(ht, hts) and torch.equal(y[:, keep], ys)
        got = dict(zip(GRADS, ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], **scan_kw(masked, g))))
        assert all(torch.isfinite(got[m]).all() for m in GRADS if got[m] is not None)
        assert (got["ddt"][0, 10:30] == 0).all() and (got["dB"][0, 10:30] == 0).all()


def test_non_finite_values_stay_in_their_sequence():
    c = make_scan(950, 1, 0, 40, 16, 1, "bf16", lens=[20, 30, 25])
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
    r = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], **kw)
    for m in ("x", "dt", "B", "C", "z"):
        bad = dict(g)
        bad[m] = g[m].clone()
        bad[m][0, 25:27] = float("nan")
        k = dict(kw, z=bad["z"])
        y2, ht2 = ck.scan_fwd(bad["x"], bad["dt"], bad["A"], bad["B"], bad["C"], **k)
        r2 = ck.scan_bwd(bad["x"], bad["dt"], bad["A"], bad["B"], bad["C"], bad["dy"], **k)
        other = np.r_[0:20, 50:75]
        assert torch.equal(y[:, other], y2[:, other]) and torch.equal(ht[[0, 2]], ht2[[0, 2]]), m
        assert not torch.isfinite(y2[0, 25]).all(), m
        for i in (0, 1, 3, 4, 6):  # dx, ddt, dB, dC, dz
            assert torch.equal(r[i][:, other], r2[i][:, other]), (m, i)


def test_states_in_place_and_repeated_calls_agree():
    """h0 and ht in one buffer, whole and cut sequences; the same bits every time."""
    for T, D in ((60, 40), (700, 24)):
        c = make_scan(970, 2, T, D, 16, 1, "bf16")
        g = scan_tensors(c)
        kw = scan_kw(c, g)
        y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
        first = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)
        again = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        state = g["h0"].clone()
        y2, ht2 = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], final_state=state, **dict(kw, h0=state))
        torch.cuda.synchronize()
        assert ht2 is state and torch.equal(y, y2) and torch.equal(ht, ht2)


def test_prompt_then_steps_are_one_prompt():
    """A prompt continued a token at a time; both halves against the whole."""
    c = make_scan(980, 2, 30, 40, 16, 1, "f32")
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    want = scan_reference(c, False)
    cut = {m: g[m][:, :22].contiguous() for m in ("x", "dt", "z", "B", "C")}
    y, st = ck.scan_fwd(cut["x"], cut["dt"], g["A"], cut["B"], cut["C"], **dict(kw, z=cut["z"]))
    ys = [y]
    for t in range(22, 30):
        one = {m: g[m][:, t] for m in ("x", "dt", "z", "B", "C")}
        ys.append(ck.scan_step(one["x"], one["dt"], g["A"], one["B"], one["C"], st, D=g["D"], z=one["z"],
                               dt_bias=g["bias"])[:, None])
    torch.cuda.synchronize()
    within("y", torch.cat(ys, 1), *want["y"], HALF["f32"])
    within("state", st, *want["ht"], HALF["f32"])


def test_batches_of_no_tokens():
    """T = 0: the states pass through, forwards and backwards; the sums are zeros."""
    c = make_scan(990, 2, 1, 24, 16, 1, "bf16")
    g = scan_tensors(c)
    none = lambda m: g[m][:, :0]
    kw = dict(scan_kw(c, g), z=none("z"))
    y, ht = ck.scan_fwd(none("x"), none("dt"), g["A"], none("B"), none("C"), **kw)
    r = dict(zip(GRADS, ck.scan_bwd(none("x"), none("dt"), g["A"], none("B"), none("C"), none("dy"), dht=g["dht"], **kw)))
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 24) and torch.equal(ht, g["h0"]) and torch.equal(r["dh0"], g["dht"])
    assert all((r[m] == 0).all() for m in ("dA", "dD", "dbias"))
    e = ck.scan_step(none("x")[0], none("dt")[0], g["A"], none("B")[0], none("C")[0], g["h0"][:0])
    assert e.shape == (0, 24)


def test_long_rows_and_late_tokens():
    """Tokens past 2^31 elements of a tensor: the last sequence of a batch whose rows
    are far apart."""
    c = make_scan(991, 1, 40, 24, 16, 1, "bf16")
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
    stride, T = (1 << 20) + 8, 2240
    wide = torch.zeros(T * stride, device="cuda", dtype=torch.bfloat16)
    far = wide.as_strided((1, T, 24), (T * stride, stride, 1))
    far[:, -40:] = g["x"]
    assert (T - 40) * stride > 1 << 31
    put = lambda t: torch.cat([torch.zeros(1, T - 40, *t.shape[2:], device="cuda", dtype=t.dtype), t], 1)
    cu = torch.tensor([0, T - 40, T], dtype=torch.int32, device="cuda")
    two = dict(D=g["D"], z=put(g["z"]), dt_bias=g["bias"], cu_seqlens=cu, h0=torch.cat([torch.zeros_like(g["h0"]), g["h0"]]))
    y2, ht2 = ck.scan_fwd(far, put(g["dt"]), g["A"], put(g["B"]), put(g["C"]), **two)
    cy, _ = ck.conv_fwd(g["x"], torch.ones(24, 4, device="cuda"))
    cy2, _ = ck.conv_fwd(far, torch.ones(24, 4, device="cuda"), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.equal(y, y2[:, -40:]) and torch.equal(ht[0], ht2[1]) and torch.equal(cy, cy2[:, -40:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,steps", [(1, "values"), (37, "values"), (37, "logits"), (300, "values")])
def test_decay_rates_of_the_lowest_value(dtype, T, steps):
    """A of float32's lowest value forgets the state at once, whatever the step; a step
    of exactly 0 keeps it all the same."""
    c = make_scan(995 + T, 1, T, 24, 16, 1, dtype, steps=steps)
    low = np.finfo(np.float32).min
    c["A"][::3], c["A"][1::3, 5] = low, low
    check(c, cut=128 if T > 256 else 0)
    if steps == "values":
        c["dt"][:, T // 2:T // 2 + 3] = 0
        check(c, grads=False, cut=128 if T > 256 else 0)  # dL/dstep of such a step is A itself
    if T == 1:
        g, want = scan_tensors(c), scan_reference(c, False)
        state = g["h0"].clone()
        y = ck.scan_step(g["x"][:, 0], g["dt"][:, 0], g["A"], g["B"][:, 0], g["C"][:, 0], state, D=g["D"], z=g["z"][:, 0],
                         steps=steps)
        torch.cuda.synchronize()
        within("y", y[:, None], *want["y"], HALF[dtype])
        within("state", state, *want["ht"], HALF["f32"])


def test_pieces_longer_than_the_shortest():
    """Sequences in a few pieces each, the last one ending inside a tile."""
    check(make_scan(998, 4, 530, 1984, 9, 1, "bf16"), grads=False, cut=160)
