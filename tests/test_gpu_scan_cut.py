"""Sequences cut into pieces for every shape of a workgroup (up to 8, 16, 32 and 64
states), with several blocks of channels, groups and sequences: forward and gradients
against the recurrence in float64 within its bounds (scan_fp64.py)."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.ssm_util import make_scan, scan_kw, scan_tensors
from tests.test_gpu_scan import check

pytestmark = pytest.mark.gpu


def cuts(c, D, S, G):
    """Whether the forward of these sizes is cut: only then it asks for a workspace."""
    B, T = c["x"].shape[:2]
    d = ck.ScanDesc(B, T, D, S, G, c["n"], ck.BF16, 1, 0, 0, 0, 0, 0)
    return ck._load().ckda_scan_fwd_workspace_size(ctypes.byref(d), int(c["lens"] is not None)) > 0


# pieces of 128 tokens at these sizes
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [3, 8, 16, 20, 32, 50, 64])
@pytest.mark.parametrize("D,G,B,T,lens", [(130, 2, 2, 300, None), (72, 1, 2, 400, None), (12, 3, 1, 1000, None),
                                          (130, 2, 1, 0, [390, 0, 1, 257, 128]), (72, 1, 1, 0, [127, 400, 16])])
def test_shapes(dtype, S, D, G, B, T, lens):
    c = make_scan(1700 + S + D, B, T, D, S, G, dtype, lens=lens, tail=3 if lens else 0)
    assert cuts(c, D, S, G)
    check(c, cut=128)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [5, 16, 33])
def test_parts(dtype, S):
    """Without gate, states, skip and bias; steps given."""
    for k, (z, states, skip) in enumerate(((False, False, False), (True, False, True), (False, True, True))):
        check(make_scan(1800 + S + k, 1, 300, 72, S, 1, dtype, steps="values" if k else "logits", z=z, states=states,
                        skip=skip), cut=128)


# gradients in three pieces of 160 tokens (65 blocks of channels, 4 sequences), and in pieces
# of 256: T blocks / 1024 rounded up to 32 in a packed batch (3002 * 84 / 1024)
@pytest.mark.parametrize("D,S,B,T,lens,cut", [(4160, 1, 4, 390, None, 160), (4160, 9, 4, 390, None, 160),
                                              (5376, 1, 1, 0, [1500, 5, 0, 997, 500], 256)])
def test_longer_pieces(D, S, B, T, lens, cut):
    check(make_scan(1900 + S, B, T, D, S, 1, "bf16", lens=lens), cut=cut)


@pytest.mark.parametrize("S", [5, 16, 40])
def test_non_finite_values_stay_in_their_sequence(S):
    """NaN, infinities and the lowest value in a few tokens of the middle sequence of three,
    each of which is cut: the others keep their bits, forward and backwards."""
    c = make_scan(2100 + S, 1, 0, 72, S, 1, "bf16", lens=[300, 290, 200])
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    run = lambda t, k: (ck.scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], **k),
                        ck.scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["dy"], dht=t["dht"], **k))
    (y, ht), r = run(g, kw)
    other = np.r_[0:300, 590:790]
    for m in ("x", "dt", "B", "C", "z", "dy"):
        for value in (float("nan"), float("inf"), float("-inf"), float(torch.finfo(torch.bfloat16).min)):
            bad = dict(g)
            bad[m] = g[m].clone()
            bad[m][0, 430:433] = value
            (y2, ht2), r2 = run(bad, dict(kw, z=bad["z"]))
            torch.cuda.synchronize()
            assert torch.equal(y[:, other], y2[:, other]) and torch.equal(ht[[0, 2]], ht2[[0, 2]]), (m, value)
            for i in (0, 1, 3, 4, 6):  # dx, ddt, dB, dC, dz
                assert torch.equal(r[i][:, other], r2[i][:, other]), (m, value, i)
            assert torch.equal(r[8][[0, 2]], r2[8][[0, 2]]), (m, value)
