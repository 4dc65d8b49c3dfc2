"""Rows of the selective scan whose channels are multiples of 4 but not of 8, at
addresses that are and are not multiples of 4 elements, NaN around them."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.ssm_util import HALF, make_scan, scan_kw, scan_reference, scan_tensors, view, within
from tests.test_gpu_scan import GRADS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 2, 4])
@pytest.mark.parametrize("D,G,S,T", [(12, 1, 3, 37), (24, 2, 16, 37), (68, 1, 16, 300), (100, 1, 8, 37), (68, 1, 40, 37),
                                     (36, 3, 20, 33)])
def test_rows_of_four(dtype, pad, D, G, S, T):
    c = make_scan(2000 + D + S, 2, T, D, S, G, dtype)
    g = scan_tensors(c)
    if pad:
        for m in ("x", "dt", "z"):
            g[m] = view(c[m], dtype, pad)
    want, half, kw = scan_reference(c, True, 128 if T > 256 else 0), HALF[dtype], scan_kw(c, g)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
    got = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)
    torch.cuda.synchronize()
    within("y", y, *want["y"], half)
    within("ht", ht, *want["ht"], HALF["f32"])
    for m, t in zip(GRADS, got):
        within(m, t, *want[m], half if m in ("dx", "ddt", "dz", "dB", "dC") else HALF["f32"])
