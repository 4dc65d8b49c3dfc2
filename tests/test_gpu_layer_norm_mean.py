"""Layer norm of rows whose mean is far above their spread: the mean's own rounding
leaves no shift of the normed row.

Bounds, in half steps (EPS = 2^-24): a first mean off by m = 88 EPS of the mean
magnitude (48 additions at most a sum, the weights of scan_fp64.layer_norm), the
centred row c0 = h - mean, exact up to EPS of |c0| <= |c| + m, and the mean of c0,
which takes m back up to 88 EPS of |c0|'s mean.  So a centred element is off by
ec = 2 EPS |c0| + 90 EPS mean |c0|, which has no EPS |h| in it."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.gpu_util import announce, dev
from tests.scan_fp64 import EPS
from tests.ssm_util import HALF, within

pytestmark = pytest.mark.gpu

DEEP = 88 * EPS


def reference(x, w, b, dn, eps):
    mean = lambda t: t.mean(-1, keepdims=True)
    x, w, b, dn = (t.astype(np.float64) for t in (x, w, b, dn))
    rows = x.shape[0]
    c = x - mean(x)
    c0 = np.abs(c) + DEEP * mean(np.abs(x))
    ec = 2 * EPS * c0 + (DEEP + 2 * EPS) * mean(c0)
    var = mean(c * c)
    # formed as mean c0^2 - (mean c0)^2, both sums of c0
    evar = 2 * DEEP * mean(c0 * c0) + 2 * mean(c0 * ec) + mean(ec * ec)
    rs = 1 / np.sqrt(var + eps)
    ers = 0.5 * rs ** 3 * evar + 4 * EPS * rs
    cn = c * rs
    ecn = ec * rs + np.abs(c) * ers + ec * ers + EPS * np.abs(cn)
    out = {"n": (cn * w + b, ecn * np.abs(w) + 2 * EPS * (np.abs(cn * w) + np.abs(b)))}
    m = dn * w
    mm, mc = mean(m), mean(m * cn)
    emm = (DEEP + EPS) * mean(np.abs(m))
    # mean m c from the sums of m c0 and of m
    emc = mean(np.abs(m) * ecn) + 2 * DEEP * mean(np.abs(m)) * (np.abs(c0) * rs).max(-1, keepdims=True)
    ein = EPS * 4 * (np.abs(m) + np.abs(mm) + np.abs(cn * mc)) + emm + ecn * np.abs(mc) + np.abs(cn) * emc + ecn * emc
    inner = m - mm - cn * mc
    dx = rs * inner
    out["dx"] = (dx, rs * ein + ers * np.abs(inner) + 2 * EPS * np.abs(dx))
    many = (rows + 96) * EPS
    out["dw"] = ((dn * cn).sum(0), (np.abs(dn) * (ecn + many * np.abs(cn))).sum(0))
    return out


@pytest.mark.parametrize("d", [24, 100, 128, 1001, 2048, 4099, 8192, 16383])
@pytest.mark.parametrize("mean", [1e3, 1.7e4, -3.3e5])
def test_a_far_mean_leaves_no_shift(d, mean):
    rng = np.random.default_rng(d)
    x = (mean * (1 + 0.01 * rng.standard_normal((9, 1))) + rng.standard_normal((9, d))).astype(np.float32)
    w, b = (f.astype(np.float32) for f in (1 + 0.3 * rng.standard_normal(d), 0.3 * rng.standard_normal(d)))
    dn = rng.standard_normal((9, d)).astype(np.float32)
    want = reference(x, w, b, dn, 1e-5)
    n, _ = ck.layer_norm(dev(x), dev(w), dev(b))
    dx, dw, db = ck.layer_norm_bwd(dev(x), dev(w), dev(dn))
    torch.cuda.synchronize()
    at = [within(m, t, *want[m], HALF["f32"]) for m, t in (("n", n), ("dx", dx), ("dw", dw))]
    announce("at %s of the bounds" % " ".join("%.2g" % a for a in at))


@pytest.mark.parametrize("d", [7, 100, 1001, 4099, 16383])
def test_far_rows_of_one_value(d):
    """A row of one value is 0 once centred, whatever the value: the mean's rounding,
    88 EPS of the value at most, is taken back to 90 EPS of itself, and
    sqrt(eps) bounds the spread from below."""
    value = np.float32(77777.7)
    x = torch.full((5, d), float(value), device="cuda")
    n, _ = ck.layer_norm(x, None)
    torch.cuda.synchronize()
    shift = DEEP * value
    assert n.abs().max() <= (DEEP + 2 * EPS) * shift / np.sqrt(1e-5), n.abs().max()
