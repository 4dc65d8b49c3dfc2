"""Layer norm on the GPU against the formulas in float64 with their bounds
(scan_fp64.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests import scan_fp64 as ref
from tests.gpu_util import announce, dev
from tests.ssm_util import HALF, rounded, within

pytestmark = pytest.mark.gpu


def check(seed, rows, d, dtype, parts="wbr", mean=0.5, eps=1e-5):
    rng = np.random.default_rng(seed)
    r = lambda m=0.0: rounded(m + 1.5 * rng.standard_normal((rows, d)), dtype)
    x, dn, dh = r(mean), r(), r()
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32) if "w" in parts else None
    b = (0.3 * rng.standard_normal(d)).astype(np.float32) if "b" in parts else None
    res = r() if "r" in parts else None
    put = lambda a, t="f32": None if a is None else dev(a, t)
    gx, gw, gb, gr = put(x, dtype), put(w), put(b), put(res, dtype)
    n, h = ck.layer_norm(gx, gw, gb, residual=gr, eps=eps)
    half = HALF[dtype]
    want = ref.layer_norm(x, w, b, res, eps)
    at = [within("n", n, *want["n"], half)]
    assert (h is None) == (res is None)
    if h is not None:
        at.append(within("h", h, *want["h"], half))
        over_r, over_x = gr.clone(), gx.clone()  # the stream in place, over either summand
        for src, add, buf in ((gx, over_r, over_r), (over_x, gr, over_x)):
            n2, h2 = ck.layer_norm(src, gw, gb, residual=add, eps=eps, residual_out=buf)
            torch.cuda.synchronize()
            assert h2 is buf and torch.equal(n, n2) and torch.equal(h, h2)
    dx, dw, db = ck.layer_norm_bwd(gx, gw, put(dn, dtype), dh=put(dh, dtype) if "r" in parts else None, eps=eps,
                                   output_dbias="b" in parts)
    torch.cuda.synchronize()
    want = ref.layer_norm(x, w, None, None, eps, dn, dh if "r" in parts else None)
    at.append(within("dx", dx, *want["dx"], half))
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    if dw is not None:
        at.append(within("dw", dw, *want["dw"], HALF["f32"]))
    if db is not None:
        at.append(within("db", db, *want["db"], HALF["f32"]))
    announce("at %s of the bounds" % " ".join("%.2g" % a for a in at))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [2, 3, 7, 8, 24, 33, 64, 100, 128, 256, 1000, 1001, 1002, 1024, 2048, 2050, 4096, 5000,
                               8192, 8200, 16383, 16384])
def test_widths(dtype, d):
    check(d, 5, d, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", ["", "w", "b", "wb", "r", "wr"])
def test_parts(dtype, parts):
    check(3, 37, 64, dtype, parts)
    check(4, 3, 1536, dtype, parts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 128), (63, 128), (65, 16), (2049, 24), (9000, 40), (3000, 512), (1500, 2048)])
def test_rows(dtype, rows, d):
    check(rows, rows, d, dtype)


def test_a_mean_far_above_the_spread():
    """The variance is that of the centred row: rows of 1000 +- 1.5 keep the digits
    that their own rounding and the mean's leave."""
    check(7, 20, 512, "f32", "wb", mean=1000.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(5, 64), (37, 128), (3, 24), (70, 1001)])
def test_no_eps_and_rows_that_leave_threads_idle(dtype, rows, d):
    """eps = 0 with rows that do not fill a workgroup: the sums over rows hold
    nothing of the idle threads."""
    check(rows + d, rows, d, dtype, "wbr", eps=0.0)


def test_rows_of_one_value_and_no_rows():
    x = torch.full((4, 64), 3.0, device="cuda")
    w = torch.ones(64, device="cuda")
    n, _ = ck.layer_norm(x, w, w)
    assert (n == 1).all()
    dx, dw, db = ck.layer_norm_bwd(x, w, x)
    assert (dx == 0).all() and (dw == 0).all() and (db == 12).all()
    one = torch.full((4, 1), 3.0, device="cuda")
    assert (ck.layer_norm(one, None)[0] == 0).all()
    e = x[:0]
    assert ck.layer_norm(e, w, residual=e)[1].shape == (0, 64)
    dx, dw, db = ck.layer_norm_bwd(e, w, e)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
