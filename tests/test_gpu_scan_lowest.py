"""Rates of float32's lowest value (a state that forgets at once) together with steps
of exactly 0, forward and gradients."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.ssm_util import HALF, make_scan, scan_kw, scan_reference, scan_tensors, within
from tests.test_gpu_scan import GRADS, check

pytestmark = pytest.mark.gpu

LOW = np.finfo(np.float32).min
MOST = np.float32(3.4028234663852886e38 / 1.4426950408889634)  # rates beyond count as this one


def lowest(seed, T, dtype, steps, S=16):
    c = make_scan(seed, 1, T, 24, S, 1, dtype, steps=steps)
    c["A"][::3], c["A"][1::3, 1] = LOW, LOW
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,S", [(37, 16), (300, 16), (37, 5), (37, 30), (37, 64)])
@pytest.mark.parametrize("logit", [-np.inf, "lowest", -200.0])
def test_masked_tokens_have_no_gradient_of_their_step(dtype, T, S, logit):
    """The slope of such a logit is 0, however large the rates that the decay's gradient
    is multiplied by: ddt is 0 there, and the bias sums the other tokens."""
    c = lowest(1400 + T + S, T, dtype, "logits", S)
    low = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    c["C"], c["dht"] = 8 * c["C"], 8 * c["dht"]
    at = slice(T // 2, T // 2 + 5)
    c["dt"][0, at] = low if logit == "lowest" else logit
    g = scan_tensors(c)
    got = dict(zip(GRADS, ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **scan_kw(c, g))))
    torch.cuda.synchronize()
    assert all(torch.isfinite(got[m]).all() for m in GRADS), [m for m in GRADS if not torch.isfinite(got[m]).all()]
    assert (got["ddt"][0, at] == 0).all()
    if not np.isinf(logit if logit != "lowest" else 0.0):
        check(c, cut=128 if T > 256 else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [37, 300])
def test_steps_of_zero_are_worth_the_rate(dtype, T):
    """dL/dstep of a given step of 0 is x (G . B) + w . A, with the rates the kernels use."""
    c = lowest(1500 + T, T, dtype, "values")
    c["dt"][:, T // 2:T // 2 + 3] = 0
    c["dy"] = (c["dy"] * 2.0 ** -14).astype(np.float32)
    c["dht"] = c["dht"] * np.float32(2.0 ** -14)
    c["A"] = np.maximum(c["A"], -MOST)
    assert np.abs(scan_reference(c)["ddt"][0]).max() > 1e32  # the rates' share is there
    check(c, cut=128 if T > 256 else 0)
    # the lowest value itself counts as that rate, up to its rounding (1.5 EPS of w . A, of
    # whose sum the bounds allow S + 10)
    g = scan_tensors(dict(c, A=np.where(c["A"] == -MOST, LOW, c["A"])))
    got = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **scan_kw(c, g))[1]
    torch.cuda.synchronize()
    within("ddt", got, *scan_reference(c, True, 128 if T > 256 else 0)["ddt"], HALF[dtype])
