"""The selective scan with rates that grow (A > 0, or steps below zero) in sequences
cut into pieces of 128 tokens, where the power over a piece leaves float32 and its
product with what enters does not: outputs and gradients against the recurrence in
float64, within the bounds carried along with it (scan_fp64.py)."""
import numpy as np
import pytest

from tests.ssm_util import make_scan
from tests.test_gpu_scan import check

pytestmark = pytest.mark.gpu

TINY = 1e-30  # a state or an adjoint that growth by e^100 leaves well inside float32


def rates(c, sign):
    """Of 24 channels, every state's rate in [0.5, 1], every third one decaying instead."""
    rng = np.random.default_rng(7)
    A = rng.uniform(0.5, 1.0, c["A"].shape).astype(np.float32)
    A[:, 2::3] *= -1
    c["A"] = sign * A


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T", [257, 1000])
def test_nothing_stays_nothing(dtype, sign, T):
    """No input before the last 20 tokens and no gradient after the first 20: states and
    adjoints of 0 in between, growing by e^128 a piece."""
    c = make_scan(1100 + T, 1, T, 24, 16, 1, dtype, steps="values", states=False)
    rates(c, sign)
    c["dt"][:] = sign
    c["x"][:, :-20] = 0
    c["dy"][:, 20:] = 0
    check(c, cut=128)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("S,lens", [(3, None), (16, None), (20, None), (50, None), (16, [300, 5, 0, 290])])
def test_tiny_states_grow(dtype, sign, S, lens):
    """States and adjoints of 1e-30 that grow by up to e^102 over one piece, and inside it."""
    c = make_scan(1200 + S, 1, 300, 24, S, 1, dtype, lens=lens, steps="values")
    rates(c, sign)
    c["h0"], c["dht"] = TINY * c["h0"], TINY * c["dht"]
    c["dt"] = sign * np.abs(c["dt"]).clip(2.0 ** -9, 2.0 ** -7).astype(np.float32)
    for _, lo, hi in c["spans"]:
        c["dt"][:, lo + 128:min(lo + 256, hi)] = sign * 0.796875  # 51 / 64
        c["x"][:, lo:min(lo + 256, hi)] = 0
        c["dy"][:, min(lo + 128, hi):hi] = 0
    check(c, cut=128)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growth_everywhere(dtype):
    """Inputs and gradients at every token, states that grow by up to e^30."""
    c = make_scan(1300, 1, 700, 24, 16, 1, dtype, steps="values")
    rates(c, 1)
    c["dt"] = (np.abs(c["dt"]).clip(0.0, 2.0 ** -5) * 1).astype(np.float32)
    check(c, cut=128)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_whose_sum_is_past_float32(dtype):
    """Two steps of 2^127 without an input reset the states that decay and leave those
    of rate 0 as they are, in whole sequences and in cut ones."""
    for T in (40, 300):
        c = make_scan(1400 + T, 1, T, 24, 16, 1, dtype, steps="values")
        c["A"][:, ::4] = 0
        c["dy"], c["dht"] = (np.float32(2.0 ** -20) * c[m] for m in ("dy", "dht"))
        for t in (5, 20):
            c["dt"][:, t], c["x"][:, t] = 2.0 ** 127, 0
        check(c, cut=128 if T > 256 else 0)
