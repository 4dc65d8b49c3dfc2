"""Decay linear attention on the GPU against the float64 recurrence of
decay_fp64.py: chunked forward, gradients and single-token step, elementwise
within the bounds derived there."""
import numpy as np
import pytest
import torch

from tests import decay_fp64 as ref
import gated_delta_rule_ckda_amd as ck
from gated_delta_rule_ckda_amd.inputs import round_bf16
from tests.gpu_util import DEV, announce, dev, host

pytestmark = pytest.mark.gpu


def make(seed, B, T, H, Hk, dk, dv, dtype, kind="values", gate="ckda", lens=None, h0=False,
         per_head=False, zeros=0.0, strong=False):
    rng = np.random.default_rng(seed)
    rnd = round_bf16 if dtype == "bf16" else (lambda x: np.asarray(x, dtype=np.float32))
    c = dict(dtype=dtype, kind=kind, gate=gate, scale=dk ** -0.5)
    c["cu"] = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = B if lens is None else len(lens)
    c["q"], c["k"] = (rnd(rng.standard_normal((B, T, Hk, dk), dtype=np.float32)) for _ in range(2))
    c["v"], c["do"] = (rnd(rng.standard_normal((B, T, H, dv), dtype=np.float32)) for _ in range(2))
    shape = (H,) if per_head else (B, T, H)
    x = rng.normal(3, 2, shape).astype(np.float32)
    if strong:
        x = rng.normal(-3, 4, shape).astype(np.float32)
    if kind == "logits":
        a = rnd(x)
        if zeros and gate == "ckda":
            a[rng.random(shape) < zeros] = 0.0
    else:
        a = (np.tanh(x / 2) if gate == "ckda" else 1 / (1 + np.exp(-x))).astype(np.float32)
        a[rng.random(shape) < zeros] = 0.0
    c["alpha"] = a
    c["h0"] = rng.standard_normal((n, H, dk, dv)).astype(np.float32) if h0 else None
    c["dht"] = rng.standard_normal((n, H, dk, dv)).astype(np.float32) if h0 else None
    return c


def gates_of(c):
    a, d = ref.gates(c["alpha"], c["kind"], c["gate"] == "ckda")
    full = c["v"].shape[:3]
    return np.broadcast_to(a, full), np.broadcast_to(d, full)


def on_gpu(c):
    dt = c["dtype"]
    g = {m: dev(c[m], dt) for m in ("q", "k", "v", "do")}
    g["alpha"] = dev(c["alpha"], dt if c["kind"] == "logits" else "f32")
    for m in ("h0", "dht"):
        g[m] = None if c[m] is None else dev(c[m])
    g["cu"] = None if c["cu"] is None else torch.from_numpy(c["cu"]).to(DEV)
    return g


def run_fwd(c, **kw):
    g = on_gpu(c)
    o, ht = ck.decay_fwd(g["q"], g["k"], g["v"], g["alpha"], h0=g["h0"], cu_seqlens=g["cu"],
                         gate=c["gate"], gates=c["kind"], scale=c["scale"], **kw)
    torch.cuda.synchronize()
    return o, ht


def run_bwd(c, **kw):
    g = on_gpu(c)
    r = ck.decay_bwd(g["q"], g["k"], g["v"], g["alpha"], g["do"], h0=g["h0"], dht=g["dht"],
                     cu_seqlens=g["cu"], gate=c["gate"], gates=c["kind"], scale=c["scale"], **kw)
    torch.cuda.synchronize()
    return r


def within(name, x, want, bound):
    x = host(x).reshape(want.shape)
    assert np.isfinite(x).all(), name
    off = np.abs(x - want) / bound
    i = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert off.size == 0 or off[i] <= 1, "%s: %.3g of the bound at %s (%g, want %g)" % (
        name, off[i], i, x[i], want[i])
    return float(off.max()) if off.size else 0.0


def check_fwd(c):
    T, dk = c["v"].shape[1], c["q"].shape[-1]
    o, ht = run_fwd(c)
    ro, rh, om, hm = ref.fwd(c["q"], c["k"], c["v"], gates_of(c)[0], c["h0"], c["cu"], c["scale"])
    a = within("o", o, ro, ref.bound_out(c["dtype"], ro, om, dk, T))
    b = within("ht", ht, rh, ref.bound_state(c["dtype"], hm, dk, T))
    announce("o at %.2g of its bound, ht at %.2g" % (a, b))


def check_bwd(c):
    T, H = c["v"].shape[1:3]
    n = max(c["q"].shape[-1], c["v"].shape[-1])
    got = run_bwd(c)
    a, da = gates_of(c)
    want, mag = ref.bwd(c["q"], c["k"], c["v"], a, c["do"], c["h0"], c["dht"], c["cu"], c["scale"])
    want[3], mag[3] = want[3] * da, mag[3] * da
    if c["alpha"].ndim == 1:
        want[3], mag[3] = want[3].sum((0, 1)), mag[3].sum((0, 1))
    at = []
    for i, m in enumerate(("dq", "dk", "dv", "dalpha", "dh0")):
        # a group's heads are added up in float32, the gate's sums run over two chunks' worth
        bound = (ref.bound_state(c["dtype"], mag[i], n, T) if m == "dh0"
                 else ref.bound_out(c["dtype"], want[i], mag[i], 4 * n if m == "dalpha" else n, T))
        at.append(within(m, got[i], want[i], bound))
    announce("dq dk dv dalpha dh0 at %s of their bounds" % " ".join("%.2g" % x for x in at))


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 200]
HEADS = [(8, 8), (16, 24), (64, 64), (48, 128), (128, 40), (72, 72), (128, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_fwd_lengths(dtype, T):
    check_fwd(make(T, 2, T, 2, 2, 64, 64, dtype, h0=T % 2 == 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_fwd_head_sizes(dtype, dk, dv):
    check_fwd(make(dk + dv, 1, 150, 2, 1, dk, dv, dtype, h0=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,gate,per_head", [("values", "kda", True), ("logits", "kda", False),
                                                ("logits", "ckda", False), ("logits", "ckda", True),
                                                ("values", "ckda", False)])
def test_fwd_gates(dtype, kind, gate, per_head):
    check_fwd(make(5, 2, 140, 4, 2, 64, 32, dtype, kind, gate, per_head=per_head, h0=True,
                   zeros=0.03))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,gate", [("values", "kda"), ("logits", "kda"), ("values", "ckda")])
def test_fwd_strong_decays(dtype, kind, gate):
    """Gates down to e^-15: products inside a chunk leave float's range."""
    check_fwd(make(6, 1, 200, 2, 2, 64, 64, dtype, kind, gate, strong=True, zeros=0.02))


PACKED = [[0, 1, 64, 63, 0, 65, 7, 130, 0], [5], [0], [200, 1], [1] * 70]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", PACKED)
def test_fwd_packed(dtype, lens):
    T = sum(lens)
    check_fwd(make(len(lens), 1, T, 2, 1, 64, 64, dtype, lens=lens, h0=True))
    check_fwd(make(len(lens), 1, T, 2, 2, 128, 128, dtype, lens=lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(1500, None), (1600, [700, 0, 3, 897])])
def test_fwd_segments(dtype, T, lens):
    """Long sequences are cut into segments joined by their end states."""
    c = make(8, 1, T, 1, 1, 32, 32, dtype, lens=lens, h0=True)
    desc = ck.DecayDesc(1, T, 1, 32, 32, 1 if lens is None else len(lens),
                        ck.F32 if dtype == "f32" else ck.BF16, 1, 0, 1, 0, 1.0)
    assert ck.decay_fwd_workspace_size(desc, lens is not None) > 0
    check_fwd(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_bwd_lengths(dtype, T):
    check_bwd(make(T, 2, T, 2, 2, 64, 64, dtype, h0=T % 2 == 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_bwd_head_sizes(dtype, dk, dv):
    check_bwd(make(dk + dv, 1, 150, 4, 2, dk, dv, dtype, h0=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,gate,per_head", [("values", "kda", True), ("logits", "kda", False),
                                                ("logits", "ckda", False), ("logits", "ckda", True),
                                                ("values", "ckda", False)])
def test_bwd_gates(dtype, kind, gate, per_head):
    check_bwd(make(5, 2, 140, 4, 2, 64, 32, dtype, kind, gate, per_head=per_head, h0=True,
                   zeros=0.03))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,gate", [("values", "kda"), ("logits", "kda"), ("values", "ckda")])
def test_bwd_strong_decays(dtype, kind, gate):
    check_bwd(make(6, 1, 200, 2, 2, 64, 64, dtype, kind, gate, strong=True, zeros=0.02))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", PACKED + [[700, 0, 3, 897]])
def test_bwd_packed(dtype, lens):
    check_bwd(make(len(lens), 1, sum(lens), 2, 1, 64, 64, dtype, lens=lens, h0=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 1, 1, 8, 8), (3, 4, 2, 16, 40), (2, 8, 8, 32, 64),
                                          (5, 2, 1, 64, 128), (7, 6, 3, 72, 24), (4, 4, 4, 128, 128)])
@pytest.mark.parametrize("kind,per_head", [("values", False), ("logits", False), ("values", True)])
def test_step(dtype, N, H, Hk, dk, dv, kind, per_head):
    c = make(N, N, 1, H, Hk, dk, dv, dtype, kind, h0=True, per_head=per_head, zeros=0.1)
    g = on_gpu(c)
    al = g["alpha"] if per_head else g["alpha"][:, 0].contiguous()
    new = torch.empty_like(g["h0"])
    args = (g["q"][:, 0].contiguous(), g["k"][:, 0].contiguous(), g["v"][:, 0].contiguous(), al)
    o = ck.decay_step(*args, g["h0"], gate=c["gate"], gates=kind, scale=c["scale"], new_state=new)
    o2 = ck.decay_step(*args, g["h0"], gate=c["gate"], gates=kind, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(new, g["h0"])
    ro, rh, om, hm = ref.fwd(c["q"], c["k"], c["v"], gates_of(c)[0], c["h0"], None, c["scale"])
    # the step multiplies exact operands in float32: only its output is rounded
    within("o", o, ro[:, 0], ref.HALF[dtype] * np.abs(ro[:, 0]) + 2 * ref.sums(dk, 1) * om[:, 0])
    within("state", new, rh, 2 * ref.sums(dk, 1) * hm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [64, 150])
def test_tiny_and_exact_gates(dtype, T):
    """Gates of 0, +-1, a half and down to the smallest normal float, forward
    and gradients: products of three of the small ones underflow, where the
    bounds' own terms vanish with them (2^-126 a term stands beside them)."""
    c = make(21, 2, T, 2, 2, 64, 64, dtype, h0=True)
    rng = np.random.default_rng(22)
    pool = np.array([1, 1, 1, 1, -1, 0.5, 0.999, 0, 1e-9, 1e-12, -1e-20, 1e-30, 2e-38], np.float32)
    c["alpha"] = rng.choice(pool, c["alpha"].shape).astype(np.float32)
    check_fwd(c)
    check_bwd(c)


SHUT = [-90.0, -120.0, -200.0, -2e7, -1e9, -1e30, "lowest", -np.inf]


def shut(c, low, share=0.04):
    """Some of the logits set to `low` ("lowest": the type's lowest value)."""
    if low == "lowest":
        low = torch.finfo(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32).min
    rng = np.random.default_rng(31)
    a = c["alpha"]
    a[rng.random(a.shape) < share] = low
    if a.ndim > 1:
        a[:, 10] = a[:, 11] = a[:, 75] = low
    else:
        a[0] = low
    c["alpha"] = round_bf16(a) if c["dtype"] == "bf16" else a
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", SHUT)
@pytest.mark.parametrize("per_head", [False, True])
def test_logits_that_shut_a_gate(dtype, low, per_head):
    """Logits so low that the gate is zero in float32 restart the state, as a
    gate of zero does: prefill and gradients, within the same bounds."""
    c = shut(make(30, 2, 150, 4, 2, 64, 64, dtype, "logits", "kda", h0=True, per_head=per_head), low)
    check_fwd(c)
    check_bwd(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e9, "lowest", -np.inf])
def test_shut_gates_across_segments_and_in_steps(dtype, low):
    """The same in a prompt that is cut into segments, and one token at a time."""
    c = shut(make(32, 1, 1500, 1, 1, 32, 32, dtype, "logits", "kda", h0=True), low, 0.01)
    check_fwd(c)
    c = shut(make(33, 2, 80, 2, 2, 32, 32, dtype, "logits", "kda", h0=True), low)
    g = on_gpu(c)
    st = g["h0"].clone()
    for t in range(80):
        at = lambda z: z[:, t].contiguous()
        ck.decay_step(at(g["q"]), at(g["k"]), at(g["v"]), at(g["alpha"]), st, gate="kda", gates="logits",
                      scale=c["scale"])
    ht = run_fwd(c)[1]
    _, rh, _, hm = ref.fwd(c["q"], c["k"], c["v"], gates_of(c)[0], c["h0"], None, c["scale"])
    # a step rounds a product and a sum, its gate (one power, one reciprocal) is off by three half steps
    within("steps", st, rh, 5 * 80 * 2.0 ** -24 * hm + 1e-30)
    within("prefill", ht, rh, ref.bound_state(dtype, hm, 32, 80))


@pytest.mark.parametrize("T", [64, 150])
def test_tiny_logits_of_signed_gates(T):
    """Logits next to zero, where a signed gate is half of them, down to the
    least float32, half of which rounds to a gate of zero."""
    c = make(34, 2, T, 2, 2, 64, 64, "f32", "logits", "ckda", h0=True)
    rng = np.random.default_rng(35)
    pool = np.array([1e-45, -1e-45, 3e-45, -1e-40, 1e-38, -1e-30, 0, 4], np.float32)
    put = rng.random(c["alpha"].shape) < 0.1
    c["alpha"][put] = rng.choice(pool, int(put.sum()))
    check_fwd(c)
    check_bwd(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0, 5])
def test_no_sequences_leave_zero_gate_gradients(dtype, T):
    """A packed batch of no sequences: the sum over no tokens is zero, whatever
    its memory held before."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, v = torch.ones(1, T, 2, 16, device=DEV, dtype=dt), torch.ones(1, T, 4, 16, device=DEV, dtype=dt)
    al, cu = torch.full((4,), 0.5, device=DEV), torch.zeros(1, device=DEV, dtype=torch.int32)
    torch.cuda.synchronize()
    dirty = [torch.full((4,), float("nan"), device=DEV, dtype=dt) for _ in range(64)]
    del dirty
    dal = ck.decay_bwd(q, q, v, al, v, cu_seqlens=cu)[3]
    torch.cuda.synchronize()
    assert dal.shape == (4,) and (dal == 0).all()


CUT = [(1500, None), (1600, [700, 0, 3, 897])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", CUT)
@pytest.mark.parametrize("dk,dv", [(128, 128), (72, 104)])
def test_segments_of_wide_heads(dtype, T, lens, dk, dv):
    """Long sequences of heads over 64 x 64, whose segment sums hold all columns
    of the state in one workgroup: forward and gradients."""
    c = make(40 + dk, 1, T, 2, 1, dk, dv, dtype, lens=lens, h0=True)
    desc = ck.DecayDesc(1, T, 2, dk, dv, 1 if lens is None else len(lens),
                        ck.F32 if dtype == "f32" else ck.BF16, 1, 0, 1, 0, 1.0)
    assert ck.decay_fwd_workspace_size(desc, lens is not None) > 0
    check_fwd(c)
    check_bwd(c)
