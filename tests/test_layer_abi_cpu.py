"""The decay and norm calls reject bad arguments on the host before any HIP call
(dummy, never-dereferenced pointers; no GPU is touched), and the binding before
the library; the float64 references behind the parity tests against differences."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests import decay_fp64 as dref
from tests import norm_fp64 as nref

BASE = 0x7F0000000000
NAMES = ["q", "k", "v", "alpha", "h0", "o", "ht", "dout", "dht", "dq", "dk", "dv", "dalpha", "dh0", "ws"]
P = {n: ctypes.c_void_p(BASE + i * (1 << 33)) for i, n in enumerate(NAMES)}
CU = ctypes.c_void_p(BASE + 40 * (1 << 33))


def desc(**kw):
    d = dict(B=2, T=64, H=4, dk=128, dv=128, num_seqs=2, io_dtype=ck.BF16, gate_range=ck.GATE_KDA,
             gate_input=ck.GATES_F32, qk_heads=2, alpha_per_head=0, scale=1.0)
    d.update(kw)
    return ck.DecayDesc(**d)


def call(which, d, cu=None, bytes_=1 << 33, **over):
    p = dict(P, **over)
    lib = ck._load()
    ref = None if d is None else ctypes.byref(d)
    if which == "fwd":
        st = lib.ckda_decay_fwd(ref, p["q"], p["k"], p["v"], p["alpha"], cu, p["h0"], p["o"], p["ht"],
                                p["ws"], bytes_, None)
    else:
        st = lib.ckda_decay_bwd(ref, p["q"], p["k"], p["v"], p["alpha"], cu, p["h0"], p["dout"],
                                p["dht"], p["dq"], p["dk"], p["dv"], p["dalpha"], p["dh0"], p["ws"],
                                bytes_, None)
    return st, lib.ckda_last_error().decode()


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("over,status,needle", [
    (dict(B=0), 1, "non-positive"), (dict(T=-1), 1, "non-positive"), (dict(dv=0), 1, "non-positive"),
    (dict(io_dtype=3), 1, "io_dtype"), (dict(gate_range=2), 1, "gate_range"),
    (dict(gate_input=4), 1, "gate_input"), (dict(alpha_per_head=2), 1, "alpha_per_head"),
    (dict(qk_heads=3), 1, "qk_heads"), (dict(num_seqs=3), 1, "num_seqs"),
    (dict(dk=12), 2, "multiples of 8"), (dict(dv=136), 2, "multiples of 8"),
    (dict(B=1 << 16, num_seqs=1 << 16, T=1 << 15), 2, "too many"),
    (dict(H=1 << 16, qk_heads=1 << 16), 2, "2^22"),
])
def test_decay_rejects_bad_descriptors(which, over, status, needle):
    st, msg = call(which, desc(**over))
    assert st == status and needle in msg, msg


def test_decay_null_alignment_overlap():
    assert call("fwd", None)[0] == 1
    for n in ("q", "k", "v", "alpha", "o"):
        st, msg = call("fwd", desc(), **{n: None})
        assert st == 1 and n + " must not be NULL" in msg
    st, msg = call("fwd", desc(), k=ctypes.c_void_p(P["k"].value + 8))
    assert st == 1 and "aligned" in msg
    for n in ("q", "v", "alpha", "h0"):
        st, msg = call("fwd", desc(), o=P[n])
        assert st == 1 and "o overlaps " + n in msg
    st, msg = call("fwd", desc(), ht=ctypes.c_void_p(P["h0"].value + 64))
    assert st == 1 and "overlaps" in msg
    for n in ("dq", "dk", "dv", "dout"):
        st, msg = call("bwd", desc(), **{n: None})
        assert st == 1 and n in msg
    st, msg = call("bwd", desc(), dq=P["dk"])
    assert st == 1 and "overlaps" in msg
    st, msg = call("bwd", desc(), dh0=P["dht"])
    assert st == 1 and "overlaps" in msg
    st, msg = call("bwd", desc(B=1, num_seqs=1), cu=P["dv"])
    assert st == 1 and "cu_seqlens" in msg
    st, msg = call("fwd", desc(), cu=CU)
    assert st == 1 and "B=2" in msg


def test_decay_workspaces():
    d = desc(B=1, num_seqs=1, T=100000)
    lib = ck._load()
    need = lib.ckda_decay_fwd_workspace_size(ctypes.byref(d), 0)
    assert need > 0
    assert call("fwd", d, bytes_=need - 1) == (3, "workspace has %d bytes, %d needed" % (need - 1, need))
    assert call("fwd", d, ws=None)[0] == 1
    assert "256-byte" in call("fwd", d, ws=ctypes.c_void_p(P["ws"].value + 16))[1]
    assert "workspace overlaps v" in call("fwd", d, ws=P["v"])[1]
    need = lib.ckda_decay_bwd_workspace_size(ctypes.byref(desc()), 0)
    # a state and an adjoint a chunk in bf16, at least
    assert need >= 2 * 2 * 4 * 128 * 128 * 2
    assert call("bwd", desc(), bytes_=need - 1)[0] == 3
    assert lib.ckda_decay_fwd_workspace_size(None, 0) == 0
    assert lib.ckda_decay_bwd_workspace_size(ctypes.byref(desc(dk=20)), 0) == 0


def test_decay_nothing_to_do():
    assert call("fwd", desc(B=1, num_seqs=0, T=0), cu=CU)[0] == 0
    assert call("bwd", desc(B=1, num_seqs=0, T=0), cu=CU)[0] == 0


def step(N=3, H=4, Hk=2, dk=64, dv=64, io=ck.BF16, gate=0, gi=0, per=0, **over):
    p = dict(P, **over)
    lib = ck._load()
    st = lib.ckda_decay_step(N, H, Hk, dk, dv, io, gate, gi, per, 1.0, p["q"], p["k"], p["v"], p["alpha"],
                             p["h0"], p["ht"], p["o"], None)
    return st, lib.ckda_last_error().decode()


def test_step_rejections():
    assert step(N=0)[0] == 0
    for kw, status in ((dict(N=-1), 1), (dict(H=0), 1), (dict(Hk=3), 1), (dict(dk=9), 2), (dict(io=2), 1),
                       (dict(gate=5), 1), (dict(gi=3), 1), (dict(per=2), 1), (dict(N=1 << 20), 2),
                       (dict(q=None), 1), (dict(h0=None), 1), (dict(ht=None), 1), (dict(o=P["v"]), 1),
                       (dict(ht=ctypes.c_void_p(P["h0"].value + 16)), 1), (dict(ht=P["k"]), 1)):
        assert step(**kw)[0] == status, kw


def norm(rows=4, d=64, io=ck.BF16, act=1, eps=1e-6, **over):
    p = dict(y=P["q"], w=P["k"], g=P["v"], x=P["alpha"], s=P["h0"], w2=P["o"], h=P["ht"], n=P["dout"])
    p.update(over)
    lib = ck._load()
    st = lib.ckda_block_norm(rows, d, io, act, eps, *[p[m] for m in ("y", "w", "g", "x", "s", "w2", "h", "n")], None)
    return st, lib.ckda_last_error().decode()


def norm_bwd(rows=4, d=64, io=ck.BF16, act=1, eps=1e-6, bytes_=1 << 33, **over):
    p = {m: ctypes.c_void_p(BASE + (50 + i) * (1 << 33)) for i, m in enumerate(
        "y w g x s w2 dh dn dy dw dg dx ds dw2 ws".split())}
    p.update(over)
    lib = ck._load()
    st = lib.ckda_block_norm_bwd(rows, d, io, act, eps, *[p[m] for m in
                                 "y w g x s w2 dh dn dy dw dg dx ds dw2 ws".split()], bytes_, None)
    return st, lib.ckda_last_error().decode()


def test_norm_rejections():
    assert norm(rows=0)[0] == 0
    for kw, status in ((dict(rows=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(io=7), 1), (dict(act=3), 1),
                       (dict(act=0), 1), (dict(g=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                       (dict(eps=float("inf")), 1), (dict(n=None), 1), (dict(w2=None), 1), (dict(y=None), 1),
                       (dict(h=None), 1), (dict(h=P["q"]), 1), (dict(n=P["alpha"]), 1), (dict(n=P["ht"]), 1),
                       (dict(y=ctypes.c_void_p(BASE + 2)), 1), (dict(rows=1 << 45), 2)):
        assert norm(**kw)[0] == status, kw
    for kw, status in ((dict(rows=0), 1), (dict(dn=None), 1), (dict(dw2=None), 1), (dict(dw=None), 1),
                       (dict(ds=None), 1), (dict(dg=None), 1), (dict(act=0), 1), (dict(bytes_=16), 3),
                       (dict(ws=None), 1), (dict(dy=None), 1), (dict(dh=None), 1)):
        assert norm_bwd(**kw)[0] == status, kw
    p = ctypes.c_void_p(BASE + 50 * (1 << 33))
    assert norm_bwd(dx=p)[0] == 1 and "dx overlaps y" in norm_bwd(dx=p)[1]


def test_binding_rejects_before_the_library():
    """Shapes, types and devices are checked in Python (tensors on the CPU here)."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    q, v, al = z(1, 8, 2, 16), z(1, 8, 4, 16), z(1, 8, 4)
    with pytest.raises(ValueError, match="GPU"):
        ck.decay_fwd(q, q, v, al)
    for bad in (dict(k=z(1, 8, 2, 8)), dict(v=z(1, 7, 4, 16)), dict(v=z(1, 8, 3, 16)), dict(alpha=z(1, 8, 2)),
                dict(alpha=z(1, 8, 4, dt=torch.bfloat16)), dict(k=z(1, 8, 2, 16, dt=torch.bfloat16)),
                dict(cu_seqlens=z(3))):
        kw = dict(q=q, k=q, v=v, alpha=al)
        kw.update(bad)
        with pytest.raises(ValueError):
            ck.decay_fwd(**kw)
    with pytest.raises(TypeError):
        ck.decay_fwd(q.half(), q.half(), v.half(), al)
    with pytest.raises(ValueError, match="gate"):
        ck.decay_fwd(q, q, v, al, gate="relu")
    y, w = z(4, 32), z(32)
    for kw in (dict(weight=z(31)), dict(gate=z(4, 31)), dict(act="relu"), dict(residual=z(3, 32)),
               dict(scale=z(32, dt=torch.bfloat16))):
        args = dict(dict(weight=w), **kw)
        with pytest.raises(ValueError):
            ck.block_norm(y, **args)
    with pytest.raises(ValueError, match="GPU"):
        ck.block_norm(y, w)


@pytest.mark.parametrize("zeros", [0.0, 0.2])
def test_decay_reference_against_differences(zeros):
    """The reference's gradients (zero and negative gates among them) against
    central differences, exact for the gates (the loss is multilinear in them)."""
    rng = np.random.default_rng(0)
    B, T, Hk, H, dk, dv = 1, 9, 1, 2, 3, 4
    cu = np.array([0, 4, 4, 9])
    p = dict(q=rng.standard_normal((B, T, Hk, dk)), k=rng.standard_normal((B, T, Hk, dk)),
             v=rng.standard_normal((B, T, H, dv)), a=rng.uniform(-1, 1, (B, T, H)), h0=rng.standard_normal((3, H, dk, dv)))
    p["a"][rng.random(p["a"].shape) < zeros] = 0.0
    do, dht = rng.standard_normal((B, T, H, dv)), rng.standard_normal((3, H, dk, dv))

    def loss(p):
        o, ht = dref.fwd(p["q"], p["k"], p["v"], p["a"], p["h0"], cu, 0.7)[:2]
        return (o * do).sum() + (ht * dht).sum()

    got = dict(zip(("q", "k", "v", "a", "h0"), dref.bwd(p["q"], p["k"], p["v"], p["a"], do, p["h0"], dht, cu, 0.7)[0]))
    for name in got:
        for i in np.ndindex(p[name].shape):
            up, down = (dict(p, **{name: p[name].copy()}) for _ in (0, 1))
            up[name][i] += 1e-4
            down[name][i] -= 1e-4
            want = (loss(up) - loss(down)) / 2e-4
            assert abs(got[name][i] - want) < 1e-7 * max(1, abs(want)), (name, i)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_norm_reference_against_differences(act):
    rng = np.random.default_rng(1)
    p = {m: rng.standard_normal((3, 5)) for m in ("y", "g", "x")}
    p.update({m: 1 + 0.3 * rng.standard_normal(5) for m in ("w", "s", "w2")})
    dh, dn = rng.standard_normal((2, 3, 5))

    def loss(p):
        h, n = nref.fwd(p["y"], p["w"], p["g"], act, p["x"], p["s"], p["w2"], 1e-3)[0]
        return (h * dh).sum() + (n * dn).sum()

    got = nref.bwd(p["y"], p["w"], dh, dn, p["g"], act, p["x"], p["s"], p["w2"], 1e-3)[0]
    for name in p:
        for i in np.ndindex(p[name].shape):
            up, down = (dict(p, **{name: p[name].copy()}) for _ in (0, 1))
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            want = (loss(up) - loss(down)) / 2e-5
            assert abs(got["d" + name][i] - want) < 1e-7 * max(1, abs(want)), (name, i)


class FakeStream:
    """A stream to be current, without a GPU."""
    device = torch.device("cpu")

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch):
    """Two streams, the first current; what is allocated, with the stream that was
    current then; what is recorded; the streams that the library was given."""
    caller, other = FakeStream(1), FakeStream(2)
    log = dict(caller=caller, other=other, now=caller, made=[], recorded=[], launched=[])

    class current:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, log["now"] = log["now"], self.s

        def __exit__(self, *exc):
            log["now"] = self.before

    class Lib:  # the sizes from the library; calls are noted, nothing is launched
        def __getattr__(self, name):
            real = getattr(lib, name)
            if name.endswith("_size") or name.endswith("_supported"):
                return real
            return lambda *args: log["launched"].append((name, args[-1])) or 0

    def noting(make):
        def made(*args, **kw):
            t = make(*args, **kw)
            log["made"].append((t.data_ptr(), log["now"]))
            return t
        return made

    lib, fake = ck._load(), Lib()
    monkeypatch.setattr(ck, "_load", lambda: fake)
    monkeypatch.setattr(ck, "_tensors", lambda *a, **kw: None)
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: log["now"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log["recorded"].append((t.data_ptr(), s)))
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
    return log


def _calls():
    r = lambda *s: torch.ones(s)
    q, v, al, st = r(1, 1400, 2, 16), r(1, 1400, 4, 16), r(1, 1400, 4), r(3, 4, 16, 16)
    y, w = r(6, 32), r(32)
    return {"decay_fwd": (ck.decay_fwd, (q, q, v, al), {}),
            "decay_bwd": (ck.decay_bwd, (q, q, v, al, v), {}),
            "decay_step": (ck.decay_step, (r(3, 2, 16), r(3, 2, 16), r(3, 4, 16), r(3, 4), st), {}),
            "block_norm": (ck.block_norm, (y, w), dict(residual=y, next_weight=w)),
            "block_norm_bwd": (ck.block_norm_bwd, (y, w, y), dict(residual=y, dnext=y, next_weight=w))}


@pytest.mark.parametrize("name", ["decay_fwd", "decay_bwd", "decay_step", "block_norm", "block_norm_bwd"])
def test_a_given_stream_owns_what_the_call_allocates(streams, name):
    """The allocator hands a dropped workspace to the stream that it was allocated
    on: that has to be the stream that uses it."""
    fn, args, kw = _calls()[name]
    got = fn(*args, stream=streams["other"], **kw)
    assert [s for _, s in streams["launched"]] == [2] and streams["now"] is streams["caller"]
    assert streams["made"] and all(s is streams["other"] for _, s in streams["made"])
    for t in list(args) + [t for t in kw.values()]:
        assert (t.data_ptr(), streams["other"]) in streams["recorded"]
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            assert (t.data_ptr(), streams["caller"]) in streams["recorded"]


@pytest.mark.parametrize("name", ["decay_fwd", "decay_bwd", "decay_step", "block_norm", "block_norm_bwd"])
def test_no_stream_or_the_current_one(streams, name):
    fn, args, kw = _calls()[name]
    fn(*args, **kw)
    fn(*args, stream=streams["caller"], **kw)
    assert [s for _, s in streams["launched"]] == [1, 1] and not streams["recorded"]


def test_no_rows_are_zeroed_on_the_given_stream(streams, monkeypatch):
    on = []
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: on.append(streams["now"]) or t)
    e, w = torch.ones(0, 32), torch.ones(32)
    ck.block_norm_bwd(e, w, e, dnext=e, next_weight=w, stream=streams["other"])
    assert on and all(s is streams["other"] for s in on)


def test_a_stream_of_another_device_is_refused(streams):
    streams["other"].device = torch.device("meta")
    for fn, args, kw in _calls().values():
        with pytest.raises(ValueError, match="stream belongs to"):
            fn(*args, stream=streams["other"], **kw)
    assert not streams["launched"] and not streams["made"]


class Delta:
    """The delta rule's calls on ones (the device checks see a GPU's tensors)."""

    def __init__(self):
        r = lambda *s: torch.ones(s)
        q, v, a, b = r(1, 128, 2, 64), r(1, 128, 2, 64), r(1, 128, 2, 64), r(1, 128, 2)
        one = [t[0, :3].contiguous() for t in (q, q, v, a, b)]
        self.calls = {"chunk_fwd": (ck.chunk_fwd, (q, q, v, a, b)), "chunk_fwd_save": (ck.chunk_fwd_save, (q, q, v, a, b)),
                      "chunk_fwd_noalloc": (ck.chunk_fwd_noalloc, (q, q, v, a, b)),
                      "chunk_bwd": (ck.chunk_bwd, (q, q, v, a, b, v)),
                      "recurrent_step": (ck.recurrent_step, (*one, r(3, 2, 64, 64)))}
        self.inputs = (q, q, v, a, b)


@pytest.mark.parametrize("name", ["chunk_fwd", "chunk_fwd_save", "chunk_fwd_noalloc", "chunk_bwd", "recurrent_step", "plan"])
def test_a_given_stream_owns_what_the_delta_rule_calls_allocate(streams, monkeypatch, name):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    d = Delta()
    if name == "plan":
        plan = ck.ChunkFwdPlan(*d.inputs, stream=streams["other"])
        plan.prepare()
        args, got = d.inputs, plan.finish()
    else:
        fn, args = d.calls[name]
        got = fn(*args, stream=streams["other"])
    handles = [s.value if isinstance(s, ctypes.c_void_p) else s for _, s in streams["launched"]]
    assert set(handles) == {2} and streams["now"] is streams["caller"]
    assert streams["made"] and all(s is streams["other"] for _, s in streams["made"])
    for t in args:
        assert (t.data_ptr(), streams["other"]) in streams["recorded"]
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            assert (t.data_ptr(), streams["caller"]) in streams["recorded"]


def test_launches_of_two_to_the_32_threads_are_refused():
    """The last batch that fits passes the checks of sizes (and is refused for a
    NULL q behind them), the next one does not."""
    one = dict(T=1, H=1, qk_heads=1)

    def at(which, n, cu=None, **kw):
        return call(which, desc(B=n, num_seqs=n, **dict(one, **kw)), q=None)

    fits, over = (1, "q must not be NULL"), 2
    for which, n, kw in (("fwd", (1 << 32) // (768 * 2), {}), ("fwd", (1 << 32) // (512 * 4) - 1, dict(io_dtype=ck.F32)),
                         ("fwd", (1 << 32) // 768, dict(dk=64, dv=64, io_dtype=ck.F32)), ("fwd", (1 << 32) // 512 - 1, dict(dv=32)),
                         ("bwd", (1 << 32) // (512 * 2) - 1, {}), ("bwd", (1 << 32) // 256 - 1, dict(dv=24))):
        assert at(which, n, **kw) == fits, (which, n, kw)
        st, msg = at(which, n + 1, **kw)
        assert st == over and "too many" in msg, (which, n, kw)
    # the states' join of a cut batch: 16 workgroups of 256 a sequence and head
    for which in ("fwd", "bwd"):
        for n, want in (((1 << 20) - 1, 1), (1 << 20, 2)):
            assert call(which, desc(B=1, num_seqs=n, T=1 << 21, H=1, qk_heads=1), cu=CU, q=None)[0] == want
    for n, dk, dv, want in ((1 << 21, 128, 128, 2), ((1 << 21) - 1, 128, 128, 1), (1 << 21, 72, 104, 2),
                            (1 << 21, 64, 128, 1), (1 << 21, 128, 96, 1)):
        assert step(N=n, H=1, Hk=1, dk=dk, dv=dv, q=None)[0] == want, (n, dk, dv)


def test_sizes_past_32_bits_are_refused():
    """The descriptors hold 32-bit sizes: 2^32 + 64 tokens are not 64."""
    n = (1 << 32) + 64
    z = lambda *s: torch.zeros(1).expand(*s)
    for q, v, al in ((z(1, n, 1, 8), z(1, n, 1, 8), z(1)), (z(n, 1, 1, 8), z(n, 1, 1, 8), z(1)),
                     (z(1, 8, 1, n), z(1, 8, 1, 8), z(1)), (z(1, 8, 1, 8), z(1, 8, 1, n), z(1))):
        with pytest.raises(ValueError, match="below 2.31"):
            ck.decay_fwd(q, q, v, al)
        with pytest.raises(ValueError, match="below 2.31"):
            ck.decay_bwd(q, q, v, al, v)
    with pytest.raises(ValueError, match="below 2.31"):
        ck.decay_step(z(n, 1, 8), z(n, 1, 8), z(n, 1, 8), z(1), z(n, 1, 8, 8))
    with pytest.raises(ValueError, match="below 2.31"):
        ck.block_norm(z(2, n), z(n))
    with pytest.raises(ValueError, match="below 2.31"):
        ck.block_norm_bwd(z(2, n), z(n), z(2, n))
