"""The scan, convolution and layer norm calls reject bad arguments on the host
before any HIP call (dummy, never-dereferenced pointers; no GPU is touched), and
the binding before the library; the float64 references behind the parity tests
against differences."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests import scan_fp64 as ref
from tests.test_layer_abi_cpu import streams  # noqa: F401  (a fixture)

BASE = 0x7F0000000000
GAP = 1 << 34


def pointers(names):
    return {n: ctypes.c_void_p(BASE + i * GAP) for i, n in enumerate(names.split())}


SCAN = "x dt A B C D z bias cu h0 y ht ws dy dht dx ddt dA dB dC dD dz dbias dh0"
CONV = "x w bias cu h0 y ht dy dht dx dw dbias dh0 ws"
NORM = "x r w b n h dn dh dx dw db ws"


def scan_desc(**kw):
    d = dict(B=2, T=64, D=128, S=16, groups=2, num_seqs=2, io_dtype=ck.BF16, softplus=1, x_stride=0, dt_stride=0,
             z_stride=0, b_stride=0, c_stride=0)
    d.update(kw)
    return ck.ScanDesc(**d)


def scan(which, d, packed=False, bytes_=1 << 34, **over):
    p = dict(pointers(SCAN), **over)
    cu = p["cu"] if packed else None
    lib, r = ck._load(), None if d is None else ctypes.byref(d)
    if which == "fwd":
        args = [p[m] for m in "x dt A B C D z bias".split()] + [cu] + [p[m] for m in "h0 y ht ws".split()]
        st = lib.ckda_scan_fwd(r, *args, bytes_, None)
    elif which == "bwd":
        args = [p[m] for m in "x dt A B C D z bias".split()] + [cu]
        args += [p[m] for m in "h0 dy dht dx ddt dA dB dC dD dz dbias dh0 ws".split()]
        st = lib.ckda_scan_bwd(r, *args, bytes_, None)
    else:
        st = lib.ckda_scan_step(r, *[p[m] for m in "x dt A B C D z bias h0 ht y".split()], None)
    return st, lib.ckda_last_error().decode()


def conv_desc(**kw):
    d = dict(B=2, T=64, D=128, K=4, num_seqs=2, io_dtype=ck.BF16, act=2, x_stride=0)
    d.update(kw)
    return ck.ConvDesc(**d)


def conv(which, d, packed=False, bytes_=1 << 34, **over):
    p = dict(pointers(CONV), **over)
    cu = p["cu"] if packed else None
    lib, r = ck._load(), None if d is None else ctypes.byref(d)
    if which == "fwd":
        st = lib.ckda_conv_fwd(r, p["x"], p["w"], p["bias"], cu, p["h0"], p["y"], p["ht"], None)
    elif which == "bwd":
        st = lib.ckda_conv_bwd(r, p["x"], p["w"], p["bias"], cu, p["h0"], p["dy"], p["dht"], p["dx"], p["dw"],
                               p["dbias"], p["dh0"], p["ws"], bytes_, None)
    else:
        st = lib.ckda_conv_step(r, p["x"], p["w"], p["bias"], p["h0"], p["ht"], p["y"], None)
    return st, lib.ckda_last_error().decode()


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("over,status,needle", [
    (dict(B=0), 1, "non-positive"), (dict(T=-1), 1, "non-positive"), (dict(D=0), 1, "non-positive"),
    (dict(S=0), 1, "non-positive"), (dict(num_seqs=-1), 1, "non-positive"), (dict(num_seqs=3), 1, "num_seqs"),
    (dict(groups=0), 1, "groups"), (dict(groups=3), 1, "groups"), (dict(softplus=2), 1, "softplus"),
    (dict(io_dtype=2), 1, "io_dtype"), (dict(S=65), 2, "S=65"), (dict(D=(1 << 20) + 2), 2, "2^20"),
    (dict(x_stride=127), 1, "stride"), (dict(dt_stride=-5), 1, "stride"), (dict(z_stride=1), 1, "stride"),
    (dict(b_stride=31), 1, "stride"), (dict(c_stride=31), 1, "stride"), (dict(x_stride=1 << 24), 2, "2^24"),
    (dict(T=1 << 30), 2, "too many"), (dict(B=1 << 16, num_seqs=1 << 16, T=1 << 15), 2, "too many"),
    (dict(B=1 << 20, num_seqs=1 << 20, T=1, D=1 << 18), 2, "too many"),
])
def test_scan_rejects_bad_descriptors(which, over, status, needle):
    st, msg = scan(which, scan_desc(**over))
    assert st == status and needle in msg, msg
    assert ck._load().ckda_scan_bwd_workspace_size(ctypes.byref(scan_desc(**over)), 0) == 0


def test_scan_null_alignment_overlap():
    assert scan("fwd", None)[0] == 1
    for m in ("x", "dt", "A", "B", "C", "y"):
        st, msg = scan("fwd", scan_desc(), **{m: None})
        assert st == 1 and m + " must not be NULL" in msg
    p = pointers(SCAN)
    at = lambda m, off: ctypes.c_void_p(p[m].value + off)
    assert "2-byte aligned" in scan("fwd", scan_desc(), x=at("x", 1))[1]
    assert "16-byte aligned" in scan("fwd", scan_desc(), A=at("A", 8))[1]
    assert "4-byte aligned" in scan("fwd", scan_desc(io_dtype=ck.F32), B=at("B", 2))[1]
    for m in ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0"):
        st, msg = scan("fwd", scan_desc(), y=p[m])
        assert st == 1 and "overlaps" in msg, m
    assert scan("fwd", scan_desc(T=0), x=None, dt=None, B=None, C=None, z=None, y=None, h0=None, ht=None,
                packed=False, A=None)[0] == 1
    st, msg = scan("fwd", scan_desc(), ht=at("h0", 64))
    assert st == 1 and "overlaps" in msg
    # the rows of a strided x reach further than its elements
    wide = scan_desc(x_stride=1 << 16)
    assert "y overlaps x" in scan("fwd", wide, y=at("x", (2 * 64 - 1) * (1 << 17)))[1]
    one = dict(B=1, num_seqs=3)
    assert "cu_seqlens" in scan("fwd", scan_desc(), packed=True)[1]
    assert "overlaps cu_seqlens" in scan("fwd", scan_desc(**one), packed=True, y=p["cu"])[1]
    assert "not 4-byte" in scan("fwd", scan_desc(**one), packed=True, cu=at("cu", 2))[1]
    for m in ("dx", "ddt", "dA", "dB", "dC"):
        st, msg = scan("bwd", scan_desc(), **{m: None})
        assert st == 1 and m in msg, msg
        st, msg = scan("bwd", scan_desc(), **{m: p["dy"]})
        assert st == 1 and "overlaps" in msg, msg
    for given, grad in (("z", "dz"), ("D", "dD"), ("bias", "dbias")):
        for m in (given, grad):
            st, msg = scan("bwd", scan_desc(), **{m: None})
            assert st == 1 and "exactly" in msg, msg
    assert "overlaps" in scan("bwd", scan_desc(), dh0=p["dht"])[1]


def test_scan_workspaces():
    lib = ck._load()
    d = scan_desc(B=1, num_seqs=1, T=100000)
    need = lib.ckda_scan_fwd_workspace_size(ctypes.byref(d), 0)
    assert need > 0
    assert scan("fwd", d, bytes_=need - 1) == (3, "workspace has %d bytes, %d needed" % (need - 1, need))
    assert scan("fwd", d, ws=None)[0] == 1
    p = pointers(SCAN)
    assert "256-byte" in scan("fwd", d, ws=ctypes.c_void_p(p["ws"].value + 16))[1]
    assert "workspace overlaps dt" in scan("fwd", d, ws=p["dt"])[1]
    assert lib.ckda_scan_fwd_workspace_size(ctypes.byref(scan_desc(T=200)), 0) == 0
    need = lib.ckda_scan_bwd_workspace_size(ctypes.byref(scan_desc()), 0)
    assert need >= 2 * 4 * 128 * 16 * 4  # a state every 16 tokens
    assert scan("bwd", scan_desc(), bytes_=need - 1)[0] == 3
    assert lib.ckda_scan_bwd_workspace_size(None, 0) == 0
    lib.ckda_scan_fwd(None, *[None] * 13, 0, None)
    kept = lib.ckda_last_error()
    lib.ckda_scan_bwd_workspace_size(ctypes.byref(scan_desc(S=70)), 0)
    assert lib.ckda_last_error() == kept != b""


def test_step_rejections():
    one = dict(B=3, num_seqs=3, T=1)
    assert scan("step", scan_desc(B=0, num_seqs=0, T=1))[0] == 0
    p = pointers(SCAN)
    for kw, over, status in ((dict(one, T=2), {}, 1), (dict(one, S=70), {}, 2), (one, dict(h0=None), 1), (one, dict(ht=None), 1),
                             (one, dict(x=None), 1), (one, dict(y=p["z"]), 1), (one, dict(ht=p["A"]), 1),
                             (one, dict(ht=ctypes.c_void_p(p["h0"].value + 16)), 1),
                             (dict(B=1 << 16, num_seqs=1 << 16, T=1, D=1 << 12, S=16), {}, 2),
                             (dict(B=1 << 13, num_seqs=1 << 13, T=1, D=1 << 19, S=1, groups=1), dict(x=None), 2)):
        assert scan("step", scan_desc(**kw), **over)[0] == status, (kw, over)
    one = dict(B=3, num_seqs=3, T=1)
    assert conv("step", conv_desc(B=0, num_seqs=0, T=1))[0] == 0
    p = pointers(CONV)
    for kw, over, status in ((dict(one, T=2), {}, 1), (dict(one, K=5), {}, 2), (one, dict(h0=None), 1), (one, dict(w=None), 1),
                             (one, dict(y=p["x"]), 1), (one, dict(ht=ctypes.c_void_p(p["h0"].value + 16)), 1)):
        assert conv("step", conv_desc(**kw), **over)[0] == status, (kw, over)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("over,status,needle", [
    (dict(B=0), 1, "non-positive"), (dict(T=-1), 1, "non-positive"), (dict(D=0), 1, "non-positive"),
    (dict(K=0), 1, "non-positive"), (dict(K=1), 2, "K=1"), (dict(K=5), 2, "K=5"), (dict(act=1), 1, "act"),
    (dict(io_dtype=9), 1, "io_dtype"), (dict(num_seqs=5), 1, "num_seqs"), (dict(x_stride=127), 1, "x_stride"),
    (dict(x_stride=1 << 24), 2, "2^24"), (dict(D=(1 << 22) + 4), 2, "2^22"), (dict(T=1 << 30), 2, "too many"),
    (dict(B=1 << 12, num_seqs=1 << 12, T=1 << 18, D=1 << 14), 2, "too many"),
])
def test_conv_rejects_bad_descriptors(which, over, status, needle):
    st, msg = conv(which, conv_desc(**over))
    assert st == status and needle in msg, msg


def test_conv_null_alignment_overlap_workspace():
    p = pointers(CONV)
    at = lambda m, off: ctypes.c_void_p(p[m].value + off)
    assert conv("fwd", None)[0] == 1
    for m in ("x", "w", "y"):
        assert m + " must not be NULL" in conv("fwd", conv_desc(), **{m: None})[1]
    assert "2-byte aligned" in conv("fwd", conv_desc(), x=at("x", 1))[1]
    assert "16-byte aligned" in conv("fwd", conv_desc(), y=at("y", 2))[1]
    for m in ("x", "w", "bias", "h0"):
        assert "overlaps" in conv("fwd", conv_desc(), y=p[m])[1]
    assert "overlaps" in conv("fwd", conv_desc(), ht=at("h0", 64))[1]
    assert "overlaps cu_seqlens" in conv("fwd", conv_desc(B=1, num_seqs=4), packed=True, y=p["cu"])[1]
    for m in ("dy", "dx", "dw"):
        assert m in conv("bwd", conv_desc(), **{m: None})[1]
    for m in ("dx", "dw", "dbias", "dh0"):
        assert "overlaps" in conv("bwd", conv_desc(), **{m: p["x"]})[1]
    need = ck._load().ckda_conv_bwd_workspace_size(ctypes.byref(conv_desc()), 0)
    assert need >= 5 * 128 * 4
    assert conv("bwd", conv_desc(), bytes_=need - 1)[0] == 3
    assert "256-byte" in conv("bwd", conv_desc(), ws=at("ws", 16))[1]
    # a long packed batch of many sequences is no product of both
    assert conv("fwd", conv_desc(B=1, T=1 << 20, num_seqs=1 << 20, D=8), packed=True, x=None)[1] == "x must not be NULL"


def norm(rows=4, d=64, io=ck.BF16, eps=1e-5, **over):
    p = dict(pointers(NORM), **over)
    lib = ck._load()
    st = lib.ckda_layer_norm(rows, d, io, eps, *[p[m] for m in "x r w b n h".split()], None)
    return st, lib.ckda_last_error().decode()


def norm_bwd(rows=4, d=64, io=ck.BF16, eps=1e-5, bytes_=1 << 34, **over):
    p = dict(pointers(NORM), **over)
    lib = ck._load()
    st = lib.ckda_layer_norm_bwd(rows, d, io, eps, *[p[m] for m in "x w dn dh dx dw db ws".split()], bytes_, None)
    return st, lib.ckda_last_error().decode()


def test_layer_norm_rejections():
    p = pointers(NORM)
    assert norm(rows=0)[0] == 0
    for kw, status in ((dict(rows=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(io=7), 1), (dict(eps=-1.0), 1),
                       (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(n=None), 1), (dict(h=None), 1), (dict(r=None), 1),
                       (dict(n=p["x"]), 1), (dict(n=p["h"]), 1), (dict(h=p["w"]), 1),
                       (dict(h=ctypes.c_void_p(p["r"].value + 128)), 1), (dict(h=ctypes.c_void_p(p["x"].value + 128)), 1),
                       (dict(x=ctypes.c_void_p(p["x"].value + 2)), 1), (dict(rows=1 << 45), 2)):
        assert norm(**kw)[0] == status, kw
    for kw, status in ((dict(rows=0), 1), (dict(d=16385), 2), (dict(w=None), 1), (dict(dw=None), 1), (dict(dx=p["dn"]), 1),
                       (dict(dx=p["dh"]), 1), (dict(db=p["dw"]), 1), (dict(dn=None), 1), (dict(ws=None), 1), (dict(bytes_=10), 3)):
        assert norm_bwd(**kw)[0] == status, kw
    assert ck._load().ckda_layer_norm_bwd_workspace_size(0, 64, 0) == 0
    assert ck._load().ckda_layer_norm_bwd_workspace_size(5, 64, 9) == 0


# ---- the binding

def _args(N=2, T=8, D=6, S=4, G=2, t=torch.float32):
    r = lambda *s: torch.ones(s, dtype=t)
    return dict(x=r(N, T, D), dt=r(N, T, D), A=torch.ones(D, S), B=r(N, T, G, S), C=r(N, T, G, S))


def test_binding_rejections(monkeypatch):
    good = _args()
    with pytest.raises(ValueError, match="on a GPU"):
        ck.scan_fwd(**good)
    with pytest.raises(ValueError, match="on a GPU"):
        ck.conv_fwd(torch.ones(2, 8, 6), torch.ones(6, 4))
    with pytest.raises(ValueError, match="on a GPU"):
        ck.layer_norm(torch.ones(2, 6), torch.ones(6))
    one = dict(steps="logits")
    for bad, kind, match in (
            (dict(dt=good["dt"][:, :4]), ValueError, "dt must"), (dict(dt=good["dt"].bfloat16()), ValueError, "dt must"),
            (dict(x=good["x"].double()), TypeError, "bfloat16 or float32"), (dict(A=good["A"].bfloat16()), ValueError, "A must"),
            (dict(A=torch.ones(5, 4)), ValueError, "A must"), (dict(B=good["B"][..., :3]), ValueError, "B must"),
            (dict(C=good["C"][:, :, :1]), ValueError, "C must"), (dict(z=good["x"][0]), ValueError, "z must"),
            (dict(D=torch.ones(5)), ValueError, "D must"), (dict(dt_bias=torch.ones(6).bfloat16()), ValueError, "dt_bias must"),
            (dict(steps="gates"), ValueError, "steps must"), (dict(cu_seqlens=torch.zeros(3)), ValueError, "cu_seqlens"),
            (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError, "B = 1"),
            (dict(B=torch.ones(2, 8, 4, 4), C=torch.ones(2, 8, 4, 4)), ValueError, "groups must divide")):
        with pytest.raises(kind, match=match):
            ck.scan_fwd(**dict(good, **dict(one, **bad)))
        with pytest.raises(kind, match=match):
            ck.scan_bwd(**dict(good, dout=good["x"], **dict(one, **bad)))
    x, w = torch.ones(2, 8, 6), torch.ones(6, 4)
    for a, kw, match in (((x, w.bfloat16()), {}, "weight must"), ((x, torch.ones(5, 4)), {}, "weight must"),
                         ((x, w), dict(act="sigmoid"), "act must"), ((x, w), dict(bias=torch.ones(5)), "bias must"),
                         ((x[0], w), {}, "x must")):
        with pytest.raises(ValueError, match=match):
            ck.conv_fwd(*a, **kw)
    monkeypatch.setattr(ck, "_on", lambda *a: None)
    monkeypatch.setattr(ck, "_tensors", lambda *a, **kw: None)
    for kw, match in ((dict(h0=torch.ones(2, 6, 5)), "h0 must"), (dict(h0=torch.ones(2, 6, 4).bfloat16()), "h0 must"),
                      (dict(final_state=torch.ones(1, 6, 4)), "final_state must"), (dict(out=good["x"].bfloat16()), "out must")):
        with pytest.raises(ValueError, match=match):
            ck.scan_fwd(**good, **kw)
    for kw, match in ((dict(h0=torch.ones(2, 2, 6)), "h0 must"), (dict(out=torch.ones(2, 8, 5)), "out must")):
        with pytest.raises(ValueError, match=match):
            ck.conv_fwd(x, w, **kw)
    with pytest.raises(ValueError, match="residual_out needs"):
        ck.layer_norm(torch.ones(2, 6), None, residual_out=torch.ones(2, 6))
    with pytest.raises(ValueError, match="must match"):
        ck.layer_norm_bwd(torch.ones(2, 6), None, torch.ones(2, 5))


def test_row_strides():
    s = ck._row_stride
    x = torch.ones(3, 5, 12)
    assert s("x", x, 2, 12) == 12 and s("x", x[..., 2:6], 2, 4) == 12
    with pytest.raises(ValueError, match="one distance"):
        s("x", x[:, 1:, :4], 2, 4)
    with pytest.raises(ValueError, match="one distance"):
        s("x", x.transpose(0, 1)[..., :4], 2, 4)
    with pytest.raises(ValueError, match="contiguous within"):
        s("x", x[..., ::2], 2, 6)
    with pytest.raises(ValueError, match="overlap"):
        s("x", torch.ones(1, 1, 4).expand(3, 5, 4), 2, 4)
    with pytest.raises(ValueError, match="overlap"):
        s("x", torch.as_strided(torch.ones(40), (9, 4), (2, 1)), 1, 4)
    # single tokens and sequences have no distance of their own
    assert s("x", x[:1, :, :4], 2, 4) == 12 and s("x", x[:, :1, :4], 2, 4) == 60 and s("x", x[:1, :1, :4], 2, 4) == 4
    assert s("B", torch.ones(3, 5, 20)[..., 4:12].unflatten(-1, (2, 4)), 2, 8) == 20
    with pytest.raises(ValueError, match="contiguous within"):
        s("B", torch.ones(3, 5, 2, 8)[..., :4], 2, 8)
    assert s("x", torch.ones(0, 5, 12)[..., :4], 2, 4) == 4


def test_sizes_past_32_bits_are_refused():
    n = (1 << 32) + 64
    z = lambda *s: torch.zeros(1).expand(*s)
    with pytest.raises(ValueError):
        ck.conv_fwd(z(1, n, 4), torch.ones(4, 4))
    with pytest.raises(ValueError):
        ck.scan_step(z(n, 4), z(n, 4), torch.ones(4, 4), z(n, 4), z(n, 4), z(n, 4, 4))
    with pytest.raises(ValueError, match="below 2.31"):
        ck.layer_norm(z(2, n), z(n))


def _calls():
    r = lambda *s: torch.ones(s)
    a = _args(1, 1400, 16, 4, 2)
    one = {m: a[m][0, :3] for m in ("x", "dt", "B", "C")}
    A = a["A"]
    x, w = r(1, 1400, 16), r(16, 4)
    y, wn = r(6, 32), r(32)
    return {"scan_fwd": (ck.scan_fwd, (a["x"], a["dt"], A, a["B"], a["C"]), dict(z=a["x"])),
            "scan_bwd": (ck.scan_bwd, (a["x"], a["dt"], A, a["B"], a["C"], a["x"]), dict(D=r(16), dt_bias=r(16))),
            "scan_step": (ck.scan_step, (one["x"], one["dt"], A, one["B"], one["C"], r(3, 16, 4)), {}),
            "conv_fwd": (ck.conv_fwd, (x, w), dict(bias=r(16))), "conv_bwd": (ck.conv_bwd, (x, w, x), dict(bias=r(16))),
            "conv_step": (ck.conv_step, (r(3, 16), w, r(3, 3, 16)), {}),
            "layer_norm": (ck.layer_norm, (y, wn, wn), dict(residual=y)),
            "layer_norm_bwd": (ck.layer_norm_bwd, (y, wn, y), dict(dh=y))}


@pytest.fixture
def ssm_streams(streams, monkeypatch):  # noqa: F811
    monkeypatch.setattr(ck, "_on", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: streams["now"].cuda_stream, raising=False)
    return streams


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_given_stream_owns_what_the_call_allocates(ssm_streams, name):
    fn, args, kw = _calls()[name]
    got = fn(*args, stream=ssm_streams["other"], **kw)
    assert [s for _, s in ssm_streams["launched"]] == [2] and ssm_streams["now"] is ssm_streams["caller"]
    assert ssm_streams["made"] and all(s is ssm_streams["other"] for _, s in ssm_streams["made"])
    for t in list(args) + [t for t in kw.values()]:
        assert (t.data_ptr(), ssm_streams["other"]) in ssm_streams["recorded"]
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            assert (t.data_ptr(), ssm_streams["caller"]) in ssm_streams["recorded"]


@pytest.mark.parametrize("name", sorted(_calls()))
def test_no_stream_or_the_current_one(ssm_streams, monkeypatch, name):
    fn, args, kw = _calls()[name]
    fn(*args, **kw)
    fn(*args, stream=ssm_streams["caller"], **kw)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)  # by a Stream object
    fn(*args, **kw)
    assert [s for _, s in ssm_streams["launched"]] == [1, 1, 1] and not ssm_streams["recorded"]


# ---- the float64 references against differences

def _difference(f, x, i, step=1e-6):
    """The difference quotient of f's value, and how far off it may be: 1e-6 of it for
    the terms past the first, and f's own rounding.  The references' bounds hold for
    arithmetic with steps of EPS = 2^-24, so in float64 each of the two losses is off
    by their 2^-29th part at most, and the quotient by that over the step."""
    a, b = x.copy(), x.copy()
    a.flat[i] += step
    b.flat[i] -= step
    (fa, ea), (fb, eb) = f(a), f(b)
    d = (fa - fb) / (2 * step)
    return d, 1e-6 * (1 + abs(d)) + (ea + eb) * 2.0 ** -29 / (2 * step)


def _loss(*terms):
    """The sum of (value, bound) pairs' products with weights, and its bound."""
    return (sum((v * w).sum() for (v, _), w in terms), sum(((e + ref.EPS * np.abs(v)) * np.abs(w)).sum() for (v, e), w in terms))


def test_scan_reference_gradients_are_differences():
    rng = np.random.default_rng(1)
    T, D, S, G = 7, 4, 3, 2
    n = lambda *s: rng.standard_normal(s)
    c = dict(x=n(T, D), dt=n(T, D) - 1, A=-np.exp(n(D, S)), B=n(T, G, S), C=n(T, G, S), D=n(D), z=n(T, D), bias=n(D), h0=n(D, S))
    dy, dht = n(T, D), n(D, S)
    for kw in (dict(softplus=True), dict(softplus=False)):
        r = ref.scan(**c, dy=dy, dht=dht, **kw)
        names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", bias="dbias", h0="dh0")
        for m, g in names.items():
            def loss(v, m=m):
                o = ref.scan(**dict(c, **{m: v}), **kw)
                return _loss((o["y"], dy), (o["ht"], dht))
            for i in rng.choice(c[m].size, 4):
                d, off = _difference(loss, c[m], i)
                assert abs(d - r[g][0].flat[i]) < off, (m, kw)


def test_conv_reference_gradients_are_differences():
    rng = np.random.default_rng(2)
    n = lambda *s: rng.standard_normal(s)
    for T, K in ((6, 4), (2, 4), (1, 3), (5, 2)):
        c = dict(x=n(T, 3), w=n(3, K), bias=n(3), h0=n(K - 1, 3))
        dy, dht = n(T, 3), n(K - 1, 3)
        for act in ("silu", "none"):
            r = ref.conv(**c, act=act, dy=dy, dht=dht)
            for m, g in dict(x="dx", w="dw", bias="dbias", h0="dh0").items():
                def loss(v, m=m):
                    o = ref.conv(**dict(c, **{m: v}), act=act)
                    return _loss((o["y"], dy), (o["ht"], dht))
                for i in range(c[m].size):
                    d, off = _difference(loss, c[m], i)
                    assert abs(d - r[g][0].flat[i]) < off, (m, act, T, K)


def test_layer_norm_reference_gradients_are_differences():
    rng = np.random.default_rng(3)
    n = lambda *s: rng.standard_normal(s)
    c = dict(x=n(3, 9), w=n(9), b=n(9))
    dn, dh = n(3, 9), n(3, 9)
    r = ref.layer_norm(**c, dn=dn, dh=dh)
    for m, g in dict(x="dx", w="dw", b="db").items():
        def loss(v, m=m):
            o = ref.layer_norm(**dict(c, **{m: v}))
            return _loss((o["n"], dn), (o["h"], dh))
        for i in range(c[m].size):
            d, off = _difference(loss, c[m], i)
            assert abs(d - r[g][0].flat[i]) < off, m
