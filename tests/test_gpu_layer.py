"""The decay attention and the block norms as a layer uses them together: a
block's forward and gradients against float64 and against differences, prefill
then decode against one prefill, and the calls a program makes around them --
other streams, captured graphs, shared buffers, tokens past the sequences."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests import decay_fp64 as dref
from tests import norm_fp64 as nref
from tests.gpu_util import DEV, announce, dev, host

pytestmark = pytest.mark.gpu

EPS = 1e-5


def layer_inputs(seed, B, T, H, dk, dv):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    d = H * dv
    return dict(x=f(B, T, d), q=f(B, T, H, dk), k=f(B, T, H, dk), g=f(B, T, H, dv),
                alpha=(1 / (1 + np.exp(-rng.normal(3, 1, (B, T, H))))).astype(np.float32),
                w0=(1 + 0.2 * f(d)), w1=(1 + 0.2 * f(dv)), w2=(1 + 0.2 * f(d)), s=(0.5 + 0.1 * f(d)),
                up=f(B, T, d), dn=f(B, T, d))


def layer_gpu(c, H, dv, scale):
    """x -> norm -> values -> decay attention -> gated head norm -> + residual -> norm."""
    B, T, d = c["x"].shape
    n0, _ = ck.block_norm(c["x"], c["w0"])
    v = n0.view(B, T, H, dv)
    o, _ = ck.decay_fwd(c["q"], c["k"], v, c["alpha"], gate="kda", scale=scale)
    y, _ = ck.block_norm(o, c["w1"], gate=c["g"])
    h, n = ck.block_norm(y.view(B, T, d), None, residual=c["x"], scale=c["s"], next_weight=c["w2"], eps=EPS)
    return dict(n0=n0, v=v, o=o, y=y, h=h, n=n)


def layer_gpu_bwd(c, f, H, dv, scale):
    B, T, d = c["x"].shape
    dy, _, _, dx, ds, dw2 = ck.block_norm_bwd(f["y"].view(B, T, d), None, c["up"], dnext=c["dn"],
                                              residual=c["x"], scale=c["s"], next_weight=c["w2"], eps=EPS)
    do, dw1, dg, _, _, _ = ck.block_norm_bwd(f["o"], c["w1"], dy.view(B, T, H, dv), gate=c["g"])
    dq, dk, dv_, da, _ = ck.decay_bwd(c["q"], c["k"], f["v"], c["alpha"], do, gate="kda", scale=scale)
    dx0, dw0 = ck.block_norm_bwd(c["x"], c["w0"], dv_.view(B, T, d))[:2]
    return dict(x=dx + dx0, q=dq, k=dk, alpha=da, g=dg, w0=dw0, w1=dw1, w2=dw2, s=ds)


def layer_ref(c, H, dv, scale):
    B, T, d = c["x"].shape
    flat = lambda z, m: z.reshape(-1, m)
    n0 = nref.fwd(flat(c["x"], d), c["w0"])[0][0].reshape(B, T, H, dv)
    o = dref.fwd(c["q"], c["k"], n0, c["alpha"], scale=scale)[0]
    y = nref.fwd(flat(o, dv), c["w1"], flat(c["g"], dv))[0][0].reshape(B, T, d)
    return nref.fwd(flat(y, d), None, x=flat(c["x"], d), s=c["s"], w2=c["w2"], eps=EPS)[0]


def test_layer_forward_and_gradients_against_differences():
    """A layer of all four calls in float32.  The forward is compared with the
    float64 one; its gradients with central differences of the float64 loss
    along random directions (the error of a difference with step 1e-6 in
    float64 is below 1e-8 of the terms).  The chain keeps float32's relative
    accuracy a call: 1e-4 is ten calls of 100 half steps each with room for
    the sums' cancellation."""
    B, T, H, dk, dv, scale = 2, 70, 2, 16, 24, 0.25
    c = layer_inputs(1, B, T, H, dk, dv)
    g = {m: dev(a) for m, a in c.items()}
    f = layer_gpu(g, H, dv, scale)
    rh, rn = layer_ref(c, H, dv, scale)
    for got, want in ((f["h"], rh), (f["n"], rn)):
        off = np.abs(host(got).reshape(want.shape) - want).max() / np.abs(want).max()
        assert off < 1e-5, off
    grads = layer_gpu_bwd(g, f, H, dv, scale)
    c64 = {m: a.astype(np.float64) for m, a in c.items()}

    def loss(p):
        h, n = layer_ref(p, H, dv, scale)
        d = p["x"].shape[-1]
        return float((h * c64["up"].reshape(-1, d)).sum() + (n * c64["dn"].reshape(-1, d)).sum())

    rng = np.random.default_rng(5)
    for name, got in grads.items():
        e = rng.standard_normal(c[name].shape)
        step = 1e-6
        up, down = (dict(c64, **{name: c64[name] + s * step * e}) for s in (1, -1))
        want = (loss(up) - loss(down)) / (2 * step)
        have = float((host(got).reshape(e.shape) * e).sum())
        size = float(np.abs(host(got).reshape(e.shape) * e).sum())
        announce("d%s: %.3g, differences %.3g" % (name, have, want))
        assert abs(have - want) <= 1e-4 * size + 1e-6 * abs(loss(c64)), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_then_decode_equals_one_prefill(dtype):
    """The states of a prefill, carried on token by token, give the outputs of
    a longer prefill: to float32's accuracy, or half a step of bf16 each way."""
    g = torch.Generator(device=DEV).manual_seed(3)
    N, T, H, Hk, dk, dv = 3, 90, 4, 2, 64, 48
    r = lambda *s: torch.randn(s, device=DEV, generator=g).to(dtype)
    q, k, v = r(N, T, Hk, dk), r(N, T, Hk, dk), r(N, T, H, dv)
    al = (r(N, T, H) + 3).contiguous()
    kw = dict(gates="logits", gate="kda", scale=0.1)
    o, ht = ck.decay_fwd(q, k, v, al, **kw)
    cut = 70
    c = lambda t: t[:, :cut].contiguous()
    o1, st = ck.decay_fwd(c(q), c(k), c(v), c(al), **kw)
    outs = [o1]
    for t in range(cut, T):
        at = lambda z: z[:, t].contiguous()
        outs.append(ck.decay_step(at(q), at(k), at(v), at(al), st, **kw)[:, None])
    o2 = torch.cat(outs, 1).float()
    tol = 1e-5 if dtype == torch.float32 else 2 ** -6
    assert ((o.float() - o2).abs().max() / o2.abs().max()).item() < tol
    assert ((ht - st).abs().max() / ht.abs().max()).item() < 1e-5


def case(seed, dtype=torch.bfloat16, B=2, T=150, H=4, Hk=2, dk=64, dv=64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, device=DEV, generator=g)
    return dict(q=r(B, T, Hk, dk).to(dtype), k=r(B, T, Hk, dk).to(dtype), v=r(B, T, H, dv).to(dtype),
                alpha=torch.sigmoid(r(B, T, H) + 3), dout=r(B, T, H, dv).to(dtype),
                h0=r(B, H, dk, dv), dht=r(B, H, dk, dv))


def grads(c):
    return ck.decay_bwd(c["q"], c["k"], c["v"], c["alpha"], c["dout"], h0=c["h0"], dht=c["dht"])


def test_same_inputs_give_the_same_bits():
    c = case(1)
    a, b = grads(c), grads(c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    head = dict(c, alpha=c["alpha"][0, 0].contiguous())
    assert torch.equal(grads(head)[3], grads(head)[3])


def test_calls_on_two_streams_at_once():
    """Each call has its own workspace, so calls on two streams may overlap."""
    cs = [case(s, T=700, B=1) for s in (1, 2)]
    want = [ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=c["h0"]) + grads(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=c["h0"]) + grads(c))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, g))


def test_explicit_stream_and_given_buffers():
    c = case(4)
    want_o, want_h = ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=c["h0"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, fin = torch.empty_like(c["v"]), c["h0"].clone()
    torch.cuda.synchronize()
    o, h = ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=fin, out=out, final_state=fin, stream=s)
    s.synchronize()
    assert o is out and h is fin and torch.equal(o, want_o) and torch.equal(h, want_h)


@pytest.mark.parametrize("T", [100, 1400])
def test_captured_graphs_replay_the_eager_results(T):
    """A training step and a decode step captured once, replayed over changed
    inputs with eager work between; two graphs, each with its own workspace."""
    c = case(5, T=T, B=1)
    x = torch.randn(64, 512, device=DEV).to(torch.bfloat16)
    w = torch.rand(512, device=DEV) + 0.5
    st = c["h0"].clone()

    def work():
        o, ht = ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=c["h0"])
        g = grads(c)
        h, n = ck.block_norm(x, w, residual=x, next_weight=w)
        b = ck.block_norm_bwd(x, w, h, dnext=n, residual=x, next_weight=w)
        t = lambda z: z[:, 0].contiguous()
        new = torch.empty_like(st)
        s = ck.decay_step(t(c["q"]), t(c["k"]), t(c["v"]), t(c["alpha"]), st, new_state=new)
        return [o, ht, h, n, s, new] + list(g) + [z for z in b if z is not None]

    work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured = []
    with torch.cuda.stream(side):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = work()
            captured.append((graph, out))
    torch.cuda.synchronize()
    for turn in range(4):
        for z in (c["q"], c["k"], c["v"], c["dout"], x):
            z.copy_(torch.randn(z.shape, device=DEV))
        want = work()
        torch.cuda.synchronize()
        for graph, out in captured:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, out)), turn


def test_tokens_past_the_sequences_are_left_alone():
    g = torch.Generator(device=DEV).manual_seed(6)
    T, used, H, d = 200, 130, 2, 64
    r = lambda *s: torch.randn(s, device=DEV, generator=g)
    q, k, v = r(1, T, H, d), r(1, T, H, d), r(1, T, H, d)
    al = torch.sigmoid(r(1, T, H) + 2)
    for t in (q, k, v, al):
        t[:, used:] = float("nan")
    cu = torch.tensor([0, 0, 65, used], device=DEV, dtype=torch.int32)
    out = torch.full_like(v, 7.0)
    o, ht = ck.decay_fwd(q, k, v, al, cu_seqlens=cu, out=out)
    assert (o[:, used:] == 7).all() and torch.isfinite(o[:, :used]).all() and torch.isfinite(ht).all()
    cut = lambda t: t[:, :used].contiguous()
    o2, ht2 = ck.decay_fwd(cut(q), cut(k), cut(v), cut(al), cu_seqlens=cu)
    assert torch.equal(o[:, :used], o2) and torch.equal(ht, ht2)
    do = r(1, T, H, d)
    gr = ck.decay_bwd(q, k, v, al, do, cu_seqlens=cu)
    gr2 = ck.decay_bwd(cut(q), cut(k), cut(v), cut(al), cut(do), cu_seqlens=cu)
    for a, b in zip(gr[:4], gr2[:4]):
        assert torch.equal(a[:, :used], b)
    one = ck.decay_bwd(q, k, v, torch.full((H,), 0.9, device=DEV), do, cu_seqlens=cu)[3]
    assert torch.isfinite(one).all()


def test_nan_stays_in_its_sequence_and_block():
    """A NaN reaches its own block of 64 tokens, later tokens of its sequence
    and no other sequence (gradients: blocks of 64 in bf16, earlier ones too)."""
    c = case(7, B=1, T=400)
    c["h0"] = c["dht"] = None
    cu = torch.tensor([0, 150, 400], device=DEV, dtype=torch.int32)
    c["v"][0, 150 + 70] = float("nan")
    o, ht = ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], cu_seqlens=cu)
    assert torch.isfinite(o[0, :150 + 64]).all() and torch.isfinite(ht[0]).all()
    assert torch.isnan(o[0, 150 + 70:]).all()
    g = ck.decay_bwd(c["q"], c["k"], c["v"], c["alpha"], c["dout"], cu_seqlens=cu)
    assert all(torch.isfinite(t[0, :150]).all() for t in g[:4])


def test_state_beyond_two_to_the_31_elements():
    """A decode batch whose states pass 2^31 elements, in place, at its ends."""
    N, H, d = 16400, 8, 128
    g = torch.Generator(device=DEV).manual_seed(8)
    st = torch.empty((N, H, d, d), device=DEV).normal_(generator=g)
    q, k, v = (torch.randn((N, H, d), device=DEV, generator=g).to(torch.bfloat16) for _ in range(3))
    al = torch.rand((N, H), device=DEV, generator=g)
    pick = [0, 1, 8191, 16383, 16399]
    before = st[pick].clone()
    o = ck.decay_step(q, k, v, al, st)
    want = al[pick][..., None, None].double() * before.double() + k[pick].double()[..., None] * v[pick].double()[..., None, :]
    assert (st[pick].double() - want).abs().max().item() <= 4 * 2.0 ** -24 * want.abs().max().item() * 2
    ref = (want * q[pick].double()[..., None]).sum(-2)
    assert (o[pick].double() - ref).abs().max().item() <= (2 ** -8 + 1e-4) * ref.abs().max().item()


def test_many_tokens_at_the_far_end():
    """Offsets past 2^31 elements: the last sequence of a long batch equals the
    same sequence alone."""
    B, T, H, d = 260, 4160, 16, 128
    g = torch.Generator(device=DEV).manual_seed(9)
    q, k, v = (torch.randn((B, T, H, d), device=DEV, generator=g, dtype=torch.bfloat16) for _ in range(3))
    al = torch.rand((B, T, H), device=DEV, generator=g)
    assert q.numel() > 2 ** 31
    o, ht = ck.decay_fwd(q, k, v, al, scale=0.1)
    one = lambda t: t[-1:].contiguous()
    o1, h1 = ck.decay_fwd(one(q), one(k), one(v), one(al), scale=0.1)
    # the short batch is cut into segments, the long one is not
    assert ((o[-1:].float() - o1.float()).abs().max() / o1.abs().max().float()).item() < 2 ** -6
    assert ((ht[-1:] - h1).abs().max() / h1.abs().max()).item() < 1e-5


def test_calls_on_given_streams_keep_their_workspaces():
    """Calls sent to two streams from one current stream, which goes on
    allocating and writing: each call's workspace is its own until it ends."""
    cs = [case(s, T=2000, B=1, H=8, Hk=4, dk=128, dv=128) for s in (11, 12)]
    x = [torch.randn(4000, 512, device=DEV) for _ in cs]
    w = torch.rand(512, device=DEV) + 0.5

    def work(c, x, **on):
        o = ck.decay_fwd(c["q"], c["k"], c["v"], c["alpha"], h0=c["h0"], **on)
        g = ck.decay_bwd(c["q"], c["k"], c["v"], c["alpha"], c["dout"], h0=c["h0"], dht=c["dht"], **on)
        n = ck.block_norm_bwd(x, w, x, dnext=x, residual=x, next_weight=w, **on)
        return o + g + tuple(t for t in n if t is not None)

    want = [work(c, y) for c, y in zip(cs, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = []
        for c, y, s in zip(cs, x, streams):
            got.append(work(c, y, stream=s))
            junk = [torch.full((n,), float("nan"), device=DEV) for n in (1 << 10, 1 << 18, 1 << 20, 1 << 23)]
            del junk
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_delta_rule_calls_on_given_streams_keep_their_workspaces():
    """The same of the delta rule's calls."""
    g = torch.Generator(device=DEV).manual_seed(13)
    r = lambda *s: torch.randn(s, device=DEV, generator=g)

    def inputs():
        q, k, v, do = (r(1, 2000, 8, 64).to(torch.bfloat16) for _ in range(4))
        return q, k, v, torch.sigmoid(r(1, 2000, 8, 64) + 4), torch.sigmoid(r(1, 2000, 8)), do

    def work(c, **on):
        kw = dict(gate="kda", scale=0.125, **on)
        o = ck.chunk_fwd(*c[:5], **kw)
        plan = ck.ChunkFwdPlan(*c[:5], **kw)
        plan.prepare()
        return o + plan.finish() + ck.chunk_bwd(*c, **kw)

    cs = [inputs() for _ in range(2)]
    want = [work(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = []
        for c, s in zip(cs, streams):
            got.append(work(c, stream=s))
            junk = [torch.full((n,), float("nan"), device=DEV) for n in (1 << 10, 1 << 18, 1 << 20, 1 << 23)]
            del junk
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
