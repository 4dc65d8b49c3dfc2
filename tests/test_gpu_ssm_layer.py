"""The selective scan, its convolution and layer norm together, as a layer of a
model runs them: the residual norm, a projection whose halves are x and z, the
convolution, a projection to steps, B and C, the scan; a prompt, its gradients,
tokens after it; on another stream, in graphs, and two calls at once."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from tests.gpu_util import announce, max_rel_err
from tests.ssm_util import make_scan, scan_kw, scan_tensors

pytestmark = pytest.mark.gpu

D, INNER, S, R, K = 32, 48, 16, 4, 4


def weights(seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(s, device="cuda", generator=g) * std
    w = dict(norm=1 + 0.2 * r(D), normb=0.1 * r(D), win=r(D, 2 * INNER, std=D ** -0.5), conv=r(INNER, K, std=0.5),
             convb=0.1 * r(INNER), wx=r(INNER, R + 2 * S, std=INNER ** -0.5), wdt=r(R, INNER, std=R ** -0.5),
             dtb=r(INNER) - 3, A=-torch.arange(1, S + 1, device="cuda").float().expand(INNER, S).contiguous(),
             skip=1 + 0.1 * r(INNER))
    for m in ("win", "wx", "wdt"):
        w[m] = w[m].to(dtype)
    return w


def prompt(w, x, res, conv0, h0, cu=None):
    """Every value of the layer's forward."""
    v = dict(x=x, res=res, conv0=conv0, h0=h0, cu=cu)
    v["n"], v["h"] = ck.layer_norm(x, w["norm"], w["normb"], residual=res)
    v["xz"] = v["n"] @ w["win"]
    v["xc"], v["conv"] = ck.conv_fwd(v["xz"][..., :INNER], w["conv"], bias=w["convb"], h0=conv0, cu_seqlens=cu)
    v["dbc"] = v["xc"] @ w["wx"]
    v["dt"] = v["dbc"][..., :R] @ w["wdt"]
    v["y"], v["state"] = ck.scan_fwd(v["xc"], v["dt"], w["A"], v["dbc"][..., R:R + S], v["dbc"][..., R + S:], D=w["skip"],
                                     z=v["xz"][..., INNER:], dt_bias=w["dtb"], h0=h0, cu_seqlens=cu)
    return v


def gradients(w, v, dy, dh):
    """Of the forward's inputs and weights, for dL/dy and dL/dh."""
    g = {}
    (dxc, ddt, g["A"], dB, dC, g["skip"], dz, g["dtb"], g["h0"]) = ck.scan_bwd(
        v["xc"], v["dt"], w["A"], v["dbc"][..., R:R + S], v["dbc"][..., R + S:], dy, D=w["skip"],
        z=v["xz"][..., INNER:], dt_bias=w["dtb"], h0=v["h0"], cu_seqlens=v["cu"])
    flat = lambda t: t.flatten(0, -2)
    g["wdt"] = flat(v["dbc"][..., :R]).t() @ flat(ddt)
    ddbc = torch.cat([ddt @ w["wdt"].t(), dB, dC], -1)
    g["wx"] = flat(v["xc"]).t() @ flat(ddbc)
    dxc = dxc + ddbc @ w["wx"].t()
    dx, g["conv"], g["convb"], g["conv0"] = ck.conv_bwd(v["xz"][..., :INNER], w["conv"], dxc, bias=w["convb"],
                                                        h0=v["conv0"], cu_seqlens=v["cu"])
    dxz = torch.cat([dx, dz], -1)
    g["win"] = flat(v["n"]).t() @ flat(dxz)
    dn = dxz @ w["win"].t()
    g["x"], g["norm"], g["normb"] = ck.layer_norm_bwd(v["h"], w["norm"], dn, dh=dh)
    return g


def definition(w, x, res, conv0, h0):
    """The layer in float64, token by token."""
    B, T = x.shape[:2]
    h = x + res
    c = h - h.mean(-1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w["norm"] + w["normb"]
    xz = n @ w["win"]
    x, z = xz[..., :INNER], xz[..., INNER:]
    seen = torch.cat([conv0, x], 1)
    s = w["convb"] + sum(w["conv"][:, j] * seen[:, j:j + T] for j in range(K))
    x = s * torch.sigmoid(s)
    dbc = x @ w["wx"]
    d = torch.nn.functional.softplus(dbc[..., :R] @ w["wdt"] + w["dtb"])
    st, ys = h0, []
    for t in range(T):
        st = torch.exp(d[:, t, :, None] * w["A"]) * st + (d[:, t] * x[:, t])[..., None] * dbc[:, t, None, R:R + S]
        ys.append((st * dbc[:, t, None, R + S:]).sum(-1))
    y = (torch.stack(ys, 1) + w["skip"] * x) * z * torch.sigmoid(z)
    return y, h, st, seen[:, T:]


def inputs(seed, B, T, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)
    return [r(B, T, D).to(dtype), r(B, T, D).to(dtype), r(B, K - 1, INNER).to(dtype), 0.3 * r(B, INNER, S)], r(B, T, INNER).to(dtype), r(B, T, D).to(dtype)


# float32: a chain of six products over at most 96 terms and two norms; each
# operator is within its own bounds (tests beside this one), about 1e-6 of a tensor's
# largest value, and 40 times that covers what the chain multiplies them by.
TOL = 4e-5


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_layer_and_its_gradients(T):
    w = weights(1, torch.float32)
    args, dy, dh = inputs(2, 2, T)
    v = prompt(w, *args)
    g = gradients(w, v, dy, dh)
    torch.cuda.synchronize()
    W = {m: t.double().requires_grad_() for m, t in w.items()}
    X = [t.double().requires_grad_() for t in args]
    y, h, st, conv = definition(W, *X)
    errs = {"y": max_rel_err(v["y"].cpu(), y.detach().cpu()), "h": max_rel_err(v["h"].cpu(), h.detach().cpu()),
            "state": max_rel_err(v["state"].cpu(), st.detach().cpu()), "cache": max_rel_err(v["conv"].cpu(), conv.detach().cpu())}
    loss = (y * dy.double()).sum() + (h * dh.double()).sum()
    names = list(W)
    want = dict(zip(names + ["x", "res", "conv0", "h0"], torch.autograd.grad(loss, [W[m] for m in names] + X)))
    for m, r in want.items():
        errs["d" + m] = max_rel_err(g["x" if m == "res" else m].double().cpu(), r.cpu())
    announce(" ".join("%s %.1e" % e for e in errs.items()))
    assert max(errs.values()) < TOL, errs


def test_tokens_after_a_packed_prompt():
    """Prompts of several lengths in one batch, then each sequence a token at a time:
    the same as every sequence by itself to its end."""
    w = weights(3, torch.float32)
    lens, more = [7, 0, 20, 1], 4
    total = sum(lens)
    (x, res, conv0, h0), _, _ = inputs(4, 4, max(lens) + more)
    alone = [definition({m: t.double() for m, t in w.items()}, *[t.double() for t in (x[i:i + 1, :n + more], res[i:i + 1, :n + more], conv0[i:i + 1], h0[i:i + 1])])
             for i, n in enumerate(lens)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    pack = lambda t: torch.cat([t[i, :n] for i, n in enumerate(lens)])[None]
    v = prompt(w, pack(x), pack(res), conv0, h0, cu)
    conv, st = v["conv"], v["state"]
    at = 0
    for i, n in enumerate(lens):
        if n:
            assert max_rel_err(v["y"][0, at:at + n].cpu(), alone[i][0][0, :n].cpu()) < TOL
        at += n
    assert at == total
    for k in range(more):
        tok = lambda t: torch.stack([t[i, n + k] for i, n in enumerate(lens)])
        n_, _ = ck.layer_norm(tok(x), w["norm"], w["normb"], residual=tok(res))
        xz = n_ @ w["win"]
        xc = ck.conv_step(xz[:, :INNER], w["conv"], conv, bias=w["convb"])
        dbc = xc @ w["wx"]
        y = ck.scan_step(xc, dbc[:, :R] @ w["wdt"], w["A"], dbc[:, R:R + S], dbc[:, R + S:], st, D=w["skip"],
                         z=xz[:, INNER:], dt_bias=w["dtb"])
        torch.cuda.synchronize()
        for i, n in enumerate(lens):
            assert max_rel_err(y[i].cpu(), alone[i][0][0, n + k].cpu()) < TOL, (k, i)
    for i in range(4):
        assert max_rel_err(st[i].cpu(), alone[i][2][0].cpu()) < TOL


def test_in_graphs_with_eager_work_between():
    """Forward and gradients of the layer in one graph and of a cut scan in another,
    replayed in turn with new inputs and eager calls between: the eager bits."""
    w = weights(5, torch.bfloat16)
    args, dy, dh = inputs(6, 2, 300, torch.bfloat16)
    c = make_scan(7, 1, 900, 40, 16, 1, "bf16")
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    long = lambda: ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw) + ck.scan_bwd(
        g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)

    def layer():
        v = prompt(w, *args)
        # the weights' products over all tokens are torch's own: not of this test
        s = ck.scan_bwd(v["xc"], v["dt"], w["A"], v["dbc"][..., R:R + S], v["dbc"][..., R + S:], dy, D=w["skip"],
                        z=v["xz"][..., INNER:], dt_bias=w["dtb"], h0=v["h0"])
        k = ck.conv_bwd(v["xz"][..., :INNER], w["conv"], s[0], bias=w["convb"], h0=v["conv0"])
        return [v["y"], v["h"], v["state"], v["conv"], *s, *k, *ck.layer_norm_bwd(v["h"], w["norm"], dh, dh=dh)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(), long()
    torch.cuda.current_stream().wait_stream(side)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = layer()
    with torch.cuda.graph(second):
        b = long()
    for k in range(4):
        for t in (args[0], g["x"]):
            t.copy_(torch.randn_like(t.float()))
        first.replay()
        second.replay()
        eager_a, eager_b = layer(), long()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, eager_a)), k
        assert all(torch.equal(p, q) for p, q in zip(b, eager_b)), k
        second.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(b, eager_b)), k


def test_two_calls_at_once_on_two_streams():
    """Cut scans with workspaces of their own side by side, by stream= and by the
    current stream."""
    cs = [make_scan(20 + i, 1, 1500, 40, 16, 1, "bf16") for i in range(2)]
    gs = [scan_tensors(c) for c in cs]
    def both(i, **more):
        g, kw = gs[i], dict(scan_kw(cs[i], gs[i]), **more)
        return ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw) + ck.scan_bwd(
            g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], dht=g["dht"], **kw)
    want = [both(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [both(0, stream=streams[0])]
        with torch.cuda.stream(streams[1]):
            got.append(both(1))
        for s in streams:
            s.synchronize()
        torch.cuda.synchronize()
        for r, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(r, w))


def test_given_workspaces_and_outputs():
    c = make_scan(30, 1, 700, 24, 16, 1, "f32")
    g = scan_tensors(c)
    kw = scan_kw(c, g)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], **kw)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # NaN throughout
    out, fin = torch.empty_like(y), torch.empty_like(ht)
    y2, ht2 = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], workspace=ws, out=out, final_state=fin, **kw)
    assert y2 is out and ht2 is fin and torch.equal(y, y2) and torch.equal(ht, ht2)
    r = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], **kw)
    ws.fill_(255)
    r2 = ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], workspace=ws, **kw)
    assert all(torch.equal(p, q) for p, q in zip(r, r2))
    with pytest.raises(ValueError, match="workspace must"):
        ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], workspace=ws[:100], **kw)
    y, ht = ck.scan_fwd(g["x"], g["dt"], g["A"], g["B"], g["C"], output_final_state=False, **kw)
    assert ht is None and torch.equal(y, y2)
    assert ck.scan_bwd(g["x"], g["dt"], g["A"], g["B"], g["C"], g["dy"], output_dh0=False, **kw)[-1] is None
