"""The selective scan, the short convolution and layer norm in float64, forward
and gradients, every value with a bound of the error that float32 arithmetic in
the kernels' order may leave: each operation is off by half a step (EPS) of its
value, errors pass on through the formulas, and a sum of m terms is off by m EPS
of its terms' magnitudes.  `value_and_bound` results are (value, bound) pairs; a
test adds the rounding of the output's type.

What an elementary function may be off by, in EPS of its value: softplus 16 and
2 |v| for the rounding of its argument v, the sigmoid and silu 24 and 2 |v|, a
power 3 (its instruction is good to 1.4) besides what its argument's error makes
of it.  Pieces of a cut sequence are joined by powers of their steps' sums, which
are off by a piece's length in EPS: `cut` adds that to every step."""
import numpy as np

EPS = 2.0 ** -24


def f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def silu(x):
    """(silu, its bound), (slope, its bound)"""
    p = sigmoid(x)
    q = np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))) ** 2
    k = EPS * (24 + 2 * np.abs(x))
    return (x * p, np.abs(x * p) * k), (p + x * q, (p + np.abs(x) * q) * (k + 8 * EPS))


def scan(x, dt, A, B, C, D=None, z=None, bias=None, softplus=True, h0=None, dy=None, dht=None, cut=0):
    """One sequence: x, dt, z, dy [T,D]; A [D,S]; B, C [T,G,S]; h0, dht [D,S].
    Returns {name: (value, bound)}: y, ht, and with dy the gradients."""
    x, dt, A, B, C, D, z, bias, h0, dy, dht = (f64(t) for t in (x, dt, A, B, C, D, z, bias, h0, dy, dht))
    T, ch = x.shape
    S, G = A.shape[1], B.shape[1]
    rep, blocks = ch // G, -(-(ch // G) // 32)
    D = np.zeros(ch) if D is None else D
    v = dt if bias is None else dt + bias
    if softplus:
        d = np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))
        ed = EPS * (16 + 2 * np.abs(v)) * d + 1e-36
        slope, eslope = sigmoid(v), EPS * (24 + 2 * np.abs(v)) * sigmoid(v)
    else:
        d, ed = v, EPS * 2 * np.abs(v)
        slope, eslope = np.ones_like(v), np.zeros_like(v)
    u = d * x
    eu = np.abs(x) * ed + EPS * np.abs(u)
    Bc, Cc = (np.repeat(m, rep, 1) for m in (B, C))  # [T,ch,S]
    a = np.exp(d[..., None] * A)
    ea = a * (np.abs(A) * (ed + (3 + cut) * EPS * np.abs(d))[..., None] + 3 * EPS)
    h = np.zeros((T + 1, ch, S))
    H, E = np.zeros_like(h), np.zeros_like(h)
    if h0 is not None:
        h[0], H[0] = h0, np.abs(h0)
    for t in range(T):
        w = u[t][:, None] * Bc[t]
        h[t + 1] = a[t] * h[t] + w
        H[t + 1] = a[t] * H[t] + np.abs(w)
        E[t + 1] = a[t] * E[t] + ea[t] * H[t] + np.abs(Bc[t]) * eu[t][:, None] + 2 * EPS * H[t + 1]
    yp = (Cc * h[1:]).sum(-1) + D * x
    ym = (np.abs(Cc) * H[1:]).sum(-1) + np.abs(D * x)
    ey = (np.abs(Cc) * E[1:]).sum(-1) + (S + 8) * EPS * ym
    if z is None:
        act, eact = np.ones_like(x), np.zeros_like(x)
    else:
        (act, eact), (sz, esz) = silu(z)
    out = {"y": (yp * act, np.abs(act) * ey + ym * eact + EPS * np.abs(yp * act)), "ht": (h[T], E[T])}
    if dy is None:
        return out
    g = dy * act
    eg = np.abs(dy) * eact + EPS * np.abs(g)
    c = np.zeros((ch, S)) if dht is None else dht.copy()
    cm, ec = np.abs(c), np.zeros_like(c)
    gb, egb, gbm, wa, ewa = (np.zeros((T, ch)) for _ in range(5))
    dA, edA, dAm = (np.zeros((ch, S)) for _ in range(3))
    dB, edB, dC, edC = (np.zeros((T, G, S)) for _ in range(4))
    groups = lambda t: t.reshape(G, rep, S).sum(1)
    deep = (64 + blocks + 8) * EPS
    for t in reversed(range(T)):
        gC = g[t][:, None] * Cc[t]
        Gt, Gm = c + gC, cm + np.abs(gC)
        eG = ec + np.abs(Cc[t]) * eg[t][:, None] + 2 * EPS * Gm
        gb[t] = (Gt * Bc[t]).sum(-1)
        gbm[t] = (Gm * np.abs(Bc[t])).sum(-1)
        egb[t] = (eG * np.abs(Bc[t])).sum(-1) + (S + 8) * EPS * gbm[t]
        uu = u[t][:, None]
        dB[t] = groups(Gt * uu)
        edB[t] = groups(eG * np.abs(uu) + Gm * eu[t][:, None]) + deep * groups(Gm * np.abs(uu))
        gg = g[t][:, None]
        dC[t] = groups(gg * h[t + 1])
        edC[t] = groups(eg[t][:, None] * H[t + 1] + np.abs(gg) * E[t + 1]) + deep * groups(np.abs(gg) * H[t + 1])
        c = a[t] * Gt
        cm = a[t] * Gm
        ec = a[t] * eG + ea[t] * Gm + EPS * cm
        w, wm = c * h[t], cm * H[t]
        ew = ec * H[t] + cm * E[t] + EPS * wm
        wa[t] = (w * A).sum(-1)
        ewa[t] = (ew * np.abs(A)).sum(-1) + (S + 10) * EPS * (wm * np.abs(A)).sum(-1)
        dt_ = d[t][:, None]
        dA += w * dt_
        dAm += wm * np.abs(dt_)
        edA += ew * np.abs(dt_) + wm * ed[t][:, None]
    dx = d * gb + D * g
    edx = ed * gbm + np.abs(d) * egb + np.abs(D) * eg + 3 * EPS * (np.abs(d) * gbm + np.abs(D * g))
    dd = x * gb + wa
    ddm = np.abs(x) * gbm + np.abs(wa) + ewa
    edd = np.abs(x) * egb + ewa + 3 * EPS * ddm
    ddt = dd * slope
    eddt = slope * edd + ddm * eslope + EPS * np.abs(ddt)
    many = (T + 64) * EPS
    out.update(dx=(dx, edx), ddt=(ddt, eddt), dA=(dA, edA + many * dAm), dB=(dB, edB), dC=(dC, edC),
               dD=((g * x).sum(0), (eg * np.abs(x)).sum(0) + many * np.abs(g * x).sum(0)),
               dbias=(ddt.sum(0), eddt.sum(0) + many * (slope * ddm).sum(0)), dh0=(c, ec))
    if z is not None:
        dz = dy * sz * yp
        out["dz"] = (dz, np.abs(dy) * (np.abs(sz) * ey + ym * esz) + 3 * EPS * np.abs(dy * sz) * ym)
    return out


def conv(x, w, bias=None, act="silu", h0=None, dy=None, dht=None):
    """One sequence: x, dy [T,D]; w [D,K]; h0, dht [K-1,D].  Returns {name: (value, bound)}."""
    x, w, bias, h0, dy, dht = (f64(t) for t in (x, w, bias, h0, dy, dht))
    (T, D), K = x.shape, w.shape[1]
    seen = np.concatenate([np.zeros((K - 1, D)) if h0 is None else h0, x])
    b = np.zeros(D) if bias is None else bias
    s = b + sum(w[:, j] * seen[j:j + T] for j in range(K))
    sm = np.abs(b) + sum(np.abs(w[:, j] * seen[j:j + T]) for j in range(K))
    es = (K + 2) * EPS * sm
    if act == "silu":
        (y, ey), (sl, esl) = silu(s)
        ey = ey + 1.1 * es        # the slope is under 1.1, the slope's under 0.5
        esl = esl + 0.5 * es
    else:
        y, ey, sl, esl = s, es, np.ones_like(s), np.zeros_like(s)
    out = {"y": (y, ey), "ht": (seen[T:], np.zeros((K - 1, D)))}
    if dy is None:
        return out
    g = dy * sl
    eg = np.abs(dy) * esl + EPS * np.abs(g)
    dseen, e = np.zeros_like(seen), np.zeros_like(seen)
    for j in range(K):
        dseen[j:j + T] += g * w[:, j]
        e[j:j + T] += (eg + (K + 3) * EPS * np.abs(g)) * np.abs(w[:, j])
    if dht is not None:
        dseen[T:] += dht
        e[T:] += EPS * (K + 3) * np.abs(dht)
    many = (T + 64) * EPS
    dw = np.stack([(g * seen[j:j + T]).sum(0) for j in range(K)], -1)
    edw = np.stack([((eg + many * np.abs(g)) * np.abs(seen[j:j + T])).sum(0) for j in range(K)], -1)
    out.update(dx=(dseen[K - 1:], e[K - 1:]), dh0=(dseen[:K - 1], e[:K - 1]), dw=(dw, edw),
               dbias=(g.sum(0), (eg + many * np.abs(g)).sum(0)))
    return out


def layer_norm(x, w=None, b=None, r=None, eps=1e-5, dn=None, dh=None):
    """x, r, dn, dh [rows,d].  Returns {name: (value, bound)}; with dn the gradients,
    for which x is the row that is normed."""
    x, w, b, r, dn, dh = (f64(t) for t in (x, w, b, r, dn, dh))
    rows, d = x.shape
    w, b = (np.ones(d) if w is None else w), (np.zeros(d) if b is None else b)
    deep = (48 + 40) * EPS  # a thread's elements (32 at most), the trees over threads and waves, single operations
    mean = lambda t: t.mean(-1, keepdims=True)
    h = x if r is None else x + r
    eh = 0 * h if r is None else EPS * np.abs(h)
    c = h - mean(h)
    ec = eh + mean(eh) + deep * mean(np.abs(h)) + EPS * np.abs(c)
    var = mean(c * c)
    evar = 2 * mean(np.abs(c) * ec) + mean(ec * ec) + deep * var
    rs = 1 / np.sqrt(var + eps)
    ers = 0.5 * rs ** 3 * evar + 4 * EPS * rs
    cn = c * rs
    ecn = ec * rs + np.abs(c) * ers + ec * ers + EPS * np.abs(cn)
    n = cn * w + b
    out = {"h": (h, eh), "n": (n, ecn * np.abs(w) + 2 * EPS * (np.abs(cn * w) + np.abs(b)))}
    if dn is None:
        return out
    m = dn * w
    mm, mc = mean(m), mean(m * cn)
    emm = (deep + EPS) * mean(np.abs(m))
    emc = mean(np.abs(m) * ecn) + deep * mean(np.abs(m * cn))
    inner = m - mm - cn * mc
    ein = EPS * 4 * (np.abs(m) + np.abs(mm) + np.abs(cn * mc)) + emm + ecn * np.abs(mc) + np.abs(cn) * emc + ecn * emc
    dx = rs * inner
    edx = rs * ein + ers * np.abs(inner) + 2 * EPS * np.abs(dx)
    if dh is not None:
        dx, edx = dx + dh, edx + EPS * (np.abs(dx) + np.abs(dh))
    many = (rows + 96) * EPS
    out.update(dx=(dx, edx), dw=((dn * cn).sum(0), (np.abs(dn) * (ecn + many * np.abs(cn))).sum(0)),
               db=(dn.sum(0), many * np.abs(dn).sum(0)))
    return out
