"""The norms around a block in float64, forward and gradients, each value with
its magnitude (the same formula on absolute values, sums of absolute terms):
float32 arithmetic is off by at most `depth` half steps of the magnitude."""
import numpy as np


def act_of(g, act):
    if g is None:
        return 1.0, 0.0
    g = np.asarray(g, dtype=np.float64)
    e = np.exp(-np.abs(g))
    p = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
    dp = e / (1 + e) ** 2
    if act == "sigmoid":
        return p, dp
    return g * p, p + g * dp


def f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _mean(x):
    return x.mean(-1, keepdims=True)


def parts(y, w, g, act, x, s, eps):
    y = f64(y)
    r1 = 1.0 if w is None else 1 / np.sqrt(_mean(y * y) + eps)
    yn = y * r1
    u = yn * (1.0 if w is None else f64(w))
    a, da = act_of(g, act)
    sc = 1.0 if s is None else f64(s)
    v = u * a
    h = sc * v + (0.0 if x is None else f64(x))
    hm = np.abs(sc * v) + (0.0 if x is None else np.abs(f64(x)))
    return r1, yn, u, a, da, sc, v, h, hm


def fwd(y, w, g=None, act="sigmoid", x=None, s=None, w2=None, eps=1e-6):
    """(h, n), (|h|, |n|); n None without w2."""
    h, hm = parts(y, w, g, act, x, s, eps)[-2:]
    if w2 is None:
        return (h, None), (hm, None)
    r2 = 1 / np.sqrt(_mean(h * h) + eps)
    # an error e of h also moves r2, by at most mean(|h| e) r2^2 of itself
    more = np.abs(h) * _mean(np.abs(h) * hm) * r2 ** 2
    return (h, h * r2 * f64(w2)), (hm, (hm + np.abs(h) + more) * r2 * np.abs(f64(w2)))


def bwd(y, w, dh, dn=None, g=None, act="sigmoid", x=None, s=None, w2=None, eps=1e-6):
    """dict of gradients, dict of magnitudes (keys dy, dw, dg, dx, ds, dw2)."""
    r1, yn, u, a, da, sc, v, h, hm = parts(y, w, g, act, x, s, eps)
    out, mag = {}, {}
    D, M = f64(dh), np.abs(f64(dh))
    if w2 is not None:
        r2 = 1 / np.sqrt(_mean(h * h) + eps)
        hn, hnm = h * r2, (hm + np.abs(h) * (1 + _mean(np.abs(h) * hm) * r2 ** 2)) * r2
        c = f64(dn) * f64(w2)
        out["dw2"], mag["dw2"] = (f64(dn) * hn).sum(0), (np.abs(f64(dn)) * hnm).sum(0)
        D = D + r2 * (c - hn * _mean(c * hn))
        ratio = 1 + _mean(np.abs(h) * hm) * r2 ** 2
        M = M + r2 * ratio * (np.abs(c) + hnm * _mean(np.abs(c) * hnm))
    out["dx"], mag["dx"] = D, M
    out["ds"], mag["ds"] = (D * v).sum(0), (M * np.abs(v)).sum(0)
    dv, dvm = D * sc, M * np.abs(sc)
    out["dg"], mag["dg"] = dv * u * da, dvm * np.abs(u) * (np.abs(da) + np.abs(a))
    du, dum = dv * a, dvm * np.abs(a)
    out["dw"], mag["dw"] = (du * yn).sum(0), (dum * np.abs(yn)).sum(0)
    if w is None:
        out["dy"], mag["dy"] = du, dum
    else:
        c, cm = du * f64(w), dum * np.abs(f64(w))
        out["dy"] = r1 * (c - yn * _mean(c * yn))
        mag["dy"] = r1 * (cm + np.abs(yn) * _mean(cm * np.abs(yn)))
    return out, mag
