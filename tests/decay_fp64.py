"""Decay linear attention token by token in float64, with the bounds that the
parity tests hold the kernels to.

Every value comes with its magnitude: the same sum with each term's absolute
value.  A kernel that rounds its operands once to a type of half step u (and
adds up in float32) is off by at most u times the magnitude, plus u times the
value where the output is rounded to that type.
"""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def sequences(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def gates(alpha, kind, ckda):
    """(gates, their derivative by what alpha holds) in float64."""
    a = np.asarray(alpha, dtype=np.float64)
    if kind == "values":
        return a, np.ones_like(a)
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(a))
    p = np.where(a >= 0, 1 / (1 + e), e / (1 + e))
    d = e / (1 + e) ** 2
    if not ckda:
        return p, d
    return np.sign(a) * (1 - e) / (1 + e), 2 * d


def fwd(q, k, v, a, h0=None, cu=None, scale=1.0):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], a [B,T,H] -> o, ht, |o|, |ht|."""
    q, k, v, a = (np.asarray(x, dtype=np.float64) for x in (q, k, v, a))
    rep = v.shape[2] // q.shape[2]
    q, k = np.repeat(q, rep, 2), np.repeat(k, rep, 2)
    seqs = sequences(q.shape[0], q.shape[1], cu)
    o, om = np.zeros(v.shape), np.zeros(v.shape)
    hs, hm = [], []
    for n, (b, lo, hi) in enumerate(seqs):
        S = np.zeros((v.shape[2], q.shape[3], v.shape[3])) if h0 is None else np.array(h0[n], dtype=np.float64)
        M = np.abs(S)
        for t in range(lo, hi):
            S = a[b, t][:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            M = np.abs(a[b, t])[:, None, None] * M + np.abs(k[b, t])[:, :, None] * np.abs(v[b, t])[:, None, :]
            o[b, t] = scale * np.einsum("hkv,hk->hv", S, q[b, t])
            om[b, t] = abs(scale) * np.einsum("hkv,hk->hv", M, np.abs(q[b, t]))
        hs.append(S)
        hm.append(M)
    z = (0, v.shape[2], q.shape[3], v.shape[3])
    return o, np.array(hs).reshape((len(seqs),) + z[1:]), om, np.array(hm).reshape((len(seqs),) + z[1:])


def bwd(q, k, v, a, do, h0=None, dht=None, cu=None, scale=1.0):
    """Gradients (dq, dk, dv, da, dh0) and their magnitudes."""
    q, k, v, a, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, a, do))
    Hk, rep = q.shape[2], v.shape[2] // q.shape[2]
    qs, ks = np.repeat(q, rep, 2), np.repeat(k, rep, 2)
    seqs = sequences(q.shape[0], q.shape[1], cu)
    H, dk, dv = v.shape[2], q.shape[3], v.shape[3]
    out = [np.zeros(qs.shape), np.zeros(qs.shape), np.zeros(v.shape), np.zeros(a.shape), np.zeros((len(seqs), H, dk, dv))]
    mag = [np.zeros_like(x) for x in out]

    def run(res, q, k, v, a, do, scale, h0, dht):
        for n, (b, lo, hi) in enumerate(seqs):
            S = np.zeros((H, dk, dv)) if h0 is None else np.array(h0[n], dtype=np.float64)
            before = []
            for t in range(lo, hi):
                before.append(S)
                S = a[b, t][:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            A = np.zeros((H, dk, dv)) if dht is None else np.array(dht[n], dtype=np.float64)
            for t in reversed(range(lo, hi)):
                res[0][b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
                A = A + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
                res[1][b, t] = np.einsum("hkv,hv->hk", A, v[b, t])
                res[2][b, t] = np.einsum("hkv,hk->hv", A, k[b, t])
                res[3][b, t] = np.einsum("hkv,hkv->h", A, before[t - lo])
                A = a[b, t][:, None, None] * A
                S = before[t - lo]
            res[4][n] = A
        for i in (0, 1):
            res[i] = res[i].reshape(res[i].shape[:2] + (Hk, rep, dk)).sum(3)
        return res

    ab = lambda x: None if x is None else np.abs(x)
    return (run(out, qs, ks, v, a, do, scale, h0, dht),
            run(mag, ab(qs), ab(ks), ab(v), ab(a), ab(do), abs(scale), ab(h0), ab(dht)))


def sums(dk, T):
    """Float32 roundings a value passes: a sum over dk and one over a chunk,
    a product of gates and an update a chunk, and the gates' own logarithms and
    powers (16 covers them: |x| 2^-|x| is below 0.54)."""
    return (dk + 64 + 4 * (T // 32 + 1) + 16) * 2.0 ** -24


def bound_out(dtype, value, mag, dk, T):
    """An output of the io type: operands rounded once, the output once."""
    u = HALF[dtype]
    return u * (np.abs(value) + mag) + 2 * sums(dk, T) * mag + 1e-30


def bound_state(dtype, mag, dk, T):
    """A float32 state (in bf16 the weighted operand goes in as three terms, 24
    bits in all, so both types keep float32's accuracy)."""
    return 2 * sums(dk, T) * mag + 1e-30
