"""Plain 64-bit references of the low-rank adapters, the tokens' log probabilities
and the embedding, with the error bounds the kernels' arithmetic allows.  numpy on
the CPU; nothing here is shared with the library."""
import numpy as np

from tests.reference64 import BF16_HALF, F32_MIN

ADD = 2.0 ** -23               # an fp32 addition that need not round to nearest


def _its(ids, L):
    """The tokens of each adapter."""
    ids = np.asarray(ids)
    return [np.flatnonzero(ids == i) for i in range(L)]


def lora(x, a, b, ids, scale, base):
    """(y before its rounding, bound on the error before it).

    v = x A^T: K exact products summed in fp32, at most K + 40 additions (steps,
    waves, splits).  v enters the second product as two pieces that miss at most
    2^-16 of it, after one product with s; there are 2 R products and the sum with
    base."""
    x, a, b, base = (np.asarray(v, np.float64) for v in (x, a, b, base))
    s = np.ones(a.shape[0]) if scale is None else np.asarray(scale, np.float64)
    y, tol = base.copy(), ADD * np.abs(base)
    K, R = x.shape[1], a.shape[1]
    for i, t in enumerate(_its(ids, a.shape[0])):
        if t.size:
            y[t] += s[i] * (x[t] @ a[i].T) @ b[i].T
            tol[t] += abs(s[i]) * (2.0 ** -16 + ADD * (K + 2 * R + 60)) * (np.abs(x[t]) @ np.abs(a[i]).T) @ np.abs(b[i]).T
    return y, tol


def lora_backward(dy, x, a, b, ids, scale, base):
    """(dx, da, db) and the bounds on their errors before rounding: u = dy B as v
    above with N additions; da and db take u and v whole, in three pieces, and add
    3 products a token."""
    dy, x, a, b, base = (np.asarray(v, np.float64) for v in (dy, x, a, b, base))
    s = np.ones(a.shape[0]) if scale is None else np.asarray(scale, np.float64)
    dx, tx = base.copy(), ADD * np.abs(base)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    ta, tb = np.zeros(a.shape), np.zeros(b.shape)
    K, N, R = x.shape[1], dy.shape[1], a.shape[1]
    for i, t in enumerate(_its(ids, a.shape[0])):
        if not t.size:
            continue
        u, v = s[i] * (dy[t] @ b[i]), s[i] * (x[t] @ a[i].T)
        ua, va = abs(s[i]) * (np.abs(dy[t]) @ np.abs(b[i])), abs(s[i]) * (np.abs(x[t]) @ np.abs(a[i]).T)
        dx[t] += u @ a[i]
        tx[t] += (2.0 ** -16 + ADD * (N + 2 * R + 60)) * (ua @ np.abs(a[i]))
        da[i], db[i] = u.T @ x[t], dy[t].T @ v
        ta[i] = ADD * (N + 3 * t.size + 100) * (ua.T @ np.abs(x[t]))
        tb[i] = ADD * (K + 3 * t.size + 100) * (np.abs(dy[t]).T @ va)
    return (dx, da, db), (tx, ta, tb)


def rounded(ref, tol, half=BF16_HALF, least=F32_MIN):
    """A bound before rounding as one after it."""
    return half * (np.abs(ref) + tol) + tol + least


def logprobs(x, target, top):
    """(logprob, entropy, lse, top_logprob, top_id) in fp64, ties to the lowest index."""
    x, target = np.asarray(x, np.float64), np.asarray(target)
    T, V = x.shape
    out = [np.zeros(T), np.zeros(T), np.zeros(T), np.zeros((T, top)), np.full((T, top), -1, np.int32)]
    for t in range(T):
        row = x[t]
        m = row.max() if not np.isnan(row).any() else np.nan
        if m == -np.inf:
            lse, logp, entropy = -np.inf, np.full(V, -np.inf), 0.0
        elif not np.isfinite(m):
            lse, logp, entropy = np.nan, np.full(V, np.nan), np.nan
        else:
            d = row - m
            lse = m + np.log(np.exp(d).sum())
            logp = d - np.log(np.exp(d).sum())
            p = np.exp(logp)
            entropy = -(p[p > 0] * logp[p > 0]).sum()
        out[0][t] = logp[target[t]] if 0 <= target[t] < V else 0.0
        out[1][t], out[2][t] = entropy, lse
        order = np.lexsort((np.arange(V), -row))
        order = order[~np.isnan(row[order])][:top]
        out[4][t, :order.size] = order
        out[3][t, :order.size] = logp[order]
        out[3][t, order.size:] = np.nan
    return out


def logprobs_bounds(x, target, top_id):
    """Bounds on the errors of logprob, entropy, lse and top_logprob.

    S adds at most V / 256 + 32 terms a lane, rescaled once a chunk of 4096 at most
    with three roundings, then 80 lanes, waves and parts; n counts them.  A term
    e^d is off by two steps and by |d| 2^-23 relatively (d times log2 e is rounded
    before it is exponentiated).  W the same with terms e^d |d|, then ln S by
    2^-22 relatively and a rounding for each of the last operations."""
    x, target = np.asarray(x, np.float64), np.asarray(target)
    T, V = x.shape
    n = V / 256 + 3 * V / 4096 + 130
    out = [np.zeros(T), np.zeros(T), np.zeros(T), np.zeros(np.asarray(top_id).shape)]
    for t in range(T):
        m = x[t].max()
        if not np.isfinite(m):
            continue
        d = np.maximum(x[t] - m, -1e4)
        e = np.exp(d)
        S = e.sum()
        D, D2 = (e * -d).sum() / S, (e * d * d).sum() / S
        ln = ADD * (n + 4 + D) + 2.0 ** -22 * np.log(S) + F32_MIN
        at = lambda i: ADD * (np.abs(x[t][i] - m) + np.log(S))
        out[0][t] = ln + at(target[t]) if 0 <= target[t] < V else 0.0
        out[1][t] = ln + ADD * ((2 * n + 12) * D + D2) + ADD * np.log(S)
        out[2][t] = ln + ADD * (abs(m) + np.log(S))
        out[3][t] = ln + at(np.maximum(np.asarray(top_id)[t], 0))
    return out


def logprobs_backward(g, x, target, lse, entropy, h):
    """(dx, bound before rounding) in fp64 from the given lse and entropy.  p is off by
    two steps and by |x - lse| 2^-22 relatively, the bracket by three additions."""
    x, target, lse = np.asarray(x, np.float64), np.asarray(target), np.asarray(lse, np.float64)
    there = (target >= 0) & (target < x.shape[1])
    g = np.where(there, np.asarray(g, np.float64), 0.0)
    h = np.zeros_like(g) if h is None else np.asarray(h, np.float64)
    H = np.zeros_like(g) if entropy is None else np.asarray(entropy, np.float64)
    dx, tol = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(x.shape[0]):
        if (g[t] == 0 and h[t] == 0) or lse[t] == -np.inf:
            continue
        z = x[t] - lse[t]
        p = np.exp(z)
        z = np.where(p > 0, np.maximum(z, -1e4), 0.0)
        dx[t] = -p * (g[t] + h[t] * (z + H[t]))
        tol[t] = p * (abs(g[t]) + abs(h[t]) * (np.abs(z) + abs(H[t]))) * ADD * (8 + 2 * np.abs(z))
        if there[t]:
            dx[t, target[t]] += g[t]
            tol[t, target[t]] += ADD * abs(g[t])
    return dx, tol


def embedding(ids, table, row_scale, scale):
    """Rows by token in fp64; row_scale [V], [V, H / 128] or None."""
    ids, table = np.asarray(ids), np.asarray(table, np.float64)
    out = np.zeros((ids.size, table.shape[1]))
    at = np.flatnonzero((ids >= 0) & (ids < table.shape[0]))
    v = table[ids[at]] * scale
    if row_scale is not None:
        s = np.asarray(row_scale, np.float64)[ids[at]].reshape(at.size, -1)
        v = v * np.repeat(s, table.shape[1] // s.shape[1], axis=1)
    out[at] = v
    return out


def embedding_backward(dout, ids, vocab, scale, table=None):
    """(dtable, bound before rounding) in fp64: as many fp32 additions as a token has
    positions, one product, and the sum with `table` where that is given."""
    dout, ids = np.asarray(dout, np.float64), np.asarray(ids)
    out = np.zeros((vocab, dout.shape[1])) if table is None else np.array(table, np.float64)
    tol = 2.0 ** -24 * np.abs(out)
    at = np.flatnonzero((ids >= 0) & (ids < vocab))
    count = np.bincount(ids[at], minlength=vocab)
    np.add.at(out, ids[at], scale * dout[at])
    mag = np.zeros(out.shape)
    np.add.at(mag, ids[at], abs(scale) * np.abs(dout[at]))
    return out, tol + 2.0 ** -24 * (count[:, None] + 3) * mag
