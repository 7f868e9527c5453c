"""The linear attention with a decay for each head in 64 bits, token after token as its recurrence is written, and beside
each result a bound on its rounding errors in units of 2^-24.

Counted, relative to the same sums over absolute values. A decay over a span: its exponential's argument (|log2| of it),
value and product, about 1.5 |g| + 6 for a token. A state: every product added to it a rounding, three parts of a
value each (their own end 2^-25 below): 3 of its size for a token, and 8 of what the token adds. A result from a state: its
products' sums, as long as the contraction, in two parts, which end 2^-16 below (256 units); gradients of decays in
three parts. Weights of pairs in a chunk: the contraction of q and k, 8 roundings of their own, two parts.

Below 2^-126 nothing is kept: exponentials and parts of values (a value of 2^-110 has its third part there) are flushed to
zero, so that a product loses up to 2^-126 times its other factor for each of its three parts and for its weight. That is
after the decays up to the end of its chunk, so those do not shrink it: it is carried without decay (`lost`). It shows only
where whole results are near 2^-110 themselves."""
import numpy as np

U = 2.0 ** -24
LEAST = 2.0 ** -126 / U
PARTS2 = 256.0      # 2^-16 in units of 2^-24


def forward(q, k, v, g, scale, lengths, init=None):
    """out [T, H, V], its error, final [S, H, K, V], its error. g [T, H]."""
    T, H, K = q.shape
    V = v.shape[2]
    out, eo = np.zeros((T, H, V)), np.zeros((T, H, V))
    fin, ef = np.zeros((len(lengths), H, K, V)), np.zeros((len(lengths), H, K, V))
    at = 0
    for n, length in enumerate(lengths):
        S = init[n].copy() if init is not None else np.zeros((H, K, V))
        size, e, lost = np.abs(S), np.zeros((H, K, V)), np.zeros((H, K, V))
        for t in range(at, at + length):
            a = np.exp(g[t])[:, None, None]
            dec = (1.5 * np.abs(np.maximum(g[t], -200.0)) + 6)[:, None, None]
            kv = k[t][:, :, None] * v[t][:, None]
            e = a * (e + size * dec) + 8 * np.abs(kv)
            lost = lost + LEAST * (size + np.abs(k[t])[:, :, None] * (3 + np.abs(v[t])[:, None]))
            S, size = a * S + kv, a * size + np.abs(kv)
            e = e + 3 * size
            out[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
            # (the pairs' sums over q and k cancel on their own: |q| |k| |v| is in |q| size)
            eo[t] = abs(scale) * np.einsum("hk,hkv->hv", np.abs(q[t]), e + lost + (PARTS2 + 3 * K + 64) * size + LEAST * (3 + size))
            eo[t] += LEAST * 192 * np.abs(v).max()
        fin[n], ef[n] = S, e + lost + 2 * size
        at += length
    return out, eo, fin, ef


def backward(q, k, v, g, scale, lengths, do, init=None, dfin=None, window=64):
    """Gradients and their errors, as two dicts; dg [T, H]. window: tokens of a segment (sums of what passes borders run over them)."""
    T, H, K = q.shape
    V = v.shape[2]
    S0 = len(lengths)
    r = {"dq": np.zeros((T, H, K)), "dk": np.zeros((T, H, K)), "dv": np.zeros((T, H, V)), "dg": np.zeros((T, H)),
         "d_initial_state": np.zeros((S0, H, K, V))}
    err = {n: np.zeros_like(x) for n, x in r.items()}
    flow = np.zeros((T, H))         # size of a token's u and w
    end = np.zeros(T, dtype=int)
    at = 0
    for n, length in enumerate(lengths):
        X = init[n].copy() if init is not None else np.zeros((H, K, V))
        size, e, lost = np.abs(X), np.zeros((H, K, V)), np.zeros((H, K, V))
        trail = []
        for t in range(at, at + length):
            end[t] = at
            a = np.exp(g[t])[:, None, None]
            dec = (1.5 * np.abs(np.maximum(g[t], -200.0)) + 6)[:, None, None]
            kv = k[t][:, :, None] * v[t][:, None]
            lost = lost + LEAST * size
            X, e, size = a * X, a * (e + size * dec), a * size
            trail.append((X, e + lost, size))
            lost = lost + LEAST * np.abs(k[t])[:, :, None] * (3 + np.abs(v[t])[:, None])
            X, e, size = X + kv, e + 8 * np.abs(kv), size + np.abs(kv)
            e = e + 3 * size
            r["dq"][t] = scale * np.einsum("hkv,hv->hk", X, do[t])
            err["dq"][t] = abs(scale) * np.einsum("hkv,hv->hk", e + lost + (PARTS2 + 3 * V + 64) * size + LEAST * (3 + size), np.abs(do[t]))
            err["dq"][t] += LEAST * 192 * np.abs(k).max()
            flow[t] += abs(scale) * np.einsum("hkv,hk,hv->h", size, np.abs(q[t]), np.abs(do[t]))
        Y = dfin[n].copy() if dfin is not None else np.zeros((H, K, V))
        size, e, lost = np.abs(Y), np.zeros((H, K, V)), np.zeros((H, K, V))
        for t in range(at + length - 1, at - 1, -1):
            qd = scale * q[t][:, :, None] * do[t][:, None]
            lost = lost + LEAST * np.abs(q[t])[:, :, None] * (3 + np.abs(do[t])[:, None])
            Y, e, size = Y + qd, e + 9 * np.abs(qd), size + np.abs(qd)
            e = e + 3 * size
            r["dk"][t] = np.einsum("hkv,hv->hk", Y, v[t])
            err["dk"][t] = np.einsum("hkv,hv->hk", e + lost + (PARTS2 + 3 * V + 64) * size + LEAST * (3 + size), np.abs(v[t])) + LEAST * 192 * np.abs(q).max()
            r["dv"][t] = np.einsum("hkv,hk->hv", Y, k[t])
            err["dv"][t] = np.einsum("hkv,hk->hv", e + lost + (PARTS2 + 3 * K + 64) * size + LEAST * (3 + size), np.abs(k[t])) + LEAST * 192 * np.abs(do).max()
            flow[t] += np.einsum("hkv,hk,hv->h", size, np.abs(k[t]), np.abs(v[t]))
            X, ex, sx = trail[t - at]
            r["dg"][t] = (X * Y).sum((1, 2))
            err["dg"][t] = (ex * size + sx * (e + lost) + (K + V + 64) * sx * size).sum((1, 2))
            a = np.exp(g[t])[:, None, None]
            dec = (1.5 * np.abs(np.maximum(g[t], -200.0)) + 6)[:, None, None]
            lost = lost + LEAST * size
            Y, e, size = a * Y, a * (e + size * dec), a * size
        r["d_initial_state"][n], err["d_initial_state"][n] = Y, e + lost + 2 * size
        at += length
    # what passes the borders of a segment is summed token after token (u, w: a contraction in three parts and
    # one over a head, and a rounding for each token of the segment)
    for t in range(T):
        lo = max(end[t], t - window)
        err["dg"][t] += (3 * (K + V) + 2 * window) * flow[lo:t + 1].sum(0) + 3 * 64 * flow[t]
        err["dg"][t] += LEAST * window * (np.abs(q).max() * np.abs(do).max() + np.abs(k).max() * np.abs(v).max()) * (K + V) * 64
    return r, err
