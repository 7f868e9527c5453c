"""Plain 64-bit forms of the operators beside the delta rule, for their tests: written from the
definitions, on the CPU, one sequence and one row after another. Each returns its results and,
beside each, the size that rounding errors are counted against (the same sums over absolute
values)."""
import numpy as np

#: half a step of each type relative to the value, and the spacing below its smallest normal number
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}
U = 2.0 ** -24


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def silu_grad(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


def conv(x, w, b, lengths, init=None, act=True, dy=None, dfin=None):
    """Results and sizes of the short convolution; with dy, of its gradients too."""
    T, C = x.shape
    W = w.shape[1]
    out = {k: np.zeros((T, C)) for k in ("y", "y_size", "dx", "dx_size")}
    out.update({k: np.zeros((len(lengths), W - 1, C)) for k in ("final", "d_initial_state", "d_initial_state_size")})
    out.update({k: np.zeros((C, W)) for k in ("dweight", "dweight_size")})
    out.update({k: np.zeros(C) for k in ("dbias", "dbias_size")})
    b = np.zeros(C) if b is None else b
    at = 0
    for i, n in enumerate(lengths):
        line = np.concatenate([init[i] if init is not None else np.zeros((W - 1, C)), x[at:at + n]])
        dline, dsize = np.zeros_like(line), np.zeros_like(line)
        for t in range(n):
            p = b + sum(w[:, j] * line[t + j] for j in range(W))
            size = np.abs(b) + sum(np.abs(w[:, j] * line[t + j]) for j in range(W))
            out["y"][at + t] = p * sigmoid(p) if act else p
            out["y_size"][at + t] = size
            if dy is not None:
                e = dy[at + t] * (silu_grad(p) if act else 1.0)
                # a relative error of p turns into one of e: |f''| <= 1/2, |f'| <= 1.1
                esize = np.abs(e) + np.abs(dy[at + t]) * (size + 1.0 if act else 1.0)
                for j in range(W):
                    dline[t + j] += w[:, j] * e
                    dsize[t + j] += np.abs(w[:, j]) * esize
                    out["dweight"][:, j] += e * line[t + j]
                    out["dweight_size"][:, j] += esize * np.abs(line[t + j])
                out["dbias"] += e
                out["dbias_size"] += esize
        out["final"][i] = line[n:]
        if dfin is not None:
            dline[n:] += dfin[i]
            dsize[n:] += np.abs(dfin[i])
        out["d_initial_state"][i], out["d_initial_state_size"][i] = dline[:W - 1], dsize[:W - 1]
        out["dx"][at:at + n], out["dx_size"][at:at + n] = dline[W - 1:], dsize[W - 1:]
        at += n
    return out


def check(name, got, ref, size, kind, steps):
    """got is within one rounding to ``kind`` of ref, plus ``steps`` roundings of 2^-24 of ``size``."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    tol = HALF[kind] * np.abs(ref) + steps * U * size * (1 + HALF[kind]) + TINY[kind]
    off = np.abs(got - ref) / tol
    worst = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert not off.size or off[worst] <= 1.0, \
        f"{name}: {off[worst]:.3g} times the tolerance at {worst}: got {got[worst]!r}, want {ref[worst]!r}"


def softplus(x):
    return np.logaddexp(x, 0.0)


def scan(u, delta, A, B, C, D, z, bias, lengths, init=None, use_softplus=True):
    """The selective scan and, beside each result, a bound on its fp32 rounding errors in units of 2^-24.

    Roundings, relative: the step s from x = delta + bias: 3 |x| + 12 (the sum, the exponential's
    argument and value, the odd series); the decay e^{sA}: |sA| times (the step's + 4), and 7 (its
    value, its product with h, the sum, and what a tile's summed steps add: at most its length
    spread over its tokens); the input s u B: the step's + 3. They are carried by the recurrence
    itself. The output: a rounding per term of the sum over states, the skip's and the gate's."""
    T, ch = u.shape
    N, G = A.shape[1], B.shape[1]
    x = delta + (0.0 if bias is None else bias)
    s = softplus(x) if use_softplus else x
    rs = 3 * np.abs(x) + 12 if use_softplus else np.ones_like(x)
    spread = lambda v: np.repeat(v, ch // G, axis=0)  # noqa: E731
    y, ye = np.zeros((T, ch)), np.zeros((T, ch))
    fin, fe = np.zeros((len(lengths), ch, N)), np.zeros((len(lengths), ch, N))
    skip = np.zeros(ch) if D is None else D
    at = 0
    for i, n in enumerate(lengths):
        h = init[i].copy() if init is not None else np.zeros((ch, N))
        size, err = np.abs(h), np.zeros((ch, N))
        for t in range(at, at + n):
            a = np.exp(s[t][:, None] * A)
            inp = (s[t] * u[t])[:, None] * spread(B[t])
            dec = (rs[t][:, None] + 4) * np.abs(s[t][:, None] * A) + 7
            err = a * (err + size * dec) + (rs[t][:, None] + 3) * np.abs(inp)
            h, size = a * h + inp, a * size + np.abs(inp)
            Ct = np.abs(spread(C[t]))
            y[t] = (spread(C[t]) * h).sum(1)
            ye[t] = (Ct * err).sum(1) + (N + 6) * (Ct * size).sum(1)
        fin[i], fe[i] = h, err
        at += n
    y, ye = y + skip * u, ye + 3 * np.abs(skip * u)
    if z is not None:
        gate = z * sigmoid(z)
        ye = np.abs(gate) * (ye + (3 * np.abs(z) + 8) * np.abs(y))
        y = y * gate
    return y, ye, fin, fe


def attention(q, k, v, table, lens, scale, kind):
    """Attention of one token per sequence, lse, and bounds on their rounding errors (absolute, but for
    the rounding of the output). A score: a product sum of Dh terms in fp32 and three roundings; a
    probability: the score's error twice (its own and the sum's), exponential and arguments; its
    split into two 16-bit parts leaves 2^-16 (bf16), or 2^-22 and an absolute 2^-25 (fp16, whose
    small values are subnormal); sums over n tokens in fp32, 32 at a time and in pieces."""
    B, hq, dh = q.shape
    hkv, page = k.shape[2], k.shape[1]
    out, oe = np.zeros((B, hq, dh)), np.zeros((B, hq, dh))
    lse, le = np.full((B, hq), -np.inf), np.zeros((B, hq))
    rel, sub = (2.0 ** -16, 0.0) if kind == "bf16" else (2.0 ** -22, 2.0 ** -25)
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        t = np.arange(n)
        kk, vv = k[table[b, t // page], t % page], v[table[b, t // page], t % page]
        for h in range(hq):
            kh, vh = kk[:, h // (hq // hkv)], vv[:, h // (hq // hkv)]
            s = scale * (kh @ q[b, h])
            es = U * (dh + 4) * abs(scale) * (np.abs(kh) @ np.abs(q[b, h]))
            m = s.max()
            p = np.exp(s - m)
            L = p.sum()
            ep = 2 * es.max() + U * (4 * np.abs(s - m) + 2 * np.abs(s) + 8)
            out[b, h] = p @ vh / L
            size = (p[:, None] * np.abs(vh)).sum(0) / L
            oe[b, h] = ((p * ep)[:, None] * np.abs(vh)).sum(0) / L + size * ((p * ep).sum() / L + rel + U * (n / 16 + 200)) \
                + sub * np.abs(vh).sum(0) / L
            lse[b, h] = m + np.log(L)
            le[b, h] = (p * ep).sum() / L + U * (n / 16 + 200 + 4 * abs(lse[b, h]))
    return out, oe, lse, le


def scan_grads(u, delta, A, B, C, D, z, bias, lengths, init, use_softplus, dy, dfin):
    """Gradients of the selective scan by the chain rule, token by token from the end, and beside each
    a bound on its fp32 rounding errors in units of 2^-24, carried as in ``scan``: a product's error
    is each factor's times the other's size; a sum adds a rounding per term to the terms' sizes."""
    T, ch = u.shape
    N, G = A.shape[1], B.shape[1]
    per = ch // G
    x = delta + (0.0 if bias is None else bias)
    s = softplus(x) if use_softplus else x
    sig = sigmoid(x) if use_softplus else np.ones_like(x)
    rs = 3 * np.abs(x) + 12 if use_softplus else np.ones_like(x)
    spread = lambda v: np.repeat(v, per, axis=0)  # noqa: E731
    gather = lambda v: v.reshape(G, per, N).sum(1)  # noqa: E731
    skip = np.zeros(ch) if D is None else D
    z0 = np.zeros_like(u) if z is None else z
    gate = z * sigmoid(z) if z is not None else np.ones_like(u)
    rg = 3 * np.abs(z0) + 10                      # of the gate, relative
    g = dy * gate
    names = ("du", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddelta_bias", "d_initial_state")
    shapes = ((T, ch), (T, ch), (T, ch), (ch, N), (T, G, N), (T, G, N), (ch,), (ch,), (len(lengths), ch, N))
    out = {n: np.zeros(sh) for n, sh in zip(names, shapes)}
    err = {n: np.zeros(sh) for n, sh in zip(names, shapes)}
    chsum = 20 + ch / G / 32                      # roundings of a sum over a group's channels
    at = 0
    for i, n in enumerate(lengths):
        h = init[i].copy() if init is not None else np.zeros((ch, N))
        size, e = np.abs(h), np.zeros((ch, N))
        trail = []
        for t in range(at, at + n):
            a = np.exp(s[t][:, None] * A)
            inp = (s[t] * u[t])[:, None] * spread(B[t])
            dec = (rs[t][:, None] + 4) * np.abs(s[t][:, None] * A) + 7
            ah, sah, eah = a * h, a * size, a * (e + size * dec)
            h, size, e = ah + inp, sah + np.abs(inp), eah + (rs[t][:, None] + 3) * np.abs(inp)
            trail.append((a, dec, ah, sah, eah, h, size, e))
        dh = dfin[i].copy() if dfin is not None else np.zeros((ch, N))
        ds, de = np.abs(dh), np.zeros((ch, N))
        for t in range(at + n - 1, at - 1, -1):
            a, dec, ah, sah, eah, h, size, e = trail[t - at]
            Bt, Ct = spread(B[t]), spread(C[t])
            gt = g[t][:, None]
            dh, ds, de = dh + Ct * gt, ds + np.abs(Ct * gt), de + (rg[t][:, None] + 3) * np.abs(Ct * gt)
            out["dC"][t] = gather(gt * h)
            err["dC"][t] = gather(np.abs(gt) * (e + (rg[t][:, None] + chsum) * size))
            su = (s[t] * u[t])[:, None]
            out["dB"][t] = gather(dh * su)
            err["dB"][t] = gather(np.abs(su) * (de + (rs[t][:, None] + chsum) * ds))
            y = (Ct * h).sum(1) + skip * u[t]
            ey = (np.abs(Ct) * (e + (N + 6) * size)).sum(1) + 3 * np.abs(skip * u[t])
            if z is not None:
                f = dy[t] * silu_grad(z[t])
                sf = np.abs(dy[t]) * sigmoid(z[t]) * (1 + np.abs(z[t]))     # before its terms cancel
                out["dz"][t], err["dz"][t] = f * y, np.abs(f) * ey + rg[t] * sf * np.abs(y)
            into, si = (dh * Bt).sum(1), (ds * np.abs(Bt)).sum(1)
            ei = (de * np.abs(Bt)).sum(1) + (N + 6) * si
            out["du"][t] = s[t] * into + skip * g[t]
            err["du"][t] = np.abs(s[t]) * (ei + (rs[t] + 2) * si) + (rg[t] + 3) * np.abs(skip * g[t])
            q, sq = dh * ah, ds * sah
            eq = de * sah + ds * eah
            through = (q * A).sum(1) + u[t] * into
            out["ddelta"][t] = through * sig[t]
            sizes = (sq * np.abs(A)).sum(1) + np.abs(u[t]) * si
            err["ddelta"][t] = sig[t] * ((np.abs(A) * (eq + (N + 8) * sq)).sum(1) + np.abs(u[t]) * ei
                                         + (3 * np.abs(x[t]) + 12) * sizes)
            out["dA"] += q * s[t][:, None]
            err["dA"] += np.abs(s[t][:, None]) * (eq + (rs[t][:, None] + 4) * sq)
            out["dD"] += g[t] * u[t]
            err["dD"] += (rg[t] + 2) * np.abs(g[t] * u[t])
            out["ddelta_bias"] += out["ddelta"][t]
            err["ddelta_bias"] += err["ddelta"][t]
            # sums over tokens: a rounding per token of a tile and per tile, of what they add up
            many = T / 16 + 160
            err["dA"] += many * np.abs(s[t][:, None]) * sq
            err["dD"] += many * np.abs(g[t] * u[t])
            err["ddelta_bias"] += many * sizes * sig[t]
            dh, ds, de = dh * a, ds * a, a * (de + ds * dec)
        out["d_initial_state"][i], err["d_initial_state"][i] = dh, de + ds
        at += n
    return out, err
