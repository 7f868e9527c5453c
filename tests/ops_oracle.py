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
