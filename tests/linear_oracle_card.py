"""linear_oracle's recurrences and bounds with all heads at once, in 64 bits on the card, for batches whose segments hold
several chunks; and beside the gradients of decays the size that they cannot exceed. Each result comes with its bound in
units of 2^-24, counted as linear_oracle says."""
import torch

from linear_oracle import LEAST, PARTS2


def _decay(g):
    """exp(g), and the units that a decay loses in a token, over a state [H, K, V]."""
    return torch.exp(g)[:, None, None], (1.5 * g.clamp_min(-200.0).abs() + 6)[:, None, None]


def _pair(a, b):
    return a[:, :, None] * b[:, None]


def _rows(s, x):        # [H, K, V] times [H, V]
    return (s @ x[:, :, None])[:, :, 0]


def _columns(s, x):     # [H, K, V] times [H, K]
    return (x[:, None] @ s)[:, 0]


def forward_and_backward(d, lengths, do, dfin, scale):
    """Two dicts of results and bounds: out, final, dq, dk, dv, dg, d_initial_state; and for dg what it cannot exceed,
    |X| |Y| of the state before a token (decayed) and the gradient of the one that it leaves."""
    q, k, v, g = (d[n].double() for n in ("q", "k", "v", "g"))
    T, H, K = q.shape
    V = v.shape[2]
    g = g if g.dim() == 2 else g.expand(T, H)
    do, init = do.double(), d["initial_state"]
    zeros = lambda like: torch.zeros_like(like, dtype=torch.float64)  # noqa: E731
    r = dict(out=zeros(v), dq=zeros(q), dk=zeros(q), dv=zeros(v), dg=zeros(g))
    e = {n: torch.zeros_like(x) for n, x in r.items()}
    r["final"], r["d_initial_state"], e["final"], e["d_initial_state"] = ([] for _ in range(4))
    most = zeros(g)
    top = {n: x.abs().max().item() if x.numel() else 0.0 for n, x in (("q", q), ("k", k), ("v", v), ("do", do))}
    none = torch.zeros(H, K, V, dtype=torch.float64, device=q.device)
    at = 0
    for n, length in enumerate(lengths):
        X = init[n].double() if init is not None else none
        size, err, lost, trail = X.abs(), none, none, []
        for t in range(at, at + length):
            a, dec = _decay(g[t])
            kv, ak, av = _pair(k[t], v[t]), k[t].abs(), v[t].abs()
            lost = lost + LEAST * size
            X, err, size = a * X, a * (err + size * dec), a * size
            trail.append((X, err + lost, size))
            lost = lost + LEAST * ak[:, :, None] * (3 + av[:, None])
            X, err, size = X + kv, err + 8 * kv.abs(), size + kv.abs()
            err = err + 3 * size
            r["out"][t], r["dq"][t] = scale * _columns(X, q[t]), scale * _rows(X, do[t])
            each = err + lost + LEAST * (3 + size)
            e["out"][t] = abs(scale) * _columns(each + (PARTS2 + 3 * K + 64) * size, q[t].abs()) + LEAST * 192 * top["v"]
            e["dq"][t] = abs(scale) * _rows(each + (PARTS2 + 3 * V + 64) * size, do[t].abs()) + LEAST * 192 * top["k"]
        r["final"].append(X), e["final"].append(err + lost + 2 * size)
        Y = dfin[n].double() if dfin is not None else none
        size, err, lost = Y.abs(), none, none
        for t in range(at + length - 1, at - 1, -1):
            qd, aq = scale * _pair(q[t], do[t]), q[t].abs()
            lost = lost + LEAST * aq[:, :, None] * (3 + do[t].abs()[:, None])
            Y, err, size = Y + qd, err + 9 * qd.abs(), size + qd.abs()
            err = err + 3 * size
            each = err + lost + LEAST * (3 + size)
            r["dk"][t], r["dv"][t] = _rows(Y, v[t]), _columns(Y, k[t])
            e["dk"][t] = _rows(each + (PARTS2 + 3 * V + 64) * size, v[t].abs()) + LEAST * 192 * top["q"]
            e["dv"][t] = _columns(each + (PARTS2 + 3 * K + 64) * size, k[t].abs()) + LEAST * 192 * top["do"]
            x, ex, sx = trail[t - at]
            r["dg"][t] = (x * Y).sum((1, 2))
            most[t] = x.norm(dim=(1, 2)) * Y.norm(dim=(1, 2))
            # every term of the sum passes the token: contractions in three parts, a rounding for each token of a chunk
            e["dg"][t] = (ex * size + sx * (err + lost) + (3 * (K + V) + 256) * sx * size).sum((1, 2))
            a, dec = _decay(g[t])
            lost = lost + LEAST * size
            Y, err, size = a * Y, a * (err + size * dec), a * size
        r["d_initial_state"].append(Y), e["d_initial_state"].append(err + lost + 2 * size)
        at += length
    e["dg"] += LEAST * 64 * (top["q"] * top["do"] + top["k"] * top["v"]) * (K + V) * 64
    for x in (r, e):
        x["final"], x["d_initial_state"] = torch.stack(x["final"]), torch.stack(x["d_initial_state"])
    return r, e, most
