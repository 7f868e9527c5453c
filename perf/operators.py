"""The operators beside the delta-rule recurrence that a hybrid linear-attention decoder runs: the
short causal convolution in front of a recurrence, the selective state space scan, and the
attention of one new token over a paged key-value cache. Each is measured over the sizes that it
meets: the smallest calls, ordinary ones and the largest, each direction and type.

Channels are heads x 128 as in the library's own workloads (2, 8, 16 and 32 heads), tokens and
batches likewise (256, 8 x 1024, 8192, 65536, 12 skewed sequences, 256 sequences of one token).

``own`` false: the plain form (elementary torch operations in fp32). ``own`` true: the library.
"""
import math

import torch
import torch.nn.functional as F

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the convolution of one projection of an 8192-token prompt (32 heads), read in place from a
        # projection's output that is twice as wide
        dict(name="conv prompt 8192x4096", op="conv", lengths="8192", ch=4096, width=4, type="bf16", wide=2, init=False),
        # its gradients in training, 8 packed sequences, 16 heads
        dict(name="conv grad 8x1024x2048", op="conv_bwd", lengths="1024," * 7 + "1024", ch=2048, width=4, type="bf16",
             wide=1, init=True),
        # one token of each of 256 sequences (serving)
        dict(name="conv token 256x4096", op="conv_step", batch=256, ch=4096, width=4, type="bf16"),
        # the smallest prompt: latency counts
        dict(name="scan prompt 256x256", op="scan", lengths="256", ch=256, n=16, groups=1, type="bf16", gate=True,
             wide=1, init=False),
        # a prompt of ordinary length over 32 heads' channels; input and gate are halves of one projection
        dict(name="scan prompt 8192x4096", op="scan", lengths="8192", ch=4096, n=16, groups=1, type="bf16", gate=True,
             wide=2, init=False),
        # a long document over few channels: only the time axis has work for the whole card
        dict(name="scan long 65536x1024", op="scan", lengths="65536", ch=1024, n=16, groups=1, type="bf16", gate=True,
             wide=1, init=False),
        # a skewed packed batch of odd sizes in fp32, two groups, an odd state size
        dict(name="scan ragged fp32", op="scan", lengths="37,2311,1,0,409,5003,16,1283", ch=1002, n=21, groups=2,
             type="fp32", gate=False, wide=1, init=True),
        # training: gradients over 8 packed sequences with states
        dict(name="scan grad 8x1024x2048", op="scan_bwd", lengths="1024," * 7 + "1024", ch=2048, n=16, groups=1,
             type="bf16", gate=True, wide=1, init=True),
        # one token of each of 256 sequences (serving): the state is read and written once
        dict(name="scan token 256x4096", op="scan_step", batch=256, ch=4096, n=16, groups=1, type="bf16", gate=True),
        # the smallest attention call: two short sequences of two heads
        dict(name="attn token 2x256", op="attn", lengths="256,113", heads=2, kv_heads=2, dim=128, page=16, type="bf16"),
        # one long document answered token by token: only the cache's length has work for the whole card
        dict(name="attn token 1x65536", op="attn", lengths="65536", heads=32, kv_heads=8, dim=128, page=16,
             type="bf16"),
        # a serving batch with skewed lengths, an empty slot among them, pages of 32 tokens
        dict(name="attn token ragged fp16", op="attn", lengths=",".join(str(x) for x in _skewed()), heads=32,
             kv_heads=4, dim=128, page=32, type="fp16"),
    ]


def _skewed():
    """64 cache lengths spread evenly over the logarithm of 37 to 16384, an empty slot among them."""
    e = [int(37 * (16384 / 37) ** ((i * 37 % 64) / 63)) for i in range(64)]
    e[11] = 0
    return e


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total):
    """1 to 12 lengths that add up to total, some of them zero or one."""
    n = rng.choice((1, 1, 2, 3, 5, 8, 12))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(("conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_step", "attn", "attn"))
    kind = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("conv", "conv_bwd"):
        tokens = _log(rng, 1, 32768)
        ch = _log(rng, 1, max(1, min(8192, (1 << 24) // tokens)))
        return dict(op=op, lengths=_split(rng, tokens), ch=ch, width=rng.choice((2, 3, 4, 4, 4)), type=kind,
                    wide=rng.choice((1, 2, 3)), init=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, batch=_log(rng, 1, 256), ch=_log(rng, 1, 4096), width=rng.choice((2, 3, 4, 4, 4)), type=kind)
    if op in ("scan", "scan_bwd"):
        tokens = _log(rng, 1, 65536 if op == "scan" else 8192)
        n = rng.choice((16, 16, 16, 8, 64, rng.randint(1, 128)))
        most = 1 << 28
        ch = _log(rng, 1, max(1, min(4096, most // (tokens * n))))
        groups = rng.choice([g for g in (1, 1, 2, 3, 4) if ch % g == 0])
        return dict(op=op, lengths=_split(rng, tokens), ch=ch, n=n, groups=groups, type=kind,
                    gate=rng.random() < 0.6, wide=rng.choice((1, 2)), init=rng.random() < 0.5)
    if op == "scan_step":
        n = rng.choice((16, 16, 16, 8, 64, rng.randint(1, 128)))
        ch = _log(rng, 1, min(4096, 65536 // n))
        return dict(op=op, batch=_log(rng, 1, 256), ch=ch, n=n, groups=rng.choice([g for g in (1, 2, 4) if ch % g == 0]),
                    type=kind, gate=rng.random() < 0.6)
    kv = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128, 128, 256))
    batch = _log(rng, 1, 96)
    longest = _log(rng, 1, min(65536, (1 << 28) // (batch * kv * dim)))
    lens = [rng.choice((longest, _log(rng, 1, longest), _log(rng, 1, longest))) for _ in range(batch)]
    if batch > 4:
        lens[rng.randrange(batch)] = 0
    return dict(op=op, lengths=",".join(str(x) for x in lens), heads=kv * rng.choice((1, 2, 4, 5, 8, 16)), kv_heads=kv,
                dim=dim, page=rng.choice((1, 8, 16, 16, 32, 48, 64, 256)), type=rng.choice(("bf16", "fp16")))


# ---------------------------------------------------------------------------- inputs
def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]
    norm = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    s = dict(case=case)
    if op == "attn":
        lens, page = _lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        total, most = max(1, sum(need)), max(1, max(need))
        pages = total + max(1, total // 8)  # a cache is never quite full, and its pages are in no order
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
        table = torch.full((len(lens), most), -1, dtype=torch.int32)
        at = 0
        for i, k in enumerate(need):
            table[i, :k] = order[at:at + k]
            at += k
        shape = (pages, page, case["kv_heads"], case["dim"])
        s.update(q=norm(len(lens), case["heads"], case["dim"]).to(dt), k=norm(*shape).to(dt), v=norm(*shape).to(dt),
                 table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
        return s
    ch = case["ch"]
    if op.startswith("conv"):
        s.update(weight=norm(ch, case["width"]) / math.sqrt(case["width"]), bias=norm(ch) * 0.1)
        if op == "conv_step":
            s.update(x=norm(case["batch"], ch).to(dt), state=norm(case["batch"], case["width"] - 1, ch).to(dt))
            return s
    else:
        n, groups = case["n"], case["groups"]
        step = torch.exp(rand(ch) * math.log(100.0) + math.log(1e-3))  # step sizes of 1e-3 to 0.1
        s.update(A=-torch.exp(torch.log(torch.arange(1, n + 1, device=dev).float()) + 0.1 * norm(ch, n)),
                 D=1 + 0.1 * norm(ch), bias=step + torch.log(-torch.expm1(-step)))
        if op == "scan_step":
            rows = case["batch"]
        else:
            rows = sum(_lengths(case))
        s.update(B=norm(rows, groups, n).to(dt), C=norm(rows, groups, n).to(dt), delta=(0.5 * norm(rows, ch)).to(dt),
                 z=None)
        if op == "scan_step":
            s.update(x=norm(rows, ch).to(dt), state=norm(rows, ch, n) * 0.3)
            if case["gate"]:
                s["z"] = norm(rows, ch).to(dt)
            return s
    lens = _lengths(case)
    rows, seqs = sum(lens), len(lens)
    cu = torch.zeros(seqs + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    s["cu"] = cu.to(dev)
    proj = norm(rows, case["wide"] * ch).to(dt)
    s["x"] = proj[:, :ch]
    if case.get("gate"):
        s["z"] = proj[:, ch:2 * ch] if case["wide"] > 1 else norm(rows, ch).to(dt)
    s["init"] = None
    if case["init"]:
        s["init"] = norm(seqs, case["width"] - 1, ch).to(dt) if op.startswith("conv") else norm(seqs, ch, case["n"]) * 0.3
    if op.endswith("_bwd"):
        s["dy"] = norm(rows, ch).to(dt)
        s["dfin"] = norm(seqs, case["width"] - 1, ch) if op == "conv_bwd" else norm(seqs, ch, case["n"]) * 0.1
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"conv": _conv, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "scan": _scan, "scan_bwd": _scan_bwd,
            "scan_step": _scan_step, "attn": _attn}[op](s)


def _own(s, op):
    import chunked_gated_delta_kda_amd as kda

    if op == "conv":
        y, fin = kda.conv_fwd(s["x"], s["weight"], s["bias"], s["cu"], s["init"])
        return {"y": y, "final": fin}
    if op == "conv_bwd":
        return kda.conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["cu"], s["init"], s["dfin"])
    if op == "conv_step":
        y, state = kda.conv_decode(s["x"], s["weight"], s["bias"], s["state"])
        return {"y": y, "state": state}
    if op == "scan":
        y, fin = kda.ssm_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["cu"], s["init"])
        return {"y": y, "final": fin}
    if op == "scan_bwd":
        return kda.ssm_bwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["dy"], s["D"], s["z"], s["bias"], s["cu"],
                           s["init"], s["dfin"])
    if op == "scan_step":
        y, state = kda.ssm_decode(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["state"])
        return {"y": y, "state": state}
    out, lse = kda.attn_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------- plain forms
def _sequence(cu, rows):
    """For every row its sequence, its place in it, and the rows left after it."""
    row = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    start, end = cu[:-1].long()[seq], cu[1:].long()[seq]
    return seq, row - start, end - 1 - row


def _silu_grad(x):
    sg = torch.sigmoid(x)
    return sg * (1 + x * (1 - sg))


def _window(s):
    """The taps of every row, [rows, width, ch] in fp32: rows before a sequence's first are its initial state."""
    x, cu, width = s["x"].float(), s["cu"], s["case"]["width"]
    seq, pos, _ = _sequence(cu, x.shape[0])
    seqs, ch = cu.shape[0] - 1, x.shape[1]
    init = s["init"].float() if s["init"] is not None else x.new_zeros(seqs, width - 1, ch)
    both = torch.cat([init.reshape(seqs * (width - 1), ch), x])
    back = torch.arange(width - 1, -1, -1, device=x.device)
    p = pos[:, None] - back
    at = torch.where(p >= 0, seqs * (width - 1) + torch.arange(x.shape[0], device=x.device)[:, None] - back,
                     seq[:, None] * (width - 1) + p + width - 1)
    # the state after each sequence: its last width-1 rows
    p = (cu[1:] - cu[:-1]).long()[:, None] - torch.arange(width - 1, 0, -1, device=x.device)
    fin = torch.where(p >= 0, seqs * (width - 1) + cu[:-1].long()[:, None] + p,
                      torch.arange(seqs, device=x.device)[:, None] * (width - 1) + p + width - 1)
    return both, at, fin


def _conv(s):
    both, at, fin = _window(s)
    pre = (both[at] * s["weight"].t()).sum(1) + s["bias"]
    return {"y": (pre * torch.sigmoid(pre)).to(s["x"].dtype), "final": both[fin].to(s["x"].dtype)}


def _conv_bwd(s):
    both, at, fin = _window(s)
    taps = both[at]
    pre = (taps * s["weight"].t()).sum(1) + s["bias"]
    dpre = s["dy"].float() * _silu_grad(pre)
    grad = torch.zeros_like(both)
    grad.index_add_(0, fin.reshape(-1), s["dfin"].reshape(-1, grad.shape[1]))
    grad.index_add_(0, at.reshape(-1), (dpre[:, None] * s["weight"].t()).reshape(-1, grad.shape[1]))
    first = s["dfin"].shape[0] * s["dfin"].shape[1]
    return {"dx": grad[first:].to(s["x"].dtype), "dweight": (dpre[:, None] * taps).sum(0).t(), "dbias": dpre.sum(0),
            "d_initial_state": grad[:first].reshape(s["dfin"].shape)}


def _conv_step(s):
    taps = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    pre = (taps * s["weight"].t()).sum(1) + s["bias"]
    s["state"].copy_(taps[:, 1:])
    return {"y": (pre * torch.sigmoid(pre)).to(s["x"].dtype), "state": s["state"]}


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis from h = 0, by doubling the span that each row covers."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _scan_parts(s):
    """Step sizes, decays and inputs of the recurrence, the states' inputs folded in."""
    x, ch = s["x"].float(), s["x"].shape[1]
    per = ch // s["B"].shape[1]
    pre = s["delta"].float() + s["bias"]
    delta = torch.log1p(torch.exp(-pre.abs())) + pre.clamp(min=0)
    Bc = s["B"].float().repeat_interleave(per, 1)
    Cc = s["C"].float().repeat_interleave(per, 1)
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * Bc
    return x, pre, delta, Bc, Cc, a, b


def _states(s, a, b):
    """h_t of every row and h_{t-1}: a sequence's first row starts from its initial state."""
    seq, pos, left = _sequence(s["cu"], a.shape[0])
    first = (pos == 0)[:, None, None]
    init = s["init"] if s["init"] is not None else torch.zeros_like(s["A"]).expand(s["cu"].shape[0] - 1, *s["A"].shape)
    before = init[seq] if s["init"] is not None else torch.zeros_like(a)
    h = _prefix(torch.where(first, 0.0, a), torch.where(first, a * before + b, b))
    prev = torch.where(first, before, torch.cat([h[:1], h[:-1]]))
    empty = (s["cu"][1:] == s["cu"][:-1])[:, None, None]
    last = (s["cu"][1:].long() - 1).clamp(min=0)
    fin = torch.where(empty, init, h[last]) if a.shape[0] else init.clone()
    return h, prev, fin, left


def _scan(s):
    x, _, _, _, Cc, a, b = _scan_parts(s)
    h, _, fin, _ = _states(s, a, b)
    y = (h * Cc).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "final": fin}


def _scan_bwd(s):
    x, pre, delta, Bc, Cc, a, b = _scan_parts(s)
    h, prev, _, left = _states(s, a, b)
    seq, pos, _ = _sequence(s["cu"], x.shape[0])
    dt, ch, groups = s["x"].dtype, x.shape[1], s["B"].shape[1]
    g = {"dz": None}
    dy = s["dy"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = (h * Cc).sum(-1) + s["D"] * x
        g["dz"] = (dy * y * _silu_grad(z)).to(dt)
        dy = dy * z * torch.sigmoid(z)
    # dh_t = C_t dy_t + a_{t+1} dh_{t+1}; after a sequence's last row comes its final state's gradient
    last = (left == 0)[:, None, None]
    after = torch.where(last, 0.0, torch.cat([a[1:], a[:1]]))
    own_part = Cc * dy[..., None] + torch.where(last, s["dfin"][seq], 0.0)
    dh = _prefix(after.flip(0), own_part.flip(0)).flip(0)
    decay = dh * a * prev  # dL/d(log a)
    through = (dh * Bc).sum(-1)
    ddelta = (decay * s["A"]).sum(-1) + x * through
    dpre = ddelta * torch.sigmoid(pre)
    empty = (s["cu"][1:] == s["cu"][:-1])[:, None, None]
    head = s["cu"][:-1].long().clamp(max=max(0, x.shape[0] - 1))
    per = lambda v: v.reshape(v.shape[0], groups, ch // groups, -1).sum(2)  # noqa: E731
    g.update(du=(delta * through + s["D"] * dy).to(dt), ddelta=dpre.to(dt), dA=(decay * delta[..., None]).sum(0),
             dB=per(dh * (delta * x)[..., None]).to(dt), dC=per(h * dy[..., None]).to(dt), dD=(dy * x).sum(0),
             ddelta_bias=dpre.sum(0), d_initial_state=torch.where(empty, s["dfin"], a[head] * dh[head]))
    return g


def _scan_step(s):
    x, _, _, _, Cc, a, b = _scan_parts(s)
    h = a * s["state"] + b
    s["state"].copy_(h)
    y = (h * Cc).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _attn(s):
    q, table, lens = s["q"].float(), s["table"].long().clamp(min=0), s["lens"].long()
    batch, heads, dim = q.shape
    kv = s["k"].shape[2]
    k = s["k"][table].float().reshape(batch, -1, kv, dim).transpose(1, 2)
    v = s["v"][table].float().reshape(batch, -1, kv, dim).transpose(1, 2).contiguous()
    qg = q.reshape(batch, kv, heads // kv, dim) / math.sqrt(dim)
    score = torch.matmul(k, qg.transpose(2, 3).contiguous()).transpose(2, 3)
    seen = (torch.arange(k.shape[2], device=q.device) < lens[:, None])[:, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top).reshape(batch, heads)
    return {"out": out.reshape(batch, heads, dim).to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, size = case["op"], torch.finfo(TYPES[case["type"]]).bits // 8
    if op == "attn":
        lens = _lengths(case)
        tokens, batch = sum(lens), len(lens)
        bytes_ = 2 * tokens * case["kv_heads"] * case["dim"] * size + batch * case["heads"] * (2 * case["dim"] * size + 4)
        bytes_ += 4 * sum(-(-n // case["page"]) for n in lens)
        return {"bytes": bytes_, "flops": 4 * tokens * case["heads"] * case["dim"]}
    rows = case["batch"] if op.endswith("_step") else sum(_lengths(case))
    seqs = case["batch"] if op.endswith("_step") else len(_lengths(case))
    el, ch = rows * case["ch"], case["ch"]
    if op.startswith("conv"):
        w = case["width"]
        state = seqs * (w - 1) * ch
        if op == "conv_bwd":
            return {"bytes": 3 * el * size + state * (8 + size * case["init"]) + 8 * ch * (w + 1), "flops": el * (6 * w + 10)}
        states = state * size * (2 if op == "conv_step" or case["init"] else 1)
        return {"bytes": 2 * el * size + states + 4 * ch * (w + 1), "flops": el * (2 * w + 5)}
    n, gate = case["n"], bool(case["gate"])
    bc, state = 2 * rows * case["groups"] * n, seqs * ch * n * 4
    if op == "scan_bwd":
        return {"bytes": (5 + 2 * gate) * el * size + 2 * bc * size + state * (2 + case["init"]) + 8 * ch * (n + 2),
                "flops": el * (n * 21 + 30)}
    states = state * (2 if op == "scan_step" or case["init"] else 1)
    return {"bytes": (3 + gate) * el * size + bc * size + states + 4 * ch * (n + 2), "flops": el * (n * 7 + 15)}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op == "attn":
        return _exact_attn(case, d)
    if op == "conv_step":
        return _exact_conv_step(d)
    if op.startswith("conv"):
        return _exact_conv(case, d, op == "conv_bwd")
    return _exact_scan(case, d)


def _exact_attn(case, d):
    outs, lses = [], []
    share = case["heads"] // case["kv_heads"]
    for i, n in enumerate(_lengths(case)):
        q = d["q"][i]
        if n == 0:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device=q.device))
            continue
        rows = d["table"][i, :-(-n // case["page"])].long()
        k, v = (c[rows].flatten(0, 1)[:n].permute(1, 0, 2).contiguous() for c in (d["k"], d["v"]))
        o, e = [], []
        for h in range(case["heads"]):
            score = (k[h // share] @ q[h]) * case["dim"] ** -0.5
            o.append(torch.softmax(score, 0) @ v[h // share])
            e.append(torch.logsumexp(score, 0))
        outs.append(torch.stack(o))
        lses.append(torch.stack(e))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_conv_step(d):
    pre = d["bias"] + d["weight"][:, -1] * d["x"]
    for j in range(d["weight"].shape[1] - 1):
        pre = pre + d["weight"][:, j] * d["state"][:, j]
    return {"y": F.silu(pre), "state": torch.cat([d["state"][:, 1:], d["x"][:, None]], 1)}


def _exact_conv(case, d, backward):
    width, ch = case["width"], case["ch"]
    ys, fins, dxs, dinits, dw, db = [], [], [], [], 0, 0
    at = 0
    w = d["weight"]
    for i, n in enumerate(_lengths(case)):
        head = d["init"][i] if d["init"] is not None else w.new_zeros(width - 1, ch)
        line = torch.cat([head, d["x"][at:at + n]])
        pre = d["bias"] + sum(w[:, j] * line[j:j + n] for j in range(width))
        ys.append(F.silu(pre))
        fins.append(line[n:])
        if backward:
            sg = torch.sigmoid(pre)
            dpre = d["dy"][at:at + n] * (sg + pre * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for j in range(width):
                dline[j:j + n] += w[:, j] * dpre
            dline[n:] += d["dfin"][i]
            dinits.append(dline[:width - 1])
            dxs.append(dline[width - 1:])
            dw = dw + torch.stack([(dpre * line[j:j + n]).sum(0) for j in range(width)], 1)
            db = db + dpre.sum(0)
        at += n
    if backward:
        return {"dx": torch.cat(dxs), "dweight": dw, "dbias": db, "d_initial_state": torch.stack(dinits)}
    return {"y": torch.cat(ys), "final": torch.stack(fins)}


def _exact_scan(case, d):
    op = case["op"]
    ch, n, groups = case["ch"], case["n"], case["groups"]
    pre = d["delta"] + d["bias"]
    delta = torch.logaddexp(pre, torch.zeros_like(pre))
    x, A = d["x"], d["A"]
    spread = lambda v: v[:, None].expand(groups, ch // groups, n).reshape(ch, n)  # noqa: E731
    gather = lambda v: v.reshape(groups, ch // groups, n).sum(1)  # noqa: E731
    gate = None if d["z"] is None else d["z"] * torch.sigmoid(d["z"])
    if op == "scan_step":
        Bf = d["B"][:, :, None].expand(-1, groups, ch // groups, n).reshape(-1, ch, n)
        Cf = d["C"][:, :, None].expand(-1, groups, ch // groups, n).reshape(-1, ch, n)
        h = d["state"] * torch.exp(delta[..., None] * A) + (delta * x)[..., None] * Bf
        y = torch.einsum("rcn,rcn->rc", h, Cf) + d["D"] * x
        return {"y": y if gate is None else y * gate, "state": h}
    # token after token, as the recurrence is written
    bwd = op == "scan_bwd"
    y = torch.zeros_like(x)
    trail = x.new_zeros(x.shape[0], ch, n) if bwd else None  # the state before each token
    fins, at = [], 0
    for i, length in enumerate(_lengths(case)):
        h = d["init"][i].clone() if d["init"] is not None else x.new_zeros(ch, n)
        for t in range(at, at + length):
            if bwd:
                trail[t] = h
            h = h * torch.exp(delta[t, :, None] * A) + (delta[t] * x[t])[:, None] * spread(d["B"][t])
            y[t] = (h * spread(d["C"][t])).sum(1)
        fins.append(h)
        at += length
    y = y + d["D"] * x
    if not bwd:
        return {"y": y if gate is None else y * gate, "final": torch.stack(fins)}
    g = {"du": torch.zeros_like(x), "ddelta": torch.zeros_like(x), "dA": torch.zeros_like(A),
         "dB": torch.zeros_like(d["B"]), "dC": torch.zeros_like(d["C"]), "dz": None}
    dy = d["dy"]
    if gate is not None:
        sg = torch.sigmoid(d["z"])
        g["dz"] = dy * y * (sg + d["z"] * sg * (1 - sg))
        dy = dy * gate
    dinit = [None] * len(fins)
    at = x.shape[0]
    for i in range(len(fins) - 1, -1, -1):
        dh = d["dfin"][i].clone()
        for t in range(at - 1, at - 1 - _lengths(case)[i], -1):
            a, Bt, Ct = torch.exp(delta[t, :, None] * A), spread(d["B"][t]), spread(d["C"][t])
            dh = dh + dy[t][:, None] * Ct
            ah = a * trail[t]
            g["dC"][t] = gather(dy[t][:, None] * (ah + (delta[t] * x[t])[:, None] * Bt))
            g["dB"][t] = gather(dh * (delta[t] * x[t])[:, None])
            into = (dh * Bt).sum(1)
            g["du"][t] = delta[t] * into
            g["ddelta"][t] = (dh * ah * A).sum(1) + x[t] * into
            g["dA"] += dh * ah * delta[t][:, None]
            dh = dh * a
        at -= _lengths(case)[i]
        dinit[i] = dh
    g["du"] += d["D"] * dy
    g["ddelta"] *= torch.sigmoid(pre)
    g.update(dD=(dy * x).sum(0), ddelta_bias=g["ddelta"].sum(0), d_initial_state=torch.stack(dinit))
    return g
