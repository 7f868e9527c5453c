"""More operators of a hybrid decoder: linear attention with a decay for each head (prompts, gradients, single
tokens), the writer of the paged key-value cache with the position rotation on the way, and the attention of one new
token over such a cache held in 4 bits. Each is measured over the sizes that it meets: the smallest calls, ordinary
ones and the largest, each direction and type.

Heads are 128 wide (and 64) as in the library's own workloads (2, 8, 16 and 32 heads), tokens and batches likewise (256,
8 x 1024, 8192, 65536, 12 skewed sequences, 256 sequences of one token).

``own`` false: the plain form (elementary torch operations). ``own`` true: the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 64      # tokens that the plain form of the linear attention takes as one block
GROUP = 32      # elements that share a scale in the 4-bit cache


def listed():
    return [
        # the smallest prompt: latency counts
        dict(name="linear prompt 256x2", op="linear", lengths="256", heads=2, dk=128, dv=128, type="bf16", fixed=False,
             joint=False, init=False),
        # a prompt of ordinary length, 32 heads, read in place from one projection's output; slopes fixed for each head
        dict(name="linear prompt 8192x32", op="linear", lengths="8192", heads=32, dk=128, dv=128, type="bf16", fixed=True,
             joint=True, init=False),
        # a long document over few heads: only the time axis has work for the whole card; decays from the data
        dict(name="linear long 65536x8", op="linear", lengths="65536", heads=8, dk=128, dv=128, type="bf16", fixed=False,
             joint=False, init=False),
        # a skewed packed batch of odd lengths, continued from states, narrow keys
        dict(name="linear ragged fp16", op="linear", lengths="37,2311,1,0,409,5003,16,1283,64,63,65,190", heads=5, dk=64,
             dv=128, type="fp16", fixed=False, joint=False, init=True),
        # training: gradients over 8 packed sequences with states
        dict(name="linear grad 8x1024x16", op="linear_bwd", lengths="1024," * 7 + "1024", heads=16, dk=128, dv=128,
             type="bf16", fixed=False, joint=False, init=True),
        # one token of each of 256 sequences (serving): the state is read and written once
        dict(name="linear token 256x32", op="linear_step", batch=256, heads=32, dk=128, dv=128, type="bf16", fixed=False),
        # one token of each of 256 sequences goes into the cache that attention then reads
        dict(name="append token 256", op="append", past=",".join(str(1 + i * 7 % 1024) for i in range(256)),
             new=",".join(["1"] * 256), heads=32, kv_heads=8, dim=128, rot=128, pairs=False, page=16, type="bf16",
             four=False),
        # skewed prompts, some of them continued, rotation of neighbouring pairs in half of a head
        dict(name="append ragged fp16", op="append", past="0,0,17,4001,0,5,0,0,129,0,64,1",
             new="1,30,4096,17,900,2048,0,333,16,700,49,2", heads=32, kv_heads=4, dim=128, rot=64, pairs=True, page=32,
             type="fp16", four=False),
        # 8 prompts into a cache of 4 bits, which is then read back
        dict(name="append 4 bits 8x1024", op="append", past=",".join(["0"] * 8), new=",".join(["1024"] * 8), heads=32,
             kv_heads=8, dim=128, rot=128, pairs=False, page=16, type="bf16", four=True),
        # the smallest attention call: two short sequences of two heads
        dict(name="attn 4 bits 2x256", op="attn", lengths="256,113", heads=2, kv_heads=2, dim=128, page=16, type="bf16"),
        # one long document answered token by token: only the cache's length has work for the whole card
        dict(name="attn 4 bits 1x65536", op="attn", lengths="65536", heads=32, kv_heads=8, dim=128, page=16, type="bf16"),
        # a serving batch with skewed lengths, an empty slot among them, pages of 32 tokens
        dict(name="attn 4 bits ragged fp16", op="attn", lengths=",".join(str(x) for x in _skewed()), heads=32, kv_heads=4,
             dim=128, page=32, type="fp16"),
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
    op = rng.choice(("linear", "linear", "linear_bwd", "linear_step", "append", "append", "attn", "attn"))
    kind = rng.choice(("bf16", "bf16", "fp16"))
    if op.startswith("linear"):
        dims = dict(dk=rng.choice((64, 128, 128)), dv=rng.choice((64, 128, 128)), type=kind, fixed=rng.random() < 0.4)
        if op == "linear_step":
            return dict(op=op, batch=_log(rng, 1, 256), heads=rng.randint(1, 32), **dims)
        most = 1 << 19 if op == "linear" else 1 << 17
        tokens = _log(rng, 1, 65536 if op == "linear" else 8192)
        heads = rng.randint(1, max(1, min(32, most // tokens // (2 if kind == "fp16" else 1))))
        return dict(op=op, lengths=_split(rng, tokens), heads=heads, joint=rng.random() < 0.4, init=rng.random() < 0.5,
                    **dims)
    kv = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128, 128, 256))
    page = rng.choice((1, 8, 16, 16, 32, 48, 64, 256))
    if op == "append":
        batch = _log(rng, 1, 256)
        most = max(1, (1 << 21) // (batch * kv * dim))
        token = rng.random() < 0.4
        new = [1 if token else rng.choice((0, 1, _log(rng, 1, most), most)) for _ in range(batch)]
        if not sum(new):
            new[-1] = 1
        past = [rng.choice((0, _log(rng, 1, 2 * most))) for _ in range(batch)]
        return dict(op=op, past=",".join(map(str, past)), new=",".join(map(str, new)), heads=kv * rng.choice((1, 2, 4, 5, 8)),
                    kv_heads=kv, dim=dim, rot=rng.choice((dim, dim, dim // 2)), pairs=rng.random() < 0.4, page=page, type=kind,
                    four=rng.random() < 0.5)
    batch = _log(rng, 1, 96)
    longest = _log(rng, 1, min(65536, (1 << 28) // (batch * kv * dim)))
    lens = [rng.choice((longest, _log(rng, 1, longest), _log(rng, 1, longest))) for _ in range(batch)]
    if batch > 4:
        lens[rng.randrange(batch)] = 0
    return dict(op=op, lengths=",".join(str(x) for x in lens), heads=kv * rng.choice((1, 2, 4, 5, 8, 16)), kv_heads=kv,
                dim=dim, page=page, type=kind)


# ---------------------------------------------------------------------------- inputs
def _ints(text):
    return [int(x) for x in text.split(",")]


def _table(gen, lens, page):
    """Pages of sequences in no order (a cache is never quite full), and how many pages the cache has."""
    need = [-(-n // page) for n in lens]
    total, most = max(1, sum(need)), max(1, max(need))
    pages = total + max(1, total // 8)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table.cuda(), pages


def _offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    return cu.cuda()


def _cache4(x):
    """Rows in 16 or 32 bits, [pages, heads, page, dim], as codes and scales of the same order seen as [pages, page, heads, ..]."""
    code, scale = _to4(x.float())
    return code.transpose(1, 2), scale.transpose(1, 2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, dt = case["op"], TYPES[case["type"]]
    norm = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    s = dict(case=case)
    if op.startswith("linear"):
        h, dk, dv = case["heads"], case["dk"], case["dv"]
        rows = case["batch"] if op == "linear_step" else sum(_ints(case["lengths"]))
        if case.get("joint"):
            both = norm(rows, h * (2 * dk + dv)).to(dt)
            s["q"], s["k"], s["v"] = (x.unflatten(1, (h, -1)) for x in both.split([h * dk, h * dk, h * dv], 1))
        else:
            s["q"], s["k"], s["v"] = norm(rows, h, dk).to(dt), norm(rows, h, dk).to(dt), norm(rows, h, dv).to(dt)
        slope = torch.exp(rand(h) * math.log(500.0) - math.log(1000.0))     # memories of 2 to 1000 tokens
        s["g"] = -slope if case["fixed"] else -slope * torch.log1p(torch.exp(norm(rows, h)))
        if op == "linear_step":
            s["state"] = norm(rows, h, dk, dv) * 0.3
            return s
        seqs = len(_ints(case["lengths"]))
        s["cu"] = _offsets(_ints(case["lengths"]))
        s["init"] = norm(seqs, h, dk, dv) * 0.3 if case["init"] else None
        if op == "linear_bwd":
            s["do"], s["dfin"] = norm(rows, h, dv).to(dt), norm(seqs, h, dk, dv) * 0.1
        return s
    heads, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if op == "attn":
        lens = _ints(case["lengths"])
        s["table"], pages = _table(gen, lens, page)
        (s["k"], s["ks"]), (s["v"], s["vs"]) = (_cache4(norm(pages, kv, page, dim).to(dt)) for _ in range(2))
        s.update(q=norm(len(lens), heads, dim).to(dt), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
        return s
    new = _ints(case["new"])
    lens = [p + n for p, n in zip(_ints(case["past"]), new)]
    s["table"], pages = _table(gen, lens, page)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu"] = None if all(n == 1 for n in new) else _offsets(new)
    both = norm(sum(new), (heads + 2 * kv) * dim).to(dt)      # one projection's output
    s["q"], s["nk"], s["nv"] = (x.unflatten(1, (-1, dim)) for x in both.split([heads * dim, kv * dim, kv * dim], 1))
    if case["four"]:
        (s["k"], s["ks"]), (s["v"], s["vs"]) = (_cache4(norm(pages, kv, page, dim).to(dt)) for _ in range(2))
        s["all"] = torch.arange(pages, dtype=torch.int32, device=dev)[None]
        s["ends"] = _offsets([pages * page])
    else:
        s["k"], s["v"] = norm(pages, page, kv, dim).to(dt), norm(pages, page, kv, dim).to(dt)
    half = case["rot"] // 2
    turn = torch.arange(max(lens), dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    s["rope"] = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"linear": _linear, "linear_bwd": _linear_bwd, "linear_step": _linear_step, "append": _append, "attn": _attn}[op](s)


def _own(s, op):
    import chunked_gated_delta_kda_amd as kda

    if op == "linear":
        o, fin = kda.lin_fwd(s["q"], s["k"], s["v"], s["g"], None, s["cu"], s["init"])
        return {"o": o, "final": fin}
    if op == "linear_bwd":
        return kda.lin_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], None, s["cu"], s["init"], s["dfin"])
    if op == "linear_step":
        o, state = kda.lin_decode(s["q"], s["k"], s["v"], s["g"], None, s["state"])
        return {"o": o, "state": state}
    if op == "attn":
        out, lse = kda.attn_decode_fp4(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], return_lse=True)
        return {"out": out, "lse": lse}
    pairs = s["case"]["pairs"]
    if not s["case"]["four"]:
        q = kda.kv_append(s["nk"], s["nv"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["rope"], s["q"],
                          interleaved=pairs)
        return {"q": q, "k": s["k"], "v": s["v"]}
    q = kda.kv_append(s["nk"], s["nv"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["rope"], s["q"], interleaved=pairs,
                      k_scale=s["ks"], v_scale=s["vs"])
    k, v = kda.kv_read_fp4(s["k"], s["v"], s["ks"], s["vs"], s["all"], s["ends"], s["k"].shape[0] * s["k"].shape[1],
                           s["q"].dtype)
    return {"q": q, "k": k, "v": v}


# ---------------------------------------------------------------------------- plain forms
class _Blocks:
    """The packed batch as blocks of BLOCK tokens of one sequence each, [blocks, heads, BLOCK, ..], short ones filled with
    zeros; pair[h, c, b]: what is left of a state after block b where block c of the same sequence begins, 0 where it has
    none; from_start, to_end: what is left of a state of a sequence's start where block c begins, of one at block c's end at its
    sequence's end."""

    def __init__(self, s):
        cu, rows = s["cu"].long(), s["q"].shape[0]
        lens = cu[1:] - cu[:-1]
        per = (lens + BLOCK - 1) // BLOCK
        blocks = sum(-(-n // BLOCK) for n in _ints(s["case"]["lengths"]))
        self.seq = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), per, output_size=blocks)
        first = torch.cumsum(per, 0) - per
        place = torch.arange(blocks, device=cu.device) - first[self.seq]
        at = place[:, None] * BLOCK + torch.arange(BLOCK, device=cu.device)
        self.there = at < lens[self.seq][:, None]
        self.at = torch.where(self.there, cu[self.seq][:, None] + at, 0)
        self.back = self.at[self.there]      # the row of every token, block by block
        self.rows, self.first, self.last, self.empty = rows, place == 0, place == per[self.seq] - 1, lens == 0
        g = s["g"].double()
        g = self.take(g[:, :, None] if g.dim() == 2 else g[None, :, None].expand(rows, -1, -1))[..., 0]
        self.G = torch.cumsum(g, 2)                     # [blocks, heads, BLOCK]
        total = self.G[:, :, -1].t()                    # [heads, blocks]
        upto = torch.cumsum(total, 1)
        same = self.seq[:, None] == self.seq[None]
        order = torch.arange(blocks, device=cu.device)
        after = same & (order[:, None] > order[None])   # block c comes after block b
        self.pair = torch.exp(torch.where(after, (upto - total)[:, :, None] - upto[:, None], -math.inf)).float()
        start = torch.where(self.first, upto - total, -math.inf)
        begin = torch.where(same[None] & self.first[None, None], start[:, None], -math.inf).amax(2)
        end = torch.where(same[None] & self.last[None, None], upto[:, None], -math.inf).amax(2)
        self.from_start, self.to_end = torch.exp(upto - total - begin).float(), torch.exp(end - upto).float()
        self.total = torch.exp(total).float()
        low = torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=cu.device).tril()
        self.mask = torch.exp(torch.where(low, self.G[..., None] - self.G[..., None, :], -math.inf)).float()
        self.into = torch.exp(self.G).float()[..., None]                            # of the block's first state, at a token
        self.out = torch.exp(self.G[..., -1:] - self.G).float()[..., None]          # of a token, at the block's end

    def take(self, x):
        return torch.where(self.there[..., None, None], x[self.at], 0).transpose(1, 2)

    def put(self, x, dtype):
        """Rows of blocks back in their places in the packed batch."""
        y = torch.zeros(self.rows, x.shape[1], *x.shape[3:], dtype=dtype, device=x.device)
        y[self.back] = x.transpose(1, 2)[self.there].to(dtype)
        return y

    def carried(self, parts, ends, backward):
        """States where each block begins (backward: gradients where it ends) from what each block adds."""
        blocks, heads = parts.shape[:2]
        m = self.pair.transpose(1, 2).contiguous() if backward else self.pair
        x = torch.matmul(m, parts.transpose(0, 1).reshape(heads, blocks, -1)).view(heads, blocks, *parts.shape[2:]).transpose(0, 1)
        if ends is not None:
            x = x + (self.to_end if backward else self.from_start).t()[..., None, None] * ends[self.seq]
        return x

    def closed(self, value, ends, backward):
        """The state after each sequence (backward: the gradient of the one before it) from the blocks' last ones."""
        like = value.shape[1:]
        fin = torch.zeros(self.empty.shape[0], *like, device=value.device)
        if ends is not None:
            fin = torch.where(self.empty[:, None, None, None], ends, fin)
        side = self.first if backward else self.last
        fin[self.seq[side]] = value[side]
        return fin


def _tt(x):
    return x.transpose(-1, -2).contiguous()


def _linear(s):
    b, scale, dt = _Blocks(s), s["case"]["dk"] ** -0.5, s["q"].dtype
    q, k, v = (b.take(s[n].float()) for n in "qkv")
    added = torch.matmul(_tt(k * b.out), v)
    enter = b.carried(added, s["init"], False)
    o = scale * (torch.matmul(torch.matmul(q, _tt(k)) * b.mask, v) + torch.matmul(q * b.into, enter))
    leave = b.total.t()[..., None, None] * enter + added
    return {"o": b.put(o, dt), "final": b.closed(leave, s["init"], False)}


def _linear_bwd(s):
    b, scale, dt = _Blocks(s), s["case"]["dk"] ** -0.5, s["q"].dtype
    q, k, v, do = (b.take(s[n].float()) for n in ("q", "k", "v", "do"))
    X = b.carried(torch.matmul(_tt(k * b.out), v), s["init"], False)
    added = scale * torch.matmul(_tt(q * b.into), do)
    Y = b.carried(added, s["dfin"], True)
    qk, dov = torch.matmul(q, _tt(k)) * b.mask * scale, torch.matmul(do, _tt(v)) * b.mask * scale
    dq_in, dk_out = scale * b.into * torch.matmul(do, _tt(X)), b.out * torch.matmul(v, _tt(Y))
    total = b.total.t()[..., None, None]
    # dg_t: what passes from tokens before t to tokens from t on, in a block and over its borders
    w = (qk * torch.matmul(do, _tt(v))).tril(-1)
    ones = torch.ones_like(w[0, 0])
    inside = (torch.matmul(ones.triu(), w) * ones.tril(-1)).sum(-1)
    u, out = (q * dq_in).sum(-1), (k * dk_out).sum(-1)
    dg = inside + u.flip(-1).cumsum(-1).flip(-1) + out.cumsum(-1) - out + (total * X * Y).sum((-1, -2))[..., None]
    dg = b.put(dg, torch.float32)
    return {"dq": b.put(torch.matmul(dov, k) + dq_in, dt), "dk": b.put(torch.matmul(_tt(dov), q) + dk_out, dt),
            "dv": b.put(torch.matmul(_tt(qk), do) + b.out * torch.matmul(k, Y), dt),
            "dg": dg.double().sum(0).float() if s["g"].dim() == 1 else dg,
            "d_initial_state": b.closed(total * Y + added, s["dfin"], True)}


def _linear_step(s):
    q, k, v = (s[n].float() for n in "qkv")
    decay = torch.exp(s["g"]).expand(q.shape[:2])[..., None, None]
    h = decay * s["state"] + k[..., None] * v[:, :, None]
    s["state"].copy_(h)
    return {"o": (s["case"]["dk"] ** -0.5 * (q[..., None] * h).sum(2)).to(s["q"].dtype), "state": s["state"]}


def _places(s):
    """For every new token its sequence's row of the table, position, page and place in the page."""
    rows, lens, page = s["q"].shape[0], s["lens"].long(), s["case"]["page"]
    row = torch.arange(rows, device=lens.device)
    if s["cu"] is None:
        seq, pos = row, lens - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:], row, right=True)
        pos = lens[seq] - (cu[1:][seq] - row)
    return pos, s["table"].long()[seq, pos // page], pos % page


def _turn(x, rope, pairs, wide):
    """Rows of x, their first elements rotated by the rows of rope."""
    half = rope.shape[1] // 2
    c, sn = rope[:, None, :half].to(wide), rope[:, None, half:].to(wide)
    x = x.to(wide)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    a, b = a * c - b * sn, b * c + a * sn
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _to4(x):
    """fp32 rows as e2m1 codes, two to a byte (the even element in the low half), and the biased exponents of their groups'
    scales: that of the largest value less 2, so that it lies between 4 and 8, one more where it would lie over 7."""
    y = x.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1).contiguous()
    e = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 2).clamp(min=1)
    y = y.double() * torch.exp2((127 - e).double())[..., None]
    a = y.abs()
    # halfway values go to the code whose last bit is 0
    code = sum((a > b).to(torch.uint8) if even else (a >= b).to(torch.uint8)
               for b, even in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)))
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], e.to(torch.uint8)


def _of4(code, scale):
    """What codes and scales stand for, in fp32."""
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    m, e = (c & 1).float(), ((c >> 1) & 3).float()
    y = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2(e - 1), 0.5 * m)
    y = torch.where(c > 7, -y, y).unflatten(-1, (-1, GROUP)) * torch.exp2(scale.float() - 127)[..., None]
    return y.flatten(-2)


def _append(s):
    pos, page, at = _places(s)
    pairs, dt, rope = s["case"]["pairs"], s["q"].dtype, s["rope"][pos]
    q = _turn(s["q"], rope, pairs, torch.float32).to(dt)
    if not s["case"]["four"]:
        s["k"][page, at] = _turn(s["nk"], rope, pairs, torch.float32).to(dt)
        s["v"][page, at] = s["nv"]
        return {"q": q, "k": s["k"], "v": s["v"]}
    for x, code, scale in ((_turn(s["nk"], rope, pairs, torch.float64).float(), "k", "ks"), (s["nv"].float(), "v", "vs")):
        s[code][page, at], s[scale][page, at] = _to4(x)
    k, v = (_of4(s[c], s[e]).to(dt).flatten(0, 1) for c, e in (("k", "ks"), ("v", "vs")))
    return {"q": q, "k": k, "v": v}


def _attn(s):
    q, table, lens = s["q"].float(), s["table"].long().clamp(min=0), s["lens"].long()
    batch, heads, dim = q.shape
    kv = s["k"].shape[2]
    k = _of4(s["k"][table], s["ks"][table]).reshape(batch, -1, kv, dim).transpose(1, 2)
    v = _of4(s["v"][table], s["vs"][table]).reshape(batch, -1, kv, dim).transpose(1, 2).contiguous()
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
    op = case["op"]
    if op.startswith("linear"):
        h, dk, dv = case["heads"], case["dk"], case["dv"]
        rows = case["batch"] if op == "linear_step" else sum(_ints(case["lengths"]))
        seqs = case["batch"] if op == "linear_step" else len(_ints(case["lengths"]))
        decays, state = 4 * (h if case["fixed"] else rows * h), 4 * seqs * h * dk * dv
        if op == "linear_bwd":
            return {"bytes": rows * h * (4 * dk + 3 * dv) * 2 + 2 * decays + state * (2 + case["init"]), "flops": 10 * rows * h * dk * dv}
        states = state * (2 if op == "linear_step" or case["init"] else 1)
        return {"bytes": rows * h * (2 * dk + 2 * dv) * 2 + decays + states, "flops": 4 * rows * h * dk * dv}
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    row = kv * (dim // 2 + dim // GROUP)      # of a 4-bit cache
    if op == "attn":
        lens = _ints(case["lengths"])
        bytes_ = 2 * sum(lens) * row + len(lens) * (case["heads"] * (4 * dim + 4) + 4) + 4 * sum(-(-n // page) for n in lens)
        return {"bytes": bytes_, "flops": 4 * sum(lens) * case["heads"] * dim}
    new = _ints(case["new"])
    lens = [p + n for p, n in zip(_ints(case["past"]), new)]
    rows = sum(new)
    bytes_ = rows * (4 * case["heads"] * dim + 4 * kv * dim + 4 * case["rot"]) + 8 * len(new)
    bytes_ += 4 * sum(-(-n // page) - p // page for n, p in zip(lens, _ints(case["past"])))
    if case["four"]:
        need = sum(-(-n // page) for n in lens)
        tokens = (max(1, need) + max(1, need // 8)) * page      # the whole cache is read back
        bytes_ += 2 * rows * row + 2 * tokens * (row + 2 * kv * dim)
    else:
        bytes_ += 4 * rows * kv * dim
    return {"bytes": bytes_, "flops": 3 * rows * (case["heads"] + kv) * case["rot"]}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "attn":
        return _exact_attn(case, d)
    if case["op"] == "append":
        return _exact_append(case, d)
    return _exact_linear(case, d)


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _exact_of4(code, scale):
    values = torch.tensor(_VALUES, dtype=torch.float64, device=code.device)
    row = code.long()
    y = torch.empty(*code.shape[:-1], code.shape[-1] * 2, dtype=torch.float64, device=code.device)
    y[..., 0::2], y[..., 1::2] = values[row % 16], values[row // 16]
    return y * (2.0 ** (scale.double() - 127)).repeat_interleave(GROUP, -1)


def _exact_attn(case, d):
    outs, lses = [], []
    share = case["heads"] // case["kv_heads"]
    for i, n in enumerate(_ints(case["lengths"])):
        q = d["q"][i]
        if n == 0:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device=q.device))
            continue
        rows = d["table"][i, :-(-n // case["page"])].long()
        k, v = (_exact_of4(d[c][rows], d[e][rows]).flatten(0, 1)[:n].permute(1, 0, 2).contiguous()
                for c, e in (("k", "ks"), ("v", "vs")))
        o, e = [], []
        for h in range(case["heads"]):
            score = (k[h // share] @ q[h]) * case["dim"] ** -0.5
            o.append(torch.softmax(score, 0) @ v[h // share])
            e.append(torch.logsumexp(score, 0))
        outs.append(torch.stack(o))
        lses.append(torch.stack(e))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_round4(x):
    """Each group of 32 of the rows x to the nearest values that the 4-bit form holds."""
    y = x.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1, keepdim=True)
    unit = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    unit = 2.0 ** (unit - 2 + (top > 1.75 * 2.0 ** unit))
    a = (y / unit).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)       # to even halfway
    return (torch.sign(y) * a * unit).flatten(-2)


def _exact_append(case, d):
    half, pairs, page = case["rot"] // 2, case["pairs"], case["page"]
    if case["four"]:
        k, v = _exact_of4(d["k"], d["ks"]).contiguous(), _exact_of4(d["v"], d["vs"]).contiguous()
    else:
        k, v = d["k"].clone(), d["v"].clone()
    q, at = torch.empty_like(d["q"]), 0
    first = torch.arange(half, device=q.device) * (2 if pairs else 1)
    second = first + (1 if pairs else half)

    def turned(x, r):
        y = x.clone()
        c, sn = r[:, None, :half], r[:, None, half:]
        y[..., first] = x[..., first] * c - x[..., second] * sn
        y[..., second] = x[..., second] * c + x[..., first] * sn
        return y

    for i, (past, n) in enumerate(zip(_ints(case["past"]), _ints(case["new"]))):
        if n == 0:
            continue
        pos = torch.arange(past, past + n, device=q.device)
        r = d["rope"][pos]
        where = d["table"][i].long()[pos // page], pos % page
        q[at:at + n] = turned(d["q"][at:at + n], r)
        nk, nv = turned(d["nk"][at:at + n], r), d["nv"][at:at + n]
        k[where], v[where] = (_exact_round4(nk), _exact_round4(nv)) if case["four"] else (nk, nv)
        at += n
    return {"q": q, "k": k.flatten(0, 1) if case["four"] else k, "v": v.flatten(0, 1) if case["four"] else v}


def _exact_linear(case, d):
    op, scale = case["op"], case["dk"] ** -0.5
    decay = torch.exp(d["g"]).expand(d["q"].shape[:2])[..., None, None]
    q, k, v = d["q"], d["k"], d["v"]
    if op == "linear_step":
        h = d["state"] * decay + torch.einsum("bhi,bhj->bhij", k, v)
        return {"o": scale * torch.einsum("bhi,bhij->bhj", q, h), "state": h}
    # token after token, as the recurrence is written
    bwd = op == "linear_bwd"
    o, fins, at = torch.zeros_like(v), [], 0
    g = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v),
         "dg": q.new_zeros(q.shape[:2])} if bwd else None
    dinit = []
    for i, n in enumerate(_ints(case["lengths"])):
        h = d["init"][i].clone() if d["init"] is not None else q.new_zeros(case["heads"], case["dk"], case["dv"])
        trail = q.new_empty(n, *h.shape) if bwd else None      # decayed states that the tokens add to
        for t in range(n):
            h = h * decay[at + t]
            if bwd:
                trail[t] = h
            h = h + k[at + t][..., None] * v[at + t][:, None]
            if bwd:
                g["dq"][at + t] = scale * (h @ d["do"][at + t][..., None])[..., 0]
            else:
                o[at + t] = scale * (q[at + t][:, None] @ h)[:, 0]
        fins.append(h)
        if bwd:
            dh = d["dfin"][i].clone()
            for t in range(n - 1, -1, -1):
                dh = dh + scale * q[at + t][..., None] * d["do"][at + t][:, None]
                g["dk"][at + t] = (dh @ v[at + t][..., None])[..., 0]
                g["dv"][at + t] = (k[at + t][:, None] @ dh)[:, 0]
                g["dg"][at + t] = (dh * trail[t]).sum((1, 2))
                dh = dh * decay[at + t]
            dinit.append(dh)
        at += n
    if not bwd:
        return {"o": o, "final": torch.stack(fins)}
    if case["fixed"]:
        g["dg"] = g["dg"].sum(0)
    g["d_initial_state"] = torch.stack(dinit)
    return g
