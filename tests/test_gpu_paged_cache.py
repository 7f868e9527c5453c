"""The writer of the paged cache, the 4-bit cache and the attention over it on the GPU, against plain 64-bit forms: lengths of
zero, one and long ones, odd pages, padding, empty slots, bad pages, layouts, offsets past 32 bits, values that are not
finite, streams and graphs.

Tolerances. A rotated element is x c - y s in fp32 (two roundings of terms up to |x c| + |y s|: 2 units of 2^-24 of them)
rounded once to its type. Keys in 4 bits are rotated in 64 bits and rounded to fp32 before they are coded: codes are
compared for equality, against the same in numpy. Attention: what ops_oracle.attention counts, over the values that
the codes stand for (exact in the products' type)."""
import numpy as np
import pytest

import cache_oracle as co
import ops_oracle as oo

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.detach().to("cpu").double().numpy()


def rope_table(rows, rot):
    half = rot // 2
    turn = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([turn.cos(), turn.sin()], 1).float()


def make(lens, new, hq, hkv, dh, rot, page, kind, four, seed, layout="tokens", pad=0, rope_rows=None):
    import chunked_gated_delta_kda_amd as kda

    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind]
    T = sum(new) + pad
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    both = torch.randn(T, (hq + 2 * hkv) * dh, generator=g).to(dt).cuda()       # a projection's output
    q, k, v = (x.unflatten(1, (-1, dh)) for x in both.split([hq * dh, hkv * dh, hkv * dh], 1))
    d = dict(k=k, v=v, q=q, block_table=table.cuda(), seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    cu = torch.zeros(len(new) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(new), 0)
    d["cu_seqlens"] = cu.cuda()
    if rot:
        d["rope"] = rope_table(rope_rows or max(lens) + 1, rot).cuda()
    if four:
        d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"] = kda.kv_cache_fp4(pages, page, hkv, dh)
        for n in ("k_cache", "v_cache"):
            d[n].copy_(torch.randint(0, 256, d[n].shape, generator=g, dtype=torch.uint8))
        if layout == "tokens":
            for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
                d[n] = d[n].contiguous()
    else:
        kv = [torch.randn(pages, page, hkv, dh, generator=g).to(dt).cuda() for _ in range(2)]
        if layout == "heads":
            kv = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in kv]
        if layout == "joint":
            both = torch.stack(kv, 1)
            kv = [both[:, 0], both[:, 1]]
        d["k_cache"], d["v_cache"] = kv
    return d


def expected(d, lens, new, interleaved, kind):
    """q, and the caches after the call (codes and scales, or values), with the sizes that errors are counted against."""
    page, pages = d["k_cache"].shape[1], d["k_cache"].shape[0]
    rope = np64(d["rope"]) if "rope" in d else None
    four = "k_scale" in d
    q, k, v = np64(d["q"]), np64(d["k"]), np64(d["v"])
    names = ("k_cache", "v_cache", "k_scale", "v_scale") if four else ("k_cache", "v_cache")
    out = {n: (d[n].cpu().numpy().copy() if four else np64(d[n])) for n in names}
    size = np.zeros(out["k_cache"].shape)
    rq, sq = np.zeros(q.shape), np.zeros(q.shape)
    written = np.zeros(len(q), dtype=bool)
    for row, n, pos, p, at in co.places(lens, new, d["block_table"].cpu().numpy(), page, pages,
                                        None if rope is None else len(rope)):
        turn = (lambda x: co.rotate(x, rope[pos], interleaved)) if rope is not None else (lambda x: x)
        sizes = (lambda x: co.rotate_size(x, rope[pos], interleaved)) if rope is not None else np.abs
        rq[row], sq[row], written[row] = turn(q[row]), sizes(q[row]), True
        if four:
            for x, n in ((turn(k[row]), "k"), (v[row], "v")):
                out[n + "_cache"][p, at], out[n + "_scale"][p, at] = co.encode(x, kind)
        else:
            out["k_cache"][p, at], size[p, at], out["v_cache"][p, at] = turn(k[row]), sizes(k[row]), v[row]
    return rq, sq, written, out, size


def append(d, **kw):
    import chunked_gated_delta_kda_amd as kda
    return kda.kv_append(**d, **kw)


def check_append(d, lens, new, interleaved, kind, **kw):
    rq, sq, written, out, size = expected(d, lens, new, interleaved, kind)
    fill = torch.full(d["q"].shape, 7.0, dtype=d["q"].dtype, device="cuda")
    got = append(d, interleaved=interleaved, q_out=fill, **kw)
    gq = np64(got)
    oo.check("q", gq[written], rq[written], 2 * sq[written], kind, 1)
    assert (gq[~written] == 7).all()
    if "k_scale" in d:
        for n in out:
            np.testing.assert_array_equal(d[n].cpu().numpy(), out[n], err_msg=n)
    else:
        np.testing.assert_array_equal(np64(d["v_cache"]), out["v_cache"])
        oo.check("k_cache", np64(d["k_cache"]), out["k_cache"], 2 * size, kind, 1)


# lengths after, new rows, query heads, cache heads, head dim, rotated, pairs, page, type, layout
CASES = [
    ([1], [1], 1, 1, 64, 64, False, 1, "bf16", "tokens"),
    ([5, 17, 40], [1, 1, 1], 4, 2, 128, 128, False, 16, "fp16", "heads"),
    ([70, 0, 3, 33, 64], [70, 0, 1, 17, 64], 8, 1, 128, 64, True, 16, "bf16", "joint"),
    ([130, 9], [129, 9], 3, 3, 256, 256, True, 48, "fp16", "tokens"),
    ([50, 20], [20, 20], 34, 2, 64, 32, False, 3, "bf16", "heads"),
    ([12, 8], [12, 3], 5, 5, 256, 16, False, 8, "bf16", "tokens"),
    ([12, 8], [12, 3], 2, 1, 128, 0, False, 8, "fp16", "tokens"),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[1])}h{c[2]}-{c[3]}d{c[4]}r{c[5]}{'i' if c[6] else ''}p{c[7]}{c[8]}{c[9]}")
def test_append(case, four):
    lens, new, hq, hkv, dh, rot, pairs, page, kind, layout = case
    d = make(lens, new, hq, hkv, dh, rot, page, kind, four, 1, layout)
    check_append(d, lens, new, pairs, kind, check=True)


@pytest.mark.parametrize("four", [False, True])
def test_one_row_each_with_empty_slots(four):
    lens = [9, 0, 33, 1, 0]
    d = make(lens, [1] * 5, 4, 2, 128, 128, 16, "bf16", four, 2)
    del d["cu_seqlens"]
    check_append(d, lens, [1] * 5, False, "bf16", check=True)


def test_padding_rows_and_no_rows():
    lens, new = [9, 4], [5, 2]
    d = make(lens, new, 4, 2, 128, 128, 16, "bf16", False, 3, pad=6)
    check_append(d, lens, new + [], False, "bf16", check=True)
    d = make([9, 4], [0, 0], 4, 2, 128, 128, 16, "bf16", True, 3)
    before = d["k_cache"].clone()
    assert append(d, check=True).shape == (0, 4, 128) and torch.equal(before, d["k_cache"])


def test_malformed_offsets_without_rows_raise():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    d = make([9, 4], [0, 0], 4, 2, 128, 128, 16, "bf16", True, 3)
    d["cu_seqlens"] = torch.tensor([0, 5, 5], dtype=torch.int32, device="cuda")
    with pytest.raises(native.KdaDeviceError) as err:
        append(d, check=True)
    assert err.value.bits == 2
    with pytest.raises(native.KdaDeviceError) as err:
        kda.kv_read_fp4(d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], d["block_table"], d["cu_seqlens"], 0, check=True)
    assert err.value.bits == 2


def test_without_queries():
    d = make([20], [20], 2, 2, 64, 64, 8, "fp16", False, 4)
    e = dict(d, k_cache=d["k_cache"].clone(), v_cache=d["v_cache"].clone())
    append(d)
    e["q"] = None
    assert append(e) is None
    assert torch.equal(d["k_cache"], e["k_cache"]) and torch.equal(d["v_cache"], e["v_cache"])


@pytest.mark.parametrize("four", [False, True])
def test_rows_that_do_not_fit_are_left_out_and_raise(four):
    from chunked_gated_delta_kda_amd import native

    lens, new, page = [40, 20, 30], [40, 20, 30], 16
    for what in ("page -1", "page past", "page far", "short length", "past the table", "past the rotations", "negative"):
        d = make(lens, new, 4, 2, 64, 64, page, "bf16", four, 5)
        pages = d["k_cache"].shape[0]
        ls = list(lens)
        if what.startswith("page"):
            d["block_table"][0, 1] = {"page -1": -1, "page past": pages, "page far": 2 ** 31 - 1}[what]
        elif what == "short length":
            ls[1] = 7                   # 20 new rows: the first 13 would lie before position 0
        elif what == "past the table":
            ls[2] = d["block_table"].shape[1] * page + 5
        elif what == "negative":
            ls[0] = -3
        else:
            d["rope"] = d["rope"][:25].contiguous()
        d["seq_lens"] = torch.tensor(ls, dtype=torch.int32, device="cuda")
        with pytest.raises(native.KdaDeviceError) as err:
            append({**d, "k_cache": d["k_cache"].clone(), "v_cache": d["v_cache"].clone()}, check=True)
        assert err.value.bits == 4, what
        if four:
            for n in ("k_scale", "v_scale"):
                d[n].fill_(127)
        check_append(d, ls, new, False, "bf16")


def test_malformed_offsets_raise_and_stay_inside():
    from chunked_gated_delta_kda_amd import native

    for bad in ([0, 30, 20, 90], [3, 40, 60, 90], [0, 40, 60, 2 ** 31 - 1], [-2 ** 31, 40, 60, 90], [0, 2 ** 30, 60, 90]):
        d = make([40, 20, 30], [40, 20, 30], 2, 1, 64, 64, 16, "bf16", False, 6)
        d["cu_seqlens"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(native.KdaDeviceError) as err:
            append(d, check=True)
        assert err.value.bits & 2, bad


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_codes_at_borders_and_far_magnitudes(kind):
    """Halfway values, the border between two scales, zeros, the smallest and largest numbers, infinities and NaN."""
    import chunked_gated_delta_kda_amd as kda

    dt = TYPES[kind]
    rows = []
    for top in (4.0, 7.0, 7.0 + 2.0 ** -5, 6.0, 7.99, 4.5):
        rows.append([top] + [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.0, -0.0] + [0.1] * 19)
    rows += [[0.0] * 32, [-0.0] * 32, [1.0] + [0.0] * 31]
    big, small = (3.3e38, 1e-38) if kind == "bf16" else (65504.0, 6e-8)
    rows += [[big, -big] + [1.0] * 30, [small, -3 * small] + [0.0] * 30, [big * 0.9, small] + [big / 2] * 30]
    rows += [[float("inf")] + [1.0] * 31, [1.0] * 31 + [float("-inf")], [float("nan")] + [2.0] * 31]
    while len(rows) % 4:
        rows.append([1.5] * 32)
    x = torch.tensor(rows, dtype=torch.float64).to(dt)
    T = len(rows) // 4
    k = x.view(T, 1, 128).cuda()
    cache = kda.kv_cache_fp4(T, 1, 1, 128)
    table = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    kda.kv_append(k, k.clone(), cache[0], cache[1], table, cu[1:], cu, k_scale=cache[2], v_scale=cache[3], check=True)
    code, scale = co.encode(x.float().view(T, 128).numpy(), kind)
    for side in (0, 1):
        s = cache[2 + side].cpu().numpy()[:, 0, 0]
        np.testing.assert_array_equal(s, scale)
        fine = np.repeat(scale != 255, 16, -1)
        np.testing.assert_array_equal(cache[side].cpu().numpy()[:, 0, 0][fine], code[fine])
    rk, rv = kda.kv_read_fp4(*cache, table, cu, T, dt, check=True)
    want = co.decode(code, scale)
    for r in (rk, rv):
        got = np64(r)[:, 0]
        assert (np.isnan(got) == np.isnan(want)).all()
        f = ~np.isnan(want)
        assert np.isfinite(got[f]).all()        # what is finite stays finite in the type that reads it
        np.testing.assert_array_equal(got[f], torch.from_numpy(want[f]).to(dt).double().numpy())


def test_every_code_and_scale_reads_back():
    import chunked_gated_delta_kda_amd as kda

    for dh in (64, 128, 256):
        pages = 256 // (dh // 32) + 1
        cache = kda.kv_cache_fp4(pages, 16, 1, dh)
        g = torch.Generator().manual_seed(3)
        for side in (0, 1):
            cache[side].copy_(torch.randint(0, 256, cache[side].shape, generator=g, dtype=torch.uint8))
            cache[2 + side].copy_((torch.arange(cache[2 + side].numel()) % 256).to(torch.uint8).view(cache[2 + side].shape))
        n = pages * 16
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for dt in TYPES.values():
            got = kda.kv_read_fp4(*cache, table, cu, n, dt)
            for side in (0, 1):
                want = torch.from_numpy(co.decode(cache[side].cpu().numpy(), cache[2 + side].cpu().numpy())).view(n, 1, dh)
                assert torch.equal(torch.nan_to_num(got[side].cpu().double(), nan=-1e300, posinf=1e301, neginf=-1e301),
                                   torch.nan_to_num(want.to(dt).double(), nan=-1e300, posinf=1e301, neginf=-1e301))


def test_read_by_tables():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    lens = [33, 0, 5, 16]
    d = make(lens, lens, 2, 2, 128, 128, 16, "bf16", True, 8, layout="heads")
    append(d)
    rows = sum(lens)
    k = torch.full((rows + 3, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    c = (d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"])
    kda.kv_read_fp4(*c, d["block_table"], d["cu_seqlens"], rows + 3, k=k, v=v, check=True)
    assert (k[rows:] == 9).all() and (v[rows:] == 9).all()
    at = 0
    for n, length in enumerate(lens):
        for t in range(length):
            p, o = int(d["block_table"][n, t // 16]), t % 16
            for got, code, scale in ((k, c[0], c[2]), (v, c[1], c[3])):
                np.testing.assert_array_equal(np64(got[at + t]), co.decode(code[p, o].cpu().numpy(), scale[p, o].cpu().numpy()))
        at += length
    d["block_table"][0, 1] = 999
    with pytest.raises(native.KdaDeviceError):
        kda.kv_read_fp4(*c, d["block_table"], d["cu_seqlens"], rows, check=True)
    bad, _ = kda.kv_read_fp4(*c, d["block_table"], d["cu_seqlens"], rows)
    assert (bad[16:32] == 0).all() and torch.equal(bad[:16], k[:16]) and torch.equal(bad[32:rows], k[32:rows])


# ---------------------------------------------------------------------------- attention
def cache4(lens, hq, hkv, dh, page, kind, seed, layout="heads", spread=1.0):
    """A cache whose unused places hold NaN scales, pages in random order, unused table entries outside it."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
    used = np.zeros((pages, page), dtype=bool)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        for t in range(lens[i]):
            used[order[at + t // page], t % page] = True
        at += n
    out, values = [], []
    for _ in range(2):
        code, scale = co.encode((torch.randn(pages, page, hkv, dh, generator=g) * spread).numpy(), kind)
        values.append(co.decode(code, scale))
        scale[~used] = 255
        out.append((torch.from_numpy(code).cuda(), torch.from_numpy(scale).cuda()))
    (k, ks), (v, vs) = out
    if layout == "heads":
        k, ks, v, vs = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, ks, v, vs))
    if layout == "joint":
        both, bs = torch.stack([k, v], 1), torch.stack([ks, vs], 1)
        k, v, ks, vs = both[:, 0], both[:, 1], bs[:, 0], bs[:, 1]
    q = torch.randn(len(lens), hq, dh, generator=g).to(TYPES[kind]).cuda()
    return dict(q=q, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32).cuda()), values


def compare(out, lse, d, values, lens, kind, scale=None):
    dh = d["q"].shape[2]
    ro, oe, rl, le = oo.attention(np64(d["q"]), *values, d["block_table"].cpu().numpy(), lens,
                                  dh ** -0.5 if scale is None else scale, kind)
    oo.check("out", np64(out), ro, oe / oo.U, kind, 1)
    got = np64(lse)
    empty = np.array(lens) == 0
    assert np.isneginf(got[empty]).all()
    oo.check("lse", got[~empty], rl[~empty], le[~empty] / oo.U, "fp32", 1)


ATTN = [
    ([1], 1, 1, 64, 1, "bf16", "tokens"),
    ([5], 2, 2, 128, 16, "bf16", "tokens"),
    ([31, 32, 33, 0, 1], 4, 2, 128, 16, "fp16", "heads"),
    ([127, 128, 129, 255, 256, 257], 8, 1, 64, 32, "bf16", "heads"),
    ([100, 7], 5, 1, 256, 3, "bf16", "tokens"),
    ([300, 0, 64], 16, 1, 128, 48, "fp16", "joint"),
    ([70], 34, 2, 64, 16, "fp16", "heads"),
    ([513, 2], 20, 1, 128, 1, "bf16", "heads"),
    ([5000], 8, 2, 128, 16, "bf16", "heads"),
    ([3000, 1, 0, 2500, 900], 6, 3, 256, 64, "fp16", "joint"),
    ([17] * 130, 2, 1, 64, 8, "fp16", "tokens"),
    ([0, 0], 4, 4, 128, 16, "bf16", "heads"),
    ([2000] + [3] * 70, 4, 2, 64, 256, "bf16", "heads"),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}h{c[1]}-{c[2]}d{c[3]}p{c[4]}{c[5]}{c[6]}")
def test_token(case):
    import chunked_gated_delta_kda_amd as kda

    lens, hq, hkv, dh, page, kind, layout = case
    d, values = cache4(lens, hq, hkv, dh, page, kind, 1, layout)
    out, lse = kda.attn_decode_fp4(**d, return_lse=True, check=True)
    compare(out, lse, d, values, lens, kind)
    again, lagain = kda.attn_decode_fp4(**d, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lagain)


def test_sharp_and_flat_scores():
    import chunked_gated_delta_kda_amd as kda

    lens = [700, 40]
    for spread, scale in ((6.0, 1.0), (1.0, 0.0), (1.0, -0.3)):
        for kind in TYPES:
            d, values = cache4(lens, 4, 2, 128, 16, kind, 2, spread=spread)
            out, lse = kda.attn_decode_fp4(**d, scale=scale, return_lse=True)
            compare(out, lse, d, values, lens, kind, scale)


def test_the_same_as_over_the_values_in_16_bits():
    """Products and roundings are those of attn_decode over the values: results differ by the order of a few sums at most."""
    import chunked_gated_delta_kda_amd as kda

    lens = [900, 33, 0, 4000]
    d, values = cache4(lens, 8, 2, 128, 16, "bf16", 4)
    out, lse = kda.attn_decode_fp4(**d, return_lse=True)
    k, v = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in values)
    o16, l16 = kda.attn_decode(d["q"], k, v, d["block_table"], d["seq_lens"], return_lse=True)
    compare(o16, l16, d, values, lens, "bf16")
    compare(out, lse, d, values, lens, "bf16")


def test_bad_pages_and_lengths_are_left_out_and_raise():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    page, lens = 16, [100, 60, 300]
    d, _ = cache4(lens, 4, 2, 128, page, "bf16", 5)
    good = kda.attn_decode_fp4(**d, check=True)
    for bad in (-1, d["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        e = dict(d, block_table=d["block_table"].clone())
        e["block_table"][1, 3] = bad                # tokens 48 .. 59 of the second sequence: its last
        with pytest.raises(native.KdaDeviceError) as err:
            kda.attn_decode_fp4(**e, check=True)
        assert err.value.bits == 4
        out = kda.attn_decode_fp4(**e)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        f = dict(d, seq_lens=torch.tensor([100, 48, 300], dtype=torch.int32, device="cuda"))
        assert torch.equal(out[1], kda.attn_decode_fp4(**f)[1])
    for n in (-5, d["block_table"].shape[1] * page + 1):
        e = dict(d, seq_lens=torch.tensor([100, n, 300], dtype=torch.int32, device="cuda"))
        e["block_table"] = d["block_table"].clamp(min=0)
        with pytest.raises(native.KdaDeviceError):
            kda.attn_decode_fp4(**e, check=True)


def test_a_group_that_is_nan_makes_its_elements_so():
    import chunked_gated_delta_kda_amd as kda

    d, values = cache4([40], 2, 1, 128, 16, "bf16", 6)
    p = int(d["block_table"][0, 1])
    d["v_scale"][p, 3, 0, 2] = 255
    out = np64(kda.attn_decode_fp4(**d))
    assert np.isnan(out[0, :, 64:96]).all() and np.isfinite(out[0, :, :64]).all() and np.isfinite(out[0, :, 96:]).all()
    d, values = cache4([40], 2, 1, 128, 16, "bf16", 6)
    d["k_scale"][p, 3, 0, 2] = 255
    assert np.isnan(np64(kda.attn_decode_fp4(**d))).all()


def test_codes_past_4_gib():
    """A page whose bytes lie past 2^32 from the cache's base."""
    import chunked_gated_delta_kda_amd as kda

    hkv, dh, page, pages = 2, 128, 16, (1 << 32) // (2 * 16 * 64) + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GiB")
    code = torch.empty(pages, hkv, page, dh // 2, dtype=torch.uint8, device="cuda")
    vode = torch.empty(pages, hkv, page, dh // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, pages, hkv, page, dh // 32), 127, dtype=torch.uint8, device="cuda")
    c = (code.transpose(1, 2), vode.transpose(1, 2), scale[0].transpose(1, 2), scale[1].transpose(1, 2))
    g = torch.Generator().manual_seed(1)
    table = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32, device="cuda")
    n = 40
    k, v = (torch.randn(n, hkv, dh, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kda.kv_append(k, v, c[0], c[1], table, lens, cu, k_scale=c[2], v_scale=c[3], check=True)
    small = kda.kv_cache_fp4(3, page, hkv, dh)
    t3 = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    kda.kv_append(k, v, small[0], small[1], t3, lens, cu, k_scale=small[2], v_scale=small[3])
    q = torch.randn(1, 4, dh, generator=g).to(torch.bfloat16).cuda()
    assert torch.equal(kda.attn_decode_fp4(q, *c, table, lens, check=True), kda.attn_decode_fp4(q, *small, t3, lens))
    for a, b in zip(kda.kv_read_fp4(*c, table, cu, n), kda.kv_read_fp4(*small, t3, cu, n)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------- together, streams and graphs
@pytest.mark.parametrize("four", [False, True])
def test_a_captured_token_step_of_append_and_attention(four):
    """One graph of writer and reader, replayed while lengths, pages and inputs change; every replay against eager calls."""
    import chunked_gated_delta_kda_amd as kda

    B, hq, hkv, dh, page, W = 3, 8, 2, 128, 16, 8
    g = torch.Generator().manual_seed(11)
    rope = rope_table(W * page, dh).cuda()
    pages = B * W
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, W).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, (hq + 2 * hkv) * dh, dtype=torch.bfloat16, device="cuda")

    def caches():
        if four:
            c = kda.kv_cache_fp4(pages, page, hkv, dh)
            return dict(k_cache=c[0], v_cache=c[1], k_scale=c[2], v_scale=c[3])
        return dict(k_cache=torch.zeros(pages, page, hkv, dh, dtype=torch.bfloat16, device="cuda"),
                    v_cache=torch.zeros(pages, page, hkv, dh, dtype=torch.bfloat16, device="cuda"))

    def step(c, q_out=None, out=None):
        q, k, v = (x.unflatten(1, (-1, dh)) for x in new.split([hq * dh, hkv * dh, hkv * dh], 1))
        q = kda.kv_append(k, v, c["k_cache"], c["v_cache"], table, lens, rope=rope, q=q, k_scale=c.get("k_scale"),
                          v_scale=c.get("v_scale"), q_out=q_out)
        if four:
            return q, kda.attn_decode_fp4(q, **c, block_table=table, seq_lens=lens, out=out)
        return q, kda.attn_decode(q, **c, block_table=table, seq_lens=lens, out=out)

    mine, eager = caches(), caches()
    q_out = torch.zeros(B, hq, dh, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q_out)
    lens.fill_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches(), q_out, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(mine, q_out, out)
    at = torch.tensor([0, 5, 40])
    # what came before the first step
    for c in (mine, eager):
        for n in c:
            c[n].zero_() if "scale" not in n else c[n].fill_(127)
    for i in range(20):
        at = at + 1
        lens.copy_(torch.tensor([int(at[0]), int(at[1]) if i % 5 else 0, int(at[2])], dtype=torch.int32))
        new.copy_(torch.randn(new.shape, generator=g))
        q_out.zero_()
        graph.replay()
        q, want = step(eager, torch.zeros_like(q_out))
        assert torch.equal(q, q_out) and torch.equal(want, out), i
        for n in mine:
            assert torch.equal(mine[n], eager[n]), (i, n)


def test_prompt_then_tokens_equals_one_prompt():
    """A prompt in one call and the same in two prompts and tokens leave the same cache."""
    import chunked_gated_delta_kda_amd as kda

    n, page = 45, 16
    d = make([n], [n], 2, 2, 128, 64, page, "bf16", True, 13)
    e = {k: (x.clone() if k.endswith(("cache", "scale")) else x) for k, x in d.items()}
    q = append(d)
    parts = []
    for lo, hi in ((0, 7), (7, 40)):
        parts.append(kda.kv_append(**{**e, "k": e["k"][lo:hi], "v": e["v"][lo:hi], "q": e["q"][lo:hi],
                                      "seq_lens": torch.tensor([hi], dtype=torch.int32, device="cuda"),
                                      "cu_seqlens": torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")}))
    for t in range(40, n):
        parts.append(kda.kv_append(**{**e, "k": e["k"][t:t + 1], "v": e["v"][t:t + 1], "q": e["q"][t:t + 1], "cu_seqlens": None,
                                      "seq_lens": torch.tensor([t + 1], dtype=torch.int32, device="cuda")}))
    assert torch.equal(torch.cat(parts), q)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(d[name], e[name])


def test_on_another_stream():
    import chunked_gated_delta_kda_amd as kda

    d = make([40, 9], [40, 9], 4, 2, 128, 128, 16, "bf16", True, 14)
    want = append({**d, "k_cache": d["k_cache"].clone(), "v_cache": d["v_cache"].clone(), "k_scale": d["k_scale"].clone(),
                   "v_scale": d["v_scale"].clone()})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = append(d, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    last = got[[39, 48]].contiguous()
    side.wait_stream(torch.cuda.current_stream())
    args = (last, d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], d["block_table"], d["seq_lens"])
    out = kda.attn_decode_fp4(*args, stream=side)
    side.synchronize()
    assert torch.equal(out, kda.attn_decode_fp4(*args))
