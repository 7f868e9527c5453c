"""Caches that are slices of one tensor, in every order in which keys, values, codes and scales may lie between each other: the
writer, the read-back and the attentions give what they give over caches of their own, and bytes between them stay."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PAGES, PAGE, H, D = 12, 8, 2, 64
DT = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def batch(heads=H):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(DT).cuda()  # noqa: E731
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    half = torch.arange(40)[:, None] * 100.0 ** (-torch.arange(0, D, 2) / D)
    return dict(k=r(50, heads, D), v=r(50, heads, D), q=r(50, 4, D), block_table=torch.randperm(PAGES, generator=g).to(torch.int32).view(3, 4).cuda(),
                seq_lens=i([20, 0, 30]), cu_seqlens=i([0, 20, 20, 50]), rope=torch.cat([half.cos(), half.sin()], 1).float().cuda())


def pair(how, heads):
    """Both caches as slices of one tensor, and it."""
    a = lambda *s: torch.full(s, 7.0, dtype=DT, device="cuda")  # noqa: E731
    if how == "token by token":
        x = a(PAGES, PAGE, 2, heads, D)
        return x[:, :, 0], x[:, :, 1], x
    if how == "page by page":
        x = a(PAGES, 2, PAGE, heads, D)
        return x[:, 1], x[:, 0], x
    if how == "row by row":
        x = a(PAGES, PAGE, heads, 2, D)
        return x[..., 0, :], x[..., 1, :], x
    if how == "heads outermost":
        x = a(heads, 2, PAGES, PAGE, D)
        return x[:, 0].permute(1, 2, 0, 3), x[:, 1].permute(1, 2, 0, 3), x
    x = a(2 * PAGES, PAGE, heads, D)        # every second page
    return x[::2], x[1::2], x


@pytest.mark.parametrize("heads", [1, 2])
@pytest.mark.parametrize("how", ["token by token", "page by page", "row by row", "heads outermost", "every second page"])
def test_caches_in_one_tensor(how, heads):
    import chunked_gated_delta_kda_amd as kda

    b = batch(heads)
    k, v, _ = pair(how, heads)
    own = [torch.full((PAGES, PAGE, heads, D), 7.0, dtype=DT, device="cuda") for _ in range(2)]
    q = kda.kv_append(b["k"], b["v"], k, v, b["block_table"], b["seq_lens"], b["cu_seqlens"], b["rope"], b["q"], check=True)
    want = kda.kv_append(b["k"], b["v"], *own, b["block_table"], b["seq_lens"], b["cu_seqlens"], b["rope"], b["q"], check=True)
    assert torch.equal(q[:20], want[:20]) and torch.equal(k, own[0]) and torch.equal(v, own[1])
    args = (b["block_table"], b["seq_lens"])
    assert torch.equal(kda.attn_decode(b["q"][:3], k, v, *args), kda.attn_decode(b["q"][:3], *own, *args))


@pytest.mark.parametrize("how", ["blocks of a page", "rows", "codes and scales of a token"])
def test_4_bit_caches_in_one_tensor(how):
    import chunked_gated_delta_kda_amd as kda

    b = batch()
    code, sc = D // 2, D // 32
    if how == "blocks of a page":       # codes of keys, of values, scales of keys, of values
        n, m = PAGE * H * code, PAGE * H * sc
        x = torch.full((PAGES, 2 * n + 2 * m + 16 - 2 * m % 16), 9, dtype=torch.uint8, device="cuda")
        cut = lambda at, size, w: x[:, at:at + size].unflatten(1, (H, PAGE, w)).transpose(1, 2)  # noqa: E731
        four = [cut(0, n, code), cut(n, n, code), cut(2 * n, m, sc), cut(2 * n + m, m, sc)]
    elif how == "rows":                 # a row's codes and scales of both, 80 bytes with a gap
        x = torch.full((PAGES, PAGE, H, 80), 9, dtype=torch.uint8, device="cuda")
        four = [x[..., 0:32], x[..., 32:64], x[..., 64:66], x[..., 70:72]]
    else:                               # of a token, all heads' codes, then their scales
        x = torch.full((PAGES, PAGE, 2 * H * code + 16), 9, dtype=torch.uint8, device="cuda")
        cut = lambda at, w: x[..., at:at + H * w].unflatten(2, (H, w))  # noqa: E731
        four = [cut(0, code), cut(H * code, code), cut(2 * H * code, sc), cut(2 * H * code + H * sc, sc)]
    before = x.clone()
    own = [t.contiguous() for t in four]
    for c in (four, own):
        kda.kv_append(b["k"], b["v"], c[0], c[1], b["block_table"], b["seq_lens"], b["cu_seqlens"], b["rope"], k_scale=c[2], v_scale=c[3],
                      check=True)
    assert all(torch.equal(s, o) for s, o in zip(four, own))
    for s, o in zip(four, own):
        assert not torch.equal(s, torch.full_like(s, 9))
        s.fill_(9)
    assert torch.equal(x, before)       # nothing between them was written
    for s, o in zip(four, own):
        s.copy_(o)
    args = (b["block_table"], b["seq_lens"])
    assert torch.equal(kda.attn_decode_fp4(b["q"][:3], *four, *args), kda.attn_decode_fp4(b["q"][:3], *own, *args))
    for s, o in zip(kda.kv_read_fp4(*four, b["block_table"], b["cu_seqlens"], 50, check=True),
                    kda.kv_read_fp4(*own, b["block_table"], b["cu_seqlens"], 50, check=True)):
        assert torch.equal(s, o)


def test_views_that_share_bytes_are_refused():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd import native

    b = batch()
    x = torch.zeros(PAGES + 1, PAGE + 1, H, D, dtype=DT, device="cuda")
    y = torch.zeros(PAGES, PAGE, H, 64, dtype=torch.uint8, device="cuda")
    call = lambda k, v, **kw: kda.kv_append(b["k"], b["v"], k, v, b["block_table"], b["seq_lens"], b["cu_seqlens"], **kw)  # noqa: E731
    for k, v in ((x[:-1, :-1], x[1:, :-1]), (x[:-1, 1:], x[:-1, :-1])):
        with pytest.raises(native.KdaError, match="ALIAS"):
            call(k, v)
    for s in ((0, 2), (32, 34), (62, 64)):
        with pytest.raises(native.KdaError, match="ALIAS"):
            call(y[..., :32], y[..., 32:], k_scale=torch.zeros(PAGES, PAGE, H, 2, dtype=torch.uint8, device="cuda"), v_scale=y[..., slice(*s)])
    assert not x.any() and not y.any()
