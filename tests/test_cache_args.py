"""The paged cache's writer, its 4-bit form and the attention over it: what their entry points refuse before anything is
launched, in Python and in the C ABI, and the codec that their tests compare with. No GPU needed."""
import ctypes
import os

import numpy as np
import pytest

import cache_oracle as co
from chunked_gated_delta_kda_amd import native

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(1 << 30)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        pytest.skip("libkda.so not built")
    return native.load_library()


# ---------------------------------------------------------------------------- codec
def test_every_code_is_its_own_nearest():
    code = np.arange(256, dtype=np.uint8).repeat(16).reshape(256, 16)
    code[:, 15] = 0x77      # each group has a 6, so that its scale is 1
    back, scale = co.encode(co.decode(code, np.full((256, 1), 127, np.uint8)), "bf16")
    assert (scale == 127).all() and (back == code).all()


def test_codes_are_the_nearest_values():
    g = np.random.Generator(np.random.PCG64(1))
    x = (g.standard_normal((200, 64)) * np.exp(g.uniform(-20, 20, (200, 1)))).astype(np.float32)
    code, scale = co.encode(x, "bf16")
    y = co.decode(code, scale)
    unit = 2.0 ** (scale.astype(np.float64) - 127).repeat(32, -1)
    top = np.abs(x.reshape(200, 2, 32)).max(-1).repeat(32, -1) / unit
    assert ((top > 3.5) & (top <= 7)).all()
    a = np.abs(x) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
    assert (np.abs(y - x) / unit <= half * (1 + 1e-12)).all()


# ---------------------------------------------------------------------------- Python checks (tensors on the CPU)
def _append(dt=torch.bfloat16, four=False, T=6, hkv=2, hq=4, dh=128):
    a = dict(k=torch.zeros(T, hkv, dh, dtype=dt), v=torch.zeros(T, hkv, dh, dtype=dt), q=torch.zeros(T, hq, dh, dtype=dt),
             block_table=torch.zeros(3, 4, dtype=torch.int32), seq_lens=torch.zeros(3, dtype=torch.int32),
             cu_seqlens=torch.zeros(4, dtype=torch.int32), rope=torch.zeros(64, dh))
    if four:
        a.update(k_cache=torch.zeros(10, hkv, 16, dh // 2, dtype=torch.uint8).transpose(1, 2),
                 v_cache=torch.zeros(10, hkv, 16, dh // 2, dtype=torch.uint8).transpose(1, 2),
                 k_scale=torch.zeros(10, 16, hkv, dh // 32, dtype=torch.uint8),
                 v_scale=torch.zeros(10, 16, hkv, dh // 32, dtype=torch.uint8))
    else:
        a.update(k_cache=torch.zeros(10, 16, hkv, dh, dtype=dt), v_cache=torch.zeros(10, 16, hkv, dh, dtype=dt))
    return a


def test_append_good_arguments():
    from chunked_gated_delta_kda_amd.paged_cache import check_kv_append_args as check
    s = check(**_append())
    assert (s.T, s.N, s.hq, s.hkv, s.dh, s.rot, s.positions, s.pages, s.page, s.width) == (6, 3, 4, 2, 128, 128, 64, 10, 16, 4)
    assert check(**_append(four=True)).strides[6:12] == [2048, 64, 1024] * 2
    a = _append()
    a.update(q=None, rope=None)
    s = check(**a)
    assert (s.hq, s.rot) == (0, 0)
    a = _append(T=3)
    a["cu_seqlens"] = None
    assert check(**a).N == 3


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("name,bad", [
    ("k", torch.zeros(6, 2, 96, dtype=torch.bfloat16)), ("k", torch.zeros(6, 2, 128)),
    ("k", torch.zeros(6, 3, 128, dtype=torch.bfloat16)), ("v", torch.zeros(5, 2, 128, dtype=torch.bfloat16)),
    ("v", torch.zeros(6, 2, 128, dtype=torch.float16)), ("q", torch.zeros(6, 4, 64, dtype=torch.bfloat16)),
    ("q", torch.zeros(7, 4, 128, dtype=torch.bfloat16)), ("k", torch.zeros(6, 2, 132, dtype=torch.bfloat16)[..., :128]),
    ("rope", torch.zeros(64, 136)), ("rope", torch.zeros(64, 24)), ("rope", torch.zeros(64, 144)),
    ("rope", torch.zeros(64, 128, dtype=torch.bfloat16)), ("rope", torch.zeros(64, 256)[:, :128]), ("rope", torch.zeros(0, 128)),
    ("block_table", torch.zeros(2, 4, dtype=torch.int32)), ("block_table", torch.zeros(3, 4, dtype=torch.int64)),
    ("seq_lens", torch.zeros(4, dtype=torch.int32)), ("cu_seqlens", torch.zeros(4, dtype=torch.int64)),
    ("cu_seqlens", None), ("q_out", torch.zeros(6, 4, 128)), ("k_cache", torch.zeros(10, 16, 2, 128)),
    ("v_cache", torch.zeros(9, 16, 2, 128, dtype=torch.bfloat16)),
])
def test_append_rejects(name, bad, four):
    from chunked_gated_delta_kda_amd.paged_cache import check_kv_append_args as check
    a = _append(four=four)
    a[name] = bad
    with pytest.raises(ValueError):
        check(**a)


@pytest.mark.parametrize("name,bad", [
    ("k_scale", None), ("k_scale", torch.zeros(10, 16, 2, 2, dtype=torch.uint8)), ("v_scale", torch.zeros(10, 16, 2, 4)),
    ("k_cache", torch.zeros(10, 16, 2, 128, dtype=torch.uint8)), ("v_cache", torch.zeros(10, 16, 1, 64, dtype=torch.uint8)),
    ("k_cache", torch.zeros(10, 16, 2, 72, dtype=torch.uint8)[..., :64]),
    ("k_scale", torch.zeros(10, 16, 2, 5, dtype=torch.uint8)[..., :4]), ("k_cache", torch.zeros(10, 16, 2, 64, dtype=torch.int8)),
])
def test_4_bit_caches_rejected(name, bad):
    from chunked_gated_delta_kda_amd.paged_cache import check_kv_append_args, check_kv_read_fp4_args
    from chunked_gated_delta_kda_amd.paged_attention import check_attn_decode_fp4_args
    a = _append(four=True)
    a[name] = bad
    with pytest.raises(ValueError):
        check_kv_append_args(**a)
    if bad is None:
        return
    caches = [a[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    with pytest.raises(ValueError):
        check_attn_decode_fp4_args(torch.zeros(3, 4, 128, dtype=torch.bfloat16), *caches, a["block_table"], a["seq_lens"])
    with pytest.raises(ValueError):
        check_kv_read_fp4_args(*caches, a["block_table"], a["cu_seqlens"], 6, torch.bfloat16)


def test_q_out_without_q_and_device():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd.paged_cache import check_kv_append_args as check
    a = _append()
    a.update(q=None, q_out=torch.zeros(6, 4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q_out"):
        check(**a)
    with pytest.raises(ValueError, match="device"):
        kda.kv_append(**_append())
    f = _append(four=True)
    caches = [f[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    with pytest.raises(ValueError, match="device"):
        kda.attn_decode_fp4(torch.zeros(3, 4, 128, dtype=torch.bfloat16), *caches, f["block_table"], f["seq_lens"])
    with pytest.raises(ValueError, match="device"):
        kda.kv_read_fp4(*caches, f["block_table"], f["cu_seqlens"], 6)
    for kw in (dict(dtype=torch.float32), dict(cu_seqlens=None), dict(total_tokens=-1), dict(k=torch.zeros(6, 2, 128))):
        from chunked_gated_delta_kda_amd.paged_cache import check_kv_read_fp4_args
        args = dict(block_table=f["block_table"], cu_seqlens=f["cu_seqlens"], total_tokens=6, dtype=torch.bfloat16)
        args.update(kw)
        with pytest.raises(ValueError):
            check_kv_read_fp4_args(*caches, **args)


def test_a_new_cache_fits_the_operators():
    import chunked_gated_delta_kda_amd as kda
    from chunked_gated_delta_kda_amd.paged_cache import check_kv_append_args as check
    for dh in (64, 128, 256):
        a = _append(four=True, dh=dh)
        a.update(zip(("k_cache", "v_cache", "k_scale", "v_scale"), kda.kv_cache_fp4(10, 16, 2, dh, "cpu")))
        assert check(**a).pages == 10
        assert a["k_scale"].unique().tolist() == [127]
    with pytest.raises(ValueError):
        kda.kv_cache_fp4(10, 16, 2, 96, "cpu")
    with pytest.raises(ValueError):
        kda.kv_cache_fp4(0, 16, 2, 64, "cpu")


# ---------------------------------------------------------------------------- C ABI
MB = 1 << 20
SCALES = dict(k_scale_page_stride=128, k_scale_token_stride=8, k_scale_head_stride=4, v_scale_page_stride=128,
              v_scale_token_stride=8, v_scale_head_stride=4)


def kv_args(four=False, **over):
    a = dict(k=1 * MB, v=2 * MB, q=3 * MB, q_out=4 * MB, rope=5 * MB, cu_seqlens=6 * MB, block_table=7 * MB, seq_lens=8 * MB,
             k_cache=16 * MB, v_cache=32 * MB, k_stride=256, k_head_stride=128, v_stride=256, v_head_stride=128, q_stride=512,
             q_head_stride=128, k_page_stride=4096, k_token_stride=256, k_cache_head_stride=128, v_page_stride=4096,
             v_token_stride=256, v_cache_head_stride=128, table_stride=4, num_seqs=3, total_tokens=6, q_heads=4, kv_heads=2,
             head_dim=128, rot_dim=128, max_positions=64, num_pages=10, page_size=16, table_width=4, dtype=1, interleaved=0)
    if four:
        a.update(k_scale=48 * MB, v_scale=49 * MB, k_page_stride=2048, k_token_stride=128, k_cache_head_stride=64,
                 v_page_stride=2048, v_token_stride=128, v_cache_head_stride=64, **SCALES)
    a.update(over)
    return native.KdaKvArgs(**a)


@pytest.mark.parametrize("four", [False, True])
def test_append_abi_refusals(lib, four):
    call = lambda **kw: lib.kda_kv_append(ctypes.byref(kv_args(four, **kw)), None)  # noqa: E731
    assert lib.kda_kv_append(None, None) == 1
    for kw in (dict(dtype=0), dict(dtype=3), dict(head_dim=96), dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=144),
               dict(interleaved=2), dict(k_stride=260), dict(q_head_stride=4), dict(k=MB + 8), dict(q_out=4 * MB + 2), dict(rope=5 * MB + 4),
               dict(k_cache=16 * MB + 8), dict(v_token_stride=132)):
        assert call(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(total_tokens=-1), dict(kv_heads=0), dict(q_heads=0), dict(q_heads=-1), dict(q_heads=65536),
               dict(kv_heads=65536), dict(num_pages=0), dict(page_size=0), dict(table_width=0), dict(table_stride=3),
               dict(table_width=1 << 27, table_stride=1 << 27), dict(max_positions=0), dict(cu_seqlens=None), dict(k_stride=-8),
               dict(total_tokens=(1 << 27) + 1), dict(k_page_stride=-4096), dict(q=None, q_heads=4),
               dict(k_token_stride=0), dict(v_page_stride=64), dict(k_cache_head_stride=0)):
        assert call(**kw) == 2, kw
    for name in ("k", "v", "q_out", "block_table", "seq_lens", "k_cache", "v_cache"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(q_out=1 * MB), dict(q_out=16 * MB), dict(k_cache=2 * MB), dict(v_cache=5 * MB), dict(k_cache=32 * MB),
               dict(q_out=7 * MB), dict(k_cache=8 * MB), dict(q_out=6 * MB), dict(q_out=3 * MB)):
        assert call(**kw) == 7, kw


def test_append_abi_refusals_of_scales(lib):
    call = lambda **kw: lib.kda_kv_append(ctypes.byref(kv_args(True, **kw)), None)  # noqa: E731
    assert call(k_scale=None) == 1 and call(v_scale=None) == 1
    for kw in (dict(k_scale=48 * MB + 2), dict(v_scale_token_stride=6), dict(k_scale_page_stride=130)):
        assert call(**kw) == 3, kw
    for kw in (dict(k_scale_token_stride=0), dict(v_scale_page_stride=-128), dict(k_scale_head_stride=0)):
        assert call(**kw) == 2, kw
    for kw in (dict(k_scale=49 * MB), dict(q_out=48 * MB), dict(k_scale=1 * MB)):
        assert call(**kw) == 7, kw


def test_attn_fp4_abi_refusals(lib):
    def call(ws=P, n=1 << 30, **over):
        a = dict(q=1 * MB, k_cache=16 * MB, v_cache=32 * MB, block_table=48 * MB, seq_lens=49 * MB, out=50 * MB, lse=51 * MB,
                 q_stride=1024, q_head_stride=128, k_page_stride=2048, k_token_stride=128, k_head_stride=64,
                 v_page_stride=2048, v_token_stride=128, v_head_stride=64, table_stride=64, num_seqs=3, q_heads=8, kv_heads=2,
                 head_dim=128, num_pages=10, page_size=16, table_width=64, dtype=1, scale=0.1)
        s = dict(k_scale=60 * MB, v_scale=61 * MB, **SCALES)
        for k, x in over.items():
            (s if "_scale" in k else a)[k] = x
        return lib.kda_attn_decode_fp4(ctypes.byref(native.KdaAttnFp4Args(attn=native.KdaAttnArgs(**a), **s)), None, ws, n)

    assert lib.kda_attn_decode_fp4(None, None, None, 0) == 1
    for kw in (dict(dtype=0), dict(head_dim=96), dict(scale=float("nan")), dict(k_token_stride=120), dict(v_head_stride=72),
               dict(q_stride=1020), dict(q=MB + 8), dict(v_cache=32 * MB + 8), dict(k_scale=60 * MB + 2),
               dict(v_scale_token_stride=6)):
        assert call(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(q_heads=7), dict(kv_heads=0), dict(num_pages=0), dict(table_width=0), dict(table_stride=63),
               dict(k_head_stride=-16), dict(k_scale_page_stride=-4), dict(num_seqs=1 << 17), dict(k_page_stride=1 << 32),
               dict(v_scale_token_stride=1 << 32)):
        assert call(**kw) == 2, kw
    for name in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "out", "k_scale", "v_scale"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(out=1 * MB), dict(out=16 * MB), dict(lse=50 * MB), dict(lse=49 * MB), dict(out=60 * MB), dict(lse=61 * MB)):
        assert call(**kw) == 7, kw
    need = lib.kda_attn_fp4_workspace_bytes(3, 8, 2, 128, 64, 16)
    assert need > 0 and call(n=need - 1) == 4


def test_read_abi_refusals(lib):
    def call(**over):
        a = dict(k_cache=16 * MB, v_cache=32 * MB, k_scale=48 * MB, v_scale=49 * MB, block_table=50 * MB, cu_seqlens=51 * MB,
                 k=60 * MB, v=61 * MB, k_page_stride=2048, k_token_stride=128, k_head_stride=64, v_page_stride=2048,
                 v_token_stride=128, v_head_stride=64, table_stride=4, num_seqs=3, total_tokens=100, kv_heads=2, head_dim=128,
                 num_pages=10, page_size=16, table_width=4, dtype=1, **SCALES)
        a.update(over)
        return lib.kda_kv_read_fp4(ctypes.byref(native.KdaKvReadArgs(**a)), None)

    assert lib.kda_kv_read_fp4(None, None) == 1
    for kw in (dict(dtype=0), dict(head_dim=32), dict(k=60 * MB + 8), dict(k_token_stride=120), dict(k_scale=48 * MB + 1)):
        assert call(**kw) == 3, kw
    for kw in (dict(num_seqs=0), dict(total_tokens=-1), dict(kv_heads=0), dict(num_pages=0), dict(table_stride=3),
               dict(v_page_stride=-16)):
        assert call(**kw) == 2, kw
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_seqlens", "k", "v"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(k=61 * MB), dict(k=16 * MB), dict(v=49 * MB), dict(v=51 * MB), dict(k=50 * MB)):
        assert call(**kw) == 7, kw


@pytest.mark.parametrize("kw", [
    dict(v_cache=16 * MB + 4096), dict(v_cache=16 * MB - 4096),                 # a page on, a page back
    dict(v_cache=16 * MB + 256), dict(k_cache=32 * MB + 16 * 256),              # a token's row on
    dict(v_cache=16 * MB + 128),                                                # a head's
    dict(v_cache=16 * MB + 4096 * 9 * 2), dict(v_cache=16 * MB - (4096 * 9 * 2 + 15 * 512 + 256 + 240)),      # only the last page, the last bytes
    dict(v_cache=16 * MB + 8192 * 2, k_page_stride=8192, v_page_stride=8192),   # pages of a wider tensor, the same halves
    dict(v_cache=16 * MB + 512, v_page_stride=8192, v_token_stride=512),        # strides that differ
])
def test_caches_that_share_bytes_are_refused(lib, kw):
    assert lib.kda_kv_append(ctypes.byref(kv_args(False, **kw)), None) == 7


@pytest.mark.parametrize("kw", [
    dict(k_scale=16 * MB), dict(v_scale=32 * MB + 64), dict(k_scale=32 * MB), dict(v_scale=16 * MB + 2048 * 9 + 15 * 128 + 64 + 60),
    dict(v_scale=48 * MB + 4), dict(v_scale=48 * MB + 8), dict(v_cache=16 * MB + 2048), dict(v_cache=16 * MB + 64),
])
def test_4_bit_caches_that_share_bytes_are_refused(lib, kw):
    assert lib.kda_kv_append(ctypes.byref(kv_args(True, **kw)), None) == 7


def test_caches_between_each_other(lib):
    """Two caches at random in one another's gaps, byte by byte: sharing bytes is refused, and nothing else where strides are
    the same. (Only where no GPU would run what is accepted.)"""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would run")
    g = np.random.Generator(np.random.PCG64(3))
    seen = {True: 0, False: 0}
    for _ in range(600):
        n = dict(zip(("page", "token", "cache_head"), (int(x) for x in g.integers(1, 4, 3))))
        order, at, st = list(g.permutation(list(n))), 64 * int(g.integers(1, 4)), {}
        for name in order[::-1]:
            st[name] = at
            at = at * n[name] + 64 * int(g.integers(0, 3))
        shift = 64 * int(g.integers(-at // 64 - 1, at // 64 + 2))
        rows = lambda base: {base + a * st["page"] + b * st["token"] + c * st["cache_head"] + e  # noqa: E731
                             for a in range(n["page"]) for b in range(n["token"]) for c in range(n["cache_head"]) for e in range(64)}
        share = bool(rows(0) & rows(shift))
        kw = {f"{x}_{name}_stride": s for x in "kv" for name, s in st.items()}
        kw.update(head_dim=64, rot_dim=64, k_head_stride=64, k_cache=16 * MB, v_cache=16 * MB + 2 * shift, num_pages=n["page"],
                  page_size=n["token"], kv_heads=n["cache_head"])
        code = lib.kda_kv_append(ctypes.byref(kv_args(False, **kw)), None)
        assert (code == 7) == share, (n, st, shift, code)
        seen[share] += 1
    assert min(seen.values()) > 100
