"""New keys and values into the paged cache that attn_decode and attn_decode_fp4 read, rotated on the way, and the
4-bit cache itself: kda_kv_append and kda_kv_read_fp4 of include/kda.h."""
import ctypes

import torch

from . import native
from ._args import DTYPES, dense, fail, launch_on, like, offsets, on_device, ptr, run
from .paged_attention import HEAD_DIMS, _by8, check_cache_fp4, check_table

__all__ = ["kv_append", "kv_cache_fp4", "kv_read_fp4"]


def kv_cache_fp4(pages, page_size, heads, head_dim, device=None):
    """A cache of 4 bits an element, zeros in it: (k_cache, v_cache) uint8 [pages, page size, heads, head_dim / 2] and
    (k_scale, v_scale) uint8 [pages, page size, heads, head_dim / 32], in this order, with the rows of a head next to each
    other in a page, as the memory likes them best. A page of 16 tokens of one head of 128 takes 1088 bytes a side
    (4096 in 16 bits)."""
    if head_dim not in HEAD_DIMS:
        raise ValueError(f"head_dim {head_dim}; expected one of {HEAD_DIMS}")
    if min(pages, page_size, heads) < 1:
        raise ValueError("pages, page_size and heads: expected at least 1 each")
    code = torch.zeros(2, pages, heads, page_size, head_dim // 2, dtype=torch.uint8, device=device or "cuda")
    scale = torch.full((2, pages, heads, page_size, head_dim // native.FP4_GROUP), 127, dtype=torch.uint8, device=code.device)
    return tuple(x[i].transpose(1, 2) for x in (code, scale) for i in (0, 1))


def _rows(name, t, dt, heads, dh, T, dev):
    if t.dtype is not dt or t.dim() != 3 or t.shape[0] != T or t.shape[2] != dh or (heads is not None and t.shape[1] != heads) \
            or t.shape[1] < 1:
        fail(name, t, f"{dt} [{T}, {'Hq' if heads is None else heads}, {dh}]", dev)
    return _by8(name, t, dev)


class _Sizes:
    __slots__ = ("T", "N", "hq", "hkv", "dh", "rot", "positions", "pages", "page", "width", "strides")


def check_kv_append_args(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, rope=None, q=None, interleaved=False,
                         k_scale=None, v_scale=None, q_out=None):
    """Every check kv_append makes before the launch; returns the sizes it found."""
    dev, dt = k.get_device(), k.dtype
    if (dt is not torch.bfloat16 and dt is not torch.float16) or k.dim() != 3 or k.shape[2] not in HEAD_DIMS or k.shape[1] < 1:
        raise ValueError(f"k: expected bf16 or fp16 [T, Hkv, Dh] with Dh one of {HEAD_DIMS}, got {dt} {tuple(k.shape)}")
    s = _Sizes()
    s.T, s.hkv, s.dh = k.shape
    strides = _by8("k", k, dev) + _rows("v", v, dt, s.hkv, s.dh, s.T, dev)
    strides += _rows("q", q, dt, None, s.dh, s.T, dev) if q is not None else [0, 0]
    s.hq = q.shape[1] if q is not None else 0
    if q_out is not None:
        if q is None:
            raise ValueError("q_out: given without q")
        dense("q_out", q_out, dt, q.shape, dev)
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale: expected both or none")
    scales = [0] * 6
    if k_scale is not None:
        kc, ks = check_cache_fp4("k", k_cache, k_scale, s.dh, dev)
        vc, vs = check_cache_fp4("v", v_cache, v_scale, s.dh, dev, k_cache.shape)
        cache, scales = kc + vc, ks + vs
    else:
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype is not dt or t.dim() != 4 or t.shape != k_cache.shape or t.shape[3] != s.dh or min(t.shape) < 1:
                raise ValueError(f"{name}: expected {dt} [pages, page size, {s.hkv}, {s.dh}], one shape for both, got {t.dtype} "
                                 f"{tuple(t.shape)}")
        cache = _by8("k_cache", k_cache, dev) + _by8("v_cache", v_cache, dev)
    s.pages, s.page, heads, _ = k_cache.shape
    if heads != s.hkv:
        raise ValueError(f"k: {s.hkv} heads, the cache has {heads}")
    if cu_seqlens is None:
        s.N = s.T
        if s.N < 1:
            raise ValueError("k: expected at least one row without cu_seqlens")
    else:
        s.N = offsets(cu_seqlens, dev)
    s.width, table = check_table(block_table, s.N, dev)
    dense("seq_lens", seq_lens, torch.int32, (s.N,), dev)
    s.rot = s.positions = 0
    if rope is not None:
        if rope.dim() != 2 or rope.shape[0] < 1 or rope.shape[1] % 16 or not 16 <= rope.shape[1] <= s.dh:
            raise ValueError(f"rope: expected fp32 [positions, rotated elements], a multiple of 16 up to {s.dh}, got {tuple(rope.shape)}")
        dense("rope", rope, torch.float32, rope.shape, dev)
        if rope.data_ptr() % 16:
            raise ValueError("rope: expected a base aligned to 16 bytes")
        s.positions, s.rot = rope.shape
    s.strides = strides + cache + scales + [table]
    return s


def kv_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, rope=None, q=None, *, interleaved=False,
              k_scale=None, v_scale=None, q_out=None, stream=None, check=False):
    """Writes the new keys and values of each sequence into its last places in a paged cache, on the current HIP device:
    the j-th of a sequence's n new rows goes to position seq_lens - n + j. What attn_decode (attn_decode_fp4) then reads with
    the same table and lengths.

    k, v: bf16 or fp16 [T, Hkv, Dh], Dh 64, 128 or 256, any strides that are multiples of 8 elements (slices of a projection
    are read in place); k_cache, v_cache: [pages, page size, Hkv, Dh] of k's dtype as attn_decode takes them, or with
    k_scale and v_scale the codes of a 4-bit cache (``kv_cache_fp4``); block_table: int32 [N, W]; seq_lens: int32 [N], cached tokens,
    the new ones included, 0 for an empty slot, whose rows are passed over; cu_seqlens: int32 [N+1] on the device (rows behind
    the last offset are padding), or None: one row for each of N = T sequences; rope: fp32 [positions, R], R a multiple of 16 up to
    Dh, R/2 cosines and R/2 sines of each position, or None for no rotation; interleaved: neighbouring elements turn
    together, else i and i + R/2; the elements behind R stay; q: [T, Hq, Dh], rotated likewise; q_out: buffer for it or None.
    Caches and scales may be slices of one tensor that lie between each other, but share no bytes.
    check: as in fwd; rows that do not fit the table, the cache or the table of rotations are left out and raise.
    Returns the rotated q [T, Hq, Dh] (None without q); rows that are padding or left out are not written there, nor in the
    cache. A tensor that the call allocates belongs to its stream.
    """
    lib = native.load_library()
    dev = k.get_device()
    on_device("kda.kv_append", dev)
    s = check_kv_append_args(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens, rope, q, interleaved, k_scale, v_scale,
                             q_out)
    with launch_on(dev, stream) as st:
        if q is not None and q_out is None:
            q_out = like(q, q.shape)
        args = native.KdaKvArgs(k.data_ptr(), v.data_ptr(), ptr(q), ptr(q_out), ptr(rope), ptr(cu_seqlens), block_table.data_ptr(),
                                seq_lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ptr(k_scale), ptr(v_scale),
                                *s.strides, s.N, s.T, s.hq, s.hkv, s.dh, s.rot, s.positions, s.pages, s.page, s.width,
                                DTYPES[k.dtype], int(bool(interleaved)))
        run(check, st, lib.kda_kv_append, ctypes.byref(args), st)
    return q_out


def check_kv_read_fp4_args(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, total_tokens, dtype, k=None, v=None):
    """Every check kv_read_fp4 makes before the launch; returns (N, Hkv, Dh, pages, page size, table width, strides)."""
    dev = k_cache.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"dtype: expected bf16 or fp16, got {dtype}")
    if k_cache.dim() != 4 or k_cache.shape[3] * 2 not in HEAD_DIMS:
        raise ValueError(f"k_cache: expected uint8 [pages, page size, Hkv, Dh / 2] with Dh one of {HEAD_DIMS}, got {tuple(k_cache.shape)}")
    dh = k_cache.shape[3] * 2
    kc, ks = check_cache_fp4("k", k_cache, k_scale, dh, dev)
    vc, vs = check_cache_fp4("v", v_cache, v_scale, dh, dev, k_cache.shape)
    if cu_seqlens is None:
        raise ValueError("cu_seqlens: expected the offsets of the sequences' rows")
    if total_tokens < 0:
        raise ValueError("total_tokens: expected 0 or more")
    N = offsets(cu_seqlens, dev)
    width, table = check_table(block_table, N, dev)
    pages, page, hkv, _ = k_cache.shape
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            dense(name, t, dtype, (total_tokens, hkv, dh), dev)
    return N, hkv, dh, pages, page, width, kc + vc + ks + vs + [table]


def kv_read_fp4(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, total_tokens, dtype=torch.bfloat16, *, k=None,
                v=None, stream=None, check=False):
    """The first tokens of each sequence of a 4-bit cache as packed rows, for a prompt that continues them: sequence n's
    first cu_seqlens[n+1] - cu_seqlens[n] cached tokens become rows cu_seqlens[n].. of k and v [total_tokens, Hkv, Dh], bf16
    (exact) or fp16 (exact from 2**-24 to 65504). cu_seqlens: int32 [N+1] on the device; rows behind its last offset are not
    written. Cache and table as kv_append; k, v: buffers or None. Tokens on a page outside the cache are zeros; check: as in
    fwd, they raise. Returns (k, v). Tensors that the call allocates belong to its stream."""
    lib = native.load_library()
    dev = k_cache.get_device()
    on_device("kda.kv_read_fp4", dev)
    N, hkv, dh, pages, page, width, strides = check_kv_read_fp4_args(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                                                                    total_tokens, dtype, k, v)
    with launch_on(dev, stream) as st:
        k = like(k_cache, (total_tokens, hkv, dh), dtype) if k is None else k
        v = like(k_cache, (total_tokens, hkv, dh), dtype) if v is None else v
        args = native.KdaKvReadArgs(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                    block_table.data_ptr(), cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, N,
                                    total_tokens, hkv, dh, pages, page, width, DTYPES[dtype])
        run(check, st, lib.kda_kv_read_fp4, ctypes.byref(args), st)
    return k, v
