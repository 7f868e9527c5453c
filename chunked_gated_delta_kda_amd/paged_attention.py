"""Attention of one new token per sequence over a paged key-value cache: kda_attn_decode of
include/kda.h."""
import ctypes
import math

import torch

from . import native
from ._args import DTYPES, dense, fail, launch_on, like, on_device, ptr, run, scratch

__all__ = ["attn_decode"]

HEAD_DIMS = (64, 128, 256)


def _by8(name, t, dev):
    """Rows read 16 bytes at a time: the last dimension contiguous, other strides multiples of 8 (those of
    dimensions of one entry do not matter). Returns those strides."""
    shape = t.shape
    if t.is_contiguous():       # (its strides of dimensions of one entry may be any: formed from the sizes)
        inner = shape[-1]
        strides = [shape[1] * inner, inner] if len(shape) == 3 else [shape[1] * shape[2] * inner, shape[2] * inner, inner]
        bad = False
    else:
        last = len(shape) - 1
        strides = [s if n > 1 else 0 for n, s in zip(shape[:last], t.stride())]
        bad = t.stride(last) != 1 or any(s % 8 for s in strides)
    if bad or t.data_ptr() % 16 or t.get_device() != dev:
        fail(name, t, "rows of contiguous elements, strides that are multiples of 8, a base aligned to 16 bytes", dev)
    return strides


def _check(q, k_cache, v_cache, block_table, seq_lens, scale, out, lse):
    dev, dt, shape = q.get_device(), q.dtype, q.shape
    if (dt is not torch.bfloat16 and dt is not torch.float16) or len(shape) != 3 or shape[0] < 1:
        raise ValueError(f"q: expected bf16 or fp16 [B, Hq, Dh], got {dt} {tuple(shape)}")
    B, hq, dh = shape
    if dh not in HEAD_DIMS:
        raise ValueError(f"q: head dimension {dh}; expected one of {HEAD_DIMS}")
    cache = k_cache.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not dt or len(cache) != 4 or t.shape != cache or cache[3] != dh or min(cache) < 1:
            raise ValueError(f"{name}: expected {dt} [pages, page size, Hkv, {dh}], one shape for both, got {t.dtype} "
                             f"{tuple(t.shape)}")
    strides = _by8("q", q, dev) + _by8("k_cache", k_cache, dev) + _by8("v_cache", v_cache, dev)
    pages, page, hkv, _ = cache
    if hq % hkv:
        raise ValueError(f"q: {hq} heads are not a multiple of the cache's {hkv}")
    table = block_table.shape
    if block_table.dtype is not torch.int32 or len(table) != 2 or table[0] != B or table[1] < 1 or block_table.get_device() != dev:
        fail("block_table", block_table, f"int32 [{B}, pages of the longest]", dev)
    rows, inner = block_table.stride()
    if (table[1] > 1 and inner != 1) or (B > 1 and rows < table[1]):
        fail("block_table", block_table, f"int32 [{B}, pages of the longest] with contiguous rows", dev)
    strides.append(rows if B > 1 else table[1])
    dense("seq_lens", seq_lens, torch.int32, (B,), dev)
    if scale is not None and not math.isfinite(scale):
        raise ValueError("scale: expected a finite number")
    if out is not None:
        dense("out", out, dt, shape, dev)
    if lse is not None:
        dense("lse", lse, torch.float32, (B, hq), dev)
    return B, hq, hkv, dh, pages, page, table[1], strides


def check_attn_decode_args(q, k_cache, v_cache, block_table, seq_lens, scale=None, out=None, lse=None):
    """Every check attn_decode makes before anything is launched; returns (B, Hq, Hkv, Dh, pages, page
    size, table width)."""
    return _check(q, k_cache, v_cache, block_table, seq_lens, scale, out, lse)[:7]


def attn_decode(q, k_cache, v_cache, block_table, seq_lens, scale=None, *, return_lse=False, out=None, lse=None,
                workspace=None, stream=None, check=False):
    """Attention of one new token of each of B sequences over its cached tokens, on the current
    HIP device: out[h] = sum_t softmax_t(scale q[h].k_t) v_t.

    q: bf16 or fp16 [B, Hq, Dh], B up to 65536, Dh 64, 128 or 256; k_cache, v_cache: [pages, page size, Hkv, Dh] of
    q's dtype, Hkv dividing Hq (query head h reads cache head h // (Hq // Hkv)), any strides that
    are multiples of 8 elements (a transposed layout or a slice of a joint cache is read in
    place); block_table: int32 [B, W], the pages of each sequence in order (entries past its
    length are not read); seq_lens: int32 [B], cached tokens, the new one's included, 0 for an
    empty slot (zeros, lse -inf); scale: 1/sqrt(Dh) by default. return_lse: also return fp32
    lse [B, Hq], the logarithm of the softmax's sum (to join with other parts); out, lse: caller
    buffers or None (lse is written where it is given). check: as in fwd; a page outside the
    cache, whose tokens are left out, or a length past its row of the table raise.
    Returns out [B, Hq, Dh], or (out, lse). Tensors that the call allocates belong to its stream.
    """
    lib = native.load_library()
    dev = q.get_device()
    on_device("kda.attn_decode", dev)
    B, hq, hkv, dh, pages, page, width, strides = _check(q, k_cache, v_cache, block_table, seq_lens, scale, out, lse)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(q, q.shape)
        if lse is None and return_lse:
            lse = like(q, (B, hq), torch.float32)
        workspace, wp, wn = scratch(workspace, lib.kda_attn_workspace_bytes(B, hq, hkv, dh, width, page), q)
        args = native.KdaAttnArgs(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                  seq_lens.data_ptr(), out.data_ptr(), ptr(lse), *strides, B, hq, hkv, dh, pages, page,
                                  width, DTYPES[q.dtype], 1.0 / math.sqrt(dh) if scale is None else scale)
        run(check, st, lib.kda_attn_decode, ctypes.byref(args), st, wp, wn)
    return (out, lse) if return_lse else out
