"""Attention of one new token per sequence over a paged key-value cache: kda_attn_decode and
kda_attn_decode_fp4 of include/kda.h."""
import ctypes
import math

import torch

from . import native
from ._args import DTYPES, dense, fail, launch_on, like, on_device, ptr, run, scratch

__all__ = ["attn_decode", "attn_decode_fp4"]

HEAD_DIMS = (64, 128, 256)


def _by8(name, t, dev):
    """Rows read 16 bytes at a time: the last dimension contiguous, other strides multiples of 8 (those of
    dimensions of one entry do not matter). Returns those strides."""
    shape = t.shape
    if t.is_contiguous():       # (its strides of dimensions of one entry may be any: formed from the sizes)
        inner = shape[-1]
        strides = [shape[1] * inner, inner] if len(shape) == 3 else [shape[1] * shape[2] * inner, shape[2] * inner, inner]
        bad = False
    elif len(shape) == 3:       # (written out: a loop over dimensions takes longer than all else here)
        a, b, inner = t.stride()
        strides = [a if shape[0] > 1 else 0, b if shape[1] > 1 else 0]
        bad = inner != 1 or (strides[0] | strides[1]) & 7
    else:
        a, b, c, inner = t.stride()
        strides = [a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, c if shape[2] > 1 else 0]
        bad = inner != 1 or (strides[0] | strides[1] | strides[2]) & 7
    if bad or t.data_ptr() % 16 or t.get_device() != dev:
        fail(name, t, "rows of contiguous elements, strides that are multiples of 8, a base aligned to 16 bytes", dev)
    return strides


def _check_q(q):
    dt, shape = q.dtype, q.shape
    if (dt is not torch.bfloat16 and dt is not torch.float16) or len(shape) != 3 or shape[0] < 1:
        raise ValueError(f"q: expected bf16 or fp16 [B, Hq, Dh], got {dt} {tuple(shape)}")
    if shape[2] not in HEAD_DIMS:
        raise ValueError(f"q: head dimension {shape[2]}; expected one of {HEAD_DIMS}")
    return shape


def check_table(block_table, rows, dev):
    """The width and row stride of a table of the pages of ``rows`` sequences."""
    table = block_table.shape
    if block_table.dtype is not torch.int32 or len(table) != 2 or table[0] != rows or table[1] < 1 or block_table.get_device() != dev:
        fail("block_table", block_table, f"int32 [{rows}, pages of the longest]", dev)
    stride, inner = block_table.stride()
    if (table[1] > 1 and inner != 1) or (rows > 1 and stride < table[1]):
        fail("block_table", block_table, f"int32 [{rows}, pages of the longest] with contiguous rows", dev)
    return table[1], stride if rows > 1 else table[1]


def _check(q, k_cache, v_cache, block_table, seq_lens, scale, out, lse):
    dev, dt = q.get_device(), q.dtype
    B, hq, dh = shape = _check_q(q)
    cache = k_cache.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype is not dt or len(cache) != 4 or t.shape != cache or cache[3] != dh or min(cache) < 1:
            raise ValueError(f"{name}: expected {dt} [pages, page size, Hkv, {dh}], one shape for both, got {t.dtype} "
                             f"{tuple(t.shape)}")
    strides = _by8("q", q, dev) + _by8("k_cache", k_cache, dev) + _by8("v_cache", v_cache, dev)
    pages, page, hkv, _ = cache
    width = _check_rest(q, hkv, block_table, seq_lens, scale, out, lse, strides)
    return B, hq, hkv, dh, pages, page, width, strides


def _check_rest(q, hkv, block_table, seq_lens, scale, out, lse, strides):
    """What does not depend on the form of the cache; appends the table's row stride to ``strides``, returns its width."""
    dev, (B, hq, _) = q.get_device(), q.shape
    if hq % hkv:
        raise ValueError(f"q: {hq} heads are not a multiple of the cache's {hkv}")
    width, stride = check_table(block_table, B, dev)
    strides.append(stride)
    dense("seq_lens", seq_lens, torch.int32, (B,), dev)
    if scale is not None and not math.isfinite(scale):
        raise ValueError("scale: expected a finite number")
    if out is not None:
        dense("out", out, q.dtype, q.shape, dev)
    if lse is not None:
        dense("lse", lse, torch.float32, (B, hq), dev)
    return width


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


def check_cache_fp4(name, code, scale, dh, dev, shape=None):
    """Codes and scales of one side of a 4-bit cache; returns the strides of both (bytes). ``shape``: of the other side's codes."""
    cs, ss = code.shape, scale.shape
    if code.dtype is not torch.uint8 or len(cs) != 4 or cs[3] * 2 != dh or min(cs) < 1 or (shape is not None and cs != shape) \
            or code.get_device() != dev:
        fail(f"{name}_cache", code, f"uint8 [pages, page size, Hkv, {dh // 2}], one shape for both,", dev)
    per = dh // native.FP4_GROUP
    if scale.dtype is not torch.uint8 or ss[:3] != cs[:3] or ss[3:] != (per,) or scale.get_device() != dev:
        fail(f"{name}_scale", scale, f"uint8 {(*cs[:3], per)}", dev)
    both = []
    for what, t, unit in ((f"{name}_cache", code, 16), (f"{name}_scale", scale, per)):
        a, b, c, inner = t.stride()
        strides = [a if cs[0] > 1 else 0, b if cs[1] > 1 else 0, c if cs[2] > 1 else 0]
        if inner != 1 or t.data_ptr() % unit or (strides[0] | strides[1] | strides[2]) % unit:      # (units are powers of two)
            fail(what, t, f"contiguous rows, strides that are multiples of {unit} bytes, a base aligned to {unit}", dev)
        both.append(strides)
    return both


def check_attn_decode_fp4_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale=None, out=None, lse=None):
    """Every check attn_decode_fp4 makes before anything is launched; returns (B, Hq, Hkv, Dh, pages, page
    size, table width), the strides of q, the codes and the table, and those of the scales."""
    dev = q.get_device()
    B, hq, dh = _check_q(q)
    k, ks = check_cache_fp4("k", k_cache, k_scale, dh, dev)
    v, vs = check_cache_fp4("v", v_cache, v_scale, dh, dev, k_cache.shape)
    strides = _by8("q", q, dev) + k + v
    pages, page, hkv, _ = k_cache.shape
    width = _check_rest(q, hkv, block_table, seq_lens, scale, out, lse, strides)
    return (B, hq, hkv, dh, pages, page, width), strides, ks + vs


def attn_decode_fp4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale=None, *, return_lse=False, out=None,
                    lse=None, workspace=None, stream=None, check=False):
    """attn_decode over a cache of 4 bits an element (``kv_cache_fp4``, written by ``kv_append``): k_cache, v_cache:
    uint8 [pages, page size, Hkv, Dh / 2], two e2m1 codes a byte, the even element in the low half; k_scale, v_scale: uint8
    [pages, page size, Hkv, Dh / 32], s for 2**(s - 127), 255 for NaN. Rows contiguous, other strides multiples of
    16 bytes (of a row, for scales). The rest as attn_decode; the values that the codes stand for are exact in bf16 and, from 2**-24 to
    65504, in fp16.
    Returns out [B, Hq, Dh] of q's dtype, or (out, lse). Tensors that the call allocates belong to its stream.
    """
    lib = native.load_library()
    dev = q.get_device()
    on_device("kda.attn_decode_fp4", dev)
    sizes, strides, scales = check_attn_decode_fp4_args(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale, out, lse)
    B, hq, hkv, dh, pages, page, width = sizes
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(q, q.shape)
        if lse is None and return_lse:
            lse = like(q, (B, hq), torch.float32)
        workspace, wp, wn = scratch(workspace, lib.kda_attn_fp4_workspace_bytes(B, hq, hkv, dh, width, page), q)
        args = native.KdaAttnFp4Args(native.KdaAttnArgs(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
            ptr(lse), *strides, B, hq, hkv, dh, pages, page, width, DTYPES[q.dtype],
            1.0 / math.sqrt(dh) if scale is None else scale), k_scale.data_ptr(), v_scale.data_ptr(), *scales)
        run(check, st, lib.kda_attn_decode_fp4, ctypes.byref(args), st, wp, wn)
    return (out, lse) if return_lse else out
