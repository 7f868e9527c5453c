"""Linear attention with a decay for each head: kda_lin_fwd, kda_lin_decode and kda_lin_bwd of include/kda.h."""
import ctypes
import math

import torch

from . import native
from ._args import DTYPES, dense, fail, launch_on, like, offsets, on_device, ptr, run, scratch
from .paged_attention import _by8

__all__ = ["lin_fwd", "lin_bwd", "lin_decode"]

DIMS = (64, 128)


class _Sizes:
    """What the checks found: T, H, K and V dims, S (sequences), whether g is [H], and the strides of q, k and v."""
    __slots__ = ("T", "H", "K", "V", "S", "per_head", "strides")


def _rows(name, t, dt, shape, dev):
    if t.dtype is not dt or t.shape != shape:
        fail(name, t, f"{dt} {tuple(shape)}", dev)
    return _by8(name, t, dev)


def _state(name, t, s, dev):
    dense(name, t, torch.float32, (s.S, s.H, s.K, s.V), dev)
    if t.data_ptr() % 16:
        raise ValueError(f"{name}: expected a base aligned to 16 bytes")


def _check(q, k, v, g, scale, cu_seqlens, initial_state):
    dev, dt, shape = q.get_device(), q.dtype, q.shape
    if (dt is not torch.bfloat16 and dt is not torch.float16) or len(shape) != 3 or shape[1] < 1 or shape[2] not in DIMS:
        raise ValueError(f"q: expected bf16 or fp16 [T, H, K] with K one of {DIMS}, got {dt} {tuple(shape)}")
    if v.dim() != 3 or v.shape[2] not in DIMS:
        raise ValueError(f"v: expected [T, H, V] with V one of {DIMS}, got {tuple(v.shape)}")
    s = _Sizes()
    s.T, s.H, s.K = shape
    s.V = v.shape[2]
    s.strides = _by8("q", q, dev) + _rows("k", k, dt, shape, dev) + _rows("v", v, dt, (s.T, s.H, s.V), dev)
    s.per_head = g.dim() == 1
    dense("g", g, torch.float32, (s.H,) if s.per_head else (s.T, s.H), dev)
    if scale is not None and not math.isfinite(scale):
        raise ValueError("scale: expected a finite number")
    s.S = offsets(cu_seqlens, dev)
    if initial_state is not None:
        _state("initial_state", initial_state, s, dev)
    return s


def _args(s, q, k, v, g, scale, cu_seqlens, initial_state, final_state, out):
    return native.KdaLinArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), ptr(cu_seqlens), ptr(initial_state),
                             ptr(final_state), ptr(out), *s.strides, s.S, s.T, s.H, s.K, s.V, DTYPES[q.dtype], int(s.per_head),
                             1.0 / math.sqrt(s.K) if scale is None else scale)


def check_lin_fwd_args(q, k, v, g, scale=None, cu_seqlens=None, initial_state=None, out=None, final_state=None):
    """Every check lin_fwd makes before anything is launched; returns the sizes it found."""
    s = _check(q, k, v, g, scale, cu_seqlens, initial_state)
    if out is not None:
        dense("out", out, q.dtype, (s.T, s.H, s.V), q.get_device())
    if final_state is not None:
        _state("final_state", final_state, s, q.get_device())
    return s


def lin_fwd(q, k, v, g, scale=None, cu_seqlens=None, initial_state=None, output_final_state=True, *, out=None, final_state=None,
            workspace=None, stream=None, check=False):
    """Linear attention with a decay for each head over a packed batch, on the current HIP device:

        S_t = exp(g_t) S_{t-1} + k_t v_t^T;  out_t = scale S_t^T q_t

    q, k: bf16 or fp16 [T, H, K], v: [T, H, V] of the same dtype, K and V 64 or 128 each, any strides that are multiples of
    8 elements (slices of a projection are read in place); g: fp32 natural-log decays, [T, H] from the data or [H] fixed for each
    head, meant to be 0 or less (-inf forgets what was before); scale: 1/sqrt(K) by default; cu_seqlens: int32 [S+1] on the device or
    None (one sequence); initial_state: fp32 [S, H, K, V] or None (zeros); out, final_state: caller buffers or
    None. final_state must not overlap initial_state (lin_decode updates in place). Inputs that are not finite make what hangs on
    them infinite or NaN, and nothing before them. check: as in fwd.
    Returns (out [T, H, V] of q's dtype, final_state fp32 [S, H, K, V] or None). Tensors that the call allocates
    belong to its stream.
    """
    lib = native.load_library()
    dev = q.get_device()
    on_device("kda.lin_fwd", dev)
    s = check_lin_fwd_args(q, k, v, g, scale, cu_seqlens, initial_state, out, final_state)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(q, (s.T, s.H, s.V))
        if not output_final_state:
            final_state = None
        elif final_state is None:
            final_state = like(q, (s.S, s.H, s.K, s.V), torch.float32)
        workspace, wp, wn = scratch(workspace, lib.kda_lin_workspace_bytes(s.T, s.H, s.K, s.V), q)
        args = _args(s, q, k, v, g, scale, cu_seqlens, initial_state, final_state, out)
        run(check, st, lib.kda_lin_fwd, ctypes.byref(args), st, wp, wn)
    return out, final_state


def check_lin_decode_args(q, k, v, g, scale=None, state=None, out=None, state_out="inplace"):
    """Every check lin_decode makes before the launch; returns the sizes it found."""
    s = _check(q, k, v, g, scale, None, None)
    if s.T < 1:
        raise ValueError("q: expected at least one row")
    if isinstance(state_out, str) and state_out != "inplace":
        raise ValueError('state_out: "inplace", None or a tensor')
    s.S = s.T
    for name, t in (("state", state), ("state_out", state_out)):
        if isinstance(t, torch.Tensor):
            _state(name, t, s, q.get_device())
    if out is not None:
        dense("out", out, q.dtype, (s.T, s.H, s.V), q.get_device())
    return s


def lin_decode(q, k, v, g, scale=None, state=None, *, out=None, state_out="inplace", stream=None):
    """lin_fwd for one token of each of S sequences: q, k [S, H, K], v [S, H, V], g [S, H] or [H]; state fp32
    [S, H, K, V] (None: zeros). state_out: "inplace" (update ``state``; a new tensor when state is None),
    None (not written), or a tensor. Returns (out [S, H, V], the updated state or None)."""
    lib = native.load_library()
    dev = q.get_device()
    on_device("kda.lin_decode", dev)
    s = check_lin_decode_args(q, k, v, g, scale, state, out, state_out)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(q, (s.T, s.H, s.V))
        if isinstance(state_out, str):
            state_out = state if state is not None else like(q, (s.S, s.H, s.K, s.V), torch.float32)
        args = _args(s, q, k, v, g, scale, None, state, state_out, out)
        run(False, st, lib.kda_lin_decode, ctypes.byref(args), st)
    return out, state_out


def check_lin_bwd_args(q, k, v, g, d_out, scale=None, cu_seqlens=None, initial_state=None, d_final_state=None):
    """Every check lin_bwd makes before anything is launched; returns the sizes it found and d_out's strides."""
    s = _check(q, k, v, g, scale, cu_seqlens, initial_state)
    strides = _rows("d_out", d_out, q.dtype, (s.T, s.H, s.V), q.get_device())
    if d_final_state is not None:
        _state("d_final_state", d_final_state, s, q.get_device())
    return s, strides


def lin_bwd(q, k, v, g, d_out, scale=None, cu_seqlens=None, initial_state=None, d_final_state=None, *,
            need_d_initial_state=True, workspace=None, stream=None, check=False):
    """Gradients of lin_fwd: given d_out = dL/d(out) ([T, H, V] of q's dtype, strides as q's) and optionally d_final_state =
    dL/d(final_state) (fp32 [S, H, K, V]), returns a dict of dq, dk ([T, H, K]) and dv ([T, H, V]) of q's dtype, and fp32 dg (of
    g's shape: [T, H], or [H] summed over all tokens) and d_initial_state ([S, H, K, V], or None when need_d_initial_state is
    False). Needs nothing that the forward computed. The same results from run to run. check: as in fwd."""
    lib = native.load_library()
    dev = q.get_device()
    on_device("kda.lin_bwd", dev)
    s, strides = check_lin_bwd_args(q, k, v, g, d_out, scale, cu_seqlens, initial_state, d_final_state)
    with launch_on(dev, stream) as st:
        gr = dict(dq=like(q, (s.T, s.H, s.K)), dk=like(q, (s.T, s.H, s.K)), dv=like(q, (s.T, s.H, s.V)),
                  dg=like(q, g.shape, torch.float32),
                  d_initial_state=like(q, (s.S, s.H, s.K, s.V), torch.float32) if need_d_initial_state else None)
        need = need_d_initial_state or initial_state is None
        workspace, wp, wn = scratch(workspace, lib.kda_lin_bwd_workspace_bytes(s.S, s.T, s.H, s.K, s.V, int(s.per_head), int(need)), q)
        args = _args(s, q, k, v, g, scale, cu_seqlens, initial_state, None, None)
        grads = native.KdaLinGrads(d_out.data_ptr(), ptr(d_final_state), gr["dq"].data_ptr(), gr["dk"].data_ptr(),
                                   gr["dv"].data_ptr(), gr["dg"].data_ptr(), ptr(gr["d_initial_state"]), *strides)
        run(check, st, lib.kda_lin_bwd, ctypes.byref(args), ctypes.byref(grads), st, wp, wn)
    return gr
