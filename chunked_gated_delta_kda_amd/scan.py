"""The selective state space scan: kda_ssm_fwd, kda_ssm_decode and kda_ssm_bwd of include/kda.h."""
import ctypes

import torch

from . import native
from ._args import DTYPES, dense, launch_on, like, offsets, on_device, ptr, rows, run, scratch

__all__ = ["ssm_fwd", "ssm_bwd", "ssm_decode"]


class _Sizes:
    """What the checks found: T, D, N (states), G, S (sequences) and the row strides."""
    __slots__ = ("T", "D", "N", "G", "S", "strides")


def _check(u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state):
    dev, dt, td, dn, tgn = u.get_device(), u.dtype, tuple(u.shape), A.shape, B.shape
    if dt not in DTYPES or len(td) != 2:
        raise ValueError(f"u: expected fp32, bf16 or fp16 [T, D], got {dt} {td}")
    s = _Sizes()
    s.T, s.D = td
    if len(dn) != 2 or not 1 <= dn[1] <= native.SSM_MAX_STATE:
        raise ValueError(f"A: expected fp32 [D, N] with N from 1 to {native.SSM_MAX_STATE}, got {tuple(dn)}")
    s.N = dn[1]
    if len(tgn) != 3 or tgn[1] < 1 or s.D % tgn[1]:
        raise ValueError(f"B: expected [T, G, N] with G dividing the {s.D} channels, got {tuple(tgn)}")
    s.G = tgn[1]
    tgn = (s.T, s.G, s.N)
    strides = [rows("u", u, dt, td, dev), rows("delta", delta, dt, td, dev), rows("B", B, dt, tgn, dev),
               rows("C", C, dt, tgn, dev), 0]
    dense("A", A, torch.float32, (s.D, s.N), dev)
    if D is not None:
        dense("D", D, torch.float32, (s.D,), dev)
    if z is not None:
        strides[4] = rows("z", z, dt, td, dev)
    if delta_bias is not None:
        dense("delta_bias", delta_bias, torch.float32, (s.D,), dev)
    s.strides = strides
    s.S = offsets(cu_seqlens, dev)
    if initial_state is not None:
        dense("initial_state", initial_state, torch.float32, (s.S, s.D, s.N), dev)
    return s


def check_ssm_fwd_args(u, delta, A, B, C, D=None, z=None, delta_bias=None, cu_seqlens=None, initial_state=None, out=None,
                       final_state=None):
    """Every check ssm_fwd makes before anything is launched; returns the sizes it found."""
    s = _check(u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state)
    if out is not None:
        dense("out", out, u.dtype, (s.T, s.D), u.get_device())
    if final_state is not None:
        dense("final_state", final_state, torch.float32, (s.S, s.D, s.N), u.get_device())
    return s


def _args(s, u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state, final_state, out, softplus):
    return native.KdaSsmArgs(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), ptr(D), ptr(z),
                             ptr(delta_bias), ptr(cu_seqlens), ptr(initial_state), ptr(final_state), ptr(out),
                             *s.strides, s.S, s.T, s.D, s.N, s.G, DTYPES[u.dtype], int(bool(softplus)))


def ssm_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, cu_seqlens=None, initial_state=None,
            output_final_state=True, *, delta_softplus=True, out=None, final_state=None, workspace=None, stream=None,
            check=False):
    """Selective state space scan over a packed batch, on the current HIP device. Per channel c of
    group g, state n and token t:

        s_t = softplus(delta_t + delta_bias);  h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t u_t B_t[g, n]
        out_t = (sum_n C_t[g, n] h_t[n] + D u_t) * silu(z_t)

    u, delta, z: fp32, bf16 or fp16 [T, D], B, C: [T, G, N] of the same dtype (N up to 256, G
    dividing D), rows contiguous, any row stride (slices of a projection are read in place); A:
    fp32 [D, N]; D, delta_bias: fp32 [D] or None; z: None for no gate; cu_seqlens: int32 [S+1] on the
    device or None (one sequence); initial_state: fp32 [S, D, N] or None (zeros); delta_softplus
    False: the steps are delta + delta_bias as they are; out, final_state: caller buffers or None. s_t A
    is meant to be negative or zero: where states grow past fp32's range within some hundred tokens, zeros become NaN.
    final_state must not overlap initial_state (ssm_decode updates in place). check: as in fwd.
    Returns (out [T, D] of u's dtype, final_state fp32 [S, D, N] or None). Tensors that the call
    allocates belong to its stream.
    """
    lib = native.load_library()
    dev = u.get_device()
    on_device("kda.ssm_fwd", dev)
    s = check_ssm_fwd_args(u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state, out, final_state)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(u, (s.T, s.D))
        if not output_final_state:
            final_state = None
        elif final_state is None:
            final_state = like(u, (s.S, s.D, s.N), torch.float32)
        workspace, wp, wn = scratch(workspace, lib.kda_ssm_workspace_bytes(s.S, s.T, s.D, s.N, s.G), u)
        args = _args(s, u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state, final_state, out, delta_softplus)
        run(check, st, lib.kda_ssm_fwd, ctypes.byref(args), st, wp, wn)
    return out, final_state


def check_ssm_decode_args(u, delta, A, B, C, D=None, z=None, delta_bias=None, state=None, out=None, state_out="inplace"):
    """Every check ssm_decode makes before the launch; returns the sizes it found."""
    s = _check(u, delta, A, B, C, D, z, delta_bias, None, None)
    if s.T < 1:
        raise ValueError("u: expected at least one row")
    if isinstance(state_out, str) and state_out != "inplace":
        raise ValueError('state_out: "inplace", None or a tensor')
    s.S = s.T
    for name, t in (("state", state), ("state_out", state_out)):
        if isinstance(t, torch.Tensor):
            dense(name, t, torch.float32, (s.S, s.D, s.N), u.get_device())
    if out is not None:
        dense("out", out, u.dtype, (s.T, s.D), u.get_device())
    return s


def ssm_decode(u, delta, A, B, C, D=None, z=None, delta_bias=None, state=None, *, delta_softplus=True, out=None,
               state_out="inplace", stream=None):
    """ssm_fwd for one token of each of S sequences: u, delta, z [S, D], B, C [S, G, N]; state fp32
    [S, D, N] (None: zeros). state_out: "inplace" (update ``state``; a new tensor when state is None),
    None (not written), or a tensor. Returns (out [S, D], the updated state or None)."""
    lib = native.load_library()
    dev = u.get_device()
    on_device("kda.ssm_decode", dev)
    s = check_ssm_decode_args(u, delta, A, B, C, D, z, delta_bias, state, out, state_out)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(u, (s.T, s.D))
        if isinstance(state_out, str):
            state_out = state if state is not None else like(u, (s.S, s.D, s.N), torch.float32)
        args = _args(s, u, delta, A, B, C, D, z, delta_bias, None, state, state_out, out, delta_softplus)
        run(False, st, lib.kda_ssm_decode, ctypes.byref(args), st)
    return out, state_out


def check_ssm_bwd_args(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, cu_seqlens=None, initial_state=None,
                       d_final_state=None):
    """Every check ssm_bwd makes before anything is launched; returns the sizes it found and dy's row stride."""
    s = _check(u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state)
    stride = rows("dy", dy, u.dtype, (s.T, s.D), u.get_device())
    if d_final_state is not None:
        dense("d_final_state", d_final_state, torch.float32, (s.S, s.D, s.N), u.get_device())
    return s, stride


def ssm_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, cu_seqlens=None, initial_state=None,
            d_final_state=None, *, delta_softplus=True, need_d_initial_state=True, workspace=None, stream=None):
    """Gradients of ssm_fwd: given dy = dL/d(out) ([T, D] of u's dtype, any row stride) and optionally
    d_final_state = dL/d(final_state) (fp32 [S, D, N]), returns a dict of du, ddelta, dz ([T, D]), dB, dC
    ([T, G, N]) of u's dtype, and fp32 dA ([D, N]), dD, ddelta_bias ([D]) and d_initial_state ([S, D, N], or None
    when need_d_initial_state is False); dz, dD and ddelta_bias are None without z, D and delta_bias. Needs
    nothing that the forward computed. The same results from run to run. The workspace holds a state per channel for
    every 4 tokens (2 from state sizes over 64, 1 over 128): 4.8 GiB for 65536 tokens of 4096 channels and 16 states."""
    lib = native.load_library()
    dev = u.get_device()
    on_device("kda.ssm_bwd", dev)
    s, dy_stride = check_ssm_bwd_args(u, delta, A, B, C, dy, D, z, delta_bias, cu_seqlens, initial_state, d_final_state)
    f32 = torch.float32
    with launch_on(dev, stream) as st:
        gr = dict(du=like(u, (s.T, s.D)), ddelta=like(u, (s.T, s.D)), dA=like(u, (s.D, s.N), f32), dB=like(u, (s.T, s.G, s.N)),
                  dC=like(u, (s.T, s.G, s.N)), dD=like(u, (s.D,), f32) if D is not None else None,
                  dz=like(u, (s.T, s.D)) if z is not None else None,
                  ddelta_bias=like(u, (s.D,), f32) if delta_bias is not None else None,
                  d_initial_state=like(u, (s.S, s.D, s.N), f32) if need_d_initial_state else None)
        workspace, wp, wn = scratch(workspace, lib.kda_ssm_bwd_workspace_bytes(s.T, s.D, s.N, s.G), u)
        args = _args(s, u, delta, A, B, C, D, z, delta_bias, cu_seqlens, initial_state, None, None, delta_softplus)
        grads = native.KdaSsmGrads(ptr(dy), ptr(d_final_state), ptr(gr["du"]), ptr(gr["ddelta"]), ptr(gr["dB"]), ptr(gr["dC"]),
                                   ptr(gr["dz"]), ptr(gr["dA"]), ptr(gr["dD"]), ptr(gr["ddelta_bias"]),
                                   ptr(gr["d_initial_state"]), dy_stride)
        run(False, st, lib.kda_ssm_bwd, ctypes.byref(args), ctypes.byref(grads), st, wp, wn)
    return gr
