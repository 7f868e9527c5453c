"""The short causal convolution in front of a recurrence: kda_conv_fwd, kda_conv_decode and
kda_conv_bwd of include/kda.h."""
import ctypes

import torch

from . import native
from ._args import DTYPES, dense, launch_on, like, offsets, on_device, ptr, rows, run, scratch

__all__ = ["conv_fwd", "conv_bwd", "conv_decode"]

_ACTIVATIONS = {None: 0, "silu": 1}


def _check(x, weight, bias, cu_seqlens, initial_state, activation):
    """Checks of the arguments that all three calls share; returns (T, C, W, N, row stride of x)."""
    if activation not in _ACTIVATIONS:
        raise ValueError('activation: "silu" or None')
    if x.dtype not in DTYPES or x.dim() != 2:
        raise ValueError(f"x: expected fp32, bf16 or fp16 [T, C], got {x.dtype} {tuple(x.shape)}")
    dev = x.get_device()
    T, C = x.shape
    if weight.dim() != 2 or not 2 <= weight.shape[1] <= native.CONV_MAX_WIDTH:
        raise ValueError(f"weight: expected fp32 [C, W] with W from 2 to {native.CONV_MAX_WIDTH}, got {tuple(weight.shape)}")
    W = weight.shape[1]
    stride = rows("x", x, x.dtype, (T, C), dev)
    dense("weight", weight, torch.float32, (C, W), dev)
    if bias is not None:
        dense("bias", bias, torch.float32, (C,), dev)
    N = offsets(cu_seqlens, dev)
    if initial_state is not None:
        dense("initial_state", initial_state, x.dtype, (N, W - 1, C), dev)
    return T, C, W, N, stride


def check_conv_fwd_args(x, weight, bias=None, cu_seqlens=None, initial_state=None, activation="silu", out=None,
                        final_state=None):
    """Every check conv_fwd makes before anything is launched; returns (T, C, W, N, row stride of x)."""
    T, C, W, N, stride = _check(x, weight, bias, cu_seqlens, initial_state, activation)
    if out is not None:
        dense("out", out, x.dtype, (T, C), x.get_device())
    if final_state is not None:
        dense("final_state", final_state, x.dtype, (N, W - 1, C), x.get_device())
    return T, C, W, N, stride


def conv_fwd(x, weight, bias=None, cu_seqlens=None, initial_state=None, output_final_state=True, *, activation="silu",
             out=None, final_state=None, stream=None, check=False):
    """Short causal convolution of each channel over a packed batch, on the current HIP device:
    out_t = silu(bias + sum_j weight[:, j] x_{t-W+1+j}), rows before a sequence's first taken from
    its initial state.

    x: fp32, bf16 or fp16 [T, C], rows contiguous, any row stride (a slice of a wider
    projection is read in place); weight: fp32 [C, W], W from 2 to 8, tap W-1 on the row itself;
    bias: fp32 [C] or None; cu_seqlens: int32 [N+1] on the device or None (one sequence);
    initial_state: [N, W-1, C] of x's dtype, oldest row first, or None (zeros); activation: "silu"
    or None; out, final_state: caller buffers or None. final_state must not overlap
    initial_state (conv_decode updates in place). check: as in fwd.
    Returns (out [T, C], final_state [N, W-1, C] or None), of x's dtype. Tensors that the call
    allocates belong to its stream.
    """
    lib = native.load_library()
    dev = x.get_device()
    on_device("kda.conv_fwd", dev)
    T, C, W, N, stride = check_conv_fwd_args(x, weight, bias, cu_seqlens, initial_state, activation, out, final_state)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(x, (T, C))
        if not output_final_state:
            final_state = None
        elif final_state is None:
            final_state = like(x, (N, W - 1, C))
        args = native.KdaConvArgs(x.data_ptr(), weight.data_ptr(), ptr(bias), ptr(cu_seqlens), ptr(initial_state),
                                  ptr(final_state), out.data_ptr(), stride, N, T, C, W, DTYPES[x.dtype], _ACTIVATIONS[activation])
        run(check, st, lib.kda_conv_fwd, ctypes.byref(args), st)
    return out, final_state


def check_conv_decode_args(x, weight, bias=None, state=None, activation="silu", out=None, state_out="inplace"):
    """Every check conv_decode makes before the launch; returns (N, C, W, row stride of x)."""
    T, C, W, _, stride = _check(x, weight, bias, None, None, activation)
    if T < 1:
        raise ValueError("x: expected at least one row")
    if isinstance(state_out, str) and state_out != "inplace":
        raise ValueError('state_out: "inplace", None or a tensor')
    for name, t in (("state", state), ("state_out", state_out)):
        if isinstance(t, torch.Tensor):
            dense(name, t, x.dtype, (T, W - 1, C), x.get_device())
    if out is not None:
        dense("out", out, x.dtype, (T, C), x.get_device())
    return T, C, W, stride


def conv_decode(x, weight, bias=None, state=None, *, activation="silu", out=None, state_out="inplace", stream=None):
    """conv_fwd for one row of each of N sequences: x [N, C]; state [N, W-1, C] of x's dtype holds
    the rows before it (None: zeros) and moves up by one row. state_out: "inplace" (update
    ``state``; a new tensor when state is None), None (not written), or a tensor.
    Returns (out [N, C], the updated state or None)."""
    lib = native.load_library()
    dev = x.get_device()
    on_device("kda.conv_decode", dev)
    N, C, W, stride = check_conv_decode_args(x, weight, bias, state, activation, out, state_out)
    with launch_on(dev, stream) as st:
        if out is None:
            out = like(x, (N, C))
        if isinstance(state_out, str):
            state_out = state if state is not None else like(x, (N, W - 1, C))
        args = native.KdaConvArgs(x.data_ptr(), weight.data_ptr(), ptr(bias), None, ptr(state), ptr(state_out), out.data_ptr(),
                                  stride, N, N, C, W, DTYPES[x.dtype], _ACTIVATIONS[activation])
        run(False, st, lib.kda_conv_decode, ctypes.byref(args), st)
    return out, state_out


def check_conv_bwd_args(x, weight, dy, bias=None, cu_seqlens=None, initial_state=None, d_final_state=None,
                        activation="silu"):
    """Every check conv_bwd makes before anything is launched; returns (T, C, W, N, row strides of x and dy)."""
    T, C, W, N, stride = _check(x, weight, bias, cu_seqlens, initial_state, activation)
    dy_stride = rows("dy", dy, x.dtype, (T, C), x.get_device())
    if d_final_state is not None:
        dense("d_final_state", d_final_state, torch.float32, (N, W - 1, C), x.get_device())
    return T, C, W, N, stride, dy_stride


def conv_bwd(x, weight, dy, bias=None, cu_seqlens=None, initial_state=None, d_final_state=None, *, activation="silu",
             need_d_initial_state=True, workspace=None, stream=None):
    """Gradients of conv_fwd: given dy = dL/d(out) ([T, C] of x's dtype, any row stride) and
    optionally d_final_state = dL/d(final_state) (fp32 [N, W-1, C]), returns a dict of dx ([T, C], x's
    dtype), dweight (fp32 [C, W]), dbias (fp32 [C], None without a bias) and d_initial_state (fp32
    [N, W-1, C], or None when need_d_initial_state is False). The same results from run to run."""
    lib = native.load_library()
    dev = x.get_device()
    on_device("kda.conv_bwd", dev)
    T, C, W, N, stride, dy_stride = check_conv_bwd_args(x, weight, dy, bias, cu_seqlens, initial_state, d_final_state,
                                                        activation)
    f32 = torch.float32
    with launch_on(dev, stream) as st:
        gr = dict(dx=like(x, (T, C)), dweight=like(x, (C, W), f32), dbias=like(x, (C,), f32) if bias is not None else None,
                  d_initial_state=like(x, (N, W - 1, C), f32) if need_d_initial_state else None)
        workspace, wp, wn = scratch(workspace, lib.kda_conv_bwd_workspace_bytes(T, C, W), x)
        args = native.KdaConvArgs(ptr(x), ptr(weight), ptr(bias), ptr(cu_seqlens), ptr(initial_state), None, None, stride,
                                  N, T, C, W, DTYPES[x.dtype], _ACTIVATIONS[activation])
        grads = native.KdaConvGrads(ptr(dy), ptr(d_final_state), ptr(gr["dx"]), ptr(gr["dweight"]), ptr(gr["dbias"]),
                                    ptr(gr["d_initial_state"]), dy_stride)
        run(False, st, lib.kda_conv_bwd, ctypes.byref(args), ctypes.byref(grads), st, wp, wn)
    return gr
