"""Argument checks and stream handling shared by the operators beside the delta rule."""
import contextlib

import torch

from . import native

try:    # the handle of a device's current stream, without a Stream object around it (0.1 us for 1.9 us)
    from torch._C import _cuda_getCurrentRawStream as _current_stream
except ImportError:
    def _current_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


DTYPES = {torch.float32: native.ACT_DTYPES["f32"], torch.bfloat16: native.ACT_DTYPES["bf16"],
          torch.float16: native.ACT_DTYPES["f16"]}


def fail(name, t, want, dev):
    raise ValueError(f"{name}: expected {want} on {dev}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} "
                     f"on {t.device}")


def dense(name, t, dtype, shape, dev):
    """A contiguous ``dtype`` tensor of ``shape`` on ``dev``."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        fail(name, t, f"contiguous {dtype} {tuple(shape)}", dev)


def rows(name, t, dtype, shape, dev):
    """A ``dtype`` tensor of ``shape`` whose rows (index 0) are contiguous and do not overlap; returns
    the row stride in elements."""
    if t.dtype != dtype or t.shape != shape or t.device != dev:
        fail(name, t, f"{dtype} {tuple(shape)}", dev)
    length = shape[1] if len(shape) == 2 else _row_len(shape)
    if t.is_contiguous():
        return length
    inner = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != inner:
            fail(name, t, f"{dtype} {tuple(shape)} with contiguous rows", dev)
        inner *= size
    if shape[0] > 1 and t.stride(0) < length:
        fail(name, t, f"{dtype} {tuple(shape)} with rows that do not overlap", dev)
    return max(t.stride(0), length)


def _row_len(shape):
    n = 1
    for s in shape[1:]:
        n *= s
    return n


def offsets(cu_seqlens, dev):
    """The number of sequences of ``cu_seqlens`` (None: one)."""
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1 \
            or not cu_seqlens.is_contiguous() or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens: expected a contiguous int32 vector of N+1 >= 2 offsets on the device")
    return cu_seqlens.shape[0] - 1


def on_device(what, dev):
    if dev.type != "cuda":
        raise ValueError(f"{what} needs device tensors")


def ptr(t):
    return t.data_ptr() if t is not None else None


def scratch(workspace, nbytes, dev):
    """The caller's workspace, or one of ``nbytes`` (None if none is needed); its pointer and size."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size()


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream(dev).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


class _Here:
    """The current device and its current stream."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def launch_on(dev, stream):
    """Context of one call: ``dev`` is the current device, tensors allocated inside belong to the
    call's stream (torch's allocator hands their memory on in that stream's order), and the
    value is that stream's handle. ``stream`` None: torch's current stream of ``dev``."""
    if stream is None and torch.cuda.current_device() == dev.index:
        return _Here(_current_stream(dev.index))
    return _elsewhere(dev, stream)


def checked(handle, call):
    """``call`` with the device error word cleared before it and read after (both synchronise)."""
    native.device_errors(handle, clear=True)
    call()
    bits = native.device_errors(handle, clear=True)
    if bits:
        raise native.KdaDeviceError(bits)
