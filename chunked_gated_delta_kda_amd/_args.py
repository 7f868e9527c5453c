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


def _place(index):
    return "the CPU" if index < 0 else f"cuda:{index}"


def fail(name, t, want, index):
    raise ValueError(f"{name}: expected {want} on {_place(index)}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} "
                     f"on {_place(t.get_device())}")


def dense(name, t, dtype, shape, index):
    """A contiguous ``dtype`` tensor of ``shape`` on device ``index`` (-1: the CPU)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        fail(name, t, f"contiguous {dtype} {tuple(shape)}", index)


def rows(name, t, dtype, shape, index):
    """A ``dtype`` tensor of ``shape`` whose rows (index 0) are contiguous and do not overlap; returns
    the row stride in elements."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        fail(name, t, f"{dtype} {tuple(shape)}", index)
    length = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return length
    inner = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != inner:
            fail(name, t, f"{dtype} {tuple(shape)} with contiguous rows", index)
        inner *= size
    if shape[0] > 1 and t.stride(0) < length:
        fail(name, t, f"{dtype} {tuple(shape)} with rows that do not overlap", index)
    return max(t.stride(0), length)


def offsets(cu_seqlens, index):
    """The number of sequences of ``cu_seqlens`` (None: one)."""
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dtype is not torch.int32 or cu_seqlens.get_device() != index or cu_seqlens.dim() != 1 \
            or not cu_seqlens.is_contiguous() or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens: expected a contiguous int32 vector of N+1 >= 2 offsets on the device")
    return cu_seqlens.shape[0] - 1


def on_device(what, index):
    if index < 0:
        raise ValueError(f"{what} needs device tensors")


def ptr(t):
    return None if t is None else t.data_ptr()


def like(x, shape, dtype=None):
    """A new contiguous tensor of ``shape`` on x's device, of x's dtype by default."""
    if dtype is None and x.shape == shape and x.is_contiguous():
        return torch.empty_like(x)      # the cheapest of torch's allocating calls
    return x.new_empty(shape, dtype=dtype or x.dtype)


def scratch(workspace, nbytes, x):
    """The caller's workspace, or one of ``nbytes`` on x's device (None if none is needed); its pointer and size."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        workspace = x.new_empty((nbytes,), dtype=torch.uint8)
    elif workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@contextlib.contextmanager
def _elsewhere(index, stream):
    with torch.cuda.device(index):
        if stream is None:
            yield _current_stream(index)
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


class _Here:
    """The current device and its current stream."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def launch_on(index, stream):
    """Context of one call: device ``index`` is the current one, tensors allocated inside belong to the
    call's stream (torch's allocator hands their memory on in that stream's order), and the
    value is that stream's handle. ``stream`` None: torch's current stream of the device."""
    if stream is None and torch.cuda.current_device() == index:
        return _Here(_current_stream(index))
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream: expected one of {_place(index)}, where the inputs are, got one of {stream.device}")
    return _elsewhere(index, stream)


def run(check, handle, call, *args):
    """One call of the library; ``check``: with the device error word cleared before it and read after (both
    synchronise)."""
    if not check:
        rc = call(*args)
        if rc:
            native.check(rc)
        return
    native.device_errors(handle, clear=True)
    native.check(call(*args))
    bits = native.device_errors(handle, clear=True)
    if bits:
        raise native.KdaDeviceError(bits)
