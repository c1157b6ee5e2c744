"""Device memory with unmapped addresses around it, for tests of what kernels fetch past a tensor's end."""
import ctypes

import torch

DEV = "cuda:0"


class _Location(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("id", ctypes.c_int)]


class _Properties(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("handle_types", ctypes.c_int), ("location", _Location),
                ("metadata", ctypes.c_void_p), ("flags", ctypes.c_ubyte * 8)]


class _Access(ctypes.Structure):
    _fields_ = [("location", _Location), ("flags", ctypes.c_int)]


class Region:
    """Mapped device memory with reserved, unmapped addresses before and behind it.  Kept until the process ends."""

    def __init__(self):
        cu = ctypes.CDLL("libcuda.so.1")
        torch.empty(1, device=DEV)  # the context is there and current

        def call(name, *args):
            status = getattr(cu, name)(*args)
            assert status == 0, (name, status)

        u64, size = ctypes.c_uint64, ctypes.c_size_t
        where = _Location(1, torch.device(DEV).index)  # a device
        prop = _Properties(type=1, location=where)     # pinned
        step, base, handle = size(0), u64(0), u64(0)
        call("cuMemGetAllocationGranularity", ctypes.byref(step), ctypes.byref(prop), 0)
        n = step.value
        call("cuMemAddressReserve", ctypes.byref(base), size(3 * n), size(0), u64(0), u64(0))
        call("cuMemCreate", ctypes.byref(handle), size(n), ctypes.byref(prop), u64(0))
        call("cuMemMap", u64(base.value + n), size(n), size(0), handle, u64(0))
        access = _Access(where, 3)  # read and write
        call("cuMemSetAccess", u64(base.value + n), size(n), ctypes.byref(access), size(1))
        self.bytes = n
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": "|u1", "data": (base.value + n, False), "version": 3}


def at_the_end(region, t):
    """A copy of t whose last byte is the region's."""
    raw = t.contiguous().view(-1).view(torch.uint8)
    assert raw.numel() <= region.numel()
    v = region[region.numel() - raw.numel():].view(t.dtype).view(t.shape)
    return v.copy_(t)
