"""Tensors on a GPU that is not the current one: the library launches on the
current device, so every call of the binding makes the tensors' device current
while it enqueues its work, and refuses tensors and streams of several.

Without a GPU: the tensors are headers of CUDA device 1 over host memory (made
through DLPack, nothing reads them), the current device and the library's entries
are stand-ins that record which device was current at the call."""

import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = '''
import ctypes, sys
import torch
import pytest

c = ctypes
torch.cuda._lazy_init = lambda: None
current, calls = [0], []
torch._C._cuda_getCurrentRawStream = lambda i: 0x1000 * (i + 1)
torch.cuda.current_device = lambda: current[0]
torch.cuda.device_count = lambda: 2


class device:
    def __init__(self, d):
        self.d = d if isinstance(d, int) else d.index
    def __enter__(self):
        self.before, current[0] = current[0], self.d
    def __exit__(self, *a):
        current[0] = self.before


class Stream:
    def __init__(self, i):
        self.device, self.device_index, self.cuda_stream = torch.device("cuda", i), i, 0x1000 * (i + 1)


torch.cuda.device = device
torch.cuda.current_stream = lambda d=None: Stream(current[0] if d is None else d if isinstance(d, int) else d.index)


class Dev(c.Structure):
    _fields_ = [("type", c.c_int32), ("id", c.c_int32)]
class Kind(c.Structure):
    _fields_ = [("code", c.c_uint8), ("bits", c.c_uint8), ("lanes", c.c_uint16)]
class Header(c.Structure):
    _fields_ = [("data", c.c_void_p), ("dev", Dev), ("ndim", c.c_int32), ("kind", Kind), ("shape", c.POINTER(c.c_int64)),
                ("strides", c.POINTER(c.c_int64)), ("offset", c.c_uint64), ("owner", c.c_void_p), ("deleter", c.c_void_p)]

capsule = c.pythonapi.PyCapsule_New
capsule.restype, capsule.argtypes = c.py_object, [c.c_void_p, c.c_char_p, c.c_void_p]
room = (c.c_char * (1 << 16))()
room = c.addressof(room) + (-c.addressof(room)) % 4096
ROCM, kept = 10, []
KINDS = {"bf16": (4, 16), "f32": (2, 32), "u8": (1, 8), "i32": (0, 32)}


def tensor(shape, kind, dev=1):
    n = len(shape)
    strides = [1] * n
    for i in range(n - 2, -1, -1):
        strides[i] = strides[i + 1] * shape[i + 1]
    shape, strides = (c.c_int64 * n)(*shape), (c.c_int64 * n)(*strides)
    h = Header(room, Dev(ROCM, dev), n, Kind(*KINDS[kind], 1), shape, strides, 0, None, None)
    kept.append((h, shape, strides))
    t = torch.utils.dlpack.from_dlpack(capsule(c.addressof(h), b"dltensor", None))
    assert t.get_device() == dev and t.is_cuda
    return t


import persistent_tile_scheduled_amd as tsg
real = tsg.load()


class Library:
    """Every entry that takes a stream records the device that is current."""
    def __init__(self):
        for name in tsg.EXPORTS:
            f = getattr(real, name)
            if name.endswith("_workspace"):     # none: torch's allocator has no device here
                fake = c.CFUNCTYPE(c.c_int64, *f.argtypes)(lambda *a: 0)
            elif name in ("tsgemm_create", "tsgemm_destroy", "tsgemm_last_error") or name.startswith("tsgemm_set"):
                setattr(self, name, f)
                continue
            elif name == "tsgemm_mx_packed_scale_bytes":
                fake = c.CFUNCTYPE(c.c_int64, *f.argtypes)(lambda *a: 512)
            else:
                def record(*a, name=name):
                    calls.append((name, current[0], [s for s in a if s in (0x1000, 0x2000)]))
                    return 0
                fake = c.CFUNCTYPE(c.c_int, *f.argtypes)(record)
            setattr(self, name, fake)

def get_device(out):
    out[0] = current[0]
    return 0


tsg._lib = Library()
tsg._lib.hipGetDevice = c.CFUNCTYPE(c.c_int, c.POINTER(c.c_int))(get_device)


def made(name):
    """The one call since the last question was `name`, on device 1 and its stream; device 0 is current again."""
    got = [x for x in calls if x[0] != "tsgemm_launch_info"]
    assert got == [("tsgemm_" + name, 1, [0x2000])], got
    assert all(x[1] == 1 for x in calls), calls
    assert current[0] == 0
    calls.clear()

'''


def _run(body):
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(body)], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_operators_run_on_their_tensors_device():
    _run("""
    x, v, r = tensor((4, 64), "bf16"), tensor((64,), "f32"), tensor((4,), "f32")
    codes, scales, dw = tensor((4, 64), "u8"), tensor((4, 2), "u8"), tensor((64, 64), "f32")
    for kw in ({}, {"stream": Stream(1)}):
        tsg.layer_norm(x, v, v, 1e-5, y=x, **kw)
        made("layer_norm")
        tsg.layer_norm_grad(x, x, v, r, r, x, v, v, **kw)
        made("layer_norm_grad")
        tsg.mx_quantize(x, codes, scales, **kw)
        made("mx_quantize")
        tsg.mx_dequantize(codes, scales, x, **kw)
        made("mx_dequantize")
        tsg.mx_weight_grad(x, codes, scales, dw, **kw)
        made("mx_weight_grad")
    """)


def test_the_current_device_stays_when_it_is_the_tensors():
    _run("""
    def never(d):
        raise AssertionError("device set")
    x, codes, scales = tensor((4, 64), "bf16"), tensor((4, 64), "u8"), tensor((4, 2), "u8")
    torch.cuda.device, current[0] = never, 1
    for kw in ({}, {"stream": Stream(1)}):
        tsg.mx_quantize(x, codes, scales, **kw)
    assert calls == [("tsgemm_mx_quantize", 1, [0x2000])] * 2
    # the extension module took the first call itself
    calls.clear()
    assert tsg._short.mx_quantize(x, codes, scales) == 0
    current[0] = 0
    assert tsg._short.mx_quantize(x, codes, scales) is None
    assert len(calls) == 1
    """)


def test_plans_run_on_their_tensors_device():
    _run("""
    a, b, t = tensor((128, 128), "bf16"), tensor((128, 128), "bf16"), tensor((64, 4), "i32")
    p = tsg.Plan(128, 128, 128, "bf16", 128, 128, 64, 8, 2)
    m = tsg.Plan(256, 256, 128, "mxfp8", 256, 256, 128, 8, 2)
    p._lib = m._lib = tsg._lib
    q, s, o, f = tensor((256, 128), "u8"), tensor((256, 4), "u8"), tensor((256, 256), "bf16"), tensor((512,), "u8")
    for kw in ({}, {"stream": Stream(1)}):
        p.run(a, b, a, **kw)
        made("run")
        p.run_traced(a, b, a, t, **kw)
        made("run_traced")
        m.run_mx(q, s, q, s, o, **kw)
        made("run_mx")
        m.run_mx_noalloc(q, s, q, s, o, **kw)
        made("run_mx_noalloc")
        m.run_mx_traced(q, s, q, s, o, t, **kw)
        made("run_mx_traced")
        m.mx_pack_scales(s, f, 0, **kw)
        made("mx_pack_scales")
        m.run_mx_packed(q, f, q, f, o, **kw)
        made("run_mx_packed")
    """)


def test_several_devices_are_refused():
    _run("""
    a, b, t = tensor((128, 128), "bf16"), tensor((128, 128), "bf16", dev=0), tensor((64, 4), "i32", dev=0)
    p = tsg.Plan(128, 128, 128, "bf16", 128, 128, 64, 8, 2)
    m = tsg.Plan(256, 256, 128, "mxfp8", 256, 256, 128, 8, 2)
    p._lib = m._lib = tsg._lib
    q, s, o, f = tensor((256, 128), "u8"), tensor((256, 4), "u8"), tensor((256, 256), "bf16"), tensor((512,), "u8")
    s0, o0, f0 = tensor((256, 4), "u8", dev=0), tensor((256, 256), "bf16", dev=0), tensor((512,), "u8", dev=0)
    x, v = tensor((4, 64), "bf16"), tensor((64,), "f32")
    codes, scales, dw = tensor((4, 64), "u8"), tensor((4, 2), "u8"), tensor((64, 64), "f32")
    for call in (lambda: p.run(a, b, a), lambda: p.run(a, a, b), lambda: p.run_traced(a, a, a, t), lambda: m.run_mx(q, s0, q, s, o),
                 lambda: m.run_mx_noalloc(q, s, q, s, o0), lambda: m.run_mx_traced(q, s, q, s, o, t),
                 lambda: m.mx_pack_scales(s, f0, 0), lambda: m.run_mx_packed(q, f0, q, f, o),
                 # and a stream of another device than the tensors'
                 lambda: p.run(a, a, a, stream=Stream(0)), lambda: m.run_mx(q, s, q, s, o, stream=Stream(0)),
                 lambda: tsg.layer_norm(x, v, v, 1e-5, y=x, stream=Stream(0)),
                 lambda: tsg.mx_quantize(x, codes, scales, stream=Stream(0)),
                 lambda: tsg.mx_weight_grad(x, codes, scales, dw, stream=Stream(0))):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not [x for x in calls if x[0] != "tsgemm_launch_info"] and current[0] == 0
    """)
