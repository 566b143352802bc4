"""The gated delta rule from a host program without torch (the C ABI on the
driver's memory), in one context of the device after another: the kernels'
leave for their shared memory, given once, holds in both."""
import os
import subprocess
import sys

import pytest
import torch

from delta_rule_linear_dpfp_gb300 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import ctypes
import numpy as np
from delta_rule_linear_dpfp_gb300 import build
from oracle import gated

cu, lib = ctypes.CDLL("libcuda.so.1"), ctypes.CDLL(build.LIB)
lib.fw_gated_delta_forward_workspace_size.restype = ctypes.c_size_t
lib.fw_gated_delta_backward_workspace_size.restype = ctypes.c_size_t
vp, sz, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float


def ok(rc):
    assert rc == 0, rc


def bf16(x):     # to bf16 by truncation, and what that is
    u = x.astype(np.float32).view(np.uint32) >> 16
    return u.astype(np.uint16), (u << 16).view(np.float32).astype(np.float64)


class Buffers:
    def __init__(self):
        self.held = []

    def make(self, nbytes, data=None):
        p = vp()
        ok(cu.cuMemAlloc_v2(ctypes.byref(p), sz(nbytes)))
        self.held.append(p)
        if data is not None:
            data = np.ascontiguousarray(data)
            ok(cu.cuMemcpyHtoD_v2(p, data.ctypes.data_as(vp), sz(nbytes)))
        return p

    def read(self, p, like):
        out = np.empty_like(like)
        ok(cu.cuMemcpyDtoH_v2(out.ctypes.data_as(vp), p, sz(out.nbytes)))
        return out

    def free(self):
        for p in self.held:
            ok(cu.cuMemFree_v2(p))


B, Hk, H, L, d_k, d_v = 1, 1, 2, 130, 64, 48
r = np.random.default_rng(0)
raw = [r.standard_normal((B, Hk, L, d_k)), r.standard_normal((B, Hk, L, d_k)), r.standard_normal((B, H, L, d_v)),
       -r.random((B, H, L)), r.random((B, H, L))]
dy = r.standard_normal((B, H, L, d_v))


def run(io):
    m = Buffers()
    if io:
        pairs = [bf16(x) for x in raw + [dy]]
        stored, wide, e = [p[0] for p in pairs], [p[1] for p in pairs], 2
    else:
        stored, e = [x.astype(np.float32) for x in raw + [dy]], 4
        wide = [x.astype(np.float64) for x in stored]
    ins = [m.make(x.size * e, x) for x in stored]
    y, W = m.make(B * H * L * d_v * e), m.make(B * H * d_v * d_k * 4)
    grads = [m.make(x.size * e) for x in stored[:5]]
    shape = (B, Hk, H, L, d_k, d_v)
    n = lib.fw_gated_delta_forward_workspace_size(*shape, io)
    b = lib.fw_gated_delta_backward_workspace_size(*shape, io)
    ws = m.make(max(n, b))
    rc = lib.fw_gated_delta_forward(*ins[:5], None, W, y, None, ws, sz(n), *shape, 1, f32(1.0), f32(1e-6), io, None)
    assert rc == 0, ("forward", io, rc)
    rc = lib.fw_gated_delta_backward(*ins[:5], None, ins[5], None, *grads, None, None, ws, sz(b), *shape, 1, f32(1.0), f32(1e-6),
                                     io, None)
    assert rc == 0, ("backward", io, rc)
    ok(lib.fw_device_status(None))
    yr, Wr = gated.gated_forward(*wide[:5])
    assert np.abs(m.read(W, Wr.astype(np.float32)) - Wr).max() <= 2.0 ** -12 * np.abs(Wr).max()
    got = m.read(grads[2], stored[2])
    got = (got.astype(np.uint32) << 16).view(np.float32) if io else got
    want = gated.gated_backward(*wide[:5], wide[5])[2]
    assert np.abs(got - want).max() <= 2.0 ** -7 * np.abs(want).max()
    m.free()


ok(cu.cuInit(0))
first, second = vp(), vp()
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(first), 0))
ok(cu.cuCtxCreate_v2(ctypes.byref(second), 0, 0))
for ctx in (first, second, first, second):
    ok(cu.cuCtxSetCurrent(ctx))
    for io in (0, 1):
        run(io)
print("both contexts")
"""


def test_two_contexts():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    out = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "both contexts" in out.stdout, out.stdout[-500:] + out.stderr[-2000:]
