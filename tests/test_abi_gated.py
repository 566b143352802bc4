"""Refusals of the gated delta rule's and the group norm's entry points (host
only: every call fails its checks before any CUDA call)."""
import ctypes

import pytest

from delta_rule_linear_dpfp_gb300 import binding, build

FAKE, MISALIGNED = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
E, U, OK = binding.FW_ERR_INVALID_ARG, binding.FW_ERR_UNSUPPORTED, binding.FW_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _call(fn, names, base):
    def call(**kw):
        a = dict(base)
        a.update(kw)
        return fn(*[a[n] for n in names])
    return call


SHAPE = ["B", "Hk", "H", "L", "d_k", "d_v"]
SIZES = dict(B=2, Hk=2, H=4, L=70, d_k=64, d_v=64)
OPTS = dict(l2norm=1, scale=1.0, eps=1e-6, io=1, stream=None)


def _shapes_refused(call, seq=True):
    assert call(Hk=0) == E and call(H=0) == E and call(H=5) == E and call(B=-1) == E
    assert call(d_k=0) == E and call(d_v=0) == E and call(io=2) == E
    assert call(l2norm=2) == E and call(scale=float("inf")) == E and call(eps=-1.0) == E and call(eps=float("nan")) == E
    assert call(d_k=48) == U and call(d_k=256) == U and call(d_v=24) == U and call(d_v=272) == U
    assert call(B=40000, H=2, Hk=2) == U
    if seq:
        assert call(L=-1) == E and call(L=2**31 - 1) == U


@pytest.mark.parametrize("io", [0, 1])
def test_forward_refusals(lib, io):
    need = lib.fw_gated_delta_forward_workspace_size(2, 2, 4, 70, 64, 64, io)
    assert need > 0
    ptrs = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, W0=None, Wf=None, y=FAKE, lengths=None, ws=FAKE, wsb=need)
    call = _call(lib.fw_gated_delta_forward, list(ptrs) + SHAPE + ["l2norm", "scale", "eps", "io", "stream"],
                 {**ptrs, **SIZES, **OPTS, "io": io})
    for n in ("q", "k", "v", "g", "beta", "y", "ws"):
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    for n in ("W0", "Wf", "lengths"):
        assert call(**{n: MISALIGNED}) == E, n
    assert call(wsb=need - 1) == E
    _shapes_refused(call)
    assert call(B=0, q=None, k=None, v=None, g=None, beta=None, y=None, ws=None, wsb=0) == OK
    assert call(L=0, q=None, k=None, v=None, g=None, beta=None, y=None, ws=None, wsb=0) == OK


def test_backward_refusals(lib):
    need = lib.fw_gated_delta_backward_workspace_size(2, 2, 4, 70, 64, 64, 1)
    assert need > lib.fw_gated_delta_forward_workspace_size(2, 2, 4, 70, 64, 64, 1)
    ptrs = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, W0=None, dy=FAKE, dWf=None, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE,
                dbeta=FAKE, dW0=None, lengths=None, ws=FAKE, wsb=need)
    call = _call(lib.fw_gated_delta_backward, list(ptrs) + SHAPE + ["l2norm", "scale", "eps", "io", "stream"],
                 {**ptrs, **SIZES, **OPTS})
    for n in ("q", "k", "v", "g", "beta", "dy", "dq", "dk", "dv", "dg", "dbeta", "ws"):
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    for n in ("W0", "dWf", "dW0", "lengths"):
        assert call(**{n: MISALIGNED}) == E, n
    assert call(wsb=need - 1) == E
    _shapes_refused(call)
    assert call(B=0, q=None, dq=None, ws=None, wsb=0) == OK
    assert call(L=0, q=None, dq=None, ws=None, wsb=0) == OK     # no dW0 asked for: nothing to do


def test_decode_refusals(lib):
    ptrs = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, W=FAKE, y=FAKE)
    call = _call(lib.fw_gated_delta_decode_step,
                 list(ptrs) + ["B", "Hk", "H", "d_k", "d_v", "l2norm", "scale", "eps", "io", "stream"],
                 {**ptrs, **SIZES, **OPTS})
    for n in ptrs:
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    _shapes_refused(call, seq=False)
    assert call(B=0, q=None, W=None, y=None) == OK


def test_workspace_queries(lib):
    for f in (lib.fw_gated_delta_forward_workspace_size, lib.fw_gated_delta_backward_workspace_size):
        assert f(2, 2, 4, 70, 48, 64, 1) == 0 and f(2, 3, 4, 70, 64, 64, 1) == 0 and f(2, 2, 4, 2**31 - 1, 64, 64, 1) == 0
        assert f(2, 2, 4, 1, 64, 64, 1) > 0 and f(1, 1, 1, 2**31 - 65, 16, 16, 1) > 2**32
    f = lib.fw_group_norm_act_backward_workspace_size
    assert f(2, 4, 8, 64) > 0 and f(2, 4, 8, 63) == 0 and f(0, 4, 8, 64) == 0 and f(2, 4, 8, 264) == 0


def test_norm_refusals(lib):
    sizes = dict(B=2, H=4, L=8, d=64, act=2, io=1, eps=1e-5, stream=None)
    ptrs = dict(x=FAKE, gate=None, gamma=FAKE, beta=FAKE, out=FAKE)
    call = _call(lib.fw_group_norm_act, list(ptrs) + list(sizes), {**ptrs, **sizes})
    need = lib.fw_group_norm_act_backward_workspace_size(2, 4, 8, 64)
    bptrs = dict(x=FAKE, gate=FAKE, gamma=FAKE, beta=FAKE, dout=FAKE, dx=FAKE, dgate=FAKE, dgamma=FAKE, dbeta2=FAKE, ws=FAKE,
                 wsb=need)
    back = _call(lib.fw_group_norm_act_backward, list(bptrs) + list(sizes), {**bptrs, **sizes})
    for n in ("x", "gamma", "beta", "out"):
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    assert call(gate=MISALIGNED) == E
    for n in ("x", "gamma", "beta", "dout", "dx", "dgamma", "dbeta2", "ws"):
        assert back(**{n: None}) == E and back(**{n: MISALIGNED}) == E, n
    assert back(gate=None) == E and back(dgate=None) == E        # dgate goes with gate
    assert back(wsb=need - 1) == E
    for c in (call, back):
        assert c(B=-1) == E and c(d=0) == E and c(act=4) == E and c(act=-1) == E and c(io=5) == E
        assert c(eps=-1.0) == E and c(eps=float("inf")) == E
        assert c(d=12) == U and c(d=264) == U and c(H=70000) == U
    assert call(B=0, x=None, out=None) == OK and call(L=0, x=None, out=None) == OK


def test_sizes_past_an_int_are_refused():
    """A length of 2^32 + 5 is not one of 5 (tensors without memory: the checks come before any call)."""
    import torch
    m = dict(dtype=torch.bfloat16, device="meta")
    L = 2 ** 32 + 5
    f = torch.empty(8, dtype=torch.float32, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        binding._norm_shapes(torch.empty(1, 1, L, 8, **m), f, f, None, "none")
    assert binding._norm_shapes(torch.empty(1, 1, 2 ** 31 - 1, 8, **m), f, f, None, "none") == (1, 1, 2 ** 31 - 1, 8)
    q, v, g = torch.empty(1, 1, L, 16, **m), torch.empty(1, 2, L, 16, **m), torch.empty(1, 2, L, **m)
    with pytest.raises(ValueError, match="2\\^31"):
        binding._gated_shapes("call", q, q, v, g, g, (), None)
    q, v, g = (t[:, :, :70] for t in (q, v, g))
    assert binding._gated_shapes("call", q, q, v, g, g, (), None)[3] == 70
